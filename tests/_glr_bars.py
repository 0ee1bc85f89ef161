"""Tolerances of the gated linear recurrence's outputs: bounds on the error of
fp32 arithmetic, element by element, carried through the recurrence in fp64.

With e = 2^-24 (half a step of fp32), to first order, relative errors:
- the plain factor a = exp(g): 1.5 e (its polynomial's last sum rounds once,
  and the reduction behind it adds less than half of that);
- s(z) = 1 / (1 + e^-z) through the hardware's 2^x and 1 / x, each off by one
  step (2 e): the exponent z log2 e is rounded twice (constant and product),
  1.5 e |z|; then 2 e, and e for the sum and 2 e for 1 / x: (1.5 |z| + 5) e;
- g = -rate s(r): that and e =: eg; below -87 a is held at 1.6e-38;
- e^g - 1: eg, as |g e^g / (e^g - 1)| <= 1, and 2.2 e (a polynomial off by 0.4 e
  and two roundings, 1.3e-7 at most in all);
- a = e^g as 1 + (e^g - 1): |g| eg + e / 2 and 2.2 e (1 / a - 1), which at the far
  end of what is not reduced, g = -0.69, is 2.2 e: 1.5 e + 2.5 e min(|g|, 0.7);
- m = sqrt(-(e^g - 1)(e^g + 1)): the product 2 eg + 4.4 e + 2 e, of which the root
  leaves half; 2 e for its own step, and 2 e more for m = m^2 (1 / sqrt):
  eg + 7.2 e =: em;
- u = m s(i) x: em + es(i) + 2 e.
A state's error obeys  E_t = a E_{t-1} + |a h_{t-1}| (ea + 2 e) + |u| eu + e |h|,
where 2 e is there for the tiles' products of factors (one rounding a token
and one where a product is applied); L's  E_t = e |L_t| + a E_{t+1} + |a L_{t+1}|
(ea + 2 e) with the next token's a.  Gradients add the
errors of their factors.  A sum over n tokens in fp32 by parts adds
(64 + 2) e times the sum of its terms' magnitudes, whatever n (a part is 128
tokens at most in some order of pairs, parts are summed in 64 bits).
Numbers below the smallest normal one (1.2e-38) count as it or as zero, so a
product of factors of which one is that small is off by TINY = 2e-38 times
the others, whatever its own size.  A decay gate below -87, where s(r) is
1.6e-38 or less, may count as -87 or as closed (s = 0): m, and with it s(r) / m
times the rate, is then off by at most sqrt(2 * 1.6e-38 rate) < 4e-19
sqrt(rate) =: CLOSED.
All bounds are doubled for what is second order and for sums that round at
an intermediate size.  A value stored in bf16 is off by its half step
besides.
"""
import numpy as np

from oracle import glr
from tests._gpu_util import half_ulp_bf16

E = 2.0 ** -24
TINY = 2e-38                 # factors below the smallest normal number count as it or as zero


def _eps(q):
    es = lambda z: (1.5 * np.minimum(np.abs(z), 90) + 5) * E                 # noqa: E731
    eg = es(q["r"]) + E
    ea = np.minimum(-q["g"], 90) * eg + (1.5 + 2.5 * np.minimum(-q["g"], 0.7)) * E
    em = eg + 7.2 * E
    return es(q["r"]), es(q["i"]), ea, em


def reference(b, cu, gated, grads=True):
    """{output: (values, largest error)} of a batch of fp64 arrays; b["dh"] and
    the like are wanted with grads."""
    h0 = b.get("h0")
    if gated:
        q = glr.gates(b["x"], b["r"], b["i"], b["rate"])
        esr, esi, ea, em = _eps(q)
        a, u, eu = q["a"], q["u"], em + esi + 2 * E
        closed = np.where(b["r"] < -87, 4e-19 * np.sqrt(b["rate"]), 0.0)
    else:
        a, u, ea, eu, closed = np.exp(b["g"]), b["x"], 1.5 * E, 0.0, 0.0
    ea = ea + 2 * E
    size = np.abs(b["x"])
    h, h_T, before = glr.scan(a, u, cu, h0)
    own = np.abs(a * before) * ea + np.abs(u) * eu + E * np.abs(h) + TINY * (np.abs(before) + size + 1) + closed * size
    Eh, EhT, Ebefore = glr.scan(a, own, cu)
    out = {"h": (h, 2 * Eh), "h_T": (h_T, 2 * EhT)}
    if not grads:
        return out
    dh_T = b.get("dh_T")
    L, dh0 = glr.sweep(a, b["dh"], cu, dh_T)
    # the product a L that a token hands to the one before it (or to dh0) is off by a's error, which where a is
    # below the smallest normal number is TINY itself and not a part of the product
    handed = np.abs(a * L) * ea + TINY * (np.abs(L) + 1)
    own = E * np.abs(L)
    own[:-1] += handed[1:]
    EL, Edh0 = glr.sweep(a, own, cu)
    for n, (s, e) in enumerate(zip(cu, cu[1:])):
        if e > s:
            Edh0[n] += handed[s]
    w, Ew = a * before, np.abs(a) * Ebefore + np.abs(a * before) * ea + TINY * np.abs(before)
    if not gated:
        dg = L * w
        out.update(dx=(L, 2 * EL), dg=(dg, 2 * (EL * np.abs(w) + np.abs(L) * Ew + E * np.abs(dg))))
    else:
        dx, dr, di, drate, _ = glr.glr_gated_vjp(b["x"], b["r"], b["i"], b["rate"], b["dh"], cu, h0, dh_T)
        bb = np.abs(q["m"] * q["si"])
        x = np.abs(q["x"])
        rel = lambda v, e: np.abs(v) * e                                     # noqa: E731
        Edx = EL * bb + rel(dx, eu + E) + (TINY + closed) * np.abs(L)
        Edi = Edx * x * q["rest_i"] + rel(di, esi + 3 * E) + TINY * (np.abs(L) * x + 1)
        inv = np.divide(1.0, q["m"], out=np.zeros_like(q["m"]), where=q["m"] > 0)
        c = q["si"] * q["x"] * a * a * inv
        ec = esi + 2 * ea + em + 5 * E
        Ein = Ew + np.abs(c) * ec + E * np.abs(w - c) + TINY * inv * x       # of w - c
        Edg = EL * np.abs(w - c) + np.abs(L) * Ein
        qq = q["rate"] * q["sr"] * q["rest_r"]
        Edr = Edg * qq + rel(dr, 2 * esr + 5 * E) + np.abs(L) * (closed * x + TINY * (np.abs(w - c) + 1))
        terms = np.abs(L * (w - c) * q["sr"])
        inside = np.zeros(len(x), bool)
        for s, e in zip(cu, cu[1:]):
            inside[s:e] = True
        # s(r) / m is CLOSED over the rate
        over = np.divide(closed, q["rate"], out=np.zeros_like(closed), where=closed > 0)
        Edrate = Edg * q["sr"] + terms * (esr + (3 + 66) * E) + np.abs(L) * (over * x + TINY * (np.abs(w) + 1))
        out.update(dx=(dx, 2 * Edx), dr=(dr, 2 * Edr), di=(di, 2 * Edi), drate=(drate, 2 * Edrate[inside].sum(0)))
    out["dh0"] = (dh0, 2 * Edh0)
    return out


def check(name, x, want, rows=slice(None)):
    """A device output against (values, largest error)."""
    ref, tol = want
    got = x.detach().double().cpu().numpy()[rows]
    ref, tol = ref[rows], tol[rows]
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), name
    if str(x.dtype) == "torch.bfloat16":
        # the value that is rounded is at most ref's size and its error
        tol = tol + half_ulp_bf16(np.abs(ref) + tol) + 1e-40
    d = np.abs(got - ref)
    worst = float((d / np.maximum(tol, 1e-300)).max(initial=0.0))
    scale = np.abs(ref).max(initial=0.0)
    print(f"  {name}: {worst:.2f} of what is allowed; most {d.max(initial=0.0) / max(scale, 1e-300):.1e} of the largest",
          flush=True)
    assert worst <= 1, (name, worst, np.unravel_index(np.argmax(d / np.maximum(tol, 1e-300)), d.shape))
