"""CPU pins of the gated linear recurrence's fp64 oracle: closed forms,
central differences for every gradient, and the tolerances of the GPU tests
(tests/_glr_bars.py) against arithmetic in fp32 and planted mistakes."""
import numpy as np
import pytest

from oracle import glr
from tests import _glr_bars as bars

CU = [0, 5, 5, 6, 13]


def batch(seed, D=3, rate=1.0):
    r = np.random.default_rng(seed)
    N, n = CU[-1], len(CU) - 1
    return dict(x=r.standard_normal((N, D)), g=-np.exp(r.standard_normal((N, D))), r=r.standard_normal((N, D)),
                i=r.standard_normal((N, D)), rate=rate * (0.05 + r.random(D)), h0=r.standard_normal((n, D)),
                dh=r.standard_normal((N, D)), dh_T=r.standard_normal((n, D)))


def test_closed_forms():
    b = batch(0)
    # no input: the state decays; an empty sequence keeps its own
    h, h_T = glr.glr_plain(0 * b["x"], b["g"], CU, b["h0"])
    assert np.allclose(h_T[0], np.exp(b["g"][:5].sum(0)) * b["h0"][0]) and np.array_equal(h_T[1], b["h0"][1])
    # no decay: a running sum; full decay: the input itself
    h, _ = glr.glr_plain(b["x"], 0 * b["g"], CU)
    assert np.allclose(h[6:13], np.cumsum(b["x"][6:13], 0))
    h, _ = glr.glr_plain(b["x"], np.full_like(b["g"], -np.inf), CU, b["h0"])
    assert np.array_equal(h, b["x"])
    # gated: an open decay gate at a high rate leaves the gated input, a closed one keeps the state
    h, _ = glr.glr_gated(b["x"], np.full_like(b["r"], 40.0), b["i"], np.full(3, 60.0), CU, b["h0"])
    assert np.allclose(h, glr.logistic(b["i"]) * b["x"], atol=1e-12)
    h, h_T = glr.glr_gated(b["x"], np.full_like(b["r"], -800.0), b["i"], b["rate"], CU, b["h0"])
    assert np.allclose(h_T, b["h0"]) and np.allclose(h[:5], b["h0"][0])
    # a^2 + (u / (s(i) x))^2 = 1
    q = glr.gates(b["x"], b["r"], b["i"], b["rate"])
    assert np.allclose(q["a"] ** 2 + (q["u"] / (q["si"] * b["x"])) ** 2, 1)


def test_rows_behind_the_last_sequence_do_not_matter():
    b = batch(1)
    cut = [0, 5, 5, 6, 9]
    h, h_T = glr.glr_plain(b["x"], b["g"], cut, b["h0"])
    h2, h_T2 = glr.glr_plain(b["x"][:9], b["g"][:9], cut, b["h0"])
    assert np.array_equal(h[:9], h2) and np.array_equal(h_T, h_T2) and not h[9:].any()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("seed", [2, 3])
def test_vjp_against_differences(gated, seed):
    b = batch(seed)
    names = ("x", "r", "i", "rate", "h0") if gated else ("x", "g", "h0")

    def loss(**kw):
        y = {**b, **kw}
        if gated:
            h, h_T = glr.glr_gated(y["x"], y["r"], y["i"], y["rate"], CU, y["h0"])
        else:
            h, h_T = glr.glr_plain(y["x"], y["g"], CU, y["h0"])
        return (h * b["dh"]).sum() + (h_T * b["dh_T"]).sum()

    if gated:
        grads = glr.glr_gated_vjp(b["x"], b["r"], b["i"], b["rate"], b["dh"], CU, b["h0"], b["dh_T"])
    else:
        grads = glr.glr_plain_vjp(b["x"], b["g"], b["dh"], CU, b["h0"], b["dh_T"])
    e = 1e-5
    for name, gr in zip(names, grads):
        num = np.zeros_like(b[name])
        for at in np.ndindex(num.shape):
            up, dn = b[name].copy(), b[name].copy()
            up[at] += e
            dn[at] -= e
            num[at] = (loss(**{name: up}) - loss(**{name: dn})) / (2 * e)
        # differences: e^2 times a third derivative, and 1e-16 / e of the loss
        assert np.allclose(gr, num, rtol=1e-6, atol=1e-8), name


def test_closed_gate_gradients_are_finite():
    b = batch(4)
    r = b["r"].copy()
    r[2], r[7] = -1e4, 1e4
    for x in glr.glr_gated_vjp(b["x"], r, b["i"], b["rate"], b["dh"], CU, b["h0"], b["dh_T"]):
        assert np.isfinite(x).all()
    for x in glr.glr_gated_vjp(b["x"], r, b["i"], 0 * b["rate"], b["dh"], CU, b["h0"], b["dh_T"]):
        assert np.isfinite(x).all()


def fp32_forward(b, gated, wrong=""):
    """The recurrence in fp32, with what `wrong` names planted in it."""
    f = np.float32
    x, h0 = b["x"].astype(f), b["h0"].astype(f)
    if gated:
        sr, si = (f(1) / (f(1) + np.exp(-b[k].astype(f))) for k in ("r", "i"))
        g = -b["rate"].astype(f) * sr
        a = np.exp(g)
        m = np.sqrt(f(1) - a * a) if wrong == "cancellation" else np.sqrt(-np.expm1(f(2) * g))
        u = m * si * x
    else:
        a, u = np.exp(b["g"].astype(f)), x
    h = np.zeros_like(x)
    for n in range(len(CU) - 1):
        s = h0[n] if wrong != "h0 dropped" else 0 * h0[n]
        if wrong == "carry from the last sequence" and n:
            s = h0[n] + h[CU[n] - 1]
        for t in range(CU[n], CU[n + 1]):
            s = a[t] * s + u[t]
            if wrong == "state in bf16":
                s = (s.view(np.uint32) + 0x8000 & 0xffff0000).astype(np.uint32).view(f)
            h[t] = s
    return h


@pytest.mark.parametrize("gated", [False, True])
def test_tolerances_hold_fp32_and_reject_mistakes(gated):
    for seed in range(20):
        b = batch(seed, D=8, rate=1e-3 if gated else 1.0)
        b = {k: v.astype(np.float32).astype(np.float64) for k, v in b.items()}
        ref = bars.reference(b, CU, gated, grads=False)
        over = lambda wrong: np.abs(fp32_forward(b, gated, wrong) - ref["h"][0]) > ref["h"][1]     # noqa: E731
        assert not over("").any()
        for wrong in ("h0 dropped", "carry from the last sequence", "state in bf16"):
            assert over(wrong).any(), wrong
        if gated:
            assert over("cancellation").any()
