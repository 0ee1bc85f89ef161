"""fp64 chunk form of the gated delta rule and of its gradients (the algebra at
the top of csrc/gdr_chunk.hip and csrc/gdr_grad.hip), for one sequence.

It is the oracle that mistakes are planted in: `held` rounds an operand to so
many bf16 parts, `drop` leaves terms of dg out.  With neither it has to equal
the token-by-token oracle (oracle/gdr.py).

It also says how much larger the numbers are that an output is formed from, as
squared 2-norms that add up over sequences (`growth` makes the ratios):
- "Y": the rows V and e^G K S whose difference the residuals R solve for, by R;
- "F": the rows P0^T dO and e^{G_C - G} K L whose sum Ub solves for, by Ub;
- "dg": the terms that dg_t is a sum of, over all t, by dg.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle.gdr import _f64

DG_TERMS = ("read", "erase", "late", "state", "dP", "dN")


def parts(x, n):
    """x held in n bf16 parts, each the rounding of what those before it leave."""
    if n is None:
        return x
    x = np.asarray(x, np.float64)
    left, out = x.copy(), np.zeros_like(x)
    for _ in range(n):
        h = torch.from_numpy(left).to(torch.bfloat16).double().numpy()
        out += h
        left -= h
    return out


def _tr(x):
    return np.swapaxes(x, -1, -2)


def gdr_chunked_vjp(q, k, v, g, beta, dO, scale, S0=None, dS_T=None, C=64, held=None, drop=()):
    """((o, S_T), (dq, dk, dv, dg, dbeta, dS0), norms) of one sequence.

    q, k [T, H_k, d_k], v, dO [T, H_v, d_v], g, beta [T, H_v]; held: parts of
    "S" and "L" where the chunk's rows multiply them, "U" and "Yb" where dg
    is formed; drop: some of DG_TERMS."""
    held = held or {}
    q, k, v, g, beta, dO, S0, dS_T = _f64(q, k, v, g, beta, dO, S0, dS_T)
    T, Hv, dv = v.shape
    Hk, dk = q.shape[1:]
    r = Hv // Hk
    heads = lambda x: np.moveaxis(np.repeat(x, r, 1), 0, 1)               # noqa: E731  [H_v, T, d_k]
    q, k, v, dO = heads(q), heads(k), np.moveaxis(v, 0, 1), np.moveaxis(dO, 0, 1)
    g, b = np.maximum(g, -1e4).T, beta.T
    S = np.zeros((Hv, dk, dv)) if S0 is None else S0.copy()
    cuts = [slice(c, min(c + C, T)) for c in range(0, T, C)]
    form, o = [], np.zeros_like(v)
    norms = {x: np.zeros(2) for x in ("Y", "F", "dg")}
    sq = lambda *xs: sum((x ** 2).sum() for x in xs)                       # noqa: E731
    for s in cuts:
        n = s.stop - s.start
        G = np.cumsum(g[:, s], 1)
        D = np.exp(np.minimum(G[:, :, None] - G[:, None, :], 0)) * np.tril(np.ones((n, n)))
        eG, eR, gam = np.exp(G)[..., None], np.exp(G[:, -1:] - G)[..., None], np.exp(G[:, -1])[:, None, None]
        bc = b[:, s, None]
        kk, qk = k[:, s] @ _tr(k[:, s]), q[:, s] @ _tr(k[:, s])
        N = np.tril(D, -1) * kk
        KS = eG * (k[:, s] @ parts(S, held.get("S")))
        R = np.linalg.solve(np.eye(n) + N * _tr(bc), v[:, s] - KS)
        o[:, s] = scale * eG * (q[:, s] @ S) + (scale * D * qk * _tr(bc)) @ R
        form.append((D, eG, eR, gam, bc, kk, qk, N, S, R))
        norms["Y"] += sq(v[:, s], KS), sq(R)
        S = gam * S + _tr(k[:, s]) @ (bc * eR * R)
    S_T = S
    L = np.zeros_like(S) if dS_T is None else dS_T.copy()
    dq, dkey, dval = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, db = np.zeros_like(g), np.zeros_like(b)
    for s, (D, eG, eR, gam, bc, kk, qk, N, S, R) in zip(reversed(cuts), reversed(form)):
        n = s.stop - s.start
        KL = eR * (k[:, s] @ parts(L, held.get("L")))
        PO = _tr(scale * D * qk) @ dO[:, s]
        Ub = np.linalg.solve(np.eye(n) + _tr(N * bc), PO + KL)
        norms["F"] += sq(PO, KL), sq(Ub)
        U, Yb = bc * R, bc * Ub
        Ug, Yg = parts(U, held.get("U")), parts(Yb, held.get("Yb"))
        dP = scale * D * (dO[:, s] @ _tr(U))
        dN = -np.tril(D, -1) * (Yb @ _tr(U))
        x1, x2, x3 = scale * eG * (dO[:, s] @ _tr(S)), eG * (Yb @ _tr(S)), eR * (U @ _tr(L))
        terms = {"read": (q[:, s] * x1).sum(-1), "erase": -(k[:, s] * (eG * (Yg @ _tr(S)))).sum(-1),
                 "late": (k[:, s] * (eR * (Ug @ _tr(L)))).sum(-1),
                 "state": gam[:, :, 0] * (L * S).sum((1, 2))[:, None],
                 "dP": np.tril(scale * D * (dO[:, s] @ _tr(Ug)) * qk, -1),
                 "dN": -np.tril(D, -1) * (Yg @ _tr(Ug)) * kk}
        for name in drop:
            terms[name] = 0 * terms[name]
        for t in range(n):
            of_t = [terms["read"][:, t:], terms["erase"][:, t:], terms["late"][:, :t], terms["state"]]
            of_t += [terms[x][:, t:, :t].reshape(Hv, -1) for x in ("dP", "dN")]
            dg[:, s.start + t] = sum(x.sum(1) for x in of_t)
            norms["dg"] += sq(*of_t), sq(dg[:, s.start + t])
        dval[:, s], db[:, s] = Yb, (Ub * R).sum(-1)
        dq[:, s] = x1 + dP @ k[:, s]
        dkey[:, s] = x3 - x2 + _tr(dP) @ q[:, s] + (dN + _tr(dN)) @ k[:, s]
        L = gam * L + _tr(q[:, s]) @ (scale * eG * dO[:, s]) - _tr(k[:, s]) @ (eG * Yb)
    rows = lambda x: np.moveaxis(x, 0, 1)                                  # noqa: E731
    share = lambda x: rows(x).reshape(T, Hk, r, dk).sum(2)                 # noqa: E731
    return (rows(o), S_T), (share(dq), share(dkey), rows(dval), dg.T, db.T, L), norms


def growth(norms):
    """The ratios "Y", "F" and "dg" over the norms of some sequences, 1 at least."""
    total = {x: sum((n[x] for n in norms), np.zeros(2)) for x in ("Y", "F", "dg")}
    return {x: float(max(1.0, np.sqrt(a / b))) if b > 0 else 1.0 for x, (a, b) in total.items()}
