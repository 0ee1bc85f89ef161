"""fp64 oracle of the gated delta rule (include/gdr.h): the recurrence token by
token, its reverse mode with every state kept, and the 8-bit form of q, k, v.

    S' = exp(g_t) S;  u = beta_t (v_t - S'^T k_t);  S = S' + k_t u^T;  o_t = scale S^T q_t

q, k have H_k heads, v, g, beta H_v: value head h uses key head h // (H_v // H_k).
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _f64(*xs):
    return tuple(None if x is None else np.asarray(x, np.float64) for x in xs)


def gdr_recurrent(q, k, v, g, beta, scale, S0=None, keep=False):
    """One sequence: q, k [T, H_k, d_k], v [T, H_v, d_v], g, beta [T, H_v].
    Returns (o, S_T), with keep also S', e = v - S'^T k and S of every token."""
    q, k, v, g, beta, S0 = _f64(q, k, v, g, beta, S0)
    T, Hv, dv = v.shape
    r = Hv // q.shape[1]
    q, k = np.repeat(q, r, 1), np.repeat(k, r, 1)
    S = np.zeros((Hv, q.shape[2], dv)) if S0 is None else S0.copy()
    o, kept = np.zeros((T, Hv, dv)), []
    for t in range(T):
        Sd = np.exp(g[t])[:, None, None] * S
        e = v[t] - np.einsum("hkv,hk->hv", Sd, k[t])
        S = Sd + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
        o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        if keep:
            kept.append((Sd, e, S))
    return (o, S, kept) if keep else (o, S)


def gdr_recurrent_vjp(q, k, v, g, beta, dO, scale, S0=None, dS_T=None):
    """(dq, dk, dv, dg, dbeta, dS0) of one sequence."""
    _, S, kept = gdr_recurrent(q, k, v, g, beta, scale, S0, keep=True)
    q, k, v, g, beta, dO, dS_T = _f64(q, k, v, g, beta, dO, dS_T)
    Hk, r = q.shape[1], v.shape[1] // q.shape[1]
    qr, kr = np.repeat(q, r, 1), np.repeat(k, r, 1)
    L = np.zeros_like(S) if dS_T is None else dS_T.copy()
    dq, dk, dv = np.zeros_like(qr), np.zeros_like(kr), np.zeros_like(v)
    dg, db = np.zeros_like(g), np.zeros_like(beta)
    for t in reversed(range(v.shape[0])):
        Sd, e, St = kept[t]
        b = beta[t][:, None]
        L = L + scale * qr[t][:, :, None] * dO[t][:, None, :]
        dq[t] = scale * np.einsum("hkv,hv->hk", St, dO[t])
        du = np.einsum("hkv,hk->hv", L, kr[t])
        dv[t] = b * du
        db[t] = (du * e).sum(-1)
        dk[t] = np.einsum("hkv,hv->hk", L, b * e) - np.einsum("hkv,hv->hk", Sd, b * du)
        dSd = L - kr[t][:, :, None] * (b * du)[:, None, :]
        dg[t] = (dSd * Sd).sum((1, 2))
        L = np.exp(g[t])[:, None, None] * dSd
    share = lambda x: x.reshape(x.shape[0], Hk, r, x.shape[2]).sum(2)      # noqa: E731
    return share(dq), share(dk), dv, dg, db, L


def packed(fn, cu, args, states, *rest):
    """Applies a one-sequence function to every sequence of a packed batch;
    the last output is a state, the others are rows of tokens."""
    outs = []
    for n in range(len(cu) - 1):
        sl = slice(int(cu[n]), int(cu[n + 1]))
        outs.append(fn(*(x[sl] for x in args), *rest,
                       *(None if s is None else s[n] for s in states)))
    return tuple(np.concatenate([o[i] for o in outs]) for i in range(len(outs[0]) - 1)) + \
        (np.stack([o[-1] for o in outs]),)


def kept8(x):
    """The values 8 bits keep of x: blocks of min(32, d) channels over the
    smallest power of two that brings their largest finite magnitude to 448
    or less (within 2^-110 .. 2^119), elements on the e4m3 grid, ties to
    even, infinities and NaN as NaN."""
    x = np.asarray(x, np.float64)
    blk = x.reshape(x.shape[:-1] + (-1, min(32, x.shape[-1])))
    fin = np.isfinite(blk)
    top = np.where(fin, np.abs(blk), 0.0).max(-1, keepdims=True)
    e = np.where(top > 0, np.ceil(np.log2(np.maximum(top, 1e-300) / E4M3_MAX)), -110)
    unit = 2.0 ** np.clip(e, -110, 119)
    y = np.clip(np.where(fin, blk, 0.0) / unit, -E4M3_MAX, E4M3_MAX)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))), -6) - 3)
    return np.where(fin, np.rint(y / step) * step * unit, np.nan).reshape(x.shape)
