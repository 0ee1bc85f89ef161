"""fp64 oracle of the gated linear recurrence (include/glr.h): the recurrence
token by token over a packed batch, and its reverse.

    h_t = a_t h_{t-1} + u_t
    plain  a = exp(g),             u = x
    gated  a = exp(-rate s(r)),    u = sqrt(1 - a^2) s(i) x,    s(z) = 1 / (1 + exp(-z))
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


def logistic(z):
    """s(z), from the side that does not overflow."""
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def gates(x, r, i, rate):
    """a, u and the parts that they are made of."""
    x, r, i, rate = _f64(x), _f64(r), _f64(i), _f64(rate)
    sr, si = logistic(r), logistic(i)
    g = -rate * sr
    m = np.sqrt(-np.expm1(2 * g))
    return dict(x=x, r=r, i=i, sr=sr, si=si, rest_r=logistic(-r), rest_i=logistic(-i), g=g, m=m, a=np.exp(g),
                u=m * si * x, rate=rate)


def scan(a, u, cu, h0=None):
    """(h, h_T, h_{t-1}) of a packed batch; rows of no sequence are zeros."""
    a, u, h0 = _f64(a), _f64(u), _f64(h0)
    D = u.shape[1]
    h, before = np.zeros_like(u), np.zeros_like(u)
    h_T = np.zeros((len(cu) - 1, D))
    for n in range(len(cu) - 1):
        s = np.zeros(D) if h0 is None else h0[n].copy()
        for t in range(int(cu[n]), int(cu[n + 1])):
            before[t] = s
            s = a[t] * s + u[t]
            h[t] = s
        h_T[n] = s
    return h, h_T, before


def sweep(a, dh, cu, dh_T=None):
    """(L, dh0): L_t = dh_t + a_{t+1} L_{t+1}, dh0 = a_1 L_1 (dh_T of an empty sequence)."""
    a, dh, dh_T = _f64(a), _f64(dh), _f64(dh_T)
    D = dh.shape[1]
    L, dh0 = np.zeros_like(dh), np.zeros((len(cu) - 1, D))
    for n in range(len(cu) - 1):
        m = np.zeros(D) if dh_T is None else dh_T[n].copy()
        for t in reversed(range(int(cu[n]), int(cu[n + 1]))):
            L[t] = dh[t] + m
            m = a[t] * L[t]
        dh0[n] = m
    return L, dh0


def glr_plain(x, g, cu, h0=None):
    return scan(np.exp(_f64(g)), x, cu, h0)[:2]


def glr_plain_vjp(x, g, dh, cu, h0=None, dh_T=None):
    """(dx, dg, dh0)"""
    a = np.exp(_f64(g))
    before = scan(a, x, cu, h0)[2]
    L, dh0 = sweep(a, dh, cu, dh_T)
    return L, L * a * before, dh0


def glr_gated(x, r, i, rate, cu, h0=None):
    q = gates(x, r, i, rate)
    return scan(q["a"], q["u"], cu, h0)[:2]


def glr_gated_vjp(x, r, i, rate, dh, cu, h0=None, dh_T=None):
    """(dx, dr, di, drate, dh0); where a gate is closed (m = 0) the part
    through m, whose slope is infinite there, counts as 0."""
    q = gates(x, r, i, rate)
    before = scan(q["a"], q["u"], cu, h0)[2]
    L, dh0 = sweep(q["a"], dh, cu, dh_T)
    dm = np.divide(-q["a"] ** 2, q["m"], out=np.zeros_like(q["m"]), where=q["m"] > 0)
    dg = L * (q["a"] * before + q["si"] * q["x"] * dm)
    dr = -q["rate"] * dg * q["sr"] * q["rest_r"]
    di = L * q["m"] * q["x"] * q["si"] * q["rest_i"]
    return L * q["m"] * q["si"], dr, di, -(dg * q["sr"]).sum(0), dh0
