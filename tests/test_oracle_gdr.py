"""CPU pins of the gated delta rule's fp64 oracle: against the pinned KDA
recurrence (equal decays in all channels), closed forms, central differences
for every gradient, and torch's own e4m3 conversion for the 8-bit form."""
import numpy as np
import pytest
import torch

from oracle.gdr import gdr_recurrent, gdr_recurrent_vjp, kept8, packed
from oracle.recurrence import kda_recurrent


def batch(seed, T, Hk, Hv, dk, dv):
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)      # noqa: E731
    return dict(q=unit(r.standard_normal((T, Hk, dk))), k=unit(r.standard_normal((T, Hk, dk))),
                v=r.standard_normal((T, Hv, dv)), g=-np.exp(r.standard_normal((T, Hv))),
                beta=1 / (1 + np.exp(-r.standard_normal((T, Hv)))),
                S0=r.standard_normal((Hv, dk, dv)))


def test_equals_kda_with_equal_channel_decays():
    b = batch(0, 20, 2, 4, 6, 5)
    rep = lambda x: np.repeat(x, 2, 1)                                  # noqa: E731
    g = np.broadcast_to(b["g"][:, :, None], (20, 4, 6))
    o, S = gdr_recurrent(b["q"], b["k"], b["v"], b["g"], b["beta"], 0.3, b["S0"])
    o2, S2 = kda_recurrent(rep(b["q"]), rep(b["k"]), b["v"], g, b["beta"], b["S0"])[:2]
    assert np.allclose(o, 0.3 * o2, rtol=1e-12, atol=1e-13)
    assert np.allclose(S, S2, rtol=1e-12, atol=1e-13)


def test_full_forgetting_and_pure_decay():
    b = batch(1, 7, 1, 2, 4, 3)
    g = b["g"].copy()
    g[4] = -np.inf
    o, S = gdr_recurrent(b["q"], b["k"], b["v"], g, b["beta"], 1.0, b["S0"])
    o2, S2 = gdr_recurrent(b["q"][4:], b["k"][4:], b["v"][4:], b["g"][4:], b["beta"][4:], 1.0)
    assert np.allclose(o[4:], o2) and np.allclose(S, S2)
    _, S = gdr_recurrent(b["q"], b["k"], b["v"], b["g"], 0 * b["beta"], 1.0, b["S0"])
    assert np.allclose(S, np.exp(b["g"].sum(0))[:, None, None] * b["S0"])


@pytest.mark.parametrize("seed", [3, 4])
def test_vjp_against_differences(seed):
    b = batch(seed, 5, 2, 4, 3, 4)
    r = np.random.default_rng(seed + 100)
    dO, dS = r.standard_normal(b["v"].shape), r.standard_normal(b["S0"].shape)
    scale = 0.7

    def loss(**kw):
        x = {**b, **kw}
        o, S = gdr_recurrent(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["S0"])
        return (o * dO).sum() + (S * dS).sum()

    grads = gdr_recurrent_vjp(b["q"], b["k"], b["v"], b["g"], b["beta"], dO, scale, b["S0"], dS)
    h = 1e-5
    for name, gr in zip(("q", "k", "v", "g", "beta", "S0"), grads):
        num = np.zeros_like(b[name])
        for i in np.ndindex(num.shape):
            up, dn = b[name].copy(), b[name].copy()
            up[i] += h
            dn[i] -= h
            num[i] = (loss(**{name: up}) - loss(**{name: dn})) / (2 * h)
        assert np.allclose(gr, num, rtol=1e-6, atol=1e-8), name


def test_packed_sequences_are_independent():
    b = batch(5, 9, 1, 2, 4, 4)
    cu = [0, 4, 4, 9]
    S0 = np.stack([b["S0"], 2 * b["S0"], -b["S0"]])
    o, S = packed(gdr_recurrent_one, cu, [b[x] for x in ("q", "k", "v", "g", "beta")], (S0,), 1.0)
    assert np.allclose(S[1], S0[1])
    o2, S2 = gdr_recurrent(b["q"][4:], b["k"][4:], b["v"][4:], b["g"][4:], b["beta"][4:], 1.0, -b["S0"])
    assert np.allclose(o[4:], o2) and np.allclose(S[2], S2)


def gdr_recurrent_one(q, k, v, g, beta, scale, S0):
    return gdr_recurrent(q, k, v, g, beta, scale, S0)


def test_kept8_is_e4m3_of_the_scaled_block():
    r = np.random.default_rng(7)
    x = (r.standard_normal((40, 64)) * 2.0 ** r.integers(-40, 40, (40, 1))).astype(np.float32)
    x[3, 5:9] = 448.0 * 2.0 ** np.array([0, 1, -1, -30])
    x[4, :32] = 0
    x[5, 0], x[5, 1] = np.inf, np.nan
    y = kept8(x)
    assert np.isnan(y[5, :2]).all() and np.isfinite(np.delete(y.ravel(), [5 * 64, 5 * 64 + 1])).all()
    for i, j in np.ndindex(40, 2):
        blk = x[i, 32 * j:32 * j + 32]
        fin = np.isfinite(blk)
        top = np.abs(blk[fin]).max()
        if top == 0:
            assert (y[i, 32 * j:32 * j + 32] == 0).all()
            continue
        e = next(n for n in range(-110, 120) if top <= 448.0 * 2.0 ** n)
        t = torch.from_numpy(np.where(fin, blk, 0).astype(np.float64) / 2.0 ** e).float()
        want = t.to(torch.float8_e4m3fn).double().numpy() * 2.0 ** e
        assert np.array_equal(want[fin], y[i, 32 * j:32 * j + 32][fin])
    # what is kept is a bf16 value
    z = torch.from_numpy(y[np.isfinite(y)])
    assert torch.equal(z.to(torch.bfloat16).double(), z)
