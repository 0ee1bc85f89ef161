"""GPU tests of decays at the ends of the range: the least and largest factors
that fp32 holds, factors of 0, and growth that overflows."""
import numpy as np
import pytest
import torch

from tests.test_gpu_gdr import BF, F32, lib

pytestmark = pytest.mark.gpu
# e^g from the last normal float on: below 2^-126 a factor may count as 0
FACTORS = [0.0, -0.0, -1e-30, -1e-7, -87.0, -104.0, -1e4, -1.0001e4, -3e38, -np.inf, 1e-7, 0.5, 88.0]


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 64), (F32, 64, 64), (BF, 16, 32), (F32, 128, 16)])
def test_one_token_of_pure_decay(dtype, dk, dv):
    """beta 0, one token a sequence: S_T = e^g S0 in the forward, and in the
    decode step; a factor is off by one step at most."""
    n = len(FACTORS)
    z = lambda *s, t=dtype: torch.zeros(s, dtype=t, device="cuda")                        # noqa: E731
    g = torch.tensor(FACTORS, device="cuda").view(n, 1)
    S0 = torch.randn(n, 1, dk, dv, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    k = torch.full((n, 1, dk), 0.125, dtype=dtype, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    _, S = lib().gdr_fwd_chunked(k, k, z(n, 1, dv), g, z(n, 1, t=F32), S0=S0, cu_seqlens=cu)
    pool = S0.clone()
    lib().gdr_decode_step(k, k, z(n, 1, dv), g, z(n, 1, t=F32), pool)
    torch.cuda.synchronize()
    want = S0.double().cpu().numpy() * np.exp(g.double().cpu().numpy())[:, :, None, None]
    # e^88 is 1.65e38: what it makes of a state above 2.06 is past fp32's
    # 3.40e38 (no element lies within a step of the border)
    top = float(np.finfo(np.float32).max)
    assert (np.abs(np.abs(want) / top - 1) > 1e-6).all()
    past = np.abs(want) > top
    assert past.any() and not past[:-1].any()
    # Only growth that does not overflow is promised (g > 0).  A column with an
    # infinity in it, or in its S'^T k, may be NaN: beta times the latter is 0
    # times an infinity by the formula, and so is the former times the rows of
    # zeros that fill a tile behind the sequence.
    may = np.broadcast_to((0.125 * np.abs(want).sum(2, keepdims=True) > top) | past.any(2, keepdims=True), want.shape)
    assert not may[:-1].any()
    allowed = 1.5 * 2.0 ** -23 * np.abs(want) + 2.0 ** -126 * np.abs(S0.double().cpu().numpy())
    for got in (S, pool):
        x = got.double().cpu().numpy()
        right = np.where(past, x == np.sign(want) * np.inf, np.abs(x - np.where(past, 0, want)) <= allowed)
        assert (right | (may & np.isnan(x))).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("g", [1e5, 3e38])
def test_overflow_is_not_hidden(g, dtype, d):
    """e^g past the range: nothing finite comes back from the state."""
    t = lambda *s, v=0.0, t=dtype: torch.full(s, v, dtype=t, device="cuda")               # noqa: E731
    S0 = torch.ones(1, 1, d, d, device="cuda")
    args = [t(1, 1, d, v=0.125), t(1, 1, d, v=0.125), t(1, 1, d), t(1, 1, v=g, t=F32), t(1, 1, t=F32)]
    _, S = lib().gdr_fwd_chunked(*args, S0=S0)
    lib().gdr_decode_step(*args, S0)
    torch.cuda.synchronize()
    assert not torch.isfinite(S).any() and not torch.isfinite(S0).any()
