"""GPU tests of the gated delta rule's decay factors: states that live from
them alone, and states that hardly decay and add up their errors.  Tolerances:
tests/_gdr_bars.py."""
import numpy as np
import pytest
import torch

from tests._gdr_bars import check, compare
from tests.test_gpu_gdr import BF, F32, host, lib, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d,dscale", [(300, 64, 1.0), (700, 128, 1.0), (1500, 128, 1.0), (300, 64, 2.0 ** -10)])
def test_slow_decays_in_one_chain(T, d, dscale, dtype):
    """States that forget only what the delta rule rewrites."""
    b = make(T + d, [T], 1, 1, d, d, dtype, gates="slow")
    b["dO"] *= dscale
    compare(b, dtype)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 128), (F32, 64, 64), (BF, 32, 16)])
@pytest.mark.parametrize("decays", [[-0.3], [-5.0], [-43.7], [-79.9], [-20.1, -0.7, -30.3]])
def test_states_that_only_decay(decays, dtype, dk, dv):
    """beta 0: S_T and dS0 are e^g of what they start from, and dg a product
    with it, to 24 bits however fast the decay is (an exponent held in one
    float would be off by |g| 2^-24)."""
    T = len(decays)
    b = make(24, [T, T], 1, 2, dk, dv, dtype)
    b["g"][:] = torch.tensor(decays * 2, device="cuda")[:, None]
    b["beta"][:] = 0
    b["dO"].zero_()
    tol = compare(b, dtype)
    if T == 1:
        pool, h = b["S0"].clone(), host(b)
        lib().gdr_decode_step(b["q"], b["k"], b["v"], b["g"], b["beta"], pool)
        torch.cuda.synchronize()
        check("S_T", pool, np.exp(h["g"])[:, :, None, None] * h["S0"], tol)
