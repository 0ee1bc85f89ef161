"""What keeping q, k, v in 8 bits costs the gradients, by the fp64 oracle: the
figures that the header and the README give, and the bytes beside them.

An e4m3 rounding is off by at most 2^-4 of the value and by 2^-4 / sqrt 3 in
the rms at most (2.7% where mantissas are spread evenly).  dq, dk and dv each
see the three inputs' roundings about once (sqrt 3 of them), dg and dbeta, as
products of two such, at most sqrt 5."""
import numpy as np
import pytest

import gated_delta_rule_95_amd as m
from oracle.gdr import gdr_recurrent_vjp, kept8
from tests.test_oracle_gdr_chunked import batch

ROUNDING = 2.0 ** -4 / np.sqrt(3)


def rel(x, y):
    return np.linalg.norm(x - y) / np.linalg.norm(y)


@pytest.mark.parametrize("seed,T,d,gates", [(0, 300, 128, "usual"), (1, 300, 64, "slow"), (2, 200, 128, "slow"),
                                            (3, 100, 16, "usual")])
def test_gradients_move_by_some_percent(seed, T, d, gates):
    b = batch(seed, T, 1, 2, d, d, gates, s0=False)
    args = lambda f: (f(b["q"]), f(b["k"]), f(b["v"]), b["g"], b["beta"], b["dO"], b["scale"])      # noqa: E731
    for x in "qkv":
        assert 0.02 < rel(kept8(b[x]), b[x]) < ROUNDING
    at, ref = gdr_recurrent_vjp(*args(kept8)), gdr_recurrent_vjp(*args(lambda x: x))
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), at, ref):
        print(f"  {name} {rel(x, y):.3f}")
        assert 0.03 < rel(x, y) < ROUNDING * np.sqrt(5 if name in ("dg", "dbeta") else 3), name


def test_bytes_saved_and_the_backwards_workspace():
    """16384 tokens, 32 heads on 16 of 128 x 128: 8 bits save 0.13 GB of what
    is kept between the passes; the backward's workspace is 1.6 GB."""
    N, Hk, Hv, d = 16384, 16, 32, 128
    elements = N * (2 * Hk + Hv) * d
    assert 0.129e9 < 2 * elements - elements * (1 + 1 / 32) < 0.131e9
    assert 1.60e9 < m.gdr_bwd_workspace_bytes(1, N, Hk, Hv, d, d) < 1.62e9
