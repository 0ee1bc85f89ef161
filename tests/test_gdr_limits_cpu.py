"""CPU tests of the gated delta rule's host limits: a call whose launch would
not fit one grid is refused as an argument error, with its message, and not
by the launch itself (no compute call is made here)."""
import ctypes

import pytest

from gated_delta_rule_95_amd import _lib

P = 1 << 44        # fake addresses, far enough apart for the sizes below


def bwd(n, Hk, Hv, dk, dv, dtype=1):
    """gdr_bwd_chunked of n sequences of one token (8-bit inputs: dtype None)."""
    lib = _lib.load()
    p = [P * (i + 1) for i in range(24)]
    sizes = (n, n, Hk, Hv, dk, dv, ctypes.c_float(1.0))
    rest = [p[5], None] + p[6:13] + [1 << 43, None]
    if dtype is None:
        return lib.gdr_bwd_chunked_saved8(*p[14:20], p[3], p[4], None, None, *sizes, *rest)
    return lib.gdr_bwd_chunked(*p[:5], None, None, *sizes, dtype, *rest)


@pytest.mark.parametrize("n,Hk,Hv,dk,dv,dtype", [
    (2 ** 21 - 1, 1, 1, 128, 128, 1), (2 ** 21 - 7, 1, 1, 64, 128, 1), (2 ** 21 - 1, 1, 1, 128, 128, None),
    (2 ** 20 - 1, 1, 2, 64, 128, 1)])
def test_backward_grids_count_whole_rounds_of_eight(n, Hk, Hv, dk, dv, dtype):
    """The workgroups of a key head go to the XCDs in rounds of eight, so the
    launch is as large as the rounded count."""
    assert bwd(n, Hk, Hv, dk, dv, dtype) == 1
    assert "2^21" in _lib.last_error() and "8" in _lib.last_error()
