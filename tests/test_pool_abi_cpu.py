"""CPU tests of the state pools' C ABI: the refusal of bad arguments before
anything reaches the GPU (no compute call is made here)."""
import ctypes

import pytest

from gated_delta_rule_95_amd import _lib

P = 0x1000000      # a fake, aligned address: every call below fails before any launch


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def rows(*pairs):
    words = [w or 0 for p in pairs for w in p]
    return (ctypes.c_size_t * max(len(words), 1))(*words)


def call(lib, fn, **kw):
    a = dict(pools=((20 * P, 64), (30 * P, 20)), n_pools=2, used=P, ns=100, src=2 * P, n=3, dst=3 * P, to=((40 * P, 64), (50 * P, 20)),
             ts=50, table=4 * P, nt=7, remap=5 * P, ws=6 * P, wsb=1 << 20)
    a.update(kw)
    pools, to = (None if a[k] is None else rows(*a[k]) for k in ("pools", "to"))
    if fn == "copy":
        return lib.pool_copy(pools, to, a["n_pools"], a["ns"], a["ts"], a["src"], a["dst"], a["n"], None)
    if fn == "alloc":
        return lib.pool_alloc(pools, a["n_pools"], a["used"], a["ns"], a["n"], a["dst"], None)
    if fn == "fork":
        return lib.pool_fork(pools, a["n_pools"], a["used"], a["ns"], a["src"], a["n"], a["dst"], None)
    if fn == "free":
        return lib.pool_free(a["used"], a["ns"], a["src"], a["n"], None)
    return lib.pool_compact(pools, a["n_pools"], a["used"], a["ns"], a["table"], a["nt"], a["remap"], a["ws"], a["wsb"], None)


ALL = ("copy", "alloc", "fork", "free", "compact")
POOLS = ("copy", "alloc", "fork", "compact")


@pytest.mark.parametrize("fns,kw,msg", [
    (POOLS, dict(n_pools=-1), "n_pools"), (POOLS, dict(pools=None), "is NULL"),
    (POOLS, dict(pools=((20 * P, 0), (30 * P, 20))), "row_bytes"), (POOLS, dict(pools=((None, 64), (30 * P, 20))), "is NULL"),
    (POOLS, dict(pools=((20 * P, 64), (30 * P, (1 << 40) + 1))), "row_bytes"),
    (POOLS, dict(pools=((20 * P, 64), (30 * P, 1 << 40)), ns=64), "2^46"),
    (ALL, dict(ns=-1), "must be >= 0"), (ALL, dict(ns=(1 << 24) + 1), "2^24"),
    (("copy", "alloc", "fork", "free"), dict(n=-1), "n must be >= 0"),
    (("copy", "alloc", "fork", "free"), dict(n=(1 << 24) + 1), "2^24"),
    (("alloc", "fork", "free", "compact"), dict(used=None), "used is NULL"),
    (("copy", "fork"), dict(src=None), "src is NULL"), (("free",), dict(src=None), "slots is NULL"),
    (("copy", "fork"), dict(dst=None), "dst is NULL"), (("alloc",), dict(dst=None), "slots is NULL"),
    (("copy", "fork"), dict(src=2 * P + 2), "aligned"), (("copy", "alloc", "fork"), dict(dst=3 * P + 1), "aligned"),
    (("fork",), dict(src=3 * P + 4), "overlaps"), (("alloc", "fork"), dict(dst=P + 4), "overlaps"),
    (("free",), dict(src=P + 4), "overlaps"),
    (("alloc", "fork", "compact"), dict(pools=((20 * P, 64), (20 * P + 6336, 20))), "pools[1] overlaps pools[0]"),
    (("alloc", "fork", "compact"), dict(used=30 * P + 1999), "pools[1] overlaps used"),
    (("fork",), dict(src=20 * P), "pools[0] overlaps src"),
    (("copy",), dict(dst=40 * P), "to[0] overlaps dst"), (("copy",), dict(to=((40 * P, 64), (40 * P + 3196, 20))), "to[1] overlaps to[0]"),
    (("copy",), dict(to=((40 * P, 64), (50 * P, 24))), "different sizes"),
    (("copy",), dict(to=((20 * P + 64, 64), (50 * P, 20))), "without being the same pool"),
    (("copy",), dict(to=((30 * P, 64), (50 * P, 20))), "without being the same pool"), (("copy",), dict(ts=-1), "to_slots"),
    (("compact",), dict(table=None), "table is NULL"), (("compact",), dict(remap=None), "remap is NULL"),
    (("compact",), dict(nt=-1), "n_table"), (("compact",), dict(nt=1 << 30), "2^24"), (("compact",), dict(ws=None), "workspace is NULL"),
    (("compact",), dict(wsb=100), "below"), (("compact",), dict(ws=6 * P + 4), "aligned"),
    (("compact",), dict(table=5 * P), "overlaps"), (("compact",), dict(remap=P + 96), "overlaps"),
])
def test_refusals(lib, fns, kw, msg):
    for fn in fns:
        assert call(lib, fn, **kw) == 1, fn
        assert msg in _lib.last_error(), (fn, _lib.last_error())


def test_pools_whose_bytes_are_zero_in_64_bits(lib):
    """2^40 bytes a slot and 2^24 slots, and sizes on both sides of 2^46 bytes."""
    for fn in POOLS:
        for row, ns in ((1 << 40, 1 << 24), (1 << 40, 64), ((1 << 22) + 1, 1 << 24), (1 << 22, 1 << 24)):
            assert call(lib, fn, pools=((20 * P, 64), (30 * P, row)), ns=ns, ts=ns) == 1, fn
            assert "pools[1] must be below 2^46" in _lib.last_error() or "from[1] must be below 2^46" in _lib.last_error()
    # the largest that fits is refused for something else only
    assert call(lib, "alloc", pools=((1 << 50, 1), (1 << 51, (1 << 22) - 1)), ns=1 << 24, used=None) == 1
    assert _lib.last_error() == "used is NULL"


def test_nothing_to_do_is_ok(lib):
    for fn in ("copy", "alloc", "fork", "free"):
        assert call(lib, fn, n=0) == 0 and _lib.last_error() == ""
    assert call(lib, "compact", ns=0, pools=((20 * P, 64), (30 * P, 20))) == 0
    assert call(lib, "copy", n_pools=0, pools=None, to=None) == 0


def test_workspace_sizes():
    import gated_delta_rule_95_amd as m
    a = m.pool_compact_workspace_bytes(1000)
    assert a % 256 == 0 and 4000 <= a < m.pool_compact_workspace_bytes(5000)
    assert m.pool_compact_workspace_bytes(-1) == 0 and m.pool_compact_workspace_bytes((1 << 24) + 1) == 0


def test_python_refusals():
    import gated_delta_rule_95_amd as m
    import torch
    with pytest.raises(ValueError, match="no CPU fallback"):
        m.pool_compact([torch.zeros(3, 4)], torch.zeros(3, dtype=torch.bool))
    with pytest.raises(TypeError):
        m.pool_fork([torch.zeros(3, 4)], [True, False, True], torch.zeros(1, dtype=torch.int32))
