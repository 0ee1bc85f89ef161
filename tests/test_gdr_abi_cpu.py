"""CPU tests of the gated delta rule's C ABI: exports, and the refusal of bad
arguments before anything reaches the GPU (no compute call is made here)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from gated_delta_rule_95_amd import _lib

HEADER = os.path.join(os.path.dirname(_lib.HEADER), "gdr.h")
P = 0x1000000      # a fake, aligned address: every call below fails before any launch


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_exports_match_header(lib):
    with open(HEADER) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(gdr_[a-z0-9_]+)\s*\(", src)))
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = sorted({ln.split()[-1] for ln in out.splitlines()
                       if " T " in ln and ln.split()[-1].startswith("gdr_")})
    assert exported == declared
    for name in declared:
        assert getattr(lib, name).argtypes


def fwd(lib, **kw):
    a = dict(q=P, k=2 * P, v=3 * P, g=4 * P, beta=5 * P, S0=None, cu=None, n=1, N=16, Hk=1, Hv=2, dk=16,
             dv=16, dt=1, o=6 * P, ST=None)
    a.update(kw)
    return lib.gdr_fwd_chunked(a["q"], a["k"], a["v"], a["g"], a["beta"], a["S0"], a["cu"], a["n"], a["N"],
                               a["Hk"], a["Hv"], a["dk"], a["dv"], ctypes.c_float(1.0), a["dt"], a["o"],
                               a["ST"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(q=None), 1, "q is NULL"), (dict(g=None), 1, "g is NULL"), (dict(o=None), 1, "o is NULL"),
    (dict(dk=48), 2, "d_k"), (dict(dv=256), 2, "d_k"), (dict(Hk=0), 1, "H_k"), (dict(Hk=3, Hv=4), 1, "multiple"),
    (dict(Hv=0), 1, "multiple"), (dict(n=-1), 1, "n_seqs"), (dict(N=-1), 1, "n_tokens"),
    (dict(n=3), 1, "multiple"), (dict(n=0), 1, "n_seqs == 0"), (dict(dt=7), 1, "in_dtype"),
    (dict(q=P + 8), 1, "aligned"), (dict(S0=7 * P + 4), 1, "aligned"), (dict(cu=7 * P + 2), 1, "aligned"),
    (dict(o=3 * P), 1, "overlaps"), (dict(ST=3 * P), 1, "overlaps"), (dict(ST=6 * P + 64), 1, "overlaps"),
    (dict(N=1 << 31), 1, "2^31"), (dict(n=1 << 20, N=1 << 20), 1, "2^21"), (dict(Hv=1 << 16, dk=128), 1, "2^22"),
])
def test_fwd_refusals(lib, kw, status, msg):
    assert fwd(lib, **kw) == status
    assert msg in _lib.last_error()


def test_nothing_to_do_is_ok(lib):
    assert fwd(lib, n=0, N=0) == 0 and _lib.last_error() == ""
    assert dec(lib, N=0) == 0
    assert lib.gdr_save8(None, None, None, 0, 1, 1, 16, 16, *[None] * 7) == 0
    assert lib.gdr_load8(*[None] * 6, 0, 1, 1, 16, 16, *[None] * 4) == 0


def dec(lib, **kw):
    a = dict(q=P, k=2 * P, v=3 * P, g=4 * P, beta=5 * P, S=8 * P, slots=None, ns=2, N=2, Hk=1, Hv=2, dk=16,
             dv=16, dt=1, o=6 * P)
    a.update(kw)
    return lib.gdr_decode_step(a["q"], a["k"], a["v"], a["g"], a["beta"], a["S"], a["slots"], a["ns"], a["N"],
                               a["Hk"], a["Hv"], a["dk"], a["dv"], ctypes.c_float(1.0), a["dt"], a["o"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(S=None), 1, "S is NULL"), (dict(N=-1), 1, "N must"), (dict(ns=-1), 1, "n_slots"),
    (dict(ns=1), 1, "without slots"), (dict(dk=8), 2, "d_k"), (dict(S=P), 1, "overlaps"),
    (dict(S=8 * P + 8), 1, "aligned"), (dict(slots=7 * P + 1), 1, "aligned"), (dict(o=P), 1, "overlaps"),
    (dict(slots=8 * P), 1, "overlaps"), (dict(N=1 << 20, ns=1 << 20), 1, "2^21"),
])
def test_decode_refusals(lib, kw, status, msg):
    assert dec(lib, **kw) == status
    assert msg in _lib.last_error()


def bwd(lib, **kw):
    a = dict(q=P, k=2 * P, v=3 * P, g=4 * P, beta=5 * P, S0=None, cu=None, n=1, N=16, Hk=1, Hv=2, dk=16, dv=16,
             dt=1, dO=6 * P, dST=None, dq=7 * P, dk_=8 * P, dv_=9 * P, dg=10 * P, db=11 * P, dS0=12 * P,
             ws=64 * P, wsb=1 << 30)
    a.update(kw)
    return lib.gdr_bwd_chunked(a["q"], a["k"], a["v"], a["g"], a["beta"], a["S0"], a["cu"], a["n"], a["N"],
                               a["Hk"], a["Hv"], a["dk"], a["dv"], ctypes.c_float(1.0), a["dt"], a["dO"],
                               a["dST"], a["dq"], a["dk_"], a["dv_"], a["dg"], a["db"], a["dS0"], a["ws"],
                               a["wsb"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(ws=None), 1, "workspace is NULL"), (dict(wsb=64), 1, "below"), (dict(ws=64 * P + 16), 1, "aligned"),
    (dict(dO=None), 1, "dO is NULL"), (dict(dq=None), 1, "dq is NULL"), (dict(dk_=7 * P), 1, "overlaps"),
    (dict(dq=P), 1, "overlaps"), (dict(ws=4 * P), 1, "overlaps"), (dict(dg=10 * P + 2), 1, "aligned"),
    (dict(dS0=12 * P + 4), 1, "aligned"), (dict(Hk=2, Hv=3), 1, "multiple"), (dict(dt=2), 1, "in_dtype"),
    (dict(N=1 << 30, dk=64, dv=64), 1, "2^23"), (dict(n=1 << 20, N=1 << 20), 1, "2^21"),
])
def test_bwd_refusals(lib, kw, status, msg):
    assert bwd(lib, **kw) == status
    assert msg in _lib.last_error()


def test_saved8_refusals(lib):
    p = [P * (i + 1) for i in range(9)]
    save = lambda a, N=8, dk=32: lib.gdr_save8(a[0], a[1], a[2], N, 1, 1, dk, 32, *a[3:], None)   # noqa: E731
    for i in range(9):
        assert save(p[:i] + [None] + p[i + 1:]) == 1 and "NULL" in _lib.last_error()
    assert save(p, N=-1) == 1 and save(p, dk=24) == 2
    assert save(p[:3] + [P] + p[4:]) == 1 and "overlaps" in _lib.last_error()
    assert save([P + 2] + p[1:]) == 1 and "aligned" in _lib.last_error()
    rest = [4 * P, 5 * P, None, None, 1, 16, 1, 1, 32, 32, ctypes.c_float(1.0)] + [P * (20 + i) for i in range(9)]
    rest[12] = None
    q8 = [P * (40 + i) for i in range(6)]
    q8[1] = None
    assert lib.gdr_bwd_chunked_saved8(*q8, *rest, 1 << 30, None) == 1 and "qe is NULL" in _lib.last_error()


def test_workspace_sizes():
    import gated_delta_rule_95_amd as m
    a = m.gdr_bwd_workspace_bytes(1, 1000, 1, 2, 64, 64)
    assert a % 256 == 0 and 0 < a < m.gdr_bwd_workspace_bytes(1, 2000, 1, 2, 64, 64)
    for bad in ((0, 10, 1, 1, 64, 64), (1, -1, 1, 1, 64, 64), (1, 10, 2, 3, 64, 64), (1, 10, 1, 1, 60, 64)):
        assert m.gdr_bwd_workspace_bytes(*bad) == 0


def test_python_refuses_cpu_tensors_and_types():
    import gated_delta_rule_95_amd as m
    x = torch.zeros(4, 1, 16, dtype=torch.bfloat16)
    g = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="no CPU fallback"):
        m.gdr_fwd_chunked(x, x, x, g, g)
    with pytest.raises(ValueError, match="no CPU fallback"):
        m.gdr_save8(x, x, x)
    with pytest.raises(TypeError):
        m.gdr_load8((x, x, x))
    with pytest.raises(TypeError):
        m.gdr_bwd_workspace_bytes(1, 1, 1, 1, 16, 16, torch.float16)
