"""GPU tests of calls at the edges of the gated delta rule's contract: tokens
that no sequence has, cu_seqlens tables that break their contract, empty
batches, a pool without states."""
import ctypes

import pytest
import torch

from gated_delta_rule_95_amd import _lib
from tests.test_gpu_gdr import BF, F32, bwd, fwd, lib, make

pytestmark = pytest.mark.gpu
FORMS = [(BF, 128, 128), (BF, 64, 128), (F32, 64, 64), (BF, 32, 16)]
FILL = 7.0


def guarded(shape, dtype):
    """A tensor filled with FILL between 4 KiB of it on either side."""
    n, pad = 1, 4096
    for x in shape:
        n *= x
    whole = torch.full((n + 2 * pad,), FILL, dtype=dtype, device="cuda")
    return whole, whole[pad:pad + n].view(shape)


def untouched(whole, inner):
    n = inner.numel()
    return bool((whole[:4096] == FILL).all()) and bool((whole[4096 + n:] == FILL).all())


def backward(b, cu, n_seqs, kept=None):
    """The gradients through the C ABI, in guarded outputs."""
    N, Hk, dk = b["q"].shape
    Hv, dv = b["v"].shape[1:]
    dt = b["v"].dtype
    outs = [guarded(s, t) for s, t in ((b["q"].shape, dt), (b["k"].shape, dt), (b["v"].shape, dt), ((N, Hv), F32),
                                       ((N, Hv), F32), ((n_seqs, Hv, dk, dv), F32))]
    ws = torch.empty(lib().gdr_bwd_workspace_bytes(n_seqs, N, Hk, Hv, dk, dv, dt), dtype=torch.uint8, device="cuda")
    p = lambda x: x.data_ptr()                                                                     # noqa: E731
    sizes = [n_seqs, N, Hk, Hv, dk, dv, ctypes.c_float(b["scale"])]
    tail = [p(b["dO"]), p(b["dS_T"])] + [p(x) for _, x in outs] + [p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream]
    rest = [p(b["g"]), p(b["beta"]), p(b["S0"]), p(cu)]
    if kept is not None:
        st = _lib.load().gdr_bwd_chunked_saved8(*(p(x) for x in kept), *rest, *sizes, *tail)
    else:
        st = _lib.load().gdr_bwd_chunked(p(b["q"]), p(b["k"]), p(b["v"]), *rest, *sizes, 1 if dt == BF else 0, *tail)
    assert st == 0, _lib.last_error()
    torch.cuda.synchronize()
    assert all(untouched(w, x) for w, x in outs)
    return [x for _, x in outs]


def longer(b, rows):
    """The batch with `rows` tokens of NaN behind its last sequence."""
    c = dict(b)
    for x in ("q", "k", "v", "g", "beta", "dO"):
        c[x] = torch.cat([b[x], torch.full((rows,) + b[x].shape[1:], float("nan"), dtype=b[x].dtype, device="cuda")])
    return c


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_backward_leaves_rows_of_no_sequence(dtype, dk, dv):
    b = make(15, [50, 0, 30], 1, 2, dk, dv, dtype)
    want = bwd(b)
    for i, (x, y) in enumerate(zip(backward(longer(b, 70), b["cu"], 3), want)):
        n = 3 if i == 5 else 80
        assert torch.equal(x[:n], y) and bool((x[n:] == FILL).all())


def test_backward_from_8_bits_leaves_rows_of_no_sequence():
    m = lib()
    b = make(15, [50, 0, 30], 1, 2, 128, 64)
    want = m.gdr_bwd_chunked_saved8(m.gdr_save8(b["q"], b["k"], b["v"]), b["g"], b["beta"], b["dO"], S0=b["S0"],
                                    dS_T=b["dS_T"], cu_seqlens=b["cu"], scale=b["scale"])
    c = longer(b, 70)
    for i, (x, y) in enumerate(zip(backward(c, b["cu"], 3, m.gdr_save8(c["q"], c["k"], c["v"])), want)):
        n = 3 if i == 5 else 80
        assert torch.equal(x[:n], y) and bool((x[n:] == FILL).all())


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
@pytest.mark.parametrize("cu", [[0, 300, 200], [-7, 120, 2 ** 31 - 1], [200, 100, 0], [0, -2 ** 31, 64], [150, 150, 151]])
def test_broken_tables_touch_nothing_else(cu, dtype, dk, dv):
    """200 tokens; entries count as the nearest of 0 .. 200, a sequence that
    would end before it starts is empty (checked on the CPU by the model in
    tests/test_gdr_slots_cpu.py)."""
    b = make(16, [100, 100], 1, 2, dk, dv, dtype)
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    whole, o = guarded(b["v"].shape, b["v"].dtype)
    ws, S = guarded(b["S0"].shape, F32)
    lib().gdr_fwd_chunked(b["q"], b["k"], b["v"], b["g"], b["beta"], S0=b["S0"], cu_seqlens=table, o=o, S_T=S)
    torch.cuda.synchronize()
    assert untouched(whole, o) and untouched(ws, S)
    grads = backward(b, table, 2)
    edge = [min(max(x, 0), 200) for x in cu]
    lens = [max(e - s, 0) for s, e in zip(edge, edge[1:])]
    for n in range(2):
        if lens[n] == 0:
            assert torch.equal(S[n], b["S0"][n]) and torch.equal(grads[5][n], b["dS_T"][n])
    outside = [t for t in range(200) if not any(s <= t < s + x for s, x in zip(edge, lens))]
    for x in [o] + grads[:5]:
        assert bool((x[outside] == FILL).all())
    if all(e <= s or e <= edge[n + 1] for n, (s, e) in enumerate(zip(edge, edge[1:]))):
        assert torch.isfinite(S).all()


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_empty_batches(dtype, dk, dv):
    """No sequences, sequences of no tokens in either layout."""
    m = lib()
    e = lambda *s, t=dtype: torch.empty(s, dtype=t, device="cuda")                                 # noqa: E731
    S0 = torch.randn(2, 4, dk, dv, device="cuda")
    o, S = m.gdr_fwd_chunked(e(2, 0, 2, dk), e(2, 0, 2, dk), e(2, 0, 4, dv), e(2, 0, 4, t=F32), e(2, 0, 4, t=F32), S0=S0)
    assert o.shape == (2, 0, 4, dv) and torch.equal(S, S0)
    g = m.gdr_bwd_chunked(e(2, 0, 2, dk), e(2, 0, 2, dk), e(2, 0, 4, dv), e(2, 0, 4, t=F32), e(2, 0, 4, t=F32),
                          e(2, 0, 4, dv), dS_T=S0)
    assert [x.numel() for x in g[:5]] == [0] * 5 and torch.equal(g[5], S0)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = m.gdr_fwd_chunked(e(0, 2, dk), e(0, 2, dk), e(0, 4, dv), e(0, 4, t=F32), e(0, 4, t=F32), cu_seqlens=none)
    assert o.shape == (0, 4, dv) and S.shape == (0, 4, dk, dv)
    g = m.gdr_bwd_chunked(e(0, 2, dk), e(0, 2, dk), e(0, 4, dv), e(0, 4, t=F32), e(0, 4, t=F32), e(0, 4, dv),
                          cu_seqlens=none)
    assert [x.numel() for x in g] == [0] * 6


def test_decode_from_an_empty_pool():
    """Every row is a padded one."""
    b = make(17, [1] * 3, 2, 4, 64, 128)
    pool = torch.empty(0, 4, 64, 128, device="cuda")
    slots = torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda")
    o = lib().gdr_decode_step(b["q"], b["k"], b["v"], b["g"], b["beta"], pool, slots=slots)
    torch.cuda.synchronize()
    assert bool((o == 0).all())


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_slices_along_the_tokens(dtype, dk, dv):
    """Inputs that start in the middle of larger tensors."""
    b = make(18, [5, 90, 40], 1, 2, dk, dv, dtype)
    o, S = fwd(b)
    cut = {x: b[x][5:95] for x in ("q", "k", "v", "g", "beta")}
    o1, S1 = lib().gdr_fwd_chunked(*cut.values(), S0=b["S0"][1:2], scale=b["scale"])
    torch.cuda.synchronize()
    assert torch.equal(o1, o[5:95]) and torch.equal(S1[0], S[1])
