"""GPU tests of how far a NaN or an infinity goes in the gated delta rule: to
any output of its own sequence and heads, and to none of another's."""
import pytest
import torch

from tests.test_gpu_gdr import BF, F32, bwd, fwd, lib, make

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
SEQS, AT = [100, 80, 3], 30                      # the value stands in token 30 of the first sequence
KEY = ("q", "k")                                 # inputs with a key head; the others have a value head


def put(b, name, x):
    """x in one place of token 30 (of state 0), head 1: key head 1, whose value
    heads are 2 and 3, or value head 1, whose key head is 0."""
    t = b[name]
    if name in ("S0", "dS_T"):
        t[0, 1, 3, 5] = x
    elif t.dim() == 2:
        t[AT, 1] = x
    else:
        t[AT, 1, 3] = x


def heads(name):
    """(value heads, key heads) the place above may reach."""
    return ([2, 3], [1]) if name in KEY else ([1], [0])


def same(x, y, n_heads, reached, tokens):
    """Bits are equal in the heads not reached, and in the other sequences."""
    keep = [h for h in range(n_heads) if h not in reached]
    rest = slice(SEQS[0], None) if tokens else slice(1, None)
    return torch.equal(x[:, keep], y[:, keep]) and torch.equal(x[rest], y[rest])


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 128), (F32, 64, 64), (BF, 32, 16)])
@pytest.mark.parametrize("name,x", [(n, x) for n in ("q", "k", "v", "beta", "dO", "S0", "dS_T") for x in (NAN, INF, -INF)]
                         + [("g", NAN), ("g", INF)])
def test_stays_in_its_sequence_and_heads(name, x, dtype, dk, dv):
    b = make(14, SEQS, 2, 4, dk, dv, dtype)
    clean, clean_b = fwd(b), bwd(b)
    put(b, name, x)
    hv, hk = heads(name)
    o, S = fwd(b)
    assert same(o, clean[0], 4, hv, True) and same(S, clean[1], 4, hv, False)
    if name in ("dO", "dS_T"):
        assert torch.equal(o, clean[0]) and torch.equal(S, clean[1])
    elif name != "q":
        assert not torch.isfinite(S[0, hv]).all()
    for out, y, z in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), bwd(b), clean_b):
        n, reached = (2, hk) if out in ("dq", "dk") else (4, hv)
        assert same(y, z, n, reached, out != "dS0"), out


@pytest.mark.parametrize("x", [NAN, INF])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_kept_in_8_bits(name, x):
    """Both become NaN in their own place, and spread as there."""
    b = make(14, SEQS, 2, 4, 128, 64)
    m = lib()
    args = lambda: (m.gdr_save8(b["q"], b["k"], b["v"]), b["g"], b["beta"], b["dO"])      # noqa: E731
    kw = dict(S0=b["S0"], dS_T=b["dS_T"], cu_seqlens=b["cu"])
    clean = m.gdr_bwd_chunked_saved8(*args(), **kw)
    put(b, name, x)
    got = m.gdr_bwd_chunked_saved8(*args(), **kw)
    loaded = dict(zip("qkv", m.gdr_load8(args()[0])))[name]
    torch.cuda.synchronize()
    assert torch.isnan(loaded[AT, 1, 3]) and int(torch.isnan(loaded).sum()) == 1
    hv, hk = heads(name)
    for out, y, z in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, clean):
        n, reached = (2, hk) if out in ("dq", "dk") else (4, hv)
        assert same(y, z, n, reached, out != "dS0"), out


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (F32, 64, 64), (F32, 16, 32)])
@pytest.mark.parametrize("name,x", [("k", NAN), ("v", INF), ("g", NAN), ("beta", INF), ("S", NAN), ("S", INF)])
def test_decode_stays_in_its_request(name, x, dtype, dk, dv):
    b = make(15, [1] * 6, 2, 4, dk, dv, dtype)
    pool = torch.randn(8, 4, dk, dv, device="cuda")
    slots = torch.tensor([7, 2, 5, 0, 1, 6], dtype=torch.int32, device="cuda")
    run = lambda S: lib().gdr_decode_step(b["q"], b["k"], b["v"], b["g"], b["beta"], S, slots=slots)     # noqa: E731
    S0 = pool.clone()
    o0 = run(S0)
    S1 = pool.clone()
    if name == "S":
        S1[5, 1, 3, 5] = x
    else:
        b[name][(2, 1) if b[name].dim() == 2 else (2, 1, 3)] = x
    o1 = run(S1)
    torch.cuda.synchronize()
    hv = heads(name)[0]
    keep, rows, others = [h for h in range(4) if h not in hv], [0, 1, 3, 4, 5], [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(o0[:, keep], o1[:, keep]) and torch.equal(o0[rows], o1[rows])
    assert torch.equal(S0[:, keep], S1[:, keep]) and torch.equal(S0[others], S1[others])
    assert not torch.isfinite(o1[2, hv]).all()
