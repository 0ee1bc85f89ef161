"""GPU tests of the gated delta rule (gdr_*) at the precision its kernels keep:
seeded random configurations, and the batches where errors grow or last
longest (nearly repeated keys, long sequences, many chunks in every form of
the chunk kernel).  The tolerances are those of
tests/_gdr_bars.py, which tests/test_oracle_gdr_chunked.py shows to reject
operands held in one part less."""
import random

import numpy as np
import pytest
import torch

from oracle.gdr import gdr_recurrent, kept8
from tests._gdr_bars import GRADS, check, compare, reference
from tests.test_gpu_gdr import BF, F32, fwd, host, lib, make

pytestmark = pytest.mark.gpu


def draw(seed):
    """(lengths, H_k, H_v, d_k, d_v, dtype, states, gates), some 3e7 kept state
    elements at most (what the oracle holds)."""
    r = random.Random(seed)
    dk, dv = r.choice((16, 32, 64, 64, 128, 128)), r.choice((16, 32, 64, 64, 128, 128))
    Hk, grp = r.choice((1, 1, 2, 3)), r.choice((1, 1, 2, 3))
    most = min(1200, 30_000_000 // (Hk * grp * dk * dv))
    n = r.choice((1, 1, 2, 3, 5))
    lens = [0 if r.random() < 0.1 else max(1, int(most / n * 2 ** r.uniform(-5, 0))) for _ in range(n)]
    lens[r.randrange(n)] = max(1, int(most / n * 2 ** r.uniform(-3, 0)))
    return (lens, Hk, Hk * grp, dk, dv, r.choice((BF, BF, F32)), r.random() < 0.6,
            r.choice(("usual", "usual", "slow", "fast")))


@pytest.mark.parametrize("seed", range(32))
def test_random_configurations(seed):
    lens, Hk, Hv, dk, dv, dtype, s0, gates = draw(seed)
    print(f"  seed {seed}: {draw(seed)}", flush=True)
    b = make(1000 + seed, lens, Hk, Hv, dk, dv, dtype, s0, gates)
    compare(b, dtype)


@pytest.mark.parametrize("seed", range(100, 108))
def test_random_backward_from_8_bits(seed):
    """Against the oracle's gradients at the values that 8 bits keep."""
    lens, Hk, Hv, dk, dv, _, s0, gates = draw(seed)
    print(f"  seed {seed}: {draw(seed)}", flush=True)
    b = make(1000 + seed, lens, Hk, Hv, dk, dv, BF, s0, gates)
    kept = lib().gdr_save8(b["q"], b["k"], b["v"])
    got = lib().gdr_bwd_chunked_saved8(kept, b["g"], b["beta"], b["dO"], S0=b["S0"], dS_T=b["dS_T"], cu_seqlens=b["cu"])
    torch.cuda.synchronize()
    h = host(b)
    for x in ("q", "k", "v"):
        h[x] = kept8(h[x])
    _, ref, tol = reference(h, b["cu"].tolist(), b["scale"], BF)
    for name, x, y in zip(GRADS, got, ref):
        check(name, x, y, tol)


@pytest.mark.parametrize("seed", range(200, 208))
def test_random_decode(seed):
    """One step: a column sum of d_k products in fp32 and two operations on
    top, each within 2^-24 of numbers no larger than |S'^T k| + |v|."""
    _, Hk, Hv, dk, dv, dtype, _, _ = draw(seed)
    N = random.Random(seed).choice((1, 3, 17, 64))
    b = make(1000 + seed, [1] * N, Hk, Hv, dk, dv, dtype)
    pool = torch.randn(N + 2, Hv, dk, dv, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    slots = torch.randperm(N + 2, generator=torch.Generator().manual_seed(seed))[:N].to(torch.int32)
    h, want_o, want = host(b), np.zeros((N, Hv, dv)), pool.double().cpu().numpy()
    for i, s in enumerate(slots.tolist()):
        o1, want[s] = gdr_recurrent(*(h[x][i:i + 1] for x in ("q", "k", "v", "g", "beta")), b["scale"], want[s])
        want_o[i] = o1[0]
    o = lib().gdr_decode_step(b["q"], b["k"], b["v"], b["g"], b["beta"], pool, slots=slots.cuda())
    torch.cuda.synchronize()
    tol = 2 * np.sqrt(dk) * 2.0 ** -24
    check("o", o, want_o, {"o": tol})
    check("S", pool, want, {"S": tol})


@pytest.mark.parametrize("noise", [0.1, 0.3])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nearly_repeated_keys(dtype, noise):
    """A common direction in all keys and beta 0.9: long chains in the
    triangular system, dg from larger terms."""
    b = make(8, [200, 65], 1, 2, 128, 128, dtype, s0=False, gates="slow")
    k = b["k"].float()
    base = k[:1] / k[:1].norm(dim=-1, keepdim=True)
    k = base + noise * k
    b["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dtype)
    b["beta"][:] = 0.9
    compare(b, dtype)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 128), (F32, 64, 64), (BF, 32, 64)])
@pytest.mark.parametrize("gates", ["usual", "slow"])
def test_long_forward(dtype, dk, dv, gates):
    """Some hundred chunks one after another."""
    compare(make(21, [6001, 4100], 1, 1, dk, dv, dtype, gates=gates), dtype, grads=False)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 128, 64), (F32, 64, 64)])
def test_long_backward(dtype, dk, dv):
    compare(make(22, [2600, 300], 1, 1, dk, dv, dtype, gates="slow"), dtype)


@pytest.mark.parametrize("dk", [128, 64])
@pytest.mark.parametrize("gates", ["usual", "slow"])
def test_many_chunks_in_many_chains(dk, gates):
    """144 chains of unequal lengths, up to seven chunks: the forward's wide
    form through its steady state.  Each sequence alone (16 chains, the narrow
    form) gives the same bits."""
    lens = [400, 1, 333, 64, 129, 0, 321, 65, 200]
    b = make(23, lens, 8, 16, dk, 128, BF, gates=gates)
    (o, S), cu = fwd(b), b["cu"].tolist()
    ref, _, tol = reference(host(b), cu, b["scale"], BF, grads=False)
    check("o", o, ref[0], tol)
    check("S_T", S, ref[1], tol)
    for n, (s, e) in enumerate(zip(cu, cu[1:])):
        if e > s:
            one = [b[x][s:e].contiguous() for x in ("q", "k", "v", "g", "beta")]
            o1, S1 = lib().gdr_fwd_chunked(*one, S0=b["S0"][n:n + 1].contiguous(), scale=b["scale"])
            assert torch.equal(o1, o[s:e]) and torch.equal(S1[0], S[n]), n
