"""CPU model of how the gated delta rule's kernels turn cu_seqlens into rows
and workspace slots (seq_edge, seq_of and find_chunk in csrc/gdr_device.h),
for tables that keep their contract and for tables that do not: every row and
slot stays inside what the host sized, and of a valid table every chunk has a
slot of its own, found again from its number."""
import random

import pytest


def edge(cu, n, tokens):
    return min(max(cu[n], 0), tokens)


def seq(cu, n, tokens):
    b, e = edge(cu, n, tokens), edge(cu, n + 1, tokens)
    return b, max(e - b, 0)


def find(cu, slot, C, tokens):
    lo, hi = 0, len(cu) - 2
    while lo < hi:
        mid = (lo + hi + 1) // 2
        if edge(cu, mid, tokens) // C + mid <= slot:
            lo = mid
        else:
            hi = mid - 1
    c = slot - (edge(cu, lo, tokens) // C + lo)
    return (lo, c) if c >= 0 and c * C < seq(cu, lo, tokens)[1] else None


def table(r, valid):
    n = r.randrange(1, 9)
    if valid:
        lens = [r.choice((0, 1, 63, 64, 65, r.randrange(300))) for _ in range(n)]
        cu = [sum(lens[:i]) for i in range(n + 1)]
        return cu, cu[-1]
    tokens = r.randrange(1, 500)
    return [r.choice((r.randrange(-50, 600), r.randrange(0, tokens + 1), -2 ** 31, 2 ** 31 - 1)) for _ in range(n + 1)], tokens


@pytest.mark.parametrize("C", [32, 64])
@pytest.mark.parametrize("valid", [True, False])
def test_rows_and_slots_stay_inside(valid, C):
    r = random.Random(C + valid)
    for _ in range(2000):
        cu, tokens = table(r, valid)
        n_seqs = len(cu) - 1
        slots = tokens // C + n_seqs + 1
        seen = set()
        for n in range(n_seqs):
            bos, length = seq(cu, n, tokens)
            assert 0 <= bos and bos + length <= tokens
            for c in range(-(-length // C)):
                slot = bos // C + n + c
                assert 0 <= slot < slots
                if valid:
                    assert slot not in seen and find(cu, slot, C, tokens) == (n, c)
                    seen.add(slot)
        for slot in range(slots):
            f = find(cu, slot, C, tokens)
            if f is not None:
                bos, length = seq(cu, f[0], tokens)
                assert 0 <= bos + f[1] * C and bos + min((f[1] + 1) * C, length) <= tokens
                assert not valid or slot in seen
