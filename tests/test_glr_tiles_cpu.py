"""CPU models of what the gated linear recurrence's kernels and the pools' plans
do with tables and orders: how a tile finds the sequence borders inside it
(mark_borders in csrc/glr_tiles.h), how the state that comes into a tile is
looked up from the words of the tiles before it (look_back), and how free
slots replace each other in one array (pool_take_kernel in csrc/pool.hip)."""
import random

import numpy as np
import pytest

WAVE = 64


def edge(cu, n, tokens):
    return min(max(cu[n], 0), tokens)


def ends_behind(cu, tokens, lo, t, reads):
    n_seqs = len(cu) - 1
    hi, rounds = n_seqs, 0
    while lo < hi:
        step = -(-(hi - lo) // WAVE)
        ended = 0
        for lane in range(WAVE):
            n = lo + lane * step
            at = (n if n < hi else lo) + 1
            assert 0 <= at <= n_seqs
            ended += n < hi and edge(cu, at, tokens) <= t
        nxt = lo + ended * step
        if ended:
            lo += (ended - 1) * step + 1
        hi = min(nxt, hi)
        rounds += 1
        assert rounds < 8 and 0 <= lo <= n_seqs
    reads.append(rounds)
    return lo


def borders(cu, tokens, t0, C, reads=None):
    """mark_borders, lane by lane; asserts that every index it forms is inside
    the table and the tile.  reads gets the rounds of loads that follow each
    other."""
    n_seqs = len(cu) - 1
    first, last, reads = {}, {}, [] if reads is None else reads
    base = ends_behind(cu, tokens, 0, t0, reads)
    while base < n_seqs:
        reads.append(1)
        stop = False
        for n in range(base, base + WAVE):
            b = e = t0 + C
            if n < n_seqs:
                b, e = edge(cu, n, tokens), edge(cu, n + 1, tokens)
                if e > b:
                    if t0 <= b < t0 + C:
                        first[b - t0] = n
                    if t0 <= e - 1 < t0 + C:
                        last[e - 1 - t0] = n
            stop |= b - t0 >= C
        if stop:
            break
        base += WAVE
        if e == b:
            lo, base = base, ends_behind(cu, tokens, base, e, reads)
            assert base >= lo
    return first, last


def table(r, valid):
    n = r.choice((1, 2, 5, 63, 64, 65, 300, 5000))
    if valid:
        lens = [r.choice((0, 0, 0, 1, 31, 32, 33, 127, 128, 129, r.randrange(300))) if n < 400 else r.choice((0, 0, 1, 2)) for _ in range(n)]
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        return cu, cu[-1] + r.choice((0, 0, 200))
    tokens = r.randrange(1, 500)
    return [r.choice((r.randrange(-50, 600), r.randrange(0, tokens + 1), -2 ** 31, 2 ** 31 - 1)) for _ in range(n + 1)], tokens


@pytest.mark.parametrize("C", [32, 64, 128])
@pytest.mark.parametrize("valid", [True, False])
def test_borders_of_any_table(valid, C):
    r = random.Random(C + valid)
    for _ in range(120):
        cu, tokens = table(r, valid)
        want_first, want_last = {}, {}
        for n in range(len(cu) - 1):
            if cu[n + 1] > cu[n]:
                want_first[cu[n]], want_last[cu[n + 1] - 1] = n, n
        total = edge(cu, len(cu) - 1, tokens)
        tiles = range(0, total, C)
        for t0 in tiles if len(tiles) < 40 else r.sample(list(tiles), 40):
            first, last = borders(cu, tokens, t0, C)
            assert all(0 <= k < C for k in (*first, *last))
            if valid:
                assert first == {t - t0: n for t, n in want_first.items() if t0 <= t < t0 + C}
                assert last == {t - t0: n for t, n in want_last.items() if t0 <= t < t0 + C}


@pytest.mark.parametrize("C", [32, 128])
def test_empty_sequences_cost_no_walk(C):
    """Runs of empty sequences inside a tile and behind the last token, far more
    than a wave looks at one after another."""
    run = 70000
    for cu in ([0] * run + [5] + [40] * run + [200] * run, [0, 7] + [7 + C] * run, [0] * run + [1], [0, 10, 10, 11] + [64] * run):
        tokens = cu[-1]
        for t0 in range(0, tokens, C):
            reads = []
            first, last = borders(cu, tokens, t0, C, reads)
            starts = {a - t0: n for n, (a, b) in enumerate(zip(cu, cu[1:])) if b > a and t0 <= a < t0 + C}
            ends = {b - 1 - t0: n for n, (a, b) in enumerate(zip(cu, cu[1:])) if b > a and t0 < b <= t0 + C}
            assert first == starts and last == ends
            # a search (3 rounds here) and one look for each token at which sequences end, and the first
            assert sum(reads) <= 4 * (len(ends) + 2)


def test_look_back_does_not_depend_on_progress():
    """Words of tiles in any state of progress (a map, or what the tile stores in
    the end) give the same float32 state, and a wait ends once the tiles before
    have stored theirs."""
    r = np.random.default_rng(0)
    f = np.float32

    def fma(a, b, c):
        return f(np.float64(a) * np.float64(b) + np.float64(c))

    for trial in range(300):
        n, W = int(r.integers(1, 40)), int(r.choice([4, 8]))
        maps = [(f(r.uniform(0, 1)), f(r.standard_normal())) for _ in range(n)]
        for k in [0] + list(np.flatnonzero(r.random(n) < 0.1)):
            maps[k] = (None, maps[k][1])                       # forgets
        prefix = []
        for a, b in maps:
            prefix.append(b if a is None else fma(a, prefix[-1], b))
        want = prefix[-1]
        done = int(r.integers(0, n))                           # tiles that have come to their end
        stored = int(r.integers(done, n + 1))                  # tiles that have stored a map
        waits = 0
        while True:
            word = [(None, prefix[k]) if k < done else maps[k] if k < stored else None for k in range(n)]
            near = [word[max(n - 1 - i, 0)] for i in range(W)]
            found = None
            for i, m in enumerate(near):
                if m is None:
                    break
                if m[0] is None:
                    found = i
                    break
            if found is not None:
                break
            stored, done, waits = min(stored + 1, n), min(done + 1, n), waits + 1
            assert waits <= n + 1
        h = near[found][1]
        for i in range(found - 1, -1, -1):
            a, b = near[i]
            h = b if a is None else fma(a, h, b)
        assert h == want


@pytest.mark.parametrize("PT", [4, 64])
def test_slots_replace_each_other_in_place(PT):
    """pool_take_kernel with PT threads a step: the list of free slots and the
    rows' answers share one array."""
    r = random.Random(PT)
    for _ in range(2000):
        n_slots, n = r.randrange(0, 40), r.randrange(1, 40)
        used = [r.random() < r.choice((0.2, 0.8)) for _ in range(n_slots)]
        valid = [r.random() < r.choice((0.3, 1.0)) for _ in range(n)]
        dst, nfree, base = [None] * n, 0, 0
        while base < n_slots and nfree < n:
            step = [j for j in range(base, min(base + PT, n_slots)) if not used[j]]
            for k, j in enumerate(step, nfree):
                if k < n:
                    dst[k] = j
            nfree += len(step)
            base += PT
        before = sum(valid)
        for base in range((n - 1) // PT * PT, -1, -PT):
            rows = range(base, min(base + PT, n))
            before -= sum(valid[i] for i in rows)
            got, k = [], before
            for i in rows:
                got.append(dst[k] if valid[i] and k < nfree else -1)
                k += valid[i]
            for i, x in zip(rows, got):
                dst[i] = x
        free = [j for j in range(n_slots) if not used[j]]
        want = [free.pop(0) if v and free else -1 for v in valid]
        assert dst == want
