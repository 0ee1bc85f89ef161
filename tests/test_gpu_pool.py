"""GPU tests of the state pools (pool_*) against slots moved one after another
on the host, and of a run of them with the recurrences that use the pools."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def lib():
    import gated_delta_rule_95_amd as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def make(seed, n_slots, rows, share):
    """Pools of random bytes: rows is a list of (dtype, shape of a slot)."""
    r = np.random.default_rng(seed)
    pools = []
    for dtype, shape in rows:
        size = torch.empty(0, dtype=dtype).element_size()
        raw = r.integers(0, 256, (n_slots, int(np.prod(shape)) * size), dtype=np.uint8)
        pools.append(torch.from_numpy(raw).cuda().view(dtype).view((n_slots,) + shape))
    used = r.random(n_slots) < share
    return pools, torch.from_numpy(used).cuda(), used.copy(), r


def raw(pools):
    return [p.view(torch.uint8).cpu().numpy().reshape(p.shape[0], -1).copy() if p.numel() else
            np.zeros((p.shape[0], 0), np.uint8) for p in pools]


def same(pools, want):
    torch.cuda.synchronize()
    for p, w in zip(raw(pools), want):
        assert np.array_equal(p, w)


def forked(want, used, src):
    free, dst = [j for j, x in enumerate(used) if not x], []
    for a in src:
        dst.append(free.pop(0) if 0 <= a < len(used) and used[a] and free else -1)
    for a, b in zip(src, dst):
        if b >= 0:
            used[b] = True
            for p in want:
                p[b] = p[a]
    return dst


def compacted(want, used, table):
    live, remap, hole = int(used.sum()), [j if x else -1 for j, x in enumerate(used)], 0
    for j in range(live, len(used)):
        if used[j]:
            while used[hole]:
                hole += 1
            for p in want:
                p[hole] = p[j]
            used[hole], used[j], remap[j] = True, False, hole
    return remap, [remap[j] if 0 <= j < len(used) else j for j in table]


F32, BF, I8 = torch.float32, torch.bfloat16, torch.int8
ROWS = {"one": [(F32, (64,))], "odd": [(F32, (1001,)), (BF, (77,)), (I8, (3,))], "bytes": [(I8, (1,)), (I8, (17,))],
        "states": [(F32, (4, 128, 128)), (BF, (3, 512))], "many": [(F32, (k + 1,)) for k in range(70)]}


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("n_slots", [1, 2, 63, 1030])
def test_fork_free_compact_alloc_copy(n_slots, rows):
    m = lib()
    if n_slots > 100 and rows == "states":
        n_slots = 130
    for seed, share in enumerate((0.0, 0.3, 0.9, 1.0)):
        pools, used, u, r = make(seed, n_slots, ROWS[rows], share)
        want = raw(pools)
        n = int(r.integers(1, n_slots + 3))
        src = r.integers(-2, n_slots + 2, n)
        dst = m.pool_fork(pools, used, i32(src))
        assert dst.tolist() == forked(want, u, src.tolist()) and used.tolist() == u.tolist()
        same(pools, want)

        gone = r.integers(-3, n_slots + 3, int(r.integers(0, n_slots + 1)))
        m.pool_free(used, i32(gone))
        u[[j for j in gone if 0 <= j < n_slots]] = False
        assert used.tolist() == u.tolist()

        table = r.integers(-2, n_slots + 2, (3, 5))
        t = i32(table)
        remap = m.pool_compact(pools, used, t)
        want_map, want_table = compacted(want, u, table.reshape(-1).tolist())
        assert remap.tolist() == want_map and t.reshape(-1).tolist() == want_table and used.tolist() == u.tolist()
        same(pools, want)

        n = int(r.integers(0, 6))
        slots = m.pool_alloc(pools, used, n)
        free = [j for j, x in enumerate(u) if not x][:n]
        assert slots.tolist() == free + [-1] * (n - len(free))
        u[free] = True
        for p in want:
            p[free] = 0
        assert used.tolist() == u.tolist()
        same(pools, want)

        others, _, _, _ = make(seed + 10, n_slots + 5, ROWS[rows], 0)
        kept = raw(others)
        n = int(r.integers(0, n_slots + 1))
        src, dst = r.integers(-1, n_slots + 1, n), r.permutation(np.arange(-1, n_slots + 6))[:n]
        m.pool_copy(pools, i32(src), others, i32(dst))
        for a, b in zip(src, dst):
            if 0 <= a < n_slots and 0 <= b < n_slots + 5:
                for p, q in zip(want, kept):
                    q[b] = p[a]
        same(others, kept)
        same(pools, want)


@pytest.mark.parametrize("rows,n", [([(F32, (1024,))], 64), ([(F32, (1024,))], 65), ([(F32, (1025,)), (I8, (4096,))], 21),
                                    ([(F32, (1025,)), (I8, (4096,))], 22), ([(I8, (1,))] * 32, 2), ([(I8, (1,))] * 33, 1),
                                    ([(F32, (65536,))], 1), ([(F32, (65537,))], 1), ([(BF, (2056,)), (I8, (8193,))], 12)])
def test_sizes_at_which_the_copies_get_a_launch_of_their_own(rows, n):
    m = lib()
    pools, used, u, r = make(14, 150, rows, 0.4)
    want = raw(pools)
    src = r.choice(np.flatnonzero(u), n)
    src[::5] = -1
    assert m.pool_fork(pools, used, i32(src)).tolist() == forked(want, u, src.tolist())
    same(pools, want)
    m.pool_free(used, i32(np.flatnonzero(u)[:70]))
    u[np.flatnonzero(u)[:70]] = False
    free = np.flatnonzero(~u)[:n]
    assert m.pool_alloc(pools, used, n).tolist() == free.tolist()
    u[free] = True
    for p in want:
        p[free] = 0
    assert used.tolist() == u.tolist()
    same(pools, want)


def test_copy_inside_a_pool():
    m = lib()
    pools, _, _, _ = make(3, 20, ROWS["odd"], 0)
    want = raw(pools)
    m.pool_copy(pools, i32([3, 3, 5]), pools, i32([10, 0, 19]))
    for p in want:
        p[10], p[0], p[19] = p[3], p[3], p[5]
    same(pools, want)


@pytest.mark.parametrize("n_slots,n", [(5000, 4000), (70000, 3000), (1 << 20, 200000)])
def test_large_counts(n_slots, n):
    """More slots and rows than one workgroup counts at once."""
    m = lib()
    pools, used, u, r = make(4, n_slots, [(F32, (4,)), (I8, (3,))], 0.7)
    want = raw(pools)
    src = r.integers(-5, n_slots + 5, n)
    dst = m.pool_fork(pools, used, i32(src))
    valid = (src >= 0) & (src < n_slots)
    valid[valid] = u[src[valid]]
    free = np.flatnonzero(~u)
    k = np.cumsum(valid) - 1
    ok = valid & (k < len(free))
    to = np.where(ok, free[np.minimum(k, len(free) - 1)], -1)
    for p in want:
        p[to[ok]] = p[src[ok]]
    u[to[ok]] = True
    assert np.array_equal(dst.cpu().numpy(), to) and np.array_equal(used.cpu().numpy(), u)
    same(pools, want)
    gone = r.permutation(n_slots)[:n_slots // 3]
    m.pool_free(used, i32(gone))
    u[gone] = False
    table = r.integers(-1, n_slots + 1, 30000)
    t = i32(table)
    remap = m.pool_compact(pools, used, t).cpu().numpy()
    live = int(u.sum())
    movers, holes = np.flatnonzero(u[live:]) + live, np.flatnonzero(~u[:live])
    want_map = np.where(u, np.arange(n_slots), -1)
    want_map[movers] = holes
    for p in want:
        p[holes] = p[movers]
    inside = (table >= 0) & (table < n_slots)
    assert np.array_equal(remap, want_map)
    assert np.array_equal(t.cpu().numpy(), np.where(inside, want_map[np.clip(table, 0, n_slots - 1)], table))
    assert np.array_equal(used.cpu().numpy(), np.arange(n_slots) < live)
    same(pools, want)


def test_destinations_named_twice_touch_nothing_else():
    """Such a slot may hold either row's bytes or some of both."""
    m = lib()
    pools, _, _, _ = make(11, 30, ROWS["odd"], 0)
    want = raw(pools)
    m.pool_copy(pools, i32([1, 2, 3, 4]), pools, i32([20, 20, 21, 21]))
    torch.cuda.synchronize()
    for p, w in zip(raw(pools), want):
        for at, a, b in ((20, 1, 2), (21, 3, 4)):
            assert ((p[at] == w[a]) | (p[at] == w[b])).all()
        rest = np.delete(np.arange(30), [20, 21])
        assert np.array_equal(p[rest], w[rest])


def test_two_streams_with_their_own_pools():
    m = lib()
    runs = [make(seed, 300, ROWS["odd"], 0.5) for seed in (12, 13)]
    streams = [torch.cuda.Stream() for _ in runs]
    wants, ws = [raw(p) for p, *_ in runs], [torch.empty(m.pool_compact_workspace_bytes(300), dtype=torch.uint8, device="cuda")
                                             for _ in runs]
    torch.cuda.synchronize()
    for k in range(6):
        srcs = [i32(np.flatnonzero(u)[k:k + 9]) for _, _, u, _ in runs]
        torch.cuda.synchronize()
        got = []
        for (pools, used, _, _), src, side, w in zip(runs, srcs, streams, ws):
            with torch.cuda.stream(side):
                dst = m.pool_fork(pools, used, src)
                m.pool_free(used, src)
                got.append((dst, m.pool_compact(pools, used, workspace=w)))
        torch.cuda.synchronize()
        for (pools, used, u, _), want, src, (dst, remap) in zip(runs, wants, srcs, got):
            assert dst.tolist() == forked(want, u, src.tolist())
            u[src.tolist()] = False
            assert remap.tolist() == compacted(want, u, [])[0] and used.tolist() == u.tolist()
            same(pools, want)


def test_nothing_to_do():
    m = lib()
    pools, used, u, _ = make(5, 9, ROWS["one"], 0.5)
    want = raw(pools)
    none = i32([])
    assert m.pool_fork(pools, used, none).shape == (0,) and m.pool_alloc(pools, used, 0).shape == (0,)
    m.pool_free(used, none)
    m.pool_copy(pools, none, pools, none)
    m.pool_copy([], i32([1]), [], i32([2]))
    empty, no_slots = torch.empty(0, 64, device="cuda"), torch.empty(0, dtype=torch.bool, device="cuda")
    assert m.pool_fork(empty, no_slots, i32([0, 1])).tolist() == [-1, -1]
    assert m.pool_alloc(empty, no_slots, 2).tolist() == [-1, -1]
    assert m.pool_compact(empty, no_slots).shape == (0,)
    m.pool_free(no_slots, i32([0, 5]))
    m.pool_copy(empty, i32([0]), pools, i32([1]))
    # no pools: slot numbers alone
    assert m.pool_fork([], used, i32([int(np.flatnonzero(u)[0])])).tolist() == [int(np.flatnonzero(~u)[0])]
    same(pools, want)


def test_guarded_rows():
    """Bytes around the pools stay, rows whose size and address no vector divides."""
    m = lib()
    for row, off in ((1, 1), (15, 3), (16, 16), (20, 4), (4097, 1), (65552, 16), (100004, 8)):
        whole = torch.full((64 + 40 * row,), 9, dtype=torch.uint8, device="cuda")
        pool = whole[off:off + 20 * row].view(20, row)
        pool.copy_(torch.randint(0, 255, (20, row), dtype=torch.uint8, device="cuda"))
        want = pool.cpu().clone()
        used = torch.zeros(20, dtype=torch.bool, device="cuda")
        used[:3] = True
        assert m.pool_fork(pool, used, i32([2, 0])).tolist() == [3, 4]
        want[3], want[4] = want[2], want[0]
        assert m.pool_alloc(pool, used, 1).tolist() == [5]
        want[5] = 0
        m.pool_free(used, i32([0, 2]))
        assert m.pool_compact(pool, used).tolist()[:6] == [-1, 1, -1, 3, 0, 2]
        want[0], want[2] = want[4].clone(), want[5].clone()
        torch.cuda.synchronize()
        assert torch.equal(pool.cpu(), want)
        assert bool((whole[:off] == 9).all()) and bool((whole[off + 20 * row:] == 9).all())


def test_offsets_past_2_to_the_32():
    m = lib()
    pool = torch.zeros(70000, 20000, dtype=F32, device="cuda")           # 5.6 GB
    pool[69999] = torch.arange(20000, device="cuda")
    used = torch.zeros(70000, dtype=torch.bool, device="cuda")
    used[69999] = True
    used[:60000] = True
    assert m.pool_fork(pool, used, i32([69999])).tolist() == [60000]
    torch.cuda.synchronize()
    assert torch.equal(pool[60000], pool[69999]) and not pool[60001].any()
    m.pool_free(used, i32(np.arange(60000)))
    m.pool_compact(pool, used)
    torch.cuda.synchronize()
    assert torch.equal(pool[0], pool[69999]) and torch.equal(pool[1], pool[69999]) and not pool[2].any()


def test_captured_and_replayed():
    """A fork, a step's worth of work, a free and a compaction in one graph."""
    m = lib()
    pools, used, u, r = make(6, 40, ROWS["odd"], 0.5)
    src, table = i32(np.flatnonzero(u)[:4]), i32(np.arange(-1, 41))
    m.pool_compact([p.clone() for p in pools], used.clone(), table.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dst = m.pool_fork(pools, used, src)
        m.pool_free(used, src)
        remap = m.pool_compact(pools, used, table)
    for seed in range(7, 11):
        fresh, fu, u, r = make(seed, 40, ROWS["odd"], 0.5)
        for p, q in zip(pools, fresh):
            p.copy_(q)
        used.copy_(fu)
        picked = r.permutation(np.flatnonzero(u))[:4]
        src.copy_(i32(picked))
        table.copy_(i32(np.arange(-1, 41)))
        graph.replay()
        torch.cuda.synchronize()
        want = raw(fresh)
        assert dst.tolist() == forked(want, u, picked.tolist())
        u[picked] = False
        want_map, want_table = compacted(want, u, list(range(-1, 41)))
        assert remap.tolist() == want_map and table.tolist() == want_table and used.tolist() == u.tolist()
        same(pools, want)
        m.pool_fork([p.clone() for p in pools], used.clone(), src)           # eager work between the replays


def test_a_server_with_both_recurrences():
    """Prompts through the scans, states into the pools, forks, steps, frees and
    a compaction, as a server queues them, against each request computed alone
    from its whole history."""
    m = lib()
    dev, Hk, Hv, d, D, n_slots = "cuda", 2, 4, 64, 200, 12
    gen = torch.Generator(device=dev).manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)                                    # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)                                      # noqa: E731

    def tokens(n):
        return dict(q=unit(rnd(n, Hk, d)).bfloat16(), k=unit(rnd(n, Hk, d)).bfloat16(), v=rnd(n, Hv, d).bfloat16(),
                    g=-0.1 * rnd(n, Hv).abs(), beta=rnd(n, Hv).sigmoid(), x=rnd(n, D).bfloat16(),
                    r=rnd(n, D).bfloat16(), i=rnd(n, D).bfloat16())

    rate = 0.2 * torch.rand(D, generator=gen, device=dev)
    S, H = torch.full((n_slots, Hv, d, d), 5.0, device=dev), torch.full((n_slots, D), 5.0, device=dev)
    used = torch.zeros(n_slots, dtype=torch.bool, device=dev)
    hist = {}                                                              # request -> its tokens so far

    def scan(t, cu=None):
        o, S_T = m.gdr_fwd_chunked(t["q"], t["k"], t["v"], t["g"], t["beta"], cu_seqlens=cu)
        h, h_T = m.glr_fwd_scan_gated(t["x"], t["r"], t["i"], rate, cu_seqlens=cu)
        return o, h, S_T, h_T

    lens = [70, 1, 130, 33, 64]
    batch = tokens(sum(lens))
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    _, _, S_T, h_T = scan(batch, cu)
    slots = m.pool_alloc([S, H], used, 5)
    m.pool_copy([S_T, h_T], i32(np.arange(5)), [S, H], slots)
    for a, (s, e) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        hist[a] = {k: v[s:e] for k, v in batch.items()}
    table = slots.clone()
    names = [0, 1, 2, 3, 4]

    def step():
        t = tokens(len(names))
        o = m.gdr_decode_step(t["q"], t["k"], t["v"], t["g"], t["beta"], S, slots=table)
        h = m.glr_decode_step_gated(t["x"], t["r"], t["i"], rate, H, slots=table)
        for j, a in enumerate(names):
            hist[a] = {k: torch.cat((hist[a][k], v[j:j + 1])) for k, v in t.items()}
        return o, h

    def agree(o, h):
        torch.cuda.synchronize()
        for j, a in enumerate(names):
            o1, h1, S1, h1_T = scan(hist[a])
            at = int(table[j])
            close = lambda x, y, tol: float((x.double() - y.double()).norm() / y.double().norm()) <= tol    # noqa: E731
            # the bf16 outputs' own rounding, 2^-8 of each element at most on either side; fp32 states 1e-5
            assert close(o[j], o1[-1], 2 * 2.0 ** -8) and close(h[j], h1[-1], 2 * 2.0 ** -8)
            assert close(S[at], S1[0], 1e-5) and close(H[at], h1_T[0], 1e-5)

    step()
    # requests 1 and 3 get two and one more candidates
    kids = m.pool_fork([S, H], used, table[[1, 1, 3]].contiguous())
    table = torch.cat((table, kids))
    names += [5, 6, 7]
    hist[5], hist[6], hist[7] = hist[1], hist[1], hist[3]
    agree(*step())
    # 0, 2 and 6 end
    m.pool_free(used, table[[0, 2, 6]].contiguous())
    keep = [1, 3, 4, 5, 7]
    table, names = table[keep].contiguous(), keep
    m.pool_compact([S, H], used, table)
    assert sorted(table.tolist()) == [0, 1, 2, 3, 4] and used.tolist() == [True] * 5 + [False] * 7
    agree(*step())
    # request 4's state is kept in other pools and brought back for a new request
    kept = [torch.zeros(2, Hv, d, d, device=dev), torch.zeros(2, D, device=dev)]
    m.pool_copy([S, H], table[2:3].contiguous(), kept, i32([1]))
    m.pool_free(used, table[2:3].contiguous())
    new = m.pool_alloc([S, H], used, 1)
    m.pool_copy(kept, i32([1]), [S, H], new)
    hist[8] = hist[4]
    table, names = torch.cat((table[[0, 1, 3, 4]], new)), [1, 3, 5, 7, 8]
    agree(*step())
