"""GPU tests of the gated linear recurrence (glr_*) through the Python entry
points against the fp64 oracle (oracle/glr.py), at the element-by-element
error bounds of tests/_glr_bars.py."""
import numpy as np
import pytest
import torch

from tests import _glr_bars as bars

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FILL = 7.0


def lib():
    import gated_delta_rule_95_amd as m
    return m


def make(seed, lens, D, dtype=BF, gated=True, states=True, decays="usual", behind=0):
    """A packed batch on the device; `behind` rows of no sequence at its end."""
    r = np.random.default_rng(seed)
    N, n = int(sum(lens)) + behind, len(lens)
    put = lambda x, t=F32: torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(t)     # noqa: E731
    b = dict(x=put(r.standard_normal((N, D)), dtype), dh=put(r.standard_normal((N, D)), dtype))
    if gated:
        b["r"], b["i"] = (put(3 * r.standard_normal((N, D)), dtype) for _ in range(2))
        fast = 8 * np.log1p(np.exp(r.standard_normal(D)))
        slow = -np.log(r.uniform(0.9, 0.999, D))
        b["rate"] = put({"usual": np.where(np.arange(D) % 3 == 0, fast, slow), "slow": 1e-3 * slow,
                         "fast": 40 * fast}[decays])
    else:
        z = r.standard_normal((N, D)) + 2
        b["g"] = put({"usual": -np.log1p(np.exp(-z)), "slow": -1e-5 * np.exp(z), "fast": -30 * np.exp(z)}[decays])
    b["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    b["h0"] = put(r.standard_normal((n, D))) if states else None
    b["dh_T"] = put(r.standard_normal((n, D))) if states else None
    b["gated"] = gated
    return b


def ins(b):
    return tuple(b[k] for k in (("x", "r", "i", "rate") if b["gated"] else ("x", "g")))


def fwd(b, **kw):
    f = lib().glr_fwd_scan_gated if b["gated"] else lib().glr_fwd_scan
    return f(*ins(b), h0=b["h0"], **{"cu_seqlens": b["cu"], **kw})


def bwd(b, **kw):
    f = lib().glr_bwd_scan_gated if b["gated"] else lib().glr_bwd_scan
    return f(*ins(b), b["dh"], h0=b["h0"], dh_T=b["dh_T"], **{"cu_seqlens": b["cu"], **kw})


def names(b):
    return ("dx", "dr", "di", "drate", "dh0") if b["gated"] else ("dx", "dg", "dh0")


def host(b):
    return {k: v.detach().double().cpu().numpy() for k, v in b.items() if isinstance(v, torch.Tensor)}


def compare(b, grads=True, kept=True):
    cu = b["cu"].tolist()
    want = bars.reference(host(b), cu, b["gated"], grads)
    rows = slice(0, cu[-1])
    h, h_T, left = fwd(b, keep=True)
    torch.cuda.synchronize()
    bars.check("h", h, want["h"], rows)
    bars.check("h_T", h_T, want["h_T"])
    if grads:
        for name, x in zip(names(b), bwd(b, kept=left if kept else None)):
            bars.check(name, x, want[name], rows if name in ("dx", "dg", "dr", "di") else slice(None))
    return h, h_T, left


LENS = {"one token": [1], "short": [77], "a tile": [128], "past a tile": [129], "ragged": [1, 0, 63, 64, 65, 0, 2, 300, 128],
        "empty ends": [0, 0, 200, 0], "long": [2500], "many": [3, 1, 2, 0] * 150}


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [1, 64, 77, 258])
@pytest.mark.parametrize("lens", LENS)
def test_forward_and_gradients(lens, D, dtype, gated):
    compare(make(1, LENS[lens], D, dtype, gated))


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_runs_of_empty_sequences(gated):
    """More of them at one token, and behind the last, than a wave looks at one
    after another."""
    run = [0] * 9000
    compare(make(24, run + [5] + run + [35, 0, 160] + run, 3, F32, gated))


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("decays", ["slow", "fast"])
@pytest.mark.parametrize("states", [True, False])
def test_decays_and_states(states, decays, gated):
    for dtype in (F32, BF):
        compare(make(2, [40, 700, 0, 333], 130, dtype, gated, states, decays))


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = np.random.default_rng(900 + seed)
    lens = [int(np.exp(r.uniform(0, 6.5))) - 1 for _ in range(int(r.integers(1, 30)))]
    D = int(np.exp(r.uniform(0, 6)))
    b = make(seed, lens, D, (BF, F32)[seed % 2], bool(seed // 2 % 2), bool(r.integers(2)), behind=int(r.integers(0, 300)))
    compare(b, kept=bool(r.integers(2)))


WIDE = [(BF, True, 8192), (BF, False, 8192), (F32, False, 8190), (F32, True, 8192), (BF, True, 8191)]


@pytest.mark.parametrize("dtype,gated,D", WIDE)
def test_wide_batches(dtype, gated, D):
    """Calls large enough for the forms with pairs of channels: borders of every
    kind inside, on and around the tiles' own, empty sequences, rows behind."""
    lens = [1, 0, 31, 32, 33, 500, 127, 128, 129, 0, 2, 700, 64, 0, 300, 5, 40]
    b = make(24, lens, D, dtype, gated, behind=70)
    compare(b, kept=False)
    compare({**b, "h0": None, "dh_T": None})


@pytest.mark.parametrize("dtype,gated,D", [(BF, True, 512), (BF, False, 256), (F32, False, 256)])
def test_long_batches(dtype, gated, D):
    """The same forms, many tiles of few channels in a chain."""
    compare(make(25, [33000, 1, 200], D, dtype, gated, decays="slow"))


@pytest.mark.parametrize("dtype,gated,D", WIDE[:3])
def test_wide_nonfinite_values_and_rows_of_no_sequence(dtype, gated, D):
    """As the small tests below, in the forms with pairs of channels."""
    lens = [70, 1500, 0, 300, 5, 140]
    N = sum(lens)
    b = make(26, lens, D, dtype, gated, behind=200)
    for k in ("x", "dh") + (("r", "i") if gated else ("g",)):
        b[k][N:] = float("nan")
    good_h, good = [torch.full_like(b["x"], FILL), None], bwd(b)
    _, good_hT = fwd(b, h=good_h[0])
    torch.cuda.synchronize()
    assert bool((good_h[0][N:] == FILL).all())
    for k in ("x", "dh") + (("r", "i") if gated else ("g",)):
        for bad in (float("nan"), float("inf")):
            c = dict(b, **{k: b[k].clone()})
            c[k][700, 3] = bad
            h, h_T = fwd(c, h=torch.full_like(b["x"], FILL))
            grads = bwd(c)
            torch.cuda.synchronize()
            keep = torch.ones(N, D, dtype=torch.bool, device="cuda")
            keep[70:1570, 3] = False
            n = torch.ones(len(lens), D, dtype=torch.bool, device="cuda")
            n[1, 3] = False
            if k != "dh":
                assert torch.equal(h[:N][keep], good_h[0][:N][keep]) and torch.equal(h_T[n], good_hT[n])
                if bad != bad:
                    assert bool(torch.isnan(h[700:1570, 3]).all())
            for x, y, name in zip(grads, good, names(b)):
                x, y = (x[:N], y[:N]) if x.shape[0] == N + 200 else (x, y)
                m = keep if x.shape == keep.shape else n if x.shape == n.shape else n[1]
                assert torch.equal(x[m], y[m]), (k, name)
    # gradients of outputs that are guarded: nothing behind the last sequence is written
    _, _, kept = fwd(b, keep=True)
    for x in call_bwd(b, len(lens), b["cu"], kept):
        if x.shape[0] == N + 200:
            assert bool((x[N:] == FILL).all())


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_kept_states_are_optional(gated):
    b = make(3, [100, 0, 301, 64], 66, F32, gated)
    _, _, kept = fwd(b, keep=True)
    assert kept.shape == (15, 66)
    for x, y in zip(bwd(b, kept=kept), bwd(b)):
        torch.cuda.synchronize()
        assert torch.allclose(x, y, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_layouts_agree(gated):
    """[B, T, D] with and without its table, [1, N, D], a part of the outputs."""
    b = make(4, [150] * 4, 96, BF, gated)
    h, h_T = fwd(b)
    four = {k: v.view(4, 150, 96) if isinstance(v, torch.Tensor) and v.shape == (600, 96) else v for k, v in b.items()}
    h4, h4_T = fwd(four, cu_seqlens=None)
    assert torch.equal(h4.view(600, 96), h) and torch.equal(h4_T, h_T)
    one = {k: v.view(1, 600, 96) if isinstance(v, torch.Tensor) and v.shape == (600, 96) else v for k, v in b.items()}
    h1, none = fwd(one, output_final_state=False)
    assert torch.equal(h1.view(600, 96), h) and none is None
    for x, y, z in zip(bwd(b), bwd(four, cu_seqlens=None), bwd(one)):
        assert torch.equal(x, y.view(x.shape)) and torch.equal(x, z.view(x.shape))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_slices_of_odd_rows(dtype):
    """Rows of 77 elements: a slice along the tokens starts anywhere."""
    b = make(5, [5, 91, 40], 77, dtype)
    h, h_T = fwd(b)
    grads = bwd(b)
    c = dict(b, **{k: b[k][5:96] for k in ("x", "r", "i", "dh")}, h0=b["h0"][1:2], dh_T=b["dh_T"][1:2],
             cu=torch.tensor([0, 91], dtype=torch.int32, device="cuda"))
    h1, h1_T = fwd(c)
    want = bars.reference(host(c), [0, 91], True)
    bars.check("h", h1, want["h"])
    bars.check("h_T", h1_T, want["h_T"])
    for name, x in zip(names(b), bwd(c)):
        bars.check(name, x, want[name])
    assert torch.allclose(h1_T[0], h_T[1], rtol=1e-5, atol=1e-6)
    assert torch.allclose(grads[0][5:96].float(), bwd(c)[0].float(), rtol=1e-2, atol=1e-3)


def guarded(shape, dtype):
    n, pad = int(np.prod(shape)), 4096
    whole = torch.full((n + 2 * pad,), FILL, dtype=dtype, device="cuda")
    return whole, whole[pad:pad + n].view(shape)


def untouched(whole, inner):
    return bool((whole[:4096] == FILL).all()) and bool((whole[4096 + inner.numel():] == FILL).all())


def call_bwd(b, n_seqs, cu, kept):
    """The gradients through the C ABI in guarded outputs."""
    from gated_delta_rule_95_amd import _lib
    N, D = b["x"].shape
    dt, L = b["x"].dtype, _lib.load()
    shapes = ([((N, D), dt)] * 3 + [((D,), F32)] if b["gated"] else [((N, D), dt), ((N, D), F32)]) + [((n_seqs, D), F32)]
    outs = [guarded(*s) for s in shapes]
    ws = torch.empty(max(L.glr_bwd_workspace_bytes(N, D), 256), dtype=torch.uint8, device="cuda")
    p = lambda x: None if x is None else x.data_ptr()                                              # noqa: E731
    f = L.glr_bwd_scan_gated if b["gated"] else L.glr_bwd_scan
    st = f(*(p(x) for x in ins(b)), p(b["h0"]), p(cu), n_seqs, N, D, 1 if dt == BF else 0, p(kept), p(b["dh"]), p(b["dh_T"]),
           *(p(x) for _, x in outs), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0, _lib.last_error()
    torch.cuda.synchronize()
    assert all(untouched(w, x) for w, x in outs)
    return [x for _, x in outs]


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("D", [64, 77])
def test_rows_of_no_sequence_are_left(D, gated):
    b = make(6, [50, 0, 130], D, BF, gated, behind=300)
    for k in ("x", "dh") + (("r", "i") if gated else ("g",)):
        b[k][180:] = float("nan")
    whole, h = guarded((480, D), BF)
    wT, h_T = guarded((3, D), F32)
    _, _, kept = fwd(b, keep=True, h=h, h_T=h_T)
    torch.cuda.synchronize()
    want = bars.reference(host({**b, **{k: v[:180] for k, v in b.items() if isinstance(v, torch.Tensor) and
                                       v.shape[0] == 480}}), [0, 50, 50, 180], gated)
    bars.check("h", h[:180], want["h"])
    bars.check("h_T", h_T, want["h_T"])
    assert bool((h[180:] == FILL).all()) and untouched(whole, h) and untouched(wT, h_T)
    for name, x in zip(names(b), call_bwd(b, 3, b["cu"], kept)):
        if x.shape[0] == 480:
            assert bool((x[180:] == FILL).all())
            x = x[:180]
        bars.check(name, x, want[name])


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("cu", [[0, 300, 200], [-7, 120, 2 ** 31 - 1], [200, 100, 0], [0, -2 ** 31, 64], [150, 150, 151],
                                [0, 0, 0]])
def test_broken_tables_touch_nothing_else(cu, gated):
    b = make(7, [100, 100], 65, BF, gated)
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    whole, h = guarded((200, 65), BF)
    wT, h_T = guarded((2, 65), F32)
    _, _, kept = fwd(b, cu_seqlens=table, h=h, h_T=h_T, keep=True)
    torch.cuda.synchronize()
    assert untouched(whole, h) and untouched(wT, h_T)
    for given in (kept, None):
        call_bwd(b, 2, table, given)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_empty_batches(gated):
    b = make(8, [0, 0], 33, BF, gated)
    h, h_T, kept = fwd(b, keep=True)
    assert h.shape == (0, 33) and kept.shape == (0, 33) and torch.equal(h_T, b["h0"])
    g = bwd(b)
    assert torch.equal(g[-1], b["dh_T"]) and (not gated or not g[3].any())
    h, h_T = fwd({**b, "h0": None})
    assert not h_T.any()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = {**b, "h0": None, "dh_T": None}
    h, h_T = fwd(c, cu_seqlens=none)
    g = bwd(c, cu_seqlens=none)
    assert h_T.shape == (0, 33) and g[-1].shape == (0, 33) and (not gated or not g[3].any())


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_values_stay_in_their_sequence_and_channel(bad, gated):
    lens = [70, 300, 5, 40, 200]
    for D in (6, 7):
        b = make(9, lens, D, BF, gated)
        good, gh = bwd(b), fwd(b)
        for k in ("x", "dh") + (("r", "i") if gated else ("g",)):
            c = {x: y.clone() if isinstance(y, torch.Tensor) else y for x, y in b.items()}
            c[k][90, 3] = bad
            h, h_T = fwd(c)
            grads = bwd(c)
            torch.cuda.synchronize()
            keep = torch.ones(sum(lens), D, dtype=torch.bool, device="cuda")
            keep[70:370, 3] = False
            n = torch.ones(len(lens), D, dtype=torch.bool, device="cuda")
            n[1, 3] = False
            if k != "dh":
                assert torch.equal(h[keep], gh[0][keep]) and torch.equal(h_T[n], gh[1][n])
                if bad != bad:
                    assert bool(torch.isnan(h[90:370, 3]).all())
            for x, y, name in zip(grads, good, names(b)):
                m = keep if x.shape == keep.shape else n if x.shape == n.shape else n[1]
                assert torch.equal(x[m], y[m]), (k, name)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("D", [7, 8192])
def test_nonfinite_states_stay_in_their_sequence_and_channel(D, gated):
    """Infinities and NaN in a sequence's first state and last cotangent, borders inside and between tiles."""
    lens = [70, 300, 0, 5, 40, 128, 200]
    b = make(33, lens, D, BF, gated)
    good_h, good = fwd(b), bwd(b)
    for bad in (float("nan"), float("inf"), float("-inf")):
        c = dict(b, h0=b["h0"].clone(), dh_T=b["dh_T"].clone())
        for n in (1, 2, 5):
            c["h0"][n, 3] = c["dh_T"][n, 3] = bad
        h, h_T = fwd(c)
        grads = bwd(c)
        torch.cuda.synchronize()
        keep, n = torch.ones(sum(lens), D, dtype=torch.bool, device="cuda"), torch.ones(len(lens), D, dtype=torch.bool, device="cuda")
        for k in (1, 2, 5):
            keep[sum(lens[:k]):sum(lens[:k + 1]), 3] = False
            n[k, 3] = False
        assert torch.equal(h[keep], good_h[0][keep]) and torch.equal(h_T[n], good_h[1][n])
        for x, y, name in zip(grads, good, names(b)):
            m = keep if x.shape == keep.shape else n if x.shape == n.shape else n[1]
            assert torch.equal(x[m], y[m]), name
        # an empty sequence hands both on as they are
        assert torch.equal(h_T[2], c["h0"][2]) if bad == bad else bool(torch.isnan(h_T[2, 3]))
        assert torch.equal(grads[-1][2], c["dh_T"][2]) if bad == bad else bool(torch.isnan(grads[-1][2, 3]))


@pytest.mark.parametrize("dtype,gated,lens", [(BF, True, [150, 3]), (F32, False, [20]), (F32, True, [5, 28])])
def test_widest_rows(dtype, gated, lens):
    """The most channels there can be: a wave's rows take up to 2^30 bytes.  Some channels against the oracle."""
    D, N = (1 << 24) - 1, sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(34)
    rnd = lambda t, *shape: torch.empty(shape, dtype=t, device="cuda").normal_(generator=gen)              # noqa: E731
    b = dict(x=rnd(dtype, N, D), dh=rnd(dtype, N, D), h0=rnd(F32, len(lens), D), dh_T=rnd(F32, len(lens), D), gated=gated)
    if gated:
        b.update(r=rnd(dtype, N, D), i=rnd(dtype, N, D), rate=rnd(F32, D).abs_())
    else:
        b["g"] = rnd(F32, N, D).abs_().neg_()
    b["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    cols = torch.tensor([0, 1, 63, 64, 8388607, 8388608, D - 128, D - 65, D - 64, D - 2, D - 1], device="cuda")
    some = {k: v[..., cols] if isinstance(v, torch.Tensor) and k != "cu" else v for k, v in b.items()}
    want = bars.reference(host(some), b["cu"].tolist(), gated)
    h, h_T, kept = fwd(b, keep=True)
    bars.check("h", h[:, cols], want["h"])
    bars.check("h_T", h_T[:, cols], want["h_T"])
    del h
    for name, x in zip(names(b), bwd(b, kept=kept)):
        bars.check(name, x[..., cols], want[name])


def test_forgetting_and_closed_gates():
    """g = -inf forgets; gates so closed or open that factors reach their ends."""
    b = make(10, [200, 90], 64, F32, False)
    b["g"][50] = float("-inf")
    b["g"][230] = -1e30
    compare(b)
    for value in (-1e4, -90.0, -40.0, 40.0, 1e4):
        for dtype in (F32, BF):
            b = make(11, [200, 90], 64, dtype, True)
            b["r"][30:60] = value
            b["i"][50:80] = value
            b["rate"][3] = 0
            compare(b)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_gradients_against_differences(gated):
    """The loss's change along a random direction in fp32, 2 e apart: e^2 times
    a third derivative, and the loss's rounding (2^-24 of terms some sqrt(n)
    times larger) over e: 1e-3 of the larger of the change and its parts."""
    b = make(12, [60, 130], 32, F32, gated)
    grads = bwd(b)
    keys = ("x", "r", "i", "rate", "h0") if gated else ("x", "g", "h0")
    gen = torch.Generator(device="cuda").manual_seed(5)
    for k, gr in zip(keys, grads):
        d = torch.randn(b[k].shape, generator=gen, device="cuda")
        if k == "rate":
            d *= b[k]

        def loss(e):
            h, h_T = fwd({**b, k: b[k] + e * d})
            return (h.double() * b["dh"].double()).sum() + (h_T.double() * b["dh_T"].double()).sum()

        e = 2.0 ** -7
        num, want = float((loss(e) - loss(-e)) / (2 * e)), float((gr.double() * d.double()).sum())
        size = float((gr.double() * d.double()).norm())
        print(k, num, want, size)
        assert abs(num - want) <= 1e-3 * max(abs(want), size), k


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 4096), (5, 77), (130, 258)])
def test_decode(N, D, dtype, gated):
    m = lib()
    b = make(13, [1] * N, D, dtype, gated)
    r = np.random.default_rng(14)
    n_slots = N + 4
    pool = torch.from_numpy(r.standard_normal((n_slots, D)).astype(np.float32)).cuda()
    order = r.permutation(n_slots)[:N].astype(np.int32)
    real = np.ones(N, bool)
    if N > 2:
        order[1], order[N - 1] = -1, n_slots
        real[[1, N - 1]] = False
    slots = torch.from_numpy(order).cuda()
    f = m.glr_decode_step_gated if gated else m.glr_decode_step
    c = host(b)
    c["h0"] = np.zeros((N, D))
    c["h0"][real] = pool.double().cpu().numpy()[order[real]]
    want = bars.reference(c, list(range(N + 1)), gated, grads=False)
    before = pool.clone()
    h = f(*ins(b), pool, slots=slots)
    torch.cuda.synchronize()
    bars.check("h", h[real], tuple(x[real] for x in want["h"]))
    assert not h[~torch.from_numpy(real)].any()
    bars.check("S", pool[order[real]], tuple(x[real] for x in want["h_T"]))
    rest = np.setdiff1d(np.arange(n_slots), order[real])
    assert torch.equal(pool[rest], before[rest])
    # states in order, and an output given
    pool2, out = before.clone(), torch.empty_like(b["x"])
    assert f(*ins(b), pool2, h=out) is out
    h2, h2_T = fwd({**b, "h0": before[:N].contiguous()})
    assert torch.equal(pool2[:N], h2_T) and torch.equal(out, h2) and torch.equal(pool2[N:], before[N:])


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("D", [40002, 33001])
def test_many_blocks_of_channels(D, gated):
    compare(make(30, [150, 0, 23], D, BF, gated))


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("n", [63, 64, 65, 66])
def test_counts_of_sequences_around_a_wave(n, gated):
    """Up to a wave of sequences a tile knows the borders from the start, of more it searches them."""
    lens = [(7 * k) % 5 * (k % 3) for k in range(n)]
    compare(make(31, lens, 100, BF, gated, behind=9))
    compare(make(32, [0] * (n - 1) + [300], 100, F32, gated))


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_slots_named_twice_touch_nothing_else(gated):
    """The state and rows of such a slot are undefined, everything else is as without them."""
    b = make(26, [6], 260, BF, gated)
    f = lib().glr_decode_step_gated if gated else lib().glr_decode_step
    S = torch.randn(9, 260, device="cuda")
    T, slots = S.clone(), torch.tensor([3, 7, 3, 1, -1, 8], dtype=torch.int32, device="cuda")
    h = f(*ins(b), S, slots)
    slots[2] = 20
    want = f(*ins(b), T, slots)
    torch.cuda.synchronize()
    for k in range(9):
        assert k == 3 or torch.equal(S[k], T[k])
    for n in (1, 3, 4, 5):
        assert torch.equal(h[n], want[n])


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_one_workspace_for_calls_in_order(gated):
    """A workspace given by the caller, dirty from a larger call, for forward and
    gradients in turn, eagerly and in two graphs that share it."""
    b, c = make(27, [900, 500], 130, BF, gated), make(28, [3, 700, 0, 150], 130, BF, gated)
    m = lib()
    need = max(f(1400, 130) for f in (m.glr_fwd_workspace_bytes, m.glr_bwd_workspace_bytes))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    run = lambda x, w: fwd(x, keep=True, workspace=w) + bwd(x, workspace=w)                # noqa: E731
    want = [run(b, None), run(c, None)]
    for k in (0, 1, 0):
        for x, y in zip(run((b, c)[k], ws), want[k]):
            assert torch.equal(x, y)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, x in zip(graphs, (b, c)):
        with torch.cuda.graph(g):
            outs.append(run(x, ws))
    for k in (0, 1, 1, 0, 1):
        for o in outs[k]:
            o.fill_(FILL)
        graphs[k].replay()
        torch.cuda.synchronize()
        for x, y in zip(outs[k], want[k]):
            assert torch.equal(x, y)
        run((c, b)[k], ws)                                                                  # eager work between


@pytest.mark.parametrize("dtype,gated,D", [(BF, True, 4096), (F32, True, 200)])
def test_near_and_far_rates_side_by_side(dtype, gated, D):
    """Rates on both sides of the near form's end, in one wave and in waves of their own."""
    b = make(29, [130, 2500 if D < 1000 else 1030], D, dtype, gated)
    b["rate"] = torch.linspace(0.0, 1.4, D, device="cuda")
    compare(b)
    b["rate"] = b["rate"].view(2, -1).t().reshape(-1).contiguous()
    compare(b)


def test_sizes_past_32_bits_are_refused():
    """Shapes alone: a refused call reads nothing, and mostly one element stands for all."""
    m, W = lib(), (1 << 32) + 2
    one = lambda t, *shape: torch.zeros(1, dtype=t, device="cuda").expand(*shape)          # noqa: E731
    x, f, i = one(BF, 1, W), one(F32, 1, W), torch.int32
    with pytest.raises(ValueError, match="D must be below"):
        m.glr_fwd_scan(x, f)
    with pytest.raises(ValueError, match="D must be below"):
        m.glr_bwd_scan_gated(x, x, x, f[0], x)
    with pytest.raises(ValueError, match="n_seqs must be below"):
        m.glr_fwd_scan(one(BF, W, 0, 3), one(F32, W, 0, 3))
    b = make(35, [1, 1], 3)
    with pytest.raises(ValueError, match="n_slots must be below"):
        m.glr_decode_step_gated(*ins(b), one(F32, W, 3))
    with pytest.raises(ValueError, match="N must be below"):
        m.glr_decode_step(torch.empty(W, 1, dtype=BF, device="cuda"), torch.empty(W, 1, device="cuda"),
                          torch.zeros(4, 1, device="cuda"))
    pool, used, few = torch.zeros(4, 3, device="cuda"), torch.zeros(4, dtype=torch.bool, device="cuda"), one(i, 2).contiguous()
    for call, what in ((lambda: m.pool_alloc(pool, used, W), "n"), (lambda: m.pool_fork(pool, used, one(i, W)), "length of src"),
                       (lambda: m.pool_free(one(torch.bool, W), few), "n_slots"), (lambda: m.pool_free(used, one(i, W)), "length of slots"),
                       (lambda: m.pool_copy(one(F32, W, 3), few, pool, few), "n_slots")):
        with pytest.raises(ValueError, match=what + " must be below"):
            call()


def test_decode_from_an_empty_pool():
    b = make(15, [1] * 3, 40)
    h = lib().glr_decode_step_gated(*ins(b), torch.empty(0, 40, device="cuda"),
                                    slots=torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert not h.any()


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_decode_continues_the_scan(gated):
    """A prompt by the scan, tokens after it one by one: the states of one scan
    over all of them, within the bounds of both."""
    b = make(16, [200, 131], 70, F32, gated)
    cut = torch.cat((torch.arange(190), torch.arange(200, 321))).cuda()
    part = lambda rows: {k: v[rows].contiguous() if isinstance(v, torch.Tensor) and v.shape[:1] == (331,) else v   # noqa: E731
                         for k, v in b.items()}
    _, S = fwd({**part(cut), "cu": torch.tensor([0, 190, 311], dtype=torch.int32, device="cuda")})
    f = lib().glr_decode_step_gated if gated else lib().glr_decode_step
    want = bars.reference(host(b), [0, 200, 331], gated, grads=False)["h"]
    for j in range(10):
        rows = torch.tensor([190 + j, 321 + j]).cuda()
        h = f(*ins(part(rows)), S)
        torch.cuda.synchronize()
        bars.check("h", h, tuple(x[rows.cpu().numpy()] for x in want))


def test_streams_and_devices():
    """Two streams at once, each with its own workspace from torch's allocator."""
    b, c = make(17, [3000], 256, BF, True), make(18, [2999], 256, BF, True)
    want = [fwd(b), fwd(c), bwd(b), bwd(c)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            x = [fwd(b), bwd(b)]
        with torch.cuda.stream(t):
            y = [fwd(c), bwd(c)]
        torch.cuda.synchronize()
        for got, ref in zip(x + y, (want[0], want[2], want[1], want[3])):
            for p, q in zip(got, ref):
                assert torch.equal(p, q)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("D,lens", [(64, [9000, 1, 7000]), (1024, [9000, 1, 7000]), (4096, [4000, 300])])
def test_runs_are_bit_identical(D, lens, gated):
    """However far the tiles before a tile have come when it looks: beside
    nothing and beside a stream of other work."""
    b = make(23, lens, D, BF, gated)
    want = fwd(b, keep=True) + bwd(b)
    other, side = torch.randn(4096, 4096, device="cuda"), torch.cuda.Stream()
    for k in range(6):
        if k % 2:
            with torch.cuda.stream(side):
                for _ in range(20):
                    other = other * 1.0001
        for x, y in zip(fwd(b, keep=True) + bwd(b), want):
            assert torch.equal(x, y)
    torch.cuda.synchronize()


def test_captured_and_replayed():
    """Scan, gradients and a decode step in one graph, replayed with new inputs
    and eager work between the replays."""
    b = make(19, [700, 0, 600, 33], 192, BF, True)
    pool = torch.zeros(4, 192, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            fwd(b), bwd(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, h_T, kept = fwd(b, keep=True)
        grads = bwd(b, kept=kept)
        pool.copy_(h_T)
        one = lib().glr_decode_step_gated(b["x"][:4], b["r"][:4], b["i"][:4], b["rate"], pool)
    for seed in range(20, 24):
        c = make(seed, [700, 0, 600, 33], 192, BF, True)
        for k in ("x", "r", "i", "rate", "dh", "h0", "dh_T"):
            b[k].copy_(c[k])
        graph.replay()
        torch.cuda.synchronize()
        want = bars.reference(host(b), b["cu"].tolist(), True)
        for name, x in zip(("h", "h_T") + names(b), (h, h_T) + grads):
            bars.check(name, x, want[name])
        S = h_T.clone()
        again = lib().glr_decode_step_gated(b["x"][:4], b["r"][:4], b["i"][:4], b["rate"], S)
        torch.cuda.synchronize()
        assert torch.equal(again, one) and torch.equal(S, pool)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_offsets_past_2_to_the_31(gated):
    """More than 2^31 elements in the token tensors; the last sequence's rows
    against the oracle."""
    D, N = 16384, 131072 + 515
    assert N * D > 2 ** 31
    dev = "cuda"
    x = torch.full((N, D), 0.5, dtype=BF, device=dev)
    dh = torch.full((N, D), 0.25, dtype=BF, device=dev)
    b = dict(x=x, dh=dh, gated=gated, h0=None, dh_T=None,
             cu=torch.tensor([0, 1000, N - 300, N], dtype=torch.int32, device=dev))
    small = make(21, [300], D, BF, gated, states=False)
    for k in (("r", "i") if gated else ("g",)):
        b[k] = torch.full((N, D), -2.0, dtype=BF if gated else F32, device=dev)
    if gated:
        b["rate"] = small["rate"]
    for k in ("x", "dh") + (("r", "i") if gated else ("g",)):
        b[k][N - 300:] = small[k]
    cols = np.r_[0:4, D - 4:D]
    c = {k: v[:, cols] if v.ndim == 2 else v[cols] for k, v in host(small).items() if k != "cu"}
    want = bars.reference(c, [0, 300], gated)
    h, h_T, kept = fwd(b, keep=True)
    torch.cuda.synchronize()
    bars.check("h", h[N - 300:][:, cols], want["h"])
    bars.check("h_T", h_T[2:, cols], want["h_T"])
    del h
    for name, g in zip(names(b), bwd(b, kept=kept)):
        if name == "drate":
            continue
        g = g[2:] if name == "dh0" else g[N - 300:]
        bars.check(name, g[:, cols], want[name])


def test_large_pool():
    """A pool of more than 2^31 elements."""
    D, n = 65536, 32768 + 3
    pool = torch.zeros(n, D, device="cuda")
    b = make(22, [1, 1], D)
    pool[n - 1] = 1.0
    h = lib().glr_decode_step_gated(*ins(b), pool, slots=torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    c = host(b)
    c["h0"] = np.stack([np.ones(D), np.zeros(D)])
    want = bars.reference(c, [0, 1, 2], True, grads=False)
    bars.check("h", h, want["h"])
    bars.check("S", pool[[n - 1, 0]], want["h_T"])
    assert not pool[1:n - 1].any()
