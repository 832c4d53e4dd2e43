"""Session-cache operators: rope_append, window_attend, weigh_tokens and
evict_tokens against their definitions in 64 bits, and their refusals."""
import ctypes
import math

import pytest
import torch

import prefix_aware_decode_b200 as pad
from prefix_aware_decode_b200 import _binding
from prefix_aware_decode_b200.session import SessionPool

import cache_ref as ref
from cache_ref import Cache, P

gpu = pytest.mark.gpu

# (kv lengths, new rows) of a batch
BATCHES = {
    "one token": ([1], [1]),
    "single": ([17, 33, 5, 300, 16], [1, 1, 1, 1, 1]),
    "few rows": ([40, 129, 7, 512], [3, 5, 7, 2]),
    "gaps": ([60, 0, 45, 31, 200], [4, 0, 0, 9, 1]),
    "whole prompt": ([70, 257, 128], [70, 257, 128]),
    "chunks": ([700, 333, 1025], [129, 64, 300]),
    "mixed": ([900, 20, 450], [1, 20, 200]),
    "no keys for some": ([3, 40, 0], [8, 2, 3]),  # more rows than cached tokens
}
HEADS = [(1, 1, 64), (8, 1, 128), (8, 2, 64), (4, 2, 128), (8, 8, 128), (32, 8, 128), (12, 3, 64), (10, 5, 128)]
WINDOWS = [(0, 0), (1, 0), (16, 1), (37, 20), (100, 4), (2 ** 31 - 1, 3), (5, 2 ** 31 - 1)]


def _lib_status(name, *args):
    return getattr(_binding.lib(), name)(*args)


# ------------------------------------------------------------------------------------------------ attention


def _attend_case(kv, rows, Hq, Hkv, D, window, sinks, seed=0, holes=(), scale=0.0, extra_pages=1, extra_rows=2):
    c = Cache(kv, rows, Hq, Hkv, D, seed=seed, holes=holes, extra_rows=extra_rows, extra_pages=extra_pages)
    out = torch.full((c.n + extra_rows, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.n + extra_rows, Hq), 7.0, device="cuda")
    ref.run_attend(c, window, sinks, scale, out=out, lse=lse)
    o, l, tol, ltol = ref.attend(c, window, sinks, scale or None)
    ref.check(out[:c.n], o, tol, "out")
    ref.check(lse[:c.n], l, ltol, "lse")
    assert bool((out[c.n:] == 7).all()) and bool((lse[c.n:] == 7).all()), "rows of no session were written"
    return c, out, lse


@gpu
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("batch", list(BATCHES))
def test_attend_batches_and_windows(batch, window, sinks):
    _attend_case(*BATCHES[batch], 8, 2, 64, window, sinks, seed=1)


@gpu
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("batch", ["single", "few rows", "chunks", "mixed"])
def test_attend_head_layouts(batch, heads):
    _attend_case(*BATCHES[batch], *heads, 0, 0, seed=2)
    _attend_case(*BATCHES[batch], *heads, 130, 5, seed=3)


# one or two rows a session over short caches have a form of their own; a table of more
# than 1024 pages a session, or more rows, take the form for long caches
FEW = {
    "single": ([17, 33, 5, 300, 16], [1, 1, 1, 1, 1], (), 0),
    "padded": ([17, 33, 5, 300, 16], [1, 1, 1, 1, 1], (), 2),
    "none": ([1, 0, 64, 1, 990], [1, 1, 0, 1, 2], (), 0),  # rows without keys, a session without rows
    "more": ([1, 0, 64, 3, 990, 31], [1, 2, 0, 9, 8, 4], (), 2),  # more rows than cached tokens
    "holes": ([200, 150, 31], [1, 1, 1], [(0, 0), (0, 5), (1, 3), (1, 9), (0, 12), (2, 0), (2, 1)], 0),
    "holes, more": ([200, 150, 31], [3, 7, 2], [(0, 0), (0, 5), (1, 3), (1, 9), (0, 12), (2, 0), (2, 1)], 0),
    "long": ([4000, 3], [1, 1], [(0, 0), (0, 100), (0, 249)], 0),
    "long, more": ([4000, 3], [5, 2], [(0, 0), (0, 100), (0, 249)], 1),
    "fewer pages than warps": ([129, 0, 257], [1, 1, 1], (), 0),  # of a cluster
    "mostly holes": ([1000], [2], [(0, j) for j in range(8, 63)], 0),  # nothing for some CTAs of a cluster
}


@gpu
@pytest.mark.parametrize("extra_pages", [1, 1100])
@pytest.mark.parametrize("heads", [(1, 1, 64), (8, 8, 128), (4, 2, 128), (2, 1, 64), (8, 2, 128), (16, 4, 64), (8, 1, 64), (16, 2, 128)])
@pytest.mark.parametrize("few", list(FEW))
def test_attend_few_rows(few, heads, extra_pages):
    kv, rows, holes, extra = FEW[few]
    _attend_case(kv, rows, *heads, 0, 0, seed=6, holes=holes, extra_pages=extra_pages, extra_rows=extra)
    _attend_case(kv, rows, *heads, 0, 0, seed=7, holes=holes, extra_pages=extra_pages, extra_rows=extra, scale=0.7)


@gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (15, 1), (16, 16), (17, 33), (500, 20), (975, 17), (976, 33)])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1, 0], [2, 1, 4, 9, 3]])
@pytest.mark.parametrize("heads", [(8, 2, 64), (3, 3, 128), (4, 2, 64), (8, 1, 128)])
def test_attend_few_rows_under_windows(heads, rows, window, sinks):
    # the windows' edges inside pages, sinks that meet the window, rows that see different pages
    kv = [2000, 40, 1003, 17, 530]
    _attend_case(kv, rows, *heads, window, sinks, seed=8, extra_rows=0)
    _attend_case(kv, rows, *heads, window, sinks, seed=9, holes=[(0, 0), (0, 124), (2, 40)], extra_rows=1)


@gpu
def test_attend_short_form_keeps_out_what_no_row_sees_and_resets_the_status():
    c = Cache([400, 20], [1, 1], 8, 2, 128, seed=12)
    want = ref.attend(c, 100, 4)
    for t in range(4, 300):
        c.k[c.table[0, t // P].item(), :, t % P] = math.nan
        c.v[c.table[0, t // P].item(), :, t % P] = math.inf
    q, k, table, lens, cu = c.dev("q", "k", "table", "lens", "cu")
    ws = pad.window_workspace(q, k, table, lens, cu, window=100, sinks=4)
    ws.view(torch.uint8).fill_(255)
    out, lse = ref.run_attend(c, 100, 4, workspace=ws)
    assert pad.window_status(ws) == pad.PA_OK
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")


@gpu
@pytest.mark.parametrize("kv,rows", [([20011, 7], [1, 1]), ([9000], [5]), ([5000, 4097], [300, 17]), ([2500], [2500])])
def test_attend_long(kv, rows):
    _attend_case(kv, rows, 4, 1, 128, 0, 0, seed=4)
    _attend_case(kv, rows, 2, 2, 64, 1000, 33, seed=5)


@gpu
@pytest.mark.parametrize("rows", [[1, 1], [6, 90]])
def test_attend_holes_are_not_seen(rows):
    # whole pages missing at the start, inside and at the end; all of them
    _attend_case([200, 150], rows, 8, 2, 128, 0, 0, holes=[(0, 0), (0, 5), (1, 3), (1, 9), (0, 12)])
    _attend_case([200, 150], rows, 8, 2, 64, 40, 20, holes=[(0, j) for j in range(13)])


@gpu
@pytest.mark.parametrize("rows", [[1], [40]])
def test_attend_scale_and_large_logits(rows):
    _attend_case([100], rows, 4, 2, 64, 0, 0, scale=0.5)
    c = Cache([300], rows, 4, 2, 64, seed=8)
    c.k[c.table[0, 3].item(), :, 4] *= 40  # one key far above the rest
    c.k[c.table[0, 16].item(), :, 2] *= 80
    out, lse = ref.run_attend(c)
    o, l, tol, ltol = ref.attend(c)
    ref.check(out, o, tol, "out")
    ref.check(lse, l, ltol, "lse")


@gpu
def test_attend_reads_no_token_outside_the_window():
    # tokens that no row sees may hold anything, NaN and infinities among it
    c = Cache([400], [1], 8, 2, 128, seed=9)
    want = ref.attend(c, 100, 4)
    for t in range(4, 300):
        c.k[c.table[0, t // P].item(), :, t % P] = math.nan
        c.v[c.table[0, t // P].item(), :, t % P] = math.inf
    out, lse = ref.run_attend(c, 100, 4)
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")


@gpu
@pytest.mark.parametrize("batch", ["single", "chunks"])
def test_attend_runs_alike_on_another_stream_and_twice(batch):
    c = Cache(*BATCHES[batch], 8, 2, 128, seed=10)
    out, lse = ref.run_attend(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out2, lse2 = ref.run_attend(c, stream=s)
    s.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks,lo,hi,rows", [(700, 21, 900, 6000, 1), (2500, 21, 900, 6000, 1), (0, 0, 500, 5000, 7), (300, 5, 400, 3000, 40)])
def test_attend_many_items_a_cta(window, sinks, lo, hi, rows, D):
    """Many short items in a row on every SM, whose blocks end inside pages: every run gives the same bits."""
    g = torch.Generator().manual_seed(13)
    kv = torch.randint(lo, hi, (48,), generator=g).tolist()
    c = Cache(kv, [1 + int(i) % rows for i in torch.randint(0, 99, (48,), generator=g)], 8, 8, D, seed=14)
    out, lse = ref.run_attend(c, window, sinks)
    o, l, tol, ltol = ref.attend(c, window, sinks)
    ref.check(out, o, tol, "out")
    ref.check(lse, l, ltol, "lse")
    for _ in range(8):
        again, lse2 = ref.run_attend(c, window, sinks)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@gpu
def test_attend_agrees_with_the_planned_decode():
    # one row of every session, no window: what Plan / attend compute
    c = Cache([400, 33, 1000, 16], [1, 1, 1, 1], 8, 2, 128, seed=11)
    out, lse = ref.run_attend(c)
    table = torch.where(c.table < 0, 0, c.table)
    o, l = pad.attend(c.q.cuda(), *c.dev("k", "v"), table, c.lens)
    # both are within one rounding of the weights and one of the result of the same value
    tol = ref.attend(c)[2]
    ref.check(out, o.double().cpu(), 2 * tol, "out")
    ref.check(lse, l.double().cpu(), torch.full((4, 8), 2e-4), "lse")


@gpu
@pytest.mark.parametrize("n_rows", [1, 40])
def test_captured_calls_follow_the_device_arrays(n_rows):
    """Two graphs that share one workspace, replayed as lengths, tables and row offsets change in place."""
    big = Cache([600, 600, 600], [n_rows] * 3, 8, 2, 128, seed=12)
    q, k, v, table, lens, cu = big.dev("q", "k", "v", "table", "lens", "cu")
    ws = pad.window_workspace(q, k, table, lens, cu)
    outs = []
    kw = [dict(), dict(window=50, sinks=3)]
    side = torch.cuda.Stream()
    graphs = []
    for o in kw:
        pad.window_attend(q, k, v, table, lens, cu, workspace=ws, **o)  # once outside a capture
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pad.window_attend(q, k, v, table, lens, cu, workspace=ws, out=out, lse=lse, **o)
        graphs.append(g)
        outs.append((out, lse))
    for kv, rows in [([600, 600, 600], [n_rows] * 3), ([20, 599, 1], [1, min(2, n_rows), 1]), ([0, 350, 48], [0, n_rows, n_rows])]:
        rows = [min(a, b) for a, b in zip(kv, rows)]
        big.kv, big.rows = kv, rows
        new = torch.tensor([0, rows[0], rows[0] + rows[1], sum(rows)], dtype=torch.int32)
        big.cu, big.n = new, sum(rows)
        lens.copy_(big.lens)
        cu.copy_(new)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (out, lse), o in zip(outs, kw):
            a, l, tol, ltol = ref.attend(big, o.get("window", 0), o.get("sinks", 0))
            ref.check(out[:big.n], a, tol, "out")
            ref.check(lse[:big.n], l, ltol, "lse")


@gpu
def test_two_calls_at_once_and_their_status():
    a, b = Cache([3000, 900], [200, 1], 8, 2, 128, seed=15), Cache([2000] * 3, [1, 1, 60], 8, 2, 128, seed=16)
    want = [ref.run_attend(c) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for c in (a, b):
        args = c.dev("q", "k", "v", "table", "lens", "cu")
        calls.append((args, pad.window_workspace(args[0], args[1], *args[3:])))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for (args, ws), s in zip(calls, streams):
            got.append(pad.window_attend(*args, workspace=ws, stream=s))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    for (_, ws), s in zip(calls, streams):
        assert pad.window_status(ws) == pad.window_status(ws, stream=s) == pad.PA_OK
    assert pad.weigh_status() == pad.PA_OK


# ------------------------------------------------------------------------------------------------ weights


def _weigh_case(kv, rows, Hq, Hkv, D, window, sinks, seed=0, holes=(), max_tokens=None, extra_pages=1):
    c = Cache(kv, rows, Hq, Hkv, D, seed=seed, holes=holes, extra_rows=1, extra_pages=extra_pages)
    _, lse = ref.run_attend(c, window, sinks)
    T = max_tokens or c.width * P
    s0 = torch.rand(len(kv), Hkv, T, generator=c.gen)
    scores = s0.cuda()
    q, k, table, lens, cu = c.dev("q", "k", "table", "lens", "cu")
    assert pad.weigh_tokens(q, k, lse, table, lens, cu, scores, window=window, sinks=sinks) is scores
    w, tol = ref.weigh(c, lse.cpu(), window, sinks)
    n = min(T, w.shape[2])
    want, bound = s0.double(), torch.zeros_like(s0, dtype=torch.float64)
    want[..., :n] += w[..., :n]
    bound[..., :n] = tol[..., :n] + 2.0 ** -24 * want[..., :n].abs()
    ref.check(scores, want, bound, "scores")
    for s, m in enumerate(kv):  # nothing past the cached tokens changes
        assert torch.equal(scores[s, :, m:].cpu(), s0[s, :, m:])
    return c, scores, lse


@gpu
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("batch", list(BATCHES))
def test_weigh_batches_and_windows(batch, window, sinks):
    _weigh_case(*BATCHES[batch], 8, 2, 64, window, sinks, seed=21)


@gpu
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("batch", ["single", "few rows", "chunks", "mixed"])
def test_weigh_head_layouts(batch, heads):
    _weigh_case(*BATCHES[batch], *heads, 0, 0, seed=22)


@gpu
def test_weigh_long_holes_and_a_short_score_row():
    _weigh_case([9000, 4100], [1, 3], 8, 1, 128, 0, 0, seed=23)
    _weigh_case([3000], [700], 4, 2, 128, 512, 16, seed=24)
    _weigh_case([2500, 1900], [1300, 900], 8, 4, 64, 0, 0, seed=29, extra_pages=1000)
    _weigh_case([200, 150], [30, 1], 8, 2, 64, 0, 0, seed=25, holes=[(0, 0), (0, 5), (1, 3), (0, 12)])
    _weigh_case([200, 150], [30, 1], 8, 2, 64, 0, 0, seed=26, max_tokens=77)


@gpu
@pytest.mark.parametrize("heads", [(32, 8, 128), (8, 8, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 10)])
@pytest.mark.parametrize("batch", list(BATCHES))
def test_weigh_in_a_wide_table(batch, window, sinks, heads):
    # a table wide enough that the kernel takes key blocks in pairs
    _weigh_case(*BATCHES[batch], *heads, window, sinks, seed=28, extra_pages=700)


@gpu
def test_weigh_one_long_chunk_among_single_rows():
    # few rows on average, so key blocks stream, but one session has several column tiles
    rows = [1, 1, 150, 1, 0, 1, 1, 40, 1, 1]
    kv = [300, 17, 420, 1, 50, 90, 512, 300, 33, 256]
    for extra in (1, 700):
        _weigh_case(kv, rows, 8, 2, 128, 0, 0, seed=30, extra_pages=extra)
        _weigh_case(kv, rows, 8, 8, 64, 60, 9, seed=31, extra_pages=extra)


@gpu
def test_weights_of_a_row_sum_to_one():
    c, scores, _ = _weigh_case([500, 90], [1, 60], 8, 2, 128, 0, 0, seed=27)
    q, k, table, lens, cu = c.dev("q", "k", "table", "lens", "cu")
    _, lse = ref.run_attend(c)
    s = torch.zeros_like(scores)
    pad.weigh_tokens(q, k, lse, table, lens, cu, s)
    got = s.double().sum(2).cpu()
    want = torch.tensor([[4.0, 4.0], [240.0, 240.0]], dtype=torch.float64)  # rows x heads of the group
    assert bool(((got - want).abs() <= want * 1e-4).all()), got
    again = torch.zeros_like(scores)
    pad.weigh_tokens(q, k, lse, table, lens, cu, again)
    assert torch.equal(s, again)


# ------------------------------------------------------------------------------------------------ eviction


def _evict_case(kv, Hkv, D, budget, sinks, recent, scores=None, seed=0, T=None):
    c = Cache(kv, [0] * len(kv), Hkv, Hkv, D, seed=seed, extra_pages=2)
    n_dst = -(-budget // P)
    base = c.num_pages
    pad_pages = torch.full((len(kv) * n_dst, Hkv, P, D), 3.0).bfloat16()
    k0, v0 = torch.cat([c.k, pad_pages]), torch.cat([c.v, pad_pages])
    dst = (base + torch.randperm(len(kv) * n_dst, generator=c.gen).int()).view(len(kv), n_dst)
    T = T or (c.width * P if scores is None else scores.shape[2])
    if scores is None:
        scores = torch.rand(len(kv), Hkv, T, generator=c.gen)
    c.num_pages = k0.shape[0]
    k, v = k0.cuda(), v0.cuda()
    lens, kept, out = pad.evict_tokens(scores.cuda(), k, v, *c.dev("table", "lens"), dst.cuda(), budget, sinks=sinks,
                                       recent=recent)
    want = ref.evict(scores, kv, budget, sinks, recent)
    assert lens.tolist() == [min(n, budget, T) for n in kv]
    kn, vn = k0.clone(), v0.clone()
    for s in range(len(kv)):
        for h in range(Hkv):
            ids = torch.tensor(want[s][h], dtype=torch.long)
            m = len(ids)
            assert kept[s, h, :m].tolist() == ids.tolist() and bool((kept[s, h, m:] == -1).all()), (s, h)
            x = torch.zeros(T)
            x[:m] = scores[s, h, ids]
            assert torch.equal(out[s, h].cpu().view(torch.int32), x.view(torch.int32))
            j = torch.arange(m)
            for new, old in ((kn, k0), (vn, v0)):
                new[dst[s, j // P].long(), h, j % P] = old[c.table[s, ids // P].long(), h, ids % P]
    for got, exp in ((k, kn), (v, vn)):
        assert torch.equal(got.cpu().view(torch.int16), exp.view(torch.int16)), "pool"


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,budget,sinks,recent", [
    ([100, 37, 0, 300, 1], 32, 4, 8), ([100, 37], 1, 0, 0), ([100, 37], 1, 1, 0), ([100, 37], 1, 0, 1),
    ([513, 16, 15], 16, 0, 0), ([513], 500, 250, 250), ([1500, 2049], 777, 0, 300), ([5000], 4999, 1, 0),
    ([2048, 2047], 4096, 7, 9), ([17, 400], 17, 5, 12)])
def test_evict(D, kv, budget, sinks, recent):
    _evict_case(kv, 2, D, budget, sinks, recent, seed=31)


@gpu
def test_evict_ties_and_odd_scores():
    g = torch.Generator().manual_seed(5)
    x = torch.randint(0, 4, (2, 3, 2000), generator=g).float()  # long ties
    _evict_case([2000, 1234], 3, 64, 500, 3, 17, scores=x, seed=32)
    _evict_case([2000, 1234], 3, 64, 500, 3, 17, scores=torch.zeros(2, 3, 2000), seed=33)
    y = torch.randn(2, 3, 2000, generator=g)
    y[0, :, 5::7] = math.inf
    y[0, :, 6::9] = -math.inf
    y[1, 0, 3::11] = math.nan
    y[1, 1, ::2] = -0.0
    y[1, 1, 1::2] = 0.0
    y[1, 2] *= 1e-42  # denormals
    _evict_case([2000, 1234], 3, 64, 300, 3, 17, scores=y, seed=34)


@gpu
def test_evict_long_and_short_score_rows():
    _evict_case([70001], 1, 64, 3000, 4, 100, seed=35)
    _evict_case([9001, 12000], 2, 64, 8000, 0, 1, seed=38)  # several CTAs a row
    g = torch.Generator().manual_seed(6)
    x = torch.randint(0, 3, (1, 1, 400000), generator=g).float()  # more keys than shared memory holds
    _evict_case([345678], 1, 64, 1000, 4, 100, scores=x, seed=39)
    _evict_case([400, 90], 2, 64, 100, 4, 10, seed=36, T=257)  # lengths taken as at most max_tokens


@gpu
def test_evict_skips_holes():
    c = Cache([100], [0], 1, 1, 64, seed=37, holes=[(0, 1)])
    k = torch.cat([c.k, torch.full((2, 1, P, 64), 3.0).bfloat16()]).cuda()
    v = k.clone()
    dst = torch.tensor([[c.num_pages, 10 ** 6]], dtype=torch.int32, device="cuda")  # the second page is outside the pool
    x = torch.zeros(1, 1, c.width * P)
    x[0, 0, 16:20] = 1.0
    lens, kept, _ = pad.evict_tokens(x.cuda(), k, v, *c.dev("table", "lens"), dst, 20)
    assert lens.tolist() == [20] and kept[0, 0].tolist() == list(range(20))
    got = k[c.num_pages, 0].cpu()
    assert torch.equal(got, c.k[c.table[0, 0].item(), 0])  # tokens 0-15; 16-19 are in a hole
    assert bool((k[c.num_pages + 1] == 3).all())


# ------------------------------------------------------------------------------------------------ rotary append


def _rope_case(kv, rows, Hq, Hkv, D, R, n_axes, interleaved, positions=None, seed=0, holes=(), in_place=False):
    c = Cache(kv, rows, Hq, Hkv, D, seed=seed, holes=holes)
    n = c.n + 1  # the last row belongs to no session
    fused = torch.randn(n, (Hq + 2 * Hkv) * D + 8, generator=c.gen).bfloat16()
    q = fused[:, :Hq * D].view(n, Hq, D)
    k = fused[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D)
    v = fused[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(n, Hkv, D)
    if positions is None:
        positions = torch.randint(-50, 1 << 20, (n_axes, n), generator=c.gen).int()
    inv = 10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)
    axes = [(i * n_axes) // (R // 2) for i in range(R // 2)] if n_axes > 1 else None
    f = fused.cuda()
    dq = f[:, :Hq * D].view(n, Hq, D)
    if in_place:
        dq = dq.contiguous()
    dk, dv = f[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D), f[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(n, Hkv, D)
    kp, vp = c.dev("k", "v")
    q_out = dq if in_place else torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = pad.rope_append(dq, dk, dv, positions.cuda(), inv.cuda(), kp, vp, *c.dev("table", "lens", "cu"), axes=axes,
                          interleaved=interleaved, q_out=q_out)
    assert got is q_out
    pos2 = positions if positions.dim() == 2 else positions[None]
    ax = axes or [0] * (R // 2)
    wq, tq = ref.rotate(q.double(), pos2, inv, ax, interleaved)
    wk, tk = ref.rotate(k.double(), pos2, inv, ax, interleaved)
    ref.check(got[:c.n], wq[:c.n], tq[:c.n], "q")
    last = q[c.n:] if in_place else torch.full((1, Hq, D), 7.0).bfloat16()
    assert torch.equal(got[c.n:].cpu(), last), "a row of no session was written"
    want_k, want_v, tol = c.k.double(), c.v.clone(), torch.zeros(c.k.shape, dtype=torch.float64)
    for s in range(len(kv)):
        for i in range(rows[s]):
            t, r = kv[s] - rows[s] + i, int(c.cu[s]) + i
            p = int(c.table[s, t // P]) if t >= 0 else -1
            if 0 <= p < c.num_pages:
                want_k[p, :, t % P], tol[p, :, t % P], want_v[p, :, t % P] = wk[r], tk[r], v[r]
    g = kp.double().cpu()
    same = (g.isnan() & want_k.isnan()) | ((g - want_k).abs() <= tol)
    assert bool(same.all()), "k_pool"
    assert torch.equal(vp.cpu().view(torch.int16), want_v.view(torch.int16)), "v_pool"


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,R,n_axes", [(8, 2, 64, 64, 1), (4, 4, 128, 128, 3), (8, 1, 128, 64, 4), (2, 1, 64, 16, 2),
                                               (32, 8, 128, 128, 1), (1, 1, 128, 112, 3)])
@pytest.mark.parametrize("batch", ["one token", "gaps", "few rows", "whole prompt", "no keys for some"])
def test_rope_append(batch, Hq, Hkv, D, R, n_axes, interleaved):
    _rope_case(*BATCHES[batch], Hq, Hkv, D, R, n_axes, interleaved, seed=41)


@gpu
def test_rope_many_sessions_one_axis_in_place_and_holes():
    kv = [(7 * i) % 40 for i in range(1100)]
    rows = [min(k, i % 3) for i, k in enumerate(kv)]
    _rope_case(kv, rows, 2, 1, 64, 64, 1, False, seed=42)
    n = 71
    _rope_case([100], [70], 4, 2, 64, 64, 1, False, positions=torch.arange(n).int(), seed=43, holes=[(0, 2), (0, 5)])
    _rope_case([100], [70], 4, 2, 64, 64, 1, True, positions=torch.arange(n).int() - 30, seed=44, in_place=True)
    far = torch.full((1, n), 2 ** 31 - 1).int()
    far[0, ::2] = -2 ** 31
    # angles of 2^31 radians are formed in fp64: off by 2^-21 radian, within the bound's 2^-20
    _rope_case([100], [70], 4, 2, 64, 64, 1, False, positions=far, seed=45)


# ------------------------------------------------------------------------------------------------ together


@gpu
def test_a_session_lives_through_append_attend_weigh_and_evict():
    """Prompt chunk, decode steps, eviction to a budget, and a decode step on what is left, through SessionPool."""
    Hq, Hkv, D, budget, sinks, recent = 8, 2, 64, 64, 4, 16
    g = torch.Generator().manual_seed(7)
    pool = SessionPool(64)
    kp = torch.full((64, Hkv, P, D), math.nan, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    inv = (10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).cuda()
    sids = [3, 9]
    for s in sids:
        pool.open(s)
    seen = {s: 0 for s in sids}  # tokens of the stream so far: positions keep counting over evictions
    cache = {s: [[], []] for s in sids}  # per kv head: the (k, v) rows in the cache, in order
    scores = torch.zeros(2, Hkv, 20 * P, device="cuda")
    total = torch.zeros(2, Hkv, 20 * P, dtype=torch.float64)

    def step(rows):
        n = sum(rows)
        for s, r in zip(sids, rows):
            pool.append(s, r)
        table, lens = pool.tables(sids)
        cu = torch.tensor([0, rows[0], n], dtype=torch.int32)
        x = torch.randn(n, Hq + 2 * Hkv, D, generator=g).bfloat16()
        pos = torch.cat([torch.arange(seen[s], seen[s] + r) for s, r in zip(sids, rows)]).int()
        dev = [torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), cu.cuda()]
        f = x.cuda()
        q = pad.rope_append(f[:, :Hq], f[:, Hq:Hq + Hkv], f[:, Hq + Hkv:], pos.cuda(), inv, kp, vp, *dev)
        out, lse = pad.window_attend(q, kp, vp, *dev)
        pad.weigh_tokens(q, kp, lse, *dev, scores)
        # the same from the definitions, with the rotated bf16 q and k the kernels hold
        c = Cache([0, 0], rows, Hq, Hkv, D)
        c.kv, c.table, c.num_pages = [int(t) for t in lens], torch.from_numpy(table), 64
        c.q, c.k, c.v = q.cpu(), kp.cpu(), vp.cpu()
        o, l, tol, ltol = ref.attend(c)
        ref.check(out, o, tol, "out")
        ref.check(lse, l, ltol, "lse")
        kr = ref.rotate(x[:, Hq:Hq + Hkv].double(), pos[None], inv.cpu(), [0] * (D // 2), False)
        w, _ = ref.weigh(c, lse.cpu())
        total[..., :w.shape[2]] += w
        for i, (s, r) in enumerate(zip(sids, rows)):
            for h in range(Hkv):
                for j in range(r):
                    row = int(cu[i]) + j
                    cache[s][h].append((kr[0][row, h], kr[1][row, h], x[row, Hq + Hkv + h]))
                kk = c.tokens(c.k, i, h)[1]
                vv = c.tokens(c.v, i, h)[1]
                for t, (want, bound, v) in enumerate(cache[s][h]):
                    assert bool(((kk[t] - want).abs() <= bound).all()) and torch.equal(vv[t], v.double())
            seen[s] += r
        return dev

    step([70, 33])
    step([1, 1])
    step([5, 40])
    table, lens = pool.tables(sids)
    assert float((scores.double().cpu() - total).abs().max()) < 1e-3
    new = pool.compact(sids, budget)
    dst = torch.tensor([n + [-1] * (budget // P - len(n)) for n in new], dtype=torch.int32).cuda()
    before = scores.cpu()
    lens2, kept, scores2 = pad.evict_tokens(scores, kp, vp, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(),
                                            dst, budget, sinks=sinks, recent=recent)
    want = ref.evict(before, [int(t) for t in lens], budget, sinks, recent)
    for i, s in enumerate(sids):
        assert pool.tokens(s) == int(lens2[i]) == min(int(lens[i]), budget)
        for h in range(Hkv):
            assert kept[i, h][:len(want[i][h])].tolist() == want[i][h]
            cache[s][h] = [cache[s][h][t] for t in want[i][h]]
    pool.check()
    total.copy_(scores2.double().cpu())
    scores.copy_(scores2)
    step([1, 1])
    step([3, 20])
    # the compact cache is an ordinary one: the planned decode reads it too
    for s in sids:
        pool.register(s, s)
    _, _, table, lens = pool.batch()
    c = Cache([0, 0], [1, 1], Hq, Hkv, D)
    q = torch.randn(2, Hq, D, generator=g).bfloat16().cuda()
    o, _ = pad.attend(q, kp, vp, table, lens)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    o2, _ = pad.window_attend(q, kp, vp, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), cu)
    c.kv, c.table, c.num_pages, c.q, c.k, c.v = [int(t) for t in lens], torch.from_numpy(table), 64, q.cpu(), kp.cpu(), vp.cpu()
    tol = ref.attend(c)[2]
    ref.check(o2, o.double().cpu(), 2 * tol, "decode")


@gpu
def test_a_captured_step_of_all_four_follows_the_device_arrays():
    """append, attend, weigh and evict in one graph, captured before any of them ran,
    replayed as lengths, tables, positions and row offsets change in place."""
    Hq, Hkv, D, budget = 8, 2, 128, 96
    base = Cache([500, 300, 40], [3, 70, 1], Hq, Hkv, D, seed=50)
    n = base.n
    g = torch.Generator().manual_seed(51)
    x = torch.randn(n, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    inv = (10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)).cuda()
    spare = torch.zeros(3 * budget // P, Hkv, P, D).bfloat16()
    dst = (base.num_pages + torch.arange(3 * budget // P).int()).view(3, -1).cuda()
    pools = [torch.cat([t, spare]).cuda() for t in (base.k, base.v)]
    table, lens, cu = base.dev("table", "lens", "cu")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    scores = torch.zeros(3, Hkv, base.width * P, device="cuda")

    def step(kp, vp, sc):
        q = pad.rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, inv, kp, vp, table, lens, cu)
        out, lse = pad.window_attend(q, kp, vp, table, lens, cu, window=200, sinks=4)
        pad.weigh_tokens(q, kp, lse, table, lens, cu, sc, window=200, sinks=4)
        return (q, out, lse, sc) + pad.evict_tokens(sc, kp, vp, table, lens, dst, budget, sinks=4, recent=20) + (kp, vp)

    held = [t.clone() for t in pools] + [scores.clone()]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        res = step(*held)
    for kv, rows in (([500, 300, 40], [3, 70, 1]), ([499, 17, 0], [1, 17, 0]), ([96, 300, 30], [20, 1, 30])):
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        cu.copy_(torch.tensor([0, rows[0], rows[0] + rows[1], sum(rows)], dtype=torch.int32))
        pos.copy_(torch.randint(0, 5000, (n,), generator=g).int())
        m = sum(rows)
        for t, s in zip(held, pools + [scores]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        want = step(*[t.clone() for t in pools], scores.clone())
        for i, (a, b) in enumerate(zip(res, want)):
            if i < 3:
                a, b = a[:m], b[:m]  # rows of no session are left as they were
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                               b.view(torch.int16) if b.dtype == torch.bfloat16 else b), i
    del graph


def test_session_pool_tables_and_compact():
    pool = SessionPool(20)
    pool.open(1)
    pool.append(1, 100)
    pool.fork(2, 1)
    table, lens = pool.tables([2, 1])
    assert lens.tolist() == [100, 100] and table.shape == (2, 7) and table.dtype == lens.dtype == "int32"
    assert table[0, :6].tolist() == table[1, :6].tolist() and table[0, 6] != table[1, 6]
    old = pool.pages(1)
    new, = pool.compact([1], 40)
    assert len(new) == 3 and not set(new) & set(old) and pool.pages(1) == new and pool.tokens(1) == 40
    assert pool.pages(2)[:6] == old[:6]  # the fork keeps the shared pages
    pool.check()
    assert pool.compact([1], 64) == [pool.pages(1)] and pool.tokens(1) == 40  # no more tokens than the session has
    pool.check()
    for bad in (([1], 0), ([1, 1], 40)):
        with pytest.raises(ValueError):
            pool.compact(*bad)
    pool.append(1, 16 * pool.free_pages)
    before = pool.pages(1)
    with pytest.raises(MemoryError):
        pool.compact([1], 40)
    assert pool.pages(1) == before
    pool.check()


def test_compacted_sessions_take_no_page_that_one_of_them_held():
    # one eviction call copies them all: a page written for one is not read for another
    pool = SessionPool(40)
    for s in range(4):
        pool.open(s)
        pool.append(s, 70 + 9 * s)
    old = {p for s in range(4) for p in pool.pages(s)}
    new = pool.compact([2, 0, 3, 1], 48)
    assert [len(p) for p in new] == [3, 3, 3, 3] and len({p for n in new for p in n}) == 12
    assert not old & {p for n in new for p in n}
    assert [pool.pages(s) for s in (2, 0, 3, 1)] == new
    pool.check()


# ------------------------------------------------------------------------------------------------ refusals


def _sessions(**kw):
    d = dict(n_sessions=2, num_rows=3, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, max_pages=4,
             num_pages_in_pool=9, d_block_table=4096, d_kv_lens=8192, d_cu_rows=12288)
    d.update(kw)
    return _binding.PaSessions(*[d[n] for n, _ in _binding.PaSessions._fields_])


BAD = [dict(n_sessions=0), dict(num_rows=-1), dict(num_q_heads=0), dict(num_kv_heads=0), dict(max_pages=0),
       dict(num_pages_in_pool=0), dict(d_block_table=0), dict(d_kv_lens=0), dict(d_cu_rows=0), dict(num_q_heads=7),
       dict(n_sessions=65536)]
UNBUILT = [dict(head_dim=96), dict(page_size=32), dict(num_q_heads=6), dict(num_q_heads=32), dict(max_pages=1 << 27),
           dict(num_pages_in_pool=1 << 26, num_kv_heads=8)]


@pytest.mark.parametrize("change,status", [(c, _binding.PA_ERR_INVALID) for c in BAD]
                         + [(c, _binding.PA_ERR_UNSUPPORTED) for c in UNBUILT])
def test_every_call_refuses_a_bad_batch(change, status):
    """Checked on the host before anything is enqueued: the addresses are never read."""
    b = ctypes.byref(_sessions(**change))
    n = ctypes.c_size_t()
    p = 1 << 20
    rope = ctypes.byref(_binding.PaRope(64, 1, 0, None, 4096, 4096))
    assert _lib_status("pa_window_workspace_size", b, 0, 0, ctypes.byref(n)) == status
    assert _lib_status("pa_window_attend", b, 0, 0, 0.0, p, p, p, p, 1 << 30, p, p, None) == status
    assert _lib_status("pa_weigh_tokens", b, 0, 0, 0.0, p, p, p, p, 64, None) == status
    assert _lib_status("pa_rope_append", b, rope, p, 512, p, 128, p, 128, p, p, p, None) == status
    if "d_cu_rows" not in change and "num_rows" not in change:
        assert _lib_status("pa_evict_tokens", b, p, 64, p, p, p, 4, 32, 0, 0, 2 * p, p, p, None) == status


def test_refusals_of_single_arguments():
    b, bad, nomem = ctypes.byref(_sessions()), _binding.PA_ERR_INVALID, _binding.PA_ERR_NOMEM
    p, n = 1 << 20, ctypes.c_size_t()
    assert _lib_status("pa_window_workspace_size", b, -1, 0, ctypes.byref(n)) == bad
    assert _lib_status("pa_window_workspace_size", b, 0, -1, ctypes.byref(n)) == bad
    assert _lib_status("pa_window_workspace_size", b, 0, 0, None) == bad
    assert _lib_status("pa_window_workspace_size", b, 0, 0, ctypes.byref(n)) == 0 and n.value > 0
    ok = [b, 0, 0, 0.0, p, p, p, p, n.value, p, p, None]
    for i, v, st in [(1, -1, bad), (2, -1, bad), (4, 0, bad), (4, p + 8, bad), (5, 0, bad), (5, p + 2, bad), (6, 0, bad),
                     (6, p + 2, bad), (7, 0, bad), (7, p + 16, bad), (8, n.value - 1, nomem), (9, 0, bad), (9, p + 8, bad)]:
        a = list(ok)
        a[i] = v
        assert _lib_status("pa_window_attend", *a) == st, (i, v)
    ok = [b, 0, 0, 0.0, p, p, p, p, 64, None]
    for i, v in [(1, -1), (2, -1), (4, 0), (4, p + 8), (5, 0), (5, p + 8), (6, 0), (7, 0), (8, 0)]:
        a = list(ok)
        a[i] = v
        assert _lib_status("pa_weigh_tokens", *a) == bad, (i, v)
    ok = [b, p, 64, p, p, p, 4, 32, 1, 2, 2 * p, p, p, None]
    for i, v in [(1, 0), (2, 0), (3, 0), (3, p + 8), (4, 0), (5, 0), (6, 0), (6, 1), (7, 0), (7, 65), (8, -1), (9, -1),
                 (8, 31), (9, 32), (10, 0), (10, p), (11, 0), (12, 0)]:
        a = list(ok)
        a[i] = v
        assert _lib_status("pa_evict_tokens", *a) == bad, (i, v)
    rope = dict(R=64, n_axes=1, il=0, axes=None, pos=4096, inv=4096)

    def roped(**kw):
        d = dict(rope, **kw)
        r = _binding.PaRope(d["R"], d["n_axes"], d["il"], d["axes"], d["pos"], d["inv"])
        return _lib_status("pa_rope_append", b, ctypes.byref(r), p, 512, p, 128, p, 128, p, p, p, None)

    for kw in (dict(R=0), dict(R=80), dict(R=24), dict(n_axes=0), dict(n_axes=5), dict(axes=b"\x01" * 32), dict(pos=0),
               dict(inv=0)):
        assert roped(**kw) == bad, kw
    r = ctypes.byref(_binding.PaRope(64, 1, 0, None, 4096, 4096))
    ok = [b, r, p, 512, p, 128, p, 128, p, p, p, None]
    for i, v in [(1, None), (2, 0), (2, p + 8), (3, 504), (3, 513), (4, 0), (5, 120), (5, 129), (6, 0), (7, 64), (8, 0),
                 (8, p + 8), (9, 0), (10, 0), (10, p + 8)]:
        a = list(ok)
        a[i] = v
        assert _lib_status("pa_rope_append", *a) == bad, (i, v)


def test_there_is_no_cpu_path():
    c = Cache([20, 5], [2, 1], 8, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        pad.window_attend(c.q, c.k, c.v, c.table, c.lens, c.cu)


@gpu
def test_python_refuses_what_the_library_cannot_see():
    """Wrong types, shapes, strides and devices: every call raises before anything is enqueued."""
    c = Cache([20, 5], [2, 1], 8, 2, 64)
    c.q, c.k, c.v, c.table, c.cu = c.dev("q", "k", "v", "table", "cu")
    c_lens = c.lens.cuda()
    args = [c.q, c.k, c.v, c.table, c_lens, c.cu]
    pad.window_attend(*args)
    for i, t in [(0, c.q.float()), (0, c.q[:, :, :32]), (1, c.k.half()), (1, c.k[0]), (2, c.v[1:]), (3, c.table.long()),
                 (3, c.table[0]), (4, c_lens.long()), (4, c_lens[:1]), (5, c.cu[:2]), (5, c.cu.float())]:
        a = list(args)
        a[i] = t
        with pytest.raises(ValueError):
            pad.window_attend(*a)
    for i in range(6):  # a tensor of another device
        a = list(args)
        a[i] = args[i].cpu()
        with pytest.raises(ValueError):
            pad.window_attend(*a)
    for kw in (dict(out=c.q[:2]), dict(out=c.q.float()), dict(lse=torch.zeros(3, 8)), dict(window=-1), dict(sinks=-1),
               dict(softmax_scale=-1.0), dict(softmax_scale=math.inf), dict(softmax_scale=math.nan)):
        with pytest.raises((ValueError, pad.PaError)):
            pad.window_attend(*args, **kw)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(pad.PaError):
        pad.window_attend(*args, workspace=small)
    scores = torch.zeros(2, 2, 64, device="cuda")
    lse = torch.zeros(3, 8, device="cuda")
    for kw in (dict(scores=scores[0]), dict(scores=scores[:1]), dict(scores=scores.double()), dict(lse=lse[:2]),
               dict(scores=scores.transpose(1, 2))):
        d = dict(dict(scores=scores, lse=lse), **kw)
        with pytest.raises(ValueError):
            pad.weigh_tokens(c.q, c.k, d["lse"], c.table, c_lens, c.cu, d["scores"])
    for dst in (torch.zeros(3, 4).int().cuda(), torch.zeros(2, 4).long().cuda(), torch.zeros(2).int().cuda()):
        with pytest.raises(ValueError):
            pad.evict_tokens(scores, c.k, c.v, c.table, c_lens, dst, 32)
    with pytest.raises(ValueError):
        pad.evict_tokens(scores, c.k, c.v, c.table, c_lens, torch.zeros(2, 4).int().cuda(), 0)
    kv = torch.zeros(3, 2, 64).bfloat16().cuda()
    pos, inv = torch.zeros(3).int().cuda(), torch.ones(32, dtype=torch.float64, device="cuda")
    rope = dict(q=c.q, k=kv, v=kv, positions=pos, inv_freq=inv)
    for kw in (dict(q=c.q[:2]), dict(k=kv.float()), dict(k=kv[:, :1]), dict(positions=pos.long()), dict(positions=pos[:2]),
               dict(inv_freq=inv.float()), dict(axes=[0] * 31), dict(q=c.q.transpose(1, 2)), dict(axes=[300] * 32),
               dict(v=torch.zeros(3, 2, 68).bfloat16().cuda()[..., :64])):
        d = dict(rope, **kw)
        with pytest.raises(ValueError):
            pad.rope_append(d["q"], d["k"], d["v"], d["positions"], d["inv_freq"], c.k, c.v, c.table, c_lens, c.cu,
                            axes=d.get("axes"))
