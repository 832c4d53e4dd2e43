"""Session-cache operators at their edges: the precision of the attention weights,
what no element-wise bound over random values shows, and inputs that are not
finite, not there or not allowed."""
import math

import pytest
import torch

from prefix_aware_decode_b200 import _binding
from prefix_aware_decode_b200.session import SessionPool

import cache_ref as ref
from cache_ref import Cache

gpu = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ precision


def _attend(c, window=0, sinks=0, scale=None):
    """out in 64 bits, and the bound for weights kept to about 16 bits."""
    scale = scale or 1 / math.sqrt(c.D)
    out = torch.zeros(c.n, c.Hq, c.D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for s in range(len(c.kv)):
        r = slice(int(c.cu[s]), int(c.cu[s + 1]))
        for h in range(c.Hq):
            t, x, err = ref.logits(c, s, h, window, sinks, scale)
            if not len(t) or not c.rows[s]:
                continue
            v = c.tokens(c.v, s, h // (c.Hq // c.Hkv))[1]
            l = torch.logsumexp(x, 1, keepdim=True)
            p = torch.where(l > -math.inf, (x - l).exp(), 0.0)
            o, a = p @ v, p @ v.abs()
            out[r, h] = o
            # one rounding of the result, half a step (2^-8); a weight within 2^-16 of
            # itself (two bf16 parts), moved by twice the logits' error; 2^-15 for fp32 sums
            tol[r, h] = 2.0 ** -8 * o.abs() + (2.0 ** -16 + 2 * err + 2.0 ** -15) * a * (1 + 2.0 ** -7)
    return out, tol


PRECISION = [([40, 23, 9, 65], [19, 23, 5, 40]), ([31, 12], [1, 1]), ([150, 33, 260], [4, 1, 130])]


@gpu
@pytest.mark.parametrize("extra_pages", [1, 1100])  # the second: the form for long caches, whatever the rows
@pytest.mark.parametrize("heads", [(8, 2, 64), (16, 16, 64), (32, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("kv,rows", PRECISION)
def test_attend_weights_keep_more_than_one_bf16(kv, rows, heads, extra_pages):
    c = Cache(kv, rows, *heads, seed=61, extra_pages=extra_pages)
    out, _ = ref.run_attend(c)
    want, tol = _attend(c)
    ref.check(out, want, tol, "out")
    out, _ = ref.run_attend(c, 20, 3, 0.4)
    want, tol = _attend(c, 20, 3, 0.4)
    ref.check(out, want, tol, "out")


def test_one_bf16_of_the_weights_is_outside_that_bound():
    # the plain computation with weights of one bf16, everything else in 64 bits
    for kv, rows in PRECISION:
        c = Cache(kv, rows, 8, 2, 64, seed=61, device="cpu")
        want, tol = _attend(c)
        got = torch.zeros_like(want)
        for s in range(len(kv)):
            r = slice(int(c.cu[s]), int(c.cu[s + 1]))
            for h in range(c.Hq):
                _, x, _ = ref.logits(c, s, h, 0, 0, 1 / 8.0)
                p = (x - x.amax(1, keepdim=True)).exp()
                got[r, h] = p.bfloat16().double() @ c.tokens(c.v, s, h // 4)[1] / p.sum(1, keepdim=True)
        assert bool(((got.bfloat16().double() - want).abs() > tol).any()), (kv, rows)


# ------------------------------------------------------------------------------------------------ queries that are not numbers

# the form for few rows with one CTA and with a cluster for a row, whole items of one
# and of two tiles, items cut into parts
NAN_QUERIES = {
    "one CTA a row": ([100 + i for i in range(80)], [1] * 80, 1),
    "a cluster a row": ([1000, 40], [1, 1], 1),
    "mostly empty cluster": ([20], [1], 60),
    "one tile": ([60, 33], [5, 9], 1),
    "two tiles": ([100, 20], [64, 3], 1),
    "cut": ([9000, 700], [5, 60], 1),
    "cut into many parts": ([20000], [3], 1),
}


@gpu
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128), (2, 2, 64)])
@pytest.mark.parametrize("name", list(NAN_QUERIES))
def test_attend_a_nan_query_gives_nan_and_stays_alone(name, heads):
    kv, rows, extra = NAN_QUERIES[name]
    c = Cache(kv, rows, *heads, seed=71, extra_pages=extra)
    clean, clean_lse = ref.run_attend(c)
    assert not bool(clean.isnan().any()) and not bool(clean_lse.isnan().any())
    bad = [(0, 1), (c.n - 1, heads[0] - 1)]
    for r, h in bad:
        c.q[r, h, 3] = math.nan
    out, lse = ref.run_attend(c)
    hit = torch.zeros(lse.shape, dtype=torch.bool)
    for r, h in bad:
        hit[r, h] = True
    assert torch.equal(lse.isnan().cpu(), hit), name
    assert torch.equal(out.isnan().cpu(), hit[..., None].expand(out.shape)), name
    ok = ~hit.cuda()
    assert torch.equal(out[ok], clean[ok]) and torch.equal(lse[ok], clean_lse[ok])


@gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_attend_a_row_without_keys_is_empty_even_with_a_nan_query(rows):
    c = Cache([rows + 5, 0], [rows, rows], 4, 2, 64, seed=72)
    c.q[rows:] = math.nan  # session 1 has no cached tokens
    out, lse = ref.run_attend(c)
    assert bool((out[rows:] == 0).all()) and bool((lse[rows:] == -math.inf).all())
    assert not bool(out[:rows].isnan().any())


# ------------------------------------------------------------------------------------------------ weights of single columns


def _columns(D=64):
    """16 rows of 8 heads over 144 tokens: every row sees the first 128 tokens, so the
    128 (row, head) columns and 128 keys make one full tile.  A column's lse of -inf
    takes it out (it weighs nothing), which leaves one weight per key."""
    c = Cache([144], [16], 8, 1, D, seed=81)
    c.q.zero_()
    c.q[..., 0] = c.q[..., 1] = 1.0
    c.k.zero_()
    return c


def _put(c, x):
    """The logits of the first 128 tokens, with a scale of ln 2: x octaves, in two bf16 parts."""
    t = torch.arange(128)
    hi = x.bfloat16()
    lo = (x - hi.double()).bfloat16()
    c.k[c.table[0, t // 16].long(), 0, t % 16, 0] = hi
    c.k[c.table[0, t // 16].long(), 0, t % 16, 1] = lo
    return hi.double() + lo.double()


def _weigh_column(c, col, lse=0.0):
    l = torch.full((16, 8), -math.inf, device="cuda")
    l[col // 8, col % 8] = lse
    scores = torch.zeros(1, 1, 144, device="cuda")
    q, k, table, lens, cu = c.dev("q", "k", "table", "lens", "cu")
    ref.pad.weigh_tokens(q, k, l, table, lens, cu, scores, softmax_scale=math.log(2.0))
    return scores[0, 0, :128].double().cpu()


@gpu
def test_weigh_every_column_computes_the_same_weight():
    c = _columns()
    x = _put(c, torch.linspace(-1.0, 1.0, 128, dtype=torch.float64))
    scale = torch.tensor(math.log(2.0)).float() * torch.tensor(1.4426950408889634).float()
    want = 2.0 ** (x * scale.double())
    for col in range(128):
        got = _weigh_column(c, col)
        # the argument to half a step of numbers up to 1 (2^-24, times ln 2 in the weight),
        # the exponential and its last rounding: 2^-22 in all
        assert bool(((got - want).abs() <= 2.0 ** -22 * want).all()), (col, float(((got - want) / want).abs().max()))


@gpu
def test_weigh_every_column_over_the_whole_range_of_exponents():
    c = _columns()
    x = _put(c, torch.linspace(-160.0, 100.0, 128, dtype=torch.float64))
    want = 2.0 ** x
    for col in range(128):
        got = _weigh_column(c, col)
        # the scale is ln 2 log2 e in fp32: off by 2^-24 each way, on an argument of up to 160
        tol = want * 2.0 ** -15 + torch.where(x < -125.0, 2.0 ** -126, 0.0)  # below: flushed or not
        assert bool(((got - want).abs() <= tol).all()), col
    x = _put(c, torch.linspace(129.0, 400.0, 128, dtype=torch.float64))
    for col in range(128):
        assert bool((_weigh_column(c, col) == math.inf).all()), col


@gpu
def test_weigh_a_row_of_lse_minus_infinity_weighs_nothing():
    c = _columns()
    _put(c, torch.linspace(-3.0, 3.0, 128, dtype=torch.float64))
    assert bool((_weigh_column(c, 0, -math.inf) == 0).all())


@gpu
def test_weigh_a_nan_query_or_lse_reaches_every_score_it_draws_on():
    c = _columns()
    _put(c, torch.linspace(-3.0, 3.0, 128, dtype=torch.float64))
    for col in range(128):
        assert bool(_weigh_column(c, col, math.nan).isnan().all()), col
        c.q[col // 8, col % 8, 5] = math.nan
        assert bool(_weigh_column(c, col).isnan().all()), col
        c.q[col // 8, col % 8, 5] = 0.0


@gpu
def test_weigh_a_logit_equal_to_its_lse_weighs_exactly_one():
    c = _columns()
    _put(c, torch.zeros(128, dtype=torch.float64))
    for col in range(128):
        assert bool((_weigh_column(c, col) == 1.0).all()), col


# ------------------------------------------------------------------------------------------------ eviction and holes


@gpu
@pytest.mark.parametrize("kv,budget,sinks,recent", [(100, 40, 4, 8), (30, 64, 0, 0), (1500, 700, 3, 17), (48, 48, 0, 0)])
def test_evict_brings_no_stale_memory_out_of_a_hole(kv, budget, sinks, recent):
    D, Hkv = 64, 2
    c = Cache([kv], [1], 4, Hkv, D, seed=91)
    holes = [0, 1, (kv - 1) // 16]
    n_dst = -(-budget // 16)
    base = c.num_pages
    spare = torch.full((n_dst, Hkv, 16, D), math.nan).bfloat16()  # what the pages held before
    k0, v0 = torch.cat([c.k, spare]), torch.cat([c.v, spare])
    for i, j in enumerate(holes):
        c.table[0, j] = (-1, base + n_dst, 2 ** 31 - 1)[i]
    scores = torch.rand(1, Hkv, c.width * 16, generator=c.gen)
    kept = ref.evict(scores, [kv], budget, sinks, recent)[0]
    k, v = k0.cuda(), v0.cuda()
    table, lens, cu, q = c.dev("table", "lens", "cu", "q")
    dst = (base + torch.arange(n_dst).int()).view(1, -1).cuda()
    new, got, _ = ref.pad.evict_tokens(scores.cuda(), k, v, table, lens, dst, budget, sinks=sinks, recent=recent)
    m = min(kv, budget)
    assert new.tolist() == [m]
    for h in range(Hkv):
        assert got[0, h, :m].tolist() == kept[h]
        t = torch.tensor(kept[h])
        gone = torch.tensor([j in holes for j in (t // 16).tolist()])
        for pool, old in ((k, k0), (v, v0)):
            row = pool[base:, h].reshape(-1, D)[:m].cpu()
            assert bool((row[gone] == 0).all()), "a slot kept what its page held before"
            src = old[c.table[0, t[~gone] // 16].long(), h, t[~gone] % 16]
            assert torch.equal(row[~gone], src)
    out, lse = ref.pad.window_attend(q, k, v, dst, new, cu)
    assert not bool(out.isnan().any()) and not bool(lse.isnan().any())


# ------------------------------------------------------------------------------------------------ status


@gpu
def test_window_status_of_calls_that_do_nothing():
    c = Cache([20, 5], [0, 0], 8, 2, 64, seed=95)
    q, k, v, table, lens, cu = c.dev("q", "k", "v", "table", "lens", "cu")
    ws = ref.pad.window_workspace(q, k, table, lens, cu)
    ws.fill_(255)
    out, lse = ref.pad.window_attend(q, k, v, table, lens, cu, workspace=ws)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    assert ref.pad.window_status(ws) == ref.pad.PA_OK
    fresh = ref.pad.window_workspace(q, k, table, lens, cu)
    assert ref.pad.window_status(fresh) == ref.pad.PA_OK
    small = torch.full((256,), 255, dtype=torch.uint8, device="cuda")  # nothing is done: any workspace will do
    ref.pad.window_attend(q, k, v, table, lens, cu, workspace=small)
    assert ref.pad.window_status(small) == ref.pad.PA_OK


@gpu
def test_window_status_needs_no_workspace():
    c = Cache([2000], [40], 8, 2, 64, seed=96)
    ref.run_attend(c)
    s = torch.cuda.Stream()
    assert ref.pad.window_status() == ref.pad.window_status(device="cuda:0", stream=s) == ref.pad.PA_OK


# Waits of the kernels that give up at once (pa_session_fault): the call ends, its status
# says so, and the next one is clean.  (kv lengths, new rows, heads, the waits it comes to.)
# Between them the cases come to every wait: 3 (a ring slot's last use) needs more blocks
# a CTA than the ring holds, 1, 2, 4, 9 and 11 several items a CTA, 14 a block whose last
# keys no row sees (a cut item has it in one CTA only, which may not hold a whole block)
GIVE_UP = {
    "two tiles": ([3000, 900], [300, 200], (8, 2, 128), [5, 6, 7, 8, 12, 13, 15]),
    "one tile": ([20000], [3], (8, 2, 128), [3, 5, 6, 7, 10, 12, 13, 15, 16, 17]),
    "short items": ([300 + 7 * i for i in range(90)], [5] * 90, (8, 8, 64), [1, 2, 4, 10, 11, 12, 14, 16, 17]),
    "short items of two tiles": ([300 + 7 * i for i in range(40)], [290] * 40, (8, 8, 64), [1, 2, 4, 8, 9, 12, 15]),
}


@gpu
@pytest.mark.parametrize("name,wait", [(n, w) for n, x in GIVE_UP.items() for w in x[3]])
def test_attend_ends_when_a_wait_gives_up(name, wait):
    kv, rows, heads, _ = GIVE_UP[name]
    c = Cache(kv, rows, *heads, seed=101)
    q, k, v, table, lens, cu = c.dev("q", "k", "v", "table", "lens", "cu")
    ws = ref.pad.window_workspace(q, k, table, lens, cu)
    want = ref.pad.window_attend(q, k, v, table, lens, cu, workspace=ws)
    assert ref.pad.window_status(ws) == ref.pad.window_status() == ref.pad.PA_OK
    assert _binding.lib().pa_session_fault(wait) == ref.pad.PA_OK
    ref.pad.window_attend(q, k, v, table, lens, cu, workspace=ws)
    assert ref.pad.window_status(ws) == ref.pad.PA_ERR_TIMEOUT
    assert ref.pad.window_status() == ref.pad.PA_ERR_TIMEOUT
    assert ref.pad.window_status() == ref.pad.PA_OK  # told once
    got = ref.pad.window_attend(q, k, v, table, lens, cu, workspace=ws)
    assert ref.pad.window_status(ws) == ref.pad.window_status() == ref.pad.PA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


WEIGH_GIVE_UP = {
    "keys stream": ([5000 + 64 * i for i in range(20)], [1] * 20, (8, 8, 64), [1, 3, 4, 5, 6, 7, 8, 9, 10, 11, 13, 14]),
    # 16 + 12 pairs of key blocks of 4 heads: one item a CTA, so no queue or K slot is used again (1, 4, 14)
    "rows stream": ([4000, 3000], [1000, 900], (8, 4, 128), [3, 5, 6, 7, 8, 9, 10, 11, 12, 13]),
}


@gpu
@pytest.mark.parametrize("name,wait", [(n, w) for n, x in WEIGH_GIVE_UP.items() for w in x[3]])
def test_weigh_ends_when_a_wait_gives_up(name, wait):
    kv, rows, heads, _ = WEIGH_GIVE_UP[name]
    c = Cache(kv, rows, *heads, seed=102)
    q, k, v, table, lens, cu = c.dev("q", "k", "v", "table", "lens", "cu")
    _, lse = ref.pad.window_attend(q, k, v, table, lens, cu)
    scores = [torch.zeros(len(kv), heads[1], c.width * 16, device="cuda") for _ in range(3)]
    ref.pad.weigh_tokens(q, k, lse, table, lens, cu, scores[0])
    assert ref.pad.weigh_status() == ref.pad.PA_OK
    assert _binding.lib().pa_session_fault(wait) == ref.pad.PA_OK
    ref.pad.weigh_tokens(q, k, lse, table, lens, cu, scores[1])
    assert ref.pad.weigh_status() == ref.pad.PA_ERR_TIMEOUT
    assert ref.pad.weigh_status() == ref.pad.PA_OK
    ref.pad.weigh_tokens(q, k, lse, table, lens, cu, scores[2])
    assert ref.pad.weigh_status() == ref.pad.PA_OK
    assert torch.equal(scores[0], scores[2])


# ------------------------------------------------------------------------------------------------ every page counts


def _one_dim_a_page(c):
    """V of a page is zero but in one dim, the page's index modulo D: an output dim is the
    weight of a few pages, all of one sign, so that a page that is lost or taken for
    another shows at any length (over random V a lost block of 128 keys disappears in the
    bound of 20000)."""
    g = torch.Generator().manual_seed(3)
    for s, n in enumerate(c.kv):
        for j in range(-(-n // 16)):
            p = int(c.table[s, j])
            if not 0 <= p < c.num_pages:
                continue
            c.v[p, :, :min(16, n - 16 * j)] = 0
            c.v[p, :, :min(16, n - 16 * j), j % c.D] = (1 + torch.rand(1, generator=g)).bfloat16()
    return c


LONG = [([20011, 7], [1, 1], (4, 1, 128)), ([9000], [5], (4, 1, 128)), ([5000, 4097], [300, 17], (4, 2, 64)),
        ([33000], [2], (8, 8, 64)), ([700] * 5, [1, 3, 1, 90, 1], (8, 2, 128)), ([1900, 1000], [1, 1], (8, 8, 128))]


@gpu
@pytest.mark.parametrize("kv,rows,heads", LONG)
def test_attend_counts_every_page(kv, rows, heads):
    c = _one_dim_a_page(Cache(kv, rows, *heads, seed=65))
    out, _ = ref.run_attend(c)
    want, tol = _attend(c)
    ref.check(out, want, tol, "out")
    out, _ = ref.run_attend(c, 1500, 40)
    want, tol = _attend(c, 1500, 40)
    ref.check(out, want, tol, "out")


@pytest.mark.parametrize("kv,rows,heads", LONG[:2] + LONG[3:])
def test_a_lost_or_swapped_page_is_outside_the_bound(kv, rows, heads):
    g = torch.Generator().manual_seed(4)
    c = _one_dim_a_page(Cache(kv, rows, *heads[:2], heads[2], seed=65, device="cpu"))
    want, tol = _attend(c)
    n = -(-kv[0] // 16) - 1
    for j in [0, n - 1] + torch.randint(0, n, (2,), generator=g).tolist():
        p, other = int(c.table[0, j]), int(c.table[0, (j + 1) % n])
        held = c.v.clone()
        for lost in (True, False):
            c.v[p] = 0 if lost else held[other]
            got, _ = _attend(c)
            c.v.copy_(held)
            row = slice(0, rows[0])
            bad = ((got - want).abs() > tol)[row].any(dim=2)
            assert bool(bad.all()), (j, lost)  # in every row and head


# ------------------------------------------------------------------------------------------------ a long chunk among single rows


@gpu
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 8, 64), (8, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 9)])
def test_attend_one_long_chunk_among_single_rows(heads, window, sinks):
    # few rows a session on average: the form for few rows also takes the session with many
    rows = [1] * 30 + [25, 0, 0, 1]
    kv = [40 + 17 * i for i in range(30)] + [300, 50, 0, 90]
    c = Cache(kv, rows, *heads, seed=97)
    out, _ = ref.run_attend(c, window, sinks)
    want, tol = _attend(c, window, sinks)
    ref.check(out, want, tol, "out")


# ------------------------------------------------------------------------------------------------ tables


def test_session_pool_tables_of_a_given_width():
    pool = SessionPool(40)
    for s, n in enumerate([100, 0, 17]):
        pool.open(s)
        pool.append(s, n)
    table, lens = pool.tables(max_pages=9)
    assert table.shape == (3, 9) and table.dtype == "int32" and lens.tolist() == [100, 0, 17]
    narrow, _ = pool.tables()
    assert (table[:, :7] == narrow).all() and (table[:, 7:] == -1).all()
    assert pool.tables([1], max_pages=1)[0].tolist() == [[-1]]
    for bad in (6, 0, -1):
        with pytest.raises(ValueError):
            pool.tables(max_pages=bad)


@gpu
def test_evict_into_the_pages_that_the_pool_gives():
    # every session shorter than the budget: its table is narrower than the budget's pages
    pool = SessionPool(40)
    for s, n in enumerate([37, 20]):
        pool.open(s)
        pool.append(s, n)
    budget = 64
    table, lens = (torch.from_numpy(t).cuda() for t in pool.tables())
    kp = torch.randn(40, 2, 16, 64, device="cuda").bfloat16()
    vp = torch.randn_like(kp)
    old = kp.clone()
    pool.compact([0, 1], budget)
    dst, want = pool.tables(max_pages=budget // 16)
    scores = torch.rand(2, 2, 64, device="cuda")
    new, kept, _ = ref.pad.evict_tokens(scores, kp, vp, table, lens, torch.from_numpy(dst).cuda(), budget)
    assert new.tolist() == want.tolist() == [37, 20]
    for s in range(2):
        for t in range(int(new[s])):
            assert torch.equal(kp[int(dst[s, t // 16]), :, t % 16], old[int(table[s, t // 16]), :, t % 16])


# ------------------------------------------------------------------------------------------------ autograd


@gpu
def test_tensors_that_require_grad_are_refused():
    c = Cache([20, 5], [2, 1], 8, 2, 64, seed=98)
    q, k, v, table, lens, cu = c.dev("q", "k", "v", "table", "lens", "cu")
    out, lse = ref.pad.window_attend(q, k, v, table, lens, cu)
    scores = torch.zeros(2, 2, 64, device="cuda")
    pos, inv = torch.zeros(3).int().cuda(), torch.ones(32, dtype=torch.float64, device="cuda")
    kv = torch.zeros(3, 2, 64, device="cuda").bfloat16()
    dst = torch.full((2, 4), -1).int().cuda()

    def grad(t):
        return t.clone().requires_grad_()

    calls = [lambda: ref.pad.window_attend(grad(q), k, v, table, lens, cu),
             lambda: ref.pad.window_attend(q, grad(k), v, table, lens, cu),
             lambda: ref.pad.window_attend(q, k, grad(v), table, lens, cu),
             lambda: ref.pad.window_attend(q, k, v, table, lens, cu, out=grad(out)),
             lambda: ref.pad.weigh_tokens(grad(q), k, lse, table, lens, cu, scores),
             lambda: ref.pad.weigh_tokens(q, k, grad(lse), table, lens, cu, scores),
             lambda: ref.pad.weigh_tokens(q, k, lse, table, lens, cu, grad(scores)),
             lambda: ref.pad.rope_append(grad(q), kv, kv, pos, inv, k, v, table, lens, cu),
             lambda: ref.pad.rope_append(q, kv, grad(kv), pos, inv, k, v, table, lens, cu),
             lambda: ref.pad.evict_tokens(grad(scores), k, v, table, lens, dst, 32)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="grad"):
            call()
    with torch.no_grad():  # no graph is asked for
        o, _ = ref.pad.window_attend(grad(q), k, v, table, lens, cu)
    assert torch.equal(o, out)
    with torch.inference_mode():
        o, _ = ref.pad.window_attend(q, k, v, table, lens, cu)
        ref.pad.weigh_tokens(q, k, lse, table, lens, cu, torch.zeros_like(scores))
    assert torch.equal(o, out)


@gpu
def test_tensors_that_a_call_changes_count_a_version():
    c = Cache([20, 5], [2, 1], 8, 2, 64, seed=99)
    q, k, v, table, lens, cu = c.dev("q", "k", "v", "table", "lens", "cu")
    scores = torch.zeros(2, 2, 64, device="cuda")
    pos, inv = torch.zeros(3).int().cuda(), torch.ones(32, dtype=torch.float64, device="cuda")
    kv = torch.zeros(3, 2, 64, device="cuda").bfloat16()
    out, lse = ref.pad.window_attend(q, k, v, table, lens, cu)
    x = torch.zeros_like(scores)
    dst = torch.full((2, 4), -1).int().cuda()

    def grows(call, *changed, same=()):
        before = [t._version for t in changed], [t._version for t in same]
        call()
        assert all(t._version > n for t, n in zip(changed, before[0])), "a changed tensor kept its version"
        assert [t._version for t in same] == before[1]

    grows(lambda: ref.pad.window_attend(q, k, v, table, lens, cu, out=out, lse=lse), out, lse, same=(q, k, v))
    grows(lambda: ref.pad.weigh_tokens(q, k, lse, table, lens, cu, scores), scores, same=(q, k, lse))
    grows(lambda: ref.pad.rope_append(q, kv, kv, pos, inv, k, v, table, lens, cu, q_out=q), q, k, v, same=(kv,))
    grows(lambda: ref.pad.evict_tokens(scores, k, v, table, lens, dst, 32, scores_out=x), k, v, x, same=(scores,))


# ------------------------------------------------------------------------------------------------ scale


def test_a_scale_whose_multiple_by_log2_e_overflows_is_refused():
    b = _binding.PaSessions(2, 3, 8, 2, 64, 16, 4, 9, 4096, 8192, 12288)
    p, L = 1 << 20, _binding.lib()
    for scale in (2.4e38, 3.4e38, math.inf):
        assert L.pa_window_attend(b, 0, 0, scale, p, p, p, p, 1 << 30, p, p, None) == _binding.PA_ERR_INVALID
        assert L.pa_weigh_tokens(b, 0, 0, scale, p, p, p, p, 64, None) == _binding.PA_ERR_INVALID
