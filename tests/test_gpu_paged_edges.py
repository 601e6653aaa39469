"""Paged serving at its edges: rows that reach the end of their table row, requests with fewer positions than
tokens, infinities and large values in long caches, sums near the end of fp32, many small requests."""
import math
import random

import pytest
import torch

from tests import paged_ref as R
from tests.test_gpu_paged import BF16, F16, P, compare, i32, paged_case, run_attn, run_tables  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows past the end of their table row

def test_a_row_past_its_table_row_leaves_the_others_in_place(P):
    """Row 0 holds all its 4 pages of 16 and asks for one more token: it is not served and reported, and the
    tokens of the rows after it are still those at rows 1 and 2 of the packed projections."""
    table, stack = [[0, 1, 2, 3], [5, -1, -1, -1], [4, -1, -1, -1]], [6, -1, -1, -1, -1, -1, -1]
    got = run_tables(P, 16, 3, [64, 3, 3], [1, 1, 1], [4, 1, 1], table, stack, 1)
    assert got == dict(held=[4, 1, 1], table=table, stack=stack, count=1, cu=[0, 1, 2, 3], kv=[0, 4, 4],
                       slots=[-1, 5 * 16 + 3, 4 * 16 + 3], pos=[64, 3, 3], status=True)


def test_a_row_of_negative_length_leaves_the_others_in_place(P):
    table, stack = [[0, 1, 2, 3], [5, -1, -1, -1], [4, -1, -1, -1]], [6, -1, -1, -1, -1, -1, -1]
    got = run_tables(P, 16, 4, [-2, 3, 3], [2, 1, 1], [4, 1, 1], table, stack, 1)
    assert got == dict(held=[4, 1, 1], table=table, stack=stack, count=1, cu=[0, 2, 3, 4], kv=[0, 4, 4],
                       slots=[-1, -1, 5 * 16 + 3, 4 * 16 + 3], pos=[-2, -1, 3, 3], status=True)


@pytest.mark.parametrize("B", [3, 300, 2100, 4096])
@pytest.mark.parametrize("fits", [True, False])
def test_rows_past_their_table_rows_at_random(P, B, fits):
    """Rows that ask for more than their table row holds among others, in one block and in two grids.  Where all
    tokens fit the packed rows theirs are counted; where they do not, the others' alone are (as paged_ref has it)."""
    r, page, M = random.Random(B), 16, 6
    cached, new, held, long = [], [], [], []
    for b in range(B):
        c = r.randint(0, M * page)
        over = b % 3 == 1
        n = r.randint(M * page - c + 1, M * page) if over and c > 0 else min(r.choice((0, 1, 5)), M * page - c)
        cached.append(c)
        new.append(n)
        held.append(-(-c // page))
        long.append(c + n > M * page)
    total = sum(held)
    ids = list(range(total + 40))
    r.shuffle(ids)
    at, table = 0, []
    for h in held:
        table.append([ids[at + j] if j < h else -5 for j in range(M)])
        at += h
    stack = ids[total:] + [-3] * total
    args = (cached, new, held, table, stack, 40)
    T = sum(new) if fits else sum(n for n, x in zip(new, long) if not x)
    got, want = run_tables(P, page, T, *args), R.tables(page, T, *args)
    assert any(long) and want["status"] and sum(new) > sum(n for n, x in zip(new, long) if not x)
    if fits:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        slots, pos = [], []
        for b in range(B):
            for i in range(new[b]):
                p = cached[b] + i
                pos.append(p)
                slots.append(want["table"][b][p // page] * page + p % page if want["kv"][b] > 0 else -1)
        want.update(cu=cu, slots=slots, pos=pos)
    assert not [x for x in want if got[x] != want[x]]


def test_a_full_row_does_not_move_the_others(P):
    """A captured decode loop in which row 0 reaches its last position: the other rows' keys, values and outputs
    stay those of their own projections, replay after replay."""
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    n, H, G, dh, page = 3, 4, 2, 64, 16
    cache = PagedCache(H, G, dh, n, 64, 60, 80, page_size=page, rope=P.rope_plan(dh, 0))
    torch.manual_seed(7)
    first = torch.randn(73, H + 2 * G, dh, device="cuda").half()
    cache.begin(i32([60, 10, 3]), 73, 60)
    cache.attend(0, *first.split([H, G, G], 1), torch.empty(73, H, dh, device="cuda").half())
    hist = [[first[a:b, H:]] for a, b in ((0, 60), (60, 70), (70, 73))]
    x = torch.randn(n, H + 2 * G, dh, device="cuda").half()
    out, ones = torch.empty(n, H, dh, device="cuda").half(), i32([1] * n)
    one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")

    def step():
        cache.begin(ones, n, 1)
        cache.attend(0, *x.split([H, G, G], 1), out)

    step()
    for b in range(n):
        hist[b].append(x[b:b + 1, H:].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert P.pi_last_device_status() == 0
    for i in range(20):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        assert cache.cu.tolist() == [0, 1, 2, 3]
        full = i >= 3                              # 61 + 3 positions are 64
        assert cache.cached.tolist() == [64 if full else 62 + i, 12 + i, 5 + i]
        assert P.pi_last_device_status() == (1 if full else 0)
        for b in range(n):
            if b == 0 and full:
                assert int(cache.slots[0]) == -1 and bool((out[0] == 0).all())
                continue
            hist[b].append(x[b:b + 1, H:].clone())
            kv = torch.cat(hist[b])
            t = torch.arange(kv.shape[0], device="cuda")
            ids = cache.table[b][t // page].long()
            assert torch.equal(cache.kcache[0][ids, :, t % page], kv[:, :G])
            assert torch.equal(cache.vcache[0][ids, :, t % page], kv[:, G:])
            want, _, tol, _ = R.attention(x[b:b + 1, :H], kv[:, :G].transpose(0, 1)[None], kv[:, G:].transpose(0, 1)[None],
                                          one, [0, 1], [kv.shape[0]])
            R.check(out[b:b + 1], want, tol, f"step {i} row {b}")


# ------------------------------------------------------------------ windows and requests that see nothing

@pytest.mark.parametrize("n,kv", [(200, 100), (700, 500), (900, 2)])
@pytest.mark.parametrize("window", [0, 1, 90, 2 ** 30, 2 ** 31 - 1])
def test_more_tokens_than_positions_under_any_window(P, n, kv, window):
    """A window of the largest int is no window; up to 29 items of a request whose first ones see nothing."""
    q, kc, vc, table, cu, _ = paged_case([(n, n), (1, 40)], 8, 1, 64, F16, 16, seed=21)
    compare(P, (q, kc, vc, table, cu, [kv, 40]), window=window)


@pytest.mark.parametrize("window", [0, 1, 300])
def test_requests_of_many_items(P, window):
    """Requests of 69 and more items, counted by formula: behind cached positions, and with fewer positions than tokens."""
    q, kc, vc, table, cu, kv = paged_case([(1100, 1900), (1, 500), (1300, 1300), (20, 90), (1200, 1200)], 16, 1, 64, F16, 16,
                                          seed=33, window=window)
    kv[2], kv[4] = 900, 10
    compare(P, (q, kc, vc, table, cu, kv), window=window)


@pytest.mark.parametrize("B", [385, 1500, 4096])
def test_thousands_of_small_requests(P, B):
    r = random.Random(B)
    lens = [(n, n + r.randint(0, 30)) for n in (r.choice((0, 1, 1, 1, 2)) for _ in range(B))]
    compare(P, paged_case(lens, 4, 2, 64, F16, 16, seed=B, junk=math.nan))


# ------------------------------------------------------------------ infinities, large values, sums near the end of fp32

def test_an_infinity_in_a_long_cache_costs_the_others_nothing(P):
    """400 requests over the same pages but for one, whose own page holds an infinity: its rows are exact (32 of a
    warp meet the infinity), the others keep their bits, and no wait runs out under a limit of 50 ms."""
    B, H, dh, page, keys = 400, 32, 64, 128, 40000
    g = torch.Generator(device="cuda").manual_seed(5)
    used = -(-keys // page)
    kc, vc = (torch.randn(used + 1, 1, page, dh, generator=g, device="cuda").half() for _ in range(2))
    q = torch.randn(B, H, dh, generator=g, device="cuda").half()
    table = torch.arange(used, device="cuda").int().repeat(B, 1)
    own = 7
    table[own, 2] = used
    kv, cu = [keys] * B, list(range(B + 1))
    want = run_attn(P, q, kc, vc, table, cu, kv)
    assert P.pi_last_device_status() == 0
    vc[used, 0, 3, 5] = math.inf
    P.pi_debug_set_wait_timeout(50_000_000)
    try:
        got = run_attn(P, q, kc, vc, table, cu, kv)
        torch.cuda.synchronize()
    finally:
        P.pi_debug_set_wait_timeout(0)
    assert P.pi_last_device_status() == 0
    rest = torch.arange(B, device="cuda") != own
    assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(got[1][rest], want[1][rest])
    exact, el, tol, ltol = R.attention(q[own:own + 1], kc, vc, table[own:own + 1], [0, 1], [keys])
    fine = torch.arange(dh, device="cuda") != 5
    R.check(got[0][own:own + 1][..., fine], exact[..., fine], tol[..., fine], "other elements")
    R.check(got[1][own:own + 1], el, ltol, "lse")
    assert bool((got[0][own, :, 5] == math.inf).all())


@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("lens,H,G,window", [([(300, 700)], 4, 1, 0), ([(130, 400), (1, 900)], 8, 8, 150), ([(1, 3000)], 4, 2, 0)])
def test_bad_values_among_masked_places(P, lens, H, G, window, dt, which):
    """Every 37th position holds a NaN or an infinity in one element: the rows that see one are as the formula has
    them, the others as without it."""
    q, kc, vc, table, cu, kv = paged_case(lens, H, G, 64, dt, 16, seed=17, window=window)
    clean = (q, kc, vc, table, cu, kv)
    want, wl, tol, ltol = R.attention(*clean, window)
    kb, vb = kc.clone(), vc.clone()
    hit = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    for b, n in enumerate(kv):
        new = cu[b + 1] - cu[b]
        for i, t in enumerate(range(n - 20, max(0, n - 250), -37)):
            g, e = i % G, (5 * i) % 64
            (kb, vb)[which - 1][table[b, t // 16].long(), g, t % 16, e] = math.nan if i % 2 == 0 else math.inf
            for j in range(new):
                p = n - new + j
                if t <= p and (window == 0 or t > p - window):
                    heads = slice(g * (H // G), (g + 1) * (H // G))
                    if which == 1:
                        hit[cu[b] + j, heads] = True
                    else:
                        hit[cu[b] + j, heads, e] = True
    out, lse = run_attn(P, q, kb, vb, table, cu, kv, window)
    assert P.pi_last_device_status() == 0
    R.check(out[~hit], want[~hit], tol[~hit], "the rest")
    ok = ~hit.any(-1) if which == 1 else torch.ones_like(lse, dtype=torch.bool)
    R.check(lse[ok], wl[ok], ltol[ok], "lse")
    if which == 2:
        assert not bool(torch.isfinite(out[hit]).any())
    assert 0 < int(hit.sum())


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("lens,H,G,window", [([(300, 700), (1, 90)], 8, 2, 0), ([(1, 3000)], 4, 1, 0), ([(150, 900)], 2, 2, 333)])
def test_many_bad_values_and_their_kinds(P, lens, H, G, window, dt):
    """Far more bad values than one: column 5 holds +inf from position 400 on (at every position), column 6 +inf at 401
    and -inf at 450, column 7 NaN and infinities, column 8 -inf at 640 alone.  An output element is the sum of what its
    column shows the row; the other elements and the log-sums are as without."""
    q, kc, vc, table, cu, kv = paged_case(lens, H, G, 64, dt, 16, seed=19, window=window)
    want, wl, tol, ltol = R.attention(q, kc, vc, table, cu, kv, window)
    inf, bad = math.inf, []
    n = kv[0]
    bad += [(5, t, inf) for t in range(400, n)] + [(6, 401, inf), (6, 450, -inf), (8, 640, -inf)]
    bad += [(7, t, math.nan if t % 3 == 0 else inf) for t in range(500, min(n, 560), 2)]
    for e, t, x in bad:
        vc[table[0, t // 16].long(), 0, t % 16, e] = x
    for i in range(lens[0][0]):
        p = n - lens[0][0] + i
        lo = max(0, p - window + 1) if window > 0 else 0
        for e in (5, 6, 7, 8):
            seen = [x for f, t, x in bad if f == e and lo <= t <= p]
            if seen:
                want[i, :H // G, e] = sum(seen)
    out, lse = run_attn(P, q, kc, vc, table, cu, kv, window)
    assert P.pi_last_device_status() == 0 and not bool(torch.isfinite(want).all())
    R.check(out, want, tol, "out")
    R.check(lse, wl, ltol, "lse")
    assert torch.equal(out.double()[torch.isinf(want)], want[torch.isinf(want)])    # of the right sign


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("many", [1, 200])
@pytest.mark.parametrize("lens,H,G", [([(200, 700)], 4, 2), ([(1, 3000)], 8, 1)])
def test_infinite_keys(P, lens, H, G, many, dt):
    """Keys with an infinity: rows whose query points along it have no number left, rows that point the other way are
    as with a key that they give no weight."""
    q, kc, vc, table, cu, kv = paged_case(lens, H, G, 64, dt, 16, seed=20)
    q[..., 4] = torch.where(torch.arange(H, device="cuda") % 2 == 0, -2.0, 2.0).to(dt)
    q[:, :, 4] *= torch.where(torch.arange(q.shape[0], device="cuda") % 3 == 0, -1.0, 1.0).to(dt)[:, None]
    far, n = kc.clone(), kv[0]
    at = range(100, 100 + many)
    for t in at:
        page = table[0, t // 16].long()
        far[page, :, t % 16, 4] = 2000.0       # scores of -500 and less where the query points the other way
        kc[page, :, t % 16, 4] = math.inf
    want, wl, tol, ltol = R.attention(q, far, vc, table, cu, kv)
    out, lse = run_attn(P, q, kc, vc, table, cu, kv)
    assert P.pi_last_device_status() == 0
    away = (q[..., 4] < 0)
    assert bool(away.any()) and not bool(away.all())
    R.check(out[away], want[away], tol[away], "out")
    R.check(lse[away], wl[away], ltol[away], "lse")
    assert bool(torch.isnan(out[~away]).all()) and not bool(torch.isfinite(lse[~away]).any())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_queries_that_are_not_finite(P, bad):
    """They reach their own rows only, and none where the row sees nothing."""
    q, kc, vc, table, cu, _ = paged_case([(90, 90), (1, 2000), (3, 40)], 8, 2, 64, F16, 16, seed=27)
    kv = [60, 2000, 40]                       # the first 30 tokens see nothing
    want, wl, tol, ltol = R.attention(q, kc, vc, table, cu, kv)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[10, 3] = hit[50, :] = hit[90, 5] = hit[92, 0] = True
    q[hit, 7] = bad
    out, lse = run_attn(P, q, kc, vc, table, cu, kv)
    hit[10] = False
    R.check(out[~hit], want[~hit], tol[~hit], "out")
    R.check(lse[~hit], wl[~hit], ltol[~hit], "lse")
    assert bool((out[:30] == 0).all()) and bool((lse[:30] == -math.inf).all())
    assert bool(torch.isnan(out[hit]).all()) and not bool(torch.isfinite(lse[hit]).any())
    assert P.pi_last_device_status() == 0


@pytest.mark.parametrize("a", range(1, 8))
def test_parts_whose_sums_add_up_past_fp32(P, a):
    """Two keys, 83.5 nats above the rest, in any two of eight key tiles: where their parts are summed under the
    maximum of what came before, each part's sum of weights is 2^127.5, and the two parts' is past fp32."""
    for b in range(a):
        q, kc, vc, table, cu, kv = paged_case([(1, 1001)], 1, 1, 64, BF16, 16, seed=23)
        q.zero_()
        q[..., 0] = 16.0
        kc.zero_()
        vc *= 2.0 ** -6
        for t in (128 * a + 5, 128 * b + 77):
            kc[table[0, t // 16].long(), 0, t % 16, 0] = 41.75          # q . k / 8 = 83.5
        compare(P, (q, kc, vc, table, cu, kv))


def test_two_parts_whose_sums_add_up_past_fp32(P):
    """The same in items of thirty tiles that a border cuts in two."""
    B, G, n = 12, 16, 3800
    q, kc, vc, table, cu, kv = paged_case([(1, n)] * B, G, G, 64, BF16, 16, seed=24)
    q.zero_()
    q[..., 0] = 16.0
    kc.zero_()
    vc *= 2.0 ** -6
    r = random.Random(1)
    for b in range(B):
        for g in range(G):
            for t in r.sample(range(n), 2):
                kc[table[b, t // 16].long(), g, t % 16, 0] = 41.75
    compare(P, (q, kc, vc, table, cu, kv))


@pytest.mark.parametrize("lens", [[(1, 1001), (1, 300)], [(200, 900)]])
@pytest.mark.parametrize("value", [65504.0, -65504.0])
def test_values_at_the_end_of_fp16(P, lens, value):
    """Any mean of equal values is that value: weights rounded up must not push it over the largest fp16."""
    q, kc, vc, table, cu, kv = paged_case(lens, 16, 4, 64, F16, 16, seed=25, gain=2.0)
    kc *= torch.linspace(0.1, 1.0, kc.shape[0], device="cuda")[:, None, None, None].half()
    vc.fill_(value)
    compare(P, (q, kc, vc, table, cu, kv), scale=0.5)


@pytest.mark.parametrize("lens", [[(1, 1001), (1, 300)], [(200, 900)]])
def test_values_near_the_end_of_bf16(P, lens):
    """Values of up to 3.2e38: their weighted mean is finite, whatever factor the weights carry on the way."""
    q, kc, vc, table, cu, kv = paged_case(lens, 4, 2, 64, BF16, 16, seed=26)
    vc.copy_((vc.float().clamp(-3.2, 3.2) * 1e38))
    compare(P, (q, kc, vc, table, cu, kv))


# ------------------------------------------------------------------ parts of an item that meet

@pytest.mark.parametrize("lens,H,G", [([(1, 3800)] * 12, 16, 16), ([(1, 2600 + 100 * i) for i in range(9)], 64, 8),
                                      ([(150, 1900), (70, 600), (1, 4000)], 16, 4)])
def test_parts_that_meet_give_the_same_bits(P, lens, H, G):
    """Items that one border cuts, both parts done at nearly the same time: whichever block adds them, and whether it
    finds the other part there or waits for it, every call gives one result, which is right."""
    case = paged_case(lens, H, G, 64, BF16, 16, seed=31)
    q, kc, vc, table, cu, kv = case
    d, pg = P.paged_desc(H, len(kv), q.shape[0], max(n for n, _ in lens), table.shape[1]), P.page_desc(kc, vc)
    ws = torch.zeros(P.pi_paged_workspace_bytes(d, pg), dtype=torch.uint8, device="cuda")
    first = compare(P, case, ws=ws)
    for _ in range(60):
        again = run_attn(P, *case, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------ the cache object and the binding

def test_outputs_beside_their_queries(P):
    """Queries and outputs in one buffer: alternate parts of its rows, and one after the other."""
    q, kc, vc, table, cu, kv = paged_case([(1, 700), (90, 90), (2, 33)], 8, 2, 64, F16, 16, seed=29)
    want, _ = compare(P, (q, kc, vc, table, cu, kv))
    T, row = q.shape[0], 8 * 64
    both = torch.full((T, 2 * row), 3.0, device="cuda").half()
    for a, b in ((0, row), (row, 0)):
        x, y = (both[:, i:i + row].unflatten(1, (8, 64)) for i in (a, b))
        x.copy_(q)
        run_attn(P, x, kc, vc, table, cu, kv, out=y)
        assert torch.equal(y, want) and torch.equal(x, q)
    for a, b in ((0, T), (T, 0)):
        line = both.view(2 * T, 8, 64)
        x, y = line[a:a + T], line[b:b + T]
        x.copy_(q)
        run_attn(P, x, kc, vc, table, cu, kv, out=y)
        assert torch.equal(y, want) and torch.equal(x, q)
    for y in (x, line[1:1 + T] if a == 0 else line[T - 1:2 * T - 1]):
        with pytest.raises(P.PiError):
            run_attn(P, x, kc, vc, table, cu, kv, out=y)


def test_rotation_in_place_of_packed_projections(P):
    """Queries turned where they lie, between the keys and values that the same call stores."""
    torch.manual_seed(2)
    T, H, G, dh = 75, 6, 2, 64
    packed = torch.randn(T, (H + 2 * G) * dh, device="cuda").half()
    q, k, v = (x.unflatten(1, (-1, dh)) for x in packed.split([H * dh, G * dh, G * dh], dim=1))
    pos, slots = torch.arange(T, device="cuda").int() * 77, torch.arange(T, device="cuda")
    plan, got = P.rope_plan(dh, 32), []
    for out in (torch.empty_like(q), q):
        kc, vc = (torch.zeros(5, G, 16, dh, device="cuda").half() for _ in range(2))
        P.pi_rope_store(plan, P.page_desc(kc, vc), q, k, v, pos, slots, out, kc, vc)
        got.append((out.clone(), kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and P.pi_last_device_status() == 0
    with pytest.raises(P.PiError):
        P.pi_rope_store(plan, P.page_desc(kc, vc), q, k, v, pos, slots, packed[:, 2 * dh:][:, :H * dh].unflatten(1, (H, dh)), kc, vc)


def test_block_tables_of_another_width_are_refused(P):
    """A table with more columns than the descriptor says would be read with the wrong row stride."""
    q, kc, vc, table, cu, kv = paged_case([(1, 30), (1, 60)], 2, 1, 64, F16, 16)
    wide = torch.cat([table, table], 1)
    pg, d = P.page_desc(kc, vc), P.paged_desc(2, 2, 2, 1, table.shape[1])
    ws = torch.zeros(P.pi_paged_workspace_bytes(d, pg), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="block_table"):
        P.pi_paged_attn(d, pg, q, kc, vc, wide, i32(cu), i32(kv), torch.empty_like(q), None, ws)
    with pytest.raises(ValueError, match="block_table"):
        one, two = i32([1]), i32([1, 1])
        P.pi_block_tables(P.tables_desc(2, 16, 8, 3, 2), two, two, two, two.clone(), i32([[0] * 4] * 2), i32([0] * 8), one,
                          one.clone(), i32([0] * 3), two.clone(), torch.empty(2, dtype=torch.int64, device="cuda"), two.clone())


def _small(**kw):
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    return PagedCache(4, 2, 64, 2, 64, 20, 30, page_size=16, **kw)


def _qkv(T):
    return torch.randn(T, 8, 64, device="cuda").half().split([4, 2, 2], 1)


def test_attend_takes_the_tokens_of_its_step(P):
    """Fewer rows than the step's tokens would leave the last step's queries in the rest."""
    cache = _small()
    cache.begin(i32([5, 4]), 9, 5)
    cache.attend(0, *_qkv(9), torch.empty(9, 4, 64, device="cuda").half())
    cache.begin(i32([2, 1]), 3, 2)
    for T in (2, 4, 0):
        with pytest.raises(ValueError):
            cache.attend(0, *_qkv(T), torch.empty(3, 4, 64, device="cuda").half())
    cache.attend(0, *_qkv(3), torch.empty(3, 4, 64, device="cuda").half())
    assert P.pi_last_device_status() == 0


def test_rows_keep_no_more_than_they_have(P):
    """keep above what a row has does not make positions visible that were never stored, and one below 0 (reported)
    leaves the row as it was."""
    cache = _small()
    cache.begin(i32([5, 4]), 9, 5)
    cache.attend(0, *_qkv(9), torch.empty(9, 4, 64, device="cuda").half())
    cache.begin(i32([1, 1]), 2, 1, i32([40, 3]))
    cache.attend(0, *_qkv(2), torch.empty(2, 4, 64, device="cuda").half())
    assert cache.cached.tolist() == [6, 4] and cache.kv_len.tolist() == [6, 4] and P.pi_last_device_status() == 0
    cache.begin(i32([1, 1]), 2, 1, i32([-3, 4]))
    assert cache.cu.tolist() == [0, 1, 2] and cache.kv_len.tolist() == [0, 5]
    assert P.pi_last_device_status() == 1 and cache.cached.tolist()[0] == 6
    cache.begin(i32([1, 1]), 2, 1)
    assert cache.cached.tolist()[0] == 7 and cache.kv_len.tolist()[0] == 7 and P.pi_last_device_status() == 0


def test_a_step_of_fewer_tokens_than_its_largest_chunk(P):
    """max_new is an upper bound: a loop may pass its chunk size for a step of fewer tokens."""
    a, b = _small(), _small()
    x, y = _qkv(3), torch.empty(3, 4, 64, device="cuda").half()
    a.begin(i32([2, 1]), 3, 20)
    a.attend(0, *x, y)
    z = torch.empty_like(y)
    b.begin(i32([2, 1]), 3, 2)
    b.attend(0, *x, z)
    assert torch.equal(y, z) and P.pi_last_device_status() == 0
