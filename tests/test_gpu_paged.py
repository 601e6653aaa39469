"""Parity of the paged-serving operators on the GPU: block tables exactly, rotary
positions, store and attention within bounds derived from their roundings."""
import math
import random

import pytest
import torch

from tests import paged_ref as R

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_ffn_layer_gb300 as P
    return P


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ block tables

def run_tables(P, page, max_tokens, cached, new, held, table, stack, count, in_place=False):
    B, M = len(cached), len(table[0])
    d = P.tables_desc(B, page, len(stack), M, max_tokens)
    t, s, h, c = i32(table), i32(stack), i32(held), i32([count])
    ho, co = (h, c) if in_place else (torch.full_like(h, 77), torch.full_like(c, 77))
    cu, kv = i32([77] * (B + 1)), i32([77] * B)
    slots = torch.full((max_tokens,), 77, dtype=torch.int64, device="cuda")
    pos = i32([77] * max_tokens)
    P.pi_block_tables(d, i32(cached), i32(new), h, ho, t, s, c, co, cu, kv, slots, pos)
    st = P.pi_last_device_status()
    return dict(held=ho.tolist(), table=t.tolist(), stack=s.tolist(), count=co.item(), cu=cu.tolist(), kv=kv.tolist(),
                slots=slots.tolist(), pos=pos.tolist(), status=st == 1)


def some_tables(rng, B, M, page, spare, n_hi):
    cached, new, held, table, nxt = [], [], [], [], 0
    for _ in range(B):
        h = rng.randint(0, M)
        what = rng.random()
        c = 0 if what < 0.3 else rng.randint(0, h * page)
        n = rng.choice((0, 1, 1, rng.randint(0, n_hi)))
        cached.append(c)
        new.append(min(n, M * page - c))
        held.append(h)
        table.append([nxt + j if j < h else -5 for j in range(M)])
        nxt += h
    total = nxt + spare
    ids = list(range(total))
    rng.shuffle(ids)
    table = [[ids[x] if x >= 0 else -5 for x in r] for r in table]
    return cached, new, held, table, ids[nxt:] + [-3] * nxt, spare


@pytest.mark.parametrize("B,M,page,spare,n_hi", [(1, 1, 16, 1, 1), (1, 4, 128, 5, 300), (3, 9, 16, 2, 60), (31, 5, 32, 40, 100),
                                                 (33, 40, 16, 300, 200), (1023, 6, 16, 700, 40), (1025, 7, 64, 2000, 200),
                                                 (4096, 5, 16, 6000, 30)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_match_row_by_row(P, B, M, page, spare, n_hi, in_place):
    rng = random.Random(B * 31 + M)
    args = some_tables(rng, B, M, page, spare, n_hi)
    for T in (sum(args[1]), sum(args[1]) + 7):
        assert run_tables(P, page, T, *args, in_place=in_place) == R.tables(page, T, *args)


def test_tables_without_tokens(P):
    args = ([0, 0], [0, 0], [2, 0], [[3, 4], [-1, -1]], [0, -1, -1, -1, -1], 1)
    assert run_tables(P, 16, 0, *args) == R.tables(16, 0, *args)


@pytest.mark.parametrize("what", ["negative", "long", "held", "past", "count", "overflow"])
def test_tables_inconsistent_rows(P, what):
    """Such a row is left as it is and reported; the others are served."""
    cached, new, held = [5, 16, 0, 40], [11, 3, 20, 2], [1, 1, 2, 3]
    table = [[8, -1, -1], [9, -1, -1], [10, 11, -1], [12, 13, 14]]
    stack, count, T = [1, 2, 3] + [-1] * 12, 3, 36
    if what == "negative":
        new[1] = -4
    elif what == "long":
        new[1] = 33
    elif what == "held":
        held[1] = 4
    elif what == "past":
        T = 30
    elif what == "count":
        count = 16
        stack = list(range(15))
    else:
        cached[3], new[3], stack, count = 0, 0, [1, 2, 3, 4], 3
    got, want = run_tables(P, 16, T, cached, new, held, table, stack, count), R.tables(16, T, cached, new, held, table, stack, count)
    assert want["status"] and got == want


def test_tables_grow_step_by_step(P):
    """In-place decode steps: rows cross page borders as the pool runs dry and is refilled by an ended row."""
    B, M, page = 5, 6, 16
    cached, held, table = [0] * B, [0] * B, [[-1] * M for _ in range(B)]
    stack, count = list(range(11)), 11
    for step in range(70):
        new = [1 if step % (b + 1) == 0 else 0 for b in range(B)]
        if step == 50:
            cached[0], new[0] = 0, 0
        cached = [min(c, M * page - n) for c, n in zip(cached, new)]
        got = run_tables(P, page, 5, cached, new, held, table, stack, count)
        assert got == R.tables(page, 5, cached, new, held, table, stack, count)
        cached = [k if k else c for k, c in zip(got["kv"], cached)]
        held, table, stack, count = got["held"], got["table"], got["stack"], got["count"]


# ------------------------------------------------------------------ rotary positions and store

def make_cache(pages, kv_heads, page, dh, dt, order, fill=None):
    shape = (pages, kv_heads, page, dh) if order == "hnd" else (pages, page, kv_heads, dh)
    t = torch.randn(shape, device="cuda").to(dt) if fill is None else torch.full(shape, fill, dtype=dt, device="cuda")
    return t if order == "hnd" else t.transpose(1, 2)


@pytest.mark.parametrize("T,H,G,dh,rot,inter,inp,dt,page,order,scaling", [
    (1, 1, 1, 64, 64, False, F16, F16, 16, "hnd", {}),
    (7, 12, 12, 64, 32, True, F32, F16, 16, "nhd", {}),
    (33, 64, 8, 128, 128, False, BF16, BF16, 32, "hnd", dict(scaling="ramp", factor=16.0, original_max=8192, high=32.0, mscale=1.3)),
    (130, 24, 8, 128, 48, True, F32, BF16, 64, "nhd", dict(scaling="linear", factor=3.0)),
    (65, 5, 5, 128, 16, False, F16, BF16, 128, "hnd", dict(base=500000.0)),
    (19, 96, 96, 128, 112, False, BF16, F16, 16, "nhd", dict(scaling="blend", factor=8.0, original_max=8192)),
    (64, 16, 1, 64, 0, True, F16, F16, 16, "hnd", {}),
    (515, 56, 56, 128, 128, True, F16, F16, 16, "nhd", {}),
])
def test_rope_store(P, T, H, G, dh, rot, inter, inp, dt, page, order, scaling):
    torch.manual_seed(T)
    qkv = torch.randn(T, (H + 2 * G) * dh, device="cuda").to(inp)
    q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv.split([H * dh, G * dh, G * dh], dim=1))
    pos = torch.randint(0, 1 << 20, (T,), device="cuda")
    pos[0] = (1 << 31) - 1 if T > 1 else 0
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, device="cuda")[:T]
    slots[T // 2::5] = -1
    kc, vc = make_cache(pages, G, page, dh, dt, order), make_cache(pages, G, page, dh, dt, order)
    wide = torch.full((T, H * dh + 24), 9.0, dtype=dt, device="cuda")
    qo = wide[:, 8:8 + H * dh].unflatten(1, (H, dh))
    k0, v0 = kc.clone(), vc.clone()
    plan = P.rope_plan(dh, rot, interleaved=inter, **scaling)
    P.pi_rope_store(plan, P.page_desc(kc, vc), q, k, v, pos.int(), slots, qo, kc, vc)
    assert P.pi_last_device_status() == 0
    f = R.frequencies(rot, scaling.get("base", 10000.0), scaling.get("scaling", "none"), scaling.get("factor", 1.0),
                      scaling.get("original_max", 0.0), scaling.get("low", 1.0), scaling.get("high", 4.0))
    u, tiny, ms = R.half_step(dt), 2.0 ** -25, scaling.get("mscale", 1.0)
    # the reference's own angle, p f in fp64, is off by 2^-53 p f: below 2.4e-7 for p < 2^31
    want, slack = R.rotate(q, pos, f, inter, ms)
    R.check(qo, want, u * want.abs() + (1 + u) * 1.4 * slack + tiny, "q")
    assert bool((wide[:, :8] == 9).all()) and bool((wide[:, 8 + H * dh:] == 9).all())
    want, slack = R.rotate(k, pos, f, inter, ms)
    kx, vx, sx = k0.double(), v0.clone(), torch.zeros(k0.shape, dtype=torch.float64, device="cuda")
    live = slots >= 0
    pg, off = slots[live] // page, slots[live] % page
    kx[pg, :, off], sx[pg, :, off] = want[live], (u * want.abs() + (1 + u) * 1.4 * slack + tiny)[live]
    vx[pg, :, off] = v[live].to(dt)
    R.check(kc, kx, sx, "keys")
    assert torch.equal(vc, vx)


def test_rope_in_place_and_alone(P):
    torch.manual_seed(1)
    q = torch.randn(37, 6, 64, device="cuda").half()
    cache = P.page_desc(*[make_cache(4, 2, 16, 64, F16, "hnd") for _ in range(2)])
    pos = torch.arange(37, device="cuda").int() * 1000
    out = torch.empty_like(q)
    plan = P.rope_plan(64, 32, interleaved=True)
    P.pi_rope_store(plan, cache, q, None, None, pos, None, out, None, None)
    P.pi_rope_store(plan, cache, q, None, None, pos, None, q, None, None)
    assert torch.equal(q, out)
    k, v = torch.randn(2, 37, 2, 64, device="cuda").half().unbind(0)
    kc, vc = make_cache(4, 2, 16, 64, F16, "hnd", 0.0), make_cache(4, 2, 16, 64, F16, "hnd", 0.0)
    slots = torch.arange(37, device="cuda")
    P.pi_rope_store(P.rope_plan(64, 0), P.page_desc(kc, vc), None, k, v, pos, slots, None, kc, vc)
    assert torch.equal(kc.transpose(1, 2).reshape(-1, 2, 64)[:37], k)
    assert torch.equal(vc.transpose(1, 2).reshape(-1, 2, 64)[:37], v)


def test_rope_slot_outside_the_cache(P):
    k = torch.ones(3, 1, 64, device="cuda").half()
    kc, vc = make_cache(2, 1, 16, 64, F16, "hnd", 0.0), make_cache(2, 1, 16, 64, F16, "hnd", 0.0)
    for bad in (32, 1 << 40, -2):
        P.pi_rope_store(P.rope_plan(64, 0), P.page_desc(kc, vc), None, k, k, i32([0, 0, 0]),
                        torch.tensor([5, bad, -1], device="cuda"), None, kc, vc)
        assert P.pi_last_device_status() == 1
        assert float(kc.float().sum()) == 64 and float(vc.float().sum()) == 64


# ------------------------------------------------------------------ attention

def paged_case(lens, H, G, dh, dt, page, order="hnd", seed=0, junk=None, window=0, gain=1.0, spare=3):
    """lens: (new tokens, keys) per request.  Positions that no token sees are filled with junk."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    used = [-(-k // page) for _, k in lens]
    pages, M = sum(used) + spare, max(max(used), 1) + 1
    perm = torch.randperm(pages, generator=g, device="cuda")
    kc, vc = (make_cache(pages, G, page, dh, dt, order) for _ in range(2))
    kc.copy_(torch.randn(kc.shape, generator=g, device="cuda") * gain)
    vc.copy_(torch.randn(vc.shape, generator=g, device="cuda"))
    table = torch.full((len(lens), M), -1, dtype=torch.int32, device="cuda")
    seen = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    at, cu = 0, [0]
    for b, (n, k) in enumerate(lens):
        table[b, :used[b]] = perm[at:at + used[b]].int()
        at += used[b]
        cu.append(cu[-1] + n)
        lo = max(0, k - n - window + 1) if window > 0 else 0
        t = torch.arange(lo if n > 0 else k, k, device="cuda")
        seen[table[b][t // page].long(), t % page] = True
    if junk is not None:
        hide = ~seen[:, None, :, None].expand(kc.shape)
        kc[hide] = junk
        vc[hide] = junk
    q = torch.randn(cu[-1], H, dh, generator=g, device="cuda").to(dt)
    return q, kc, vc, table, cu, [k for _, k in lens]


def run_attn(P, q, kc, vc, table, cu, kv, window=0, scale=0.0, max_new=None, extra=0, ws=None, out=None):
    T, H = q.shape[:2]
    n = max([b - a for a, b in zip(cu, cu[1:])] + [1]) if max_new is None else max_new
    d = P.paged_desc(H, len(kv), T, min(n, max(T, 1)), table.shape[1], window=window, scale=scale)
    pg = P.page_desc(kc, vc)
    ws = torch.zeros(P.pi_paged_workspace_bytes(d, pg), dtype=torch.uint8, device="cuda") if ws is None else ws
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((T, H), 5.0, device="cuda")
    P.pi_paged_attn(d, pg, q, kc, vc, table, i32(cu), i32(kv), out, lse, ws)
    return out, lse


def compare(P, case, window=0, scale=0.0, status=0, **kw):
    q, kc, vc, table, cu, kv = case
    out, lse = run_attn(P, q, kc, vc, table, cu, kv, window, scale, **kw)
    assert P.pi_last_device_status() == status
    want, wl, tol, ltol = R.attention(q, kc, vc, table, cu, kv, window, scale or None)
    R.check(out, want, tol, "out")
    R.check(lse, wl, ltol, "lse")
    return out, lse


RAGGED = [(1, 1), (1, 2), (0, 5), (1, 127), (1, 128), (1, 129), (3, 3), (2, 17), (1, 400), (5, 255), (0, 0), (1, 257)]


@pytest.mark.parametrize("H,G,dh,dt,page,order", [
    (1, 1, 64, F16, 16, "hnd"), (12, 12, 64, BF16, 32, "nhd"), (8, 1, 128, F16, 16, "nhd"), (64, 8, 128, BF16, 64, "hnd"),
    (6, 2, 128, F16, 128, "hnd"), (32, 1, 64, BF16, 16, "nhd"), (14, 2, 64, F16, 32, "hnd"), (128, 1, 128, F16, 16, "hnd")])
def test_decode_and_short_rows(P, H, G, dh, dt, page, order):
    compare(P, paged_case(RAGGED, H, G, dh, dt, page, order, junk=math.nan))


@pytest.mark.parametrize("lens,H,G,dh,dt,page", [
    ([(128, 128)], 1, 1, 128, F16, 16), ([(129, 129)], 2, 1, 64, BF16, 16), ([(257, 300)], 3, 3, 128, BF16, 32),
    ([(33, 1000)], 8, 1, 128, F16, 64), ([(100, 100), (1, 700), (31, 32)], 8, 2, 128, F16, 16),
    ([(260, 515)], 1, 1, 64, F16, 128), ([(17, 17), (64, 64), (63, 191), (1, 1)], 5, 1, 64, BF16, 16),
    ([(700, 701)], 2, 2, 128, F16, 16), ([(7, 2500)], 24, 8, 128, BF16, 32), ([(1, 5000)], 4, 4, 64, F16, 16)])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_chunks(P, lens, H, G, dh, dt, page, window):
    compare(P, paged_case(lens, H, G, dh, dt, page, seed=3, junk=math.inf, window=window), window=window)


def test_rows_that_see_nothing(P):
    """More tokens than positions: the first ones see nothing; a refused request (no positions) none."""
    q, kc, vc, table, cu, kv = paged_case([(5, 5), (40, 40), (300, 300), (2, 2)], 4, 2, 64, F16, 16, junk=math.nan)
    out, lse = compare(P, (q, kc, vc, table, cu, [3, 0, 130, 2]))
    assert bool((out[:2] == 0).all()) and bool((lse[5:45] == -math.inf).all())


@pytest.mark.parametrize("gain,scale", [(1.0, 1.0), (8.0, 0.125), (30.0, 0.3), (0.01, 0.125)])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_sharp_and_flat_scores(P, gain, scale, dt):
    """Scores of hundreds (one key takes all, maxima that keep rising) and of nearly nothing."""
    q, kc, vc, table, cu, kv = paged_case([(1, 900), (70, 640)], 6, 2, 64, dt, 16, gain=gain, seed=5)
    kc *= torch.linspace(0.1, 1.0, kc.shape[0], device="cuda")[:, None, None, None].to(dt)
    compare(P, (q, kc, vc, table, cu, kv), scale=scale)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("jump", [10.0, 60.0, 85.0, 200.0, 2000.0])
@pytest.mark.parametrize("lens,H,G", [([(1, 700)], 4, 2), ([(200, 900)], 2, 2), ([(1, 3000), (40, 1000)], 4, 1)])
def test_scores_that_jump(P, lens, H, G, dt, jump):
    """Keys whose scores lie `jump` above all before them, in the midst of a tile and at its start, and small
    values: weights relative to what was the maximum leave fp16's range, then fp32's."""
    q, kc, vc, table, cu, kv = paged_case(lens, H, G, 64, dt, 16, seed=6)
    q[..., 0] = 16.0
    kc *= 0.1
    vc *= 2.0 ** -6
    for b, n in enumerate(kv):
        for i, t in enumerate((256, 330, 512, 650)):
            if t < n:
                kc[table[b, t // 16].long(), :, t % 16, 0] = jump * (i + 1) / 2.0    # q . k / 8 = jump (i + 1)
    compare(P, (q, kc, vc, table, cu, kv))


def test_small_weights_keep_their_mass(P):
    """One key of weight 1 and 20000 of weight 2^-22 each: together 0.5 %."""
    n = 20001
    q, kc, vc, table, cu, kv = paged_case([(1, n)], 1, 1, 64, F16, 16)
    q.zero_()
    q[..., 0] = 8.0
    kc.zero_()
    vc.fill_(1.0)
    kc[..., 0] = -22.0 * math.log(2.0)
    kc[table[0, 0].long(), 0, 0, 0] = 0.0
    vc[table[0, 0].long(), 0, 0, :] = 0.0
    compare(P, (q, kc, vc, table, cu, kv))


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_value_reaches_only_the_tokens_that_see_it(P, bad):
    """Token 60 of a chunk stored a non-finite key or value: earlier tokens are as without it."""
    for which in (1, 2):
        case = paged_case([(100, 170), (1, 40)], 8, 2, 64, F16, 16, seed=9)
        page = case[3][0, 130 // 16].long()
        case[which][page, 1, 130 % 16, 3] = bad
        q, kc, vc, table, cu, kv = case
        out, lse = run_attn(P, *case)
        want, wl, tol, ltol = R.attention(q, kc, vc, table, cu, kv)
        see = torch.zeros(101, 8, dtype=torch.bool, device="cuda")
        see[60:100, 4:] = True
        R.check(out[~see], want[~see], tol[~see], "tokens before")
        R.check(lse[~see], wl[~see], ltol[~see], "lse before")
        if which == 2:
            R.check(out[see][:, :3], want[see][:, :3], tol[see][:, :3], "other elements")
        hit = out[see][:, 3] if which == 2 else out[see]
        assert not bool(torch.isfinite(hit).any()) or (which == 1 and bad == math.inf)
    assert P.pi_last_device_status() == 0


def test_strided_rows_streams_and_graphs(P):
    """Queries inside a packed projection, outputs inside a wider buffer, no lse, a side stream, a graph; the bits stay."""
    H, G, dh = 8, 2, 128
    q, kc, vc, table, cu, kv = paged_case([(1, 700), (90, 90), (1, 33)], H, G, dh, BF16, 16, "nhd", seed=2)
    ref, _ = compare(P, (q, kc, vc, table, cu, kv))
    T = q.shape[0]
    packed = torch.randn(T, (H + 2 * G) * dh, device="cuda").bfloat16()
    packed[:, :H * dh] = q.flatten(1)
    wide = torch.full((T, H * dh + 16), 3.0, device="cuda").bfloat16()
    qv, ov = packed[:, :H * dh].unflatten(1, (H, dh)), wide[:, 8:8 + H * dh].unflatten(1, (H, dh))
    d, pg = P.paged_desc(H, 3, T, 90, table.shape[1]), P.page_desc(kc, vc)
    ws = torch.zeros(P.pi_paged_workspace_bytes(d, pg), dtype=torch.uint8, device="cuda")
    cut, kvt = i32(cu), i32(kv)
    go = lambda: P.pi_paged_attn(d, pg, qv, kc, vc, table, cut, kvt, ov, None, ws)  # noqa: E731
    go()
    assert torch.equal(ov, ref) and bool((wide[:, :8] == 3).all()) and bool((wide[:, -8:] == 3).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    wide.fill_(3.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        go()
    side.synchronize()
    assert torch.equal(ov, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        wide.fill_(3.0)
        graph.replay()
        assert torch.equal(ov, ref)
    kvt[0] = 500                       # lengths are read at replay
    graph.replay()
    again, _ = run_attn(P, q, kc, vc, table, cu, [500] + kv[1:])
    assert torch.equal(ov, again)


def test_same_bits_every_time(P):
    case = paged_case([(1, 3000), (300, 1500), (1, 77), (9, 2222)], 16, 4, 64, F16, 32, seed=8)
    q, kc, vc, table, cu, kv = case
    d, pg = P.paged_desc(16, 4, q.shape[0], 300, table.shape[1]), P.page_desc(kc, vc)
    ws = torch.zeros(P.pi_paged_workspace_bytes(d, pg), dtype=torch.uint8, device="cuda")
    first = run_attn(P, *case, ws=ws)
    for _ in range(20):
        again = run_attn(P, *case, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_pages_past_4_gib(P):
    """A cache whose offsets pass 32 bits in elements and in bytes: the pages at its end."""
    G, page, dh = 8, 64, 128
    pages = (1 << 32) // (G * page * dh) + 40
    kc, vc = (torch.empty(pages, G, page, dh, dtype=F16, device="cuda") for _ in range(2))
    ids = torch.tensor([[pages - 1, 0, pages - 7, 33000 % pages], [pages - 2, pages // 2, pages - 3, 5]], dtype=torch.int32,
                       device="cuda")
    assert pages * G * page * dh > 1 << 32
    for c in (kc, vc):
        c[ids.long().flatten()] = torch.randn(8, G, page, dh, device="cuda").half()
    T = 200
    k, v = torch.randn(2, T, G, dh, device="cuda").half().unbind(0)
    q = torch.randn(T + 1, 16, dh, device="cuda").half()
    pos = torch.arange(T, device="cuda")
    slots = ids[0].long()[pos // page] * page + pos % page
    P.pi_rope_store(P.rope_plan(dh, 0), P.page_desc(kc, vc), None, k, v, pos.int(), slots, None, kc, vc)
    assert torch.equal(vc[slots // page, :, slots % page], v) and P.pi_last_device_status() == 0
    compare(P, (q, kc, vc, ids, [0, T, T + 1], [T, 250]))


def test_page_outside_the_cache_reads_as_zeros(P):
    q, kc, vc, table, cu, kv = paged_case([(1, 100), (40, 60)], 4, 2, 64, F16, 16)
    zero = 0                                 # a page of zeros that stands for the bad ids
    good = table.clone()
    kc = torch.cat([torch.zeros_like(kc[:1]), kc])
    vc = torch.cat([torch.zeros_like(vc[:1]), vc])
    good[good >= 0] += 1
    bad = good.clone()
    good[0, 2], good[1, 1] = zero, zero
    bad[0, 2], bad[1, 1] = -4, kc.shape[0] + (1 << 20)
    want = run_attn(P, q, kc, vc, good, cu, kv)
    assert P.pi_last_device_status() == 0
    got = run_attn(P, q, kc, vc, bad, cu, kv)
    assert P.pi_last_device_status() == 1
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_inconsistent_rows_are_left_out(P):
    q, kc, vc, table, cu, kv = paged_case([(2, 50), (3, 40), (1, 30)], 4, 2, 64, F16, 16)
    good, _ = run_attn(P, q, kc, vc, table, cu, kv)
    assert P.pi_last_device_status() == 0
    out, lse = run_attn(P, q, kc, vc, table, cu, [kv[0], table.shape[1] * 16 + 1, kv[2]])    # too many positions
    assert P.pi_last_device_status() == 1
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:]) and bool((out[2:5] == 0).all())
    out, _ = run_attn(P, q, kc, vc, table, [0, 2, 1, 6], kv, max_new=3)                       # decreasing, then too many
    assert P.pi_last_device_status() == 1
    assert torch.equal(out[:2], good[:2]) and bool((out[2:] == 5).all())
    out, _ = run_attn(P, q, kc, vc, table, [0, 2, 5, 9], kv, max_new=3)                       # past the rows
    assert P.pi_last_device_status() == 1
    assert torch.equal(out[:5], good[:5]) and bool((out[5:] == 5).all())


def test_rows_past_the_last_request_stay(P):
    q, kc, vc, table, cu, kv = paged_case([(2, 50), (3, 40)], 4, 2, 64, F16, 16)
    more = torch.cat([q, torch.full_like(q[:3], math.nan)])
    out, lse = run_attn(P, more, kc, vc, table, cu, kv)
    good, gl = run_attn(P, q, kc, vc, table, cu, kv)
    assert torch.equal(out[:5], good) and bool((out[5:] == 5).all()) and bool((lse[5:] == 5).all())


def test_tables_store_and_attention_together(P):
    """Two requests prefill in chunks and decode beside each other through all three operators; the last
    step's rows match dense causal attention over the rotated history."""
    torch.manual_seed(4)
    B, H, G, dh, page, M = 2, 8, 2, 64, 16, 8
    pages = 12
    kc, vc = make_cache(pages, G, page, dh, F16, "hnd", math.nan), make_cache(pages, G, page, dh, F16, "hnd", math.nan)
    pg, plan = P.page_desc(kc, vc), P.rope_plan(dh, 32)
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    stack, count, held = torch.arange(pages, device="cuda").int(), i32([pages]), i32([0, 0])
    kv, f = i32([0, 0]), R.frequencies(32, 10000.0)
    hist = [([], []) for _ in range(B)]
    for new in ([20, 7], [30, 1], [1, 40], [1, 1]):
        T = sum(new)
        td, ad = P.tables_desc(B, page, pages, M, T), P.paged_desc(H, B, T, max(new), M)
        cu, slots, pos = i32([0] * (B + 1)), torch.empty(T, dtype=torch.int64, device="cuda"), i32([0] * T)
        nkv = torch.empty_like(kv)
        P.pi_block_tables(td, kv, i32(new), held, held, table, stack, count, count, cu, nkv, slots, pos)
        q, k, v = torch.randn(T, H + 2 * G, dh, device="cuda").half().split([H, G, G], 1)
        qo, out = torch.empty(T, H, dh, device="cuda").half(), torch.empty(T, H, dh, device="cuda").half()
        P.pi_rope_store(plan, pg, q, k, v, pos, slots, qo, kc, vc)
        ws = torch.zeros(P.pi_paged_workspace_bytes(ad, pg), dtype=torch.uint8, device="cuda")
        P.pi_paged_attn(ad, pg, qo, kc, vc, table, cu, nkv, out, None, ws)
        kv, at = nkv, 0
        for b in range(B):
            p = torch.arange(T, device="cuda")[at:at + new[b]] - at + sum(x.shape[0] for x in hist[b][0])
            hist[b][0].append(R.rotate(k[at:at + new[b]], p, f, False)[0].half())
            hist[b][1].append(v[at:at + new[b]])
            kk, vv = torch.cat(hist[b][0]), torch.cat(hist[b][1])
            qq = R.rotate(q[at:at + new[b]], p, f, False)[0].half()
            n = kk.shape[0]
            one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
            want, _, tol, _ = R.attention(qq, kk.transpose(0, 1)[None], vv.transpose(0, 1)[None], one, [0, new[b]], [n])
            # a rotated value may round the other way than the reference's: one more half step on keys and queries
            # moves a score by at most 2 u scale sum |q k|, which the doubled bound and 2^-7 A cover
            R.check(out[at:at + new[b]], want, 2 * tol + 2.0 ** -7, f"request {b}")
            at += new[b]
    assert P.pi_last_device_status() == 0
    assert kv.tolist() == [52, 49] and count.item() == pages - 4 - 4


def test_paged_cache_serves_chunks_and_decodes(P):
    """Two layers behind one set of tables: prompts in chunks, then single tokens, a request that ends and one that
    takes its row, a pool that runs dry; every step's rows match the dense reference over the same history."""
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    torch.manual_seed(11)
    n, H, G, dh = 3, 6, 2, 64
    cache = PagedCache(H, G, dh, n, 100, 40, 80, layers=2, page_size=16, num_pages=9, dtype=BF16, rope=P.rope_plan(dh, 16))
    f = R.frequencies(16, 10000.0)
    hist = [[([], []) for _ in range(2)] for _ in range(n)]
    have = [0] * n
    for step, (new, keep) in enumerate([([40, 7, 0], None), ([20, 30, 5], None), ([1, 1, 1], None), ([1, 0, 40], None),
                                        ([1, 33, 1], [61 + 1, 0, 6]), ([1, 1, 40], None)]):
        if keep is not None:
            for b in range(n):
                if keep[b] < have[b]:
                    hist[b], have[b] = [([], []), ([], [])], 0
        T = sum(new)
        cache.begin(i32(new), T, max(new), None if keep is None else i32(keep))
        served = [k > 0 or m == 0 for k, m in zip(cache.kv_len.tolist(), new)]
        for layer in range(2):
            q, k, v = torch.randn(T, H + 2 * G, dh, device="cuda").split([H, G, G], 1)
            out = cache.attend(layer, q, k, v, torch.empty(T, H, dh, device="cuda").bfloat16())
            at = 0
            for b in range(n):
                rows = slice(at, at + new[b])
                at += new[b]
                if new[b] == 0:
                    continue
                if not served[b]:
                    assert bool((out[rows] == 0).all())
                    continue
                p = torch.arange(new[b], device="cuda") + have[b]
                # the stored keys are read back, so that the reference attends to the same rounded values
                slot = cache.slots[rows]
                pg, off = slot // 16, slot % 16
                kk, vv = cache.kcache[layer][pg, :, off], cache.vcache[layer][pg, :, off]
                want, slack = R.rotate(k[rows], p, f, False)
                u = R.half_step(BF16)
                R.check(kk, want, u * want.abs() + (1 + u) * 1.4 * slack + 2.0 ** -25, "stored keys")
                hist[b][layer][0].append(kk)
                hist[b][layer][1].append(vv)
                ks, vs = torch.cat(hist[b][layer][0]), torch.cat(hist[b][layer][1])
                want, _, tol, _ = R.attention(cache.q[rows], ks.transpose(0, 1)[None], vs.transpose(0, 1)[None],
                                              torch.zeros(1, 1, dtype=torch.int32, device="cuda"), [0, new[b]], [ks.shape[0]])
                R.check(out[rows], want, tol, f"step {step} layer {layer} request {b}")
        have = [h + m if s else h for h, m, s in zip(have, new, served)]
        assert cache.cached.tolist() == have
        # pages held and pages free make up the pool
        assert int(cache.held.sum()) + cache.free_count.item() == 9
    assert P.pi_last_device_status() == 0


def test_paged_example_runs(P, capsys):
    from activation_sparse_ffn_layer_gb300 import paged
    paged.main(["--config", "c1", "--requests", "3", "--prompt", "70", "--chunk", "32", "--tokens", "3", "--layers", "2"])
    assert "3 requests" in capsys.readouterr().out


def test_a_captured_decode_step_goes_on(P):
    """A decode step (tables, store, attention, state in place) replayed as a graph: every replay's outputs are the
    eager cache's bits, over page borders and past the end of the pool."""
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    n, H, G, dh, T = 3, 8, 2, 64, 20
    make = lambda: PagedCache(H, G, dh, n, 64, T, 2 * T, page_size=16, num_pages=8, rope=P.rope_plan(dh))  # noqa: E731
    a, b = make(), make()
    torch.manual_seed(3)
    first = torch.randn(T + 10 + 3, H + 2 * G, dh, device="cuda").half()
    x = torch.randn(n, H + 2 * G, dh, device="cuda").half()
    outs = []
    for c in (a, b):
        c.begin(i32([T, 10, 3]), T + 13, T)
        q, k, v = first.split([H, G, G], 1)
        c.attend(0, q, k, v, torch.empty(T + 13, H, dh, device="cuda").half())
    out = torch.empty(n, H, dh, device="cuda").half()
    ones = i32([1] * n)

    def step(c, o):
        c.begin(ones, n, 1)
        c.attend(0, *x.split([H, G, G], 1), o)

    step(b, out.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, out)
    eager = torch.empty_like(out)
    step(a, eager)
    for i in range(40):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        step(a, eager)
        assert torch.equal(out, eager) and torch.equal(a.cached, b.cached) and torch.equal(a.slots[:n], b.slots[:n]), i
    assert int((a.kv_len == 0).sum()) > 0 and P.pi_last_device_status() == 0


@pytest.mark.parametrize("H,G,lens", [(4, 4, [(1, 3000), (1, 2900)]), (2, 2, [(300, 2000)]), (8, 1, [(1, 20000)])])
@pytest.mark.parametrize("which", [1, 2])
def test_cut_items_with_bad_values(P, H, G, lens, which):
    """A non-finite key or value in one part of items that many blocks share: those rows are not finite, the others
    right, call after call on one workspace, and so is a good call after them."""
    good = paged_case(lens, H, G, 64, F16, 16, seed=12)
    q, kc, vc, table, cu, kv = good
    d, pg = P.paged_desc(H, len(kv), q.shape[0], max(n for n, _ in lens), table.shape[1]), P.page_desc(kc, vc)
    ws = torch.zeros(P.pi_paged_workspace_bytes(d, pg), dtype=torch.uint8, device="cuda")
    want = run_attn(P, *good, ws=ws)
    for at in (3, 700, kv[0] - lens[0][0] - 1):
        bad = [x.clone() if torch.is_tensor(x) else x for x in good]
        bad[which][table[0, at // 16].long(), 0, at % 16, 5] = math.nan
        for _ in range(6):
            out, lse = run_attn(P, *bad, ws=ws)
            see = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
            see[:lens[0][0], :H // G] = True
            hit = out[see][:, 5] if which == 2 else out[see]
            assert bool(torch.isnan(hit).all())
            # rows without it: the same keys in the same parts, so the same bits
            assert torch.equal(out[~see], want[0][~see]) and torch.equal(lse[~see], want[1][~see])
        again = run_attn(P, *good, ws=ws)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert P.pi_last_device_status() == 0


@pytest.mark.parametrize("lens,H,G", [([(1, 5000), (1, 300)], 8, 2), ([(300, 4000)], 4, 2)])
def test_waits_that_run_out(P, lens, H, G):
    """With a wait limit of 1 ns the first wait that is not satisfied at once gives up: the blocks wait for their own
    copies and products, free their tensor memory and return, and the status is PI_ERR_TIMEOUT.  After a zero fill of
    the workspace the same call gives the bits of a clean run."""
    case = paged_case(lens, H, G, 128, F16, 16, seed=13)
    q, kc, vc, table, cu, kv = case
    d, pg = P.paged_desc(H, len(kv), q.shape[0], max(n for n, _ in lens), table.shape[1]), P.page_desc(kc, vc)
    ws = torch.zeros(P.pi_paged_workspace_bytes(d, pg), dtype=torch.uint8, device="cuda")
    want = run_attn(P, *case, ws=ws)
    assert P.pi_last_device_status() == 0
    for limit in (1, 3000):
        P.pi_debug_set_wait_timeout(limit)
        try:
            run_attn(P, *case, ws=ws)
            torch.cuda.synchronize()
        finally:
            P.pi_debug_set_wait_timeout(0)
        assert P.pi_last_device_status() in ((4,) if limit == 1 else (0, 4))
        ws.zero_()
        for _ in range(3):
            got = run_attn(P, *case, ws=ws)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert P.pi_last_device_status() == 0


@pytest.mark.parametrize("seed", range(8))
def test_steps_of_many_sizes_on_one_workspace(P, seed):
    """Decodes, chunks and empty rows whose items the blocks' borders cut anywhere, one step after the other on one
    workspace that is filled with zeros only once."""
    r = random.Random(seed)
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    for _ in range(4):
        H, G = r.choice([(4, 4), (8, 2), (16, 1), (64, 8)])
        dh, dt, page, window = r.choice([64, 128]), r.choice([F16, BF16]), r.choice([16, 32, 128]), r.choice([0, 0, 1, 300])
        lens = []
        for _ in range(r.choice([1, 2, 5, 40])):
            n = r.choice([0, 1, 1, 1, r.randint(2, 30), r.randint(30, 400)])
            lens.append((n, n + r.choice([0, r.randint(0, 100), r.randint(100, 1500)])))
        if not any(n for n, _ in lens):
            lens.append((1, 700))
        compare(P, paged_case(lens, H, G, dh, dt, page, seed=r.randrange(1000), junk=math.nan, window=window), window=window, ws=ws)
