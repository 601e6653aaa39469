"""The 8-bit paged cache at its edges: workspaces that heads of both widths share, rows of no request, reads beside
requests that are not consistent, the store's larger windows and its queries in a launch of their own, reads of many
rows, the ends of fp16 in the attention."""
import random

import pytest
import torch

from tests import paged8_ref as R
from tests import paged_ref as R16
from tests.test_gpu_paged8 import (BF16, F16, F32, P, attn, i32, make_cache, quantised, same_codes, slots_of, starts,  # noqa: F401
                                   store_each, tables)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ one workspace for heads of both widths

@pytest.mark.parametrize("dt", [F16, BF16])
def test_heads_of_both_widths_on_one_workspace(P, dt):
    """Prompts, chunks and decode steps with heads of 64 and of 128 in turn on one workspace that is filled with zeros
    once: items that many blocks share in each, copies of pages and partials over most of the workspace between them."""
    r = random.Random(1)
    wide64 = (16, 8, 64, 16, [60] * 40, [60 + r.randint(0, 200) for _ in range(40)])
    long64 = (4, 2, 64, 32, [300] * 9 + [1], [300 + r.randint(0, 900) for _ in range(9)] + [700])
    long128 = (4, 2, 128, 32, [200] * 13 + [1], [200 + r.randint(0, 900) for _ in range(13)] + [700])
    few64 = (64, 8, 64, 16, [1] * 300, [r.randint(200, 700) for _ in range(300)])
    few128 = (64, 8, 128, 16, [1] * 300, [r.randint(200, 700) for _ in range(300)])
    some128 = (64, 8, 128, 16, [2] * 120, [r.randint(200, 700) for _ in range(120)])
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for i, (H, G, dh, page, n, kv) in enumerate([wide64, long128, few128, long64, some128, wide64, few64, long128, long64]):
        used = sum(-(-x // page) for x in kv)
        kc, ke = quantised(used, G, page, dh, "hnd", 1)
        vc, ve = quantised(used, G, page, dh, "hnd", 2)
        torch.manual_seed(i)
        q = torch.randn(sum(n), H, dh, device="cuda").to(dt)
        table, cu = tables(kv, page, used, i), starts(n)
        out, lse = attn(P, q, kc, ke, vc, ve, table, cu, kv, ws=ws)
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), cu, kv)
        R16.check(out, want, tol, f"step {i}: out")
        R16.check(lse, wl, ltol, f"step {i}: lse")
    assert P.pi_last_device_status() == 0


# ------------------------------------------------------------------ rows of no request

def test_calls_of_no_rows(P):
    """Nothing to rotate, store, read or attend to: nothing is done, and nothing refused."""
    kc, ke = make_cache(4, 2, 16, 64, "hnd", 1)
    cache, plan = P.page8_desc(kc, kc), P.rope_plan(64)
    none, slots = torch.empty(0, 2, 64, dtype=F16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    pos, before = i32([]), kc.view(torch.uint8).clone()
    P.pi_rope_store8(plan, cache, none, None, None, pos, None, none, None, None, None, None)
    P.pi_rope_store8(plan, cache, none, none, none, pos, slots, none, kc, kc, ke, ke)
    other = torch.zeros(4, 2, 16, 64, dtype=F16, device="cuda")
    P.pi_rope_store(plan, P.page_desc(other, other), none, None, None, pos, None, none, None, None)
    P.pi_page_read8(P.read8_desc(1, 4, 0), cache, kc, kc, ke, ke, i32([[0, 1, 2, 3]]), None, i32([0, 0]), none, none)
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    c = PagedCache(4, 2, 64, 2, 64, 8, 16, bits=8)
    k, v = c.read(0, None, i32([0, 0, 0]), 0)
    assert k.shape == v.shape == (0, 2, 64) and k.dtype is F16
    assert torch.equal(kc.view(torch.uint8), before) and P.pi_last_device_status() == 0


@pytest.mark.parametrize("cu,rows", [([0, 100, 8, 12], 20), ([0, 5, 3, 9], 12), ([0, -4, 2, 7], 8), ([-3, 6, 11, 13], 14),
                                     ([0, 4, 30, 5, 9], 10), ([4, 7, 7, 9], 10)])
def test_read_back_beside_inconsistent_requests(P, cu, rows):
    """Requests whose rows are in order are read, whatever others of the same call ask for."""
    G, dh, page = 2, 64, 16
    kc, ke = make_cache(8, G, page, dh, "hnd", 1)
    val, B = R.values(kc, ke).float(), len(cu) - 1
    out = torch.full((rows, G, dh), 7.0, device="cuda")
    P.pi_page_read8(P.read8_desc(B, 1, rows), P.page8_desc(kc, kc), kc, None, ke, None, i32([[b] for b in range(B)]), None,
                    i32(cu), out, None)
    fine = [b for b in range(B) if 0 <= cu[b] <= cu[b + 1] <= rows]
    assert P.pi_last_device_status() == (1 if len(fine) < B else 0)
    for row in range(rows):
        mine = [val[b, :, row - cu[b]] for b in fine if cu[b] <= row < cu[b + 1]]
        if mine:
            assert any(torch.equal(out[row], x) for x in mine), row
        else:
            assert bool((out[row] == 7).all()), row


# ------------------------------------------------------------------ the store's windows

@pytest.mark.parametrize("G,T,page,order", [(32, 1200, 32, "hnd"), (32, 1999, 16, "nhd"), (3, 1500, 64, "hnd"), (8, 5000, 128, "nhd")])
@pytest.mark.parametrize("rot,inter,dh", [(128, False, 128), (64, True, 128), (32, False, 64)])
@pytest.mark.parametrize("inp", [F16, F32])
def test_store_of_many_tokens_with_rotation(P, G, T, page, order, rot, inter, dh, inp):
    """Prompts, chunks that start inside a block and single tokens whose blocks of positions begin anywhere in a window of 4
    or of 16 tokens: values bit for bit, keys within half a step of their code and what fp32 rounds of the rotation."""
    H, base, r = 2, 10000.0, random.Random(G + T)
    runs, left = [], T
    while left > 0:
        n = min(left, r.choice((1, 1, 2, 5, 16, 17, 33, 200)))
        runs.append((r.randint(0, 1 << 18), n))
        left -= n
    pages = sum((c + n - 1) // page - c // page + 1 for c, n in runs)
    slots, pos = slots_of(page, pages, runs, 3)
    for t in r.sample([t for t, s in enumerate(slots) if s % 16 == 15], 10):   # (a block's new tokens stay in a row)
        slots[t] = -1
    torch.manual_seed(rot)
    qkv = torch.randn(T, (H + 2 * G) * dh, device="cuda").to(inp)
    q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv.split([H * dh, G * dh, G * dh], dim=1))
    (kc, ke), (vc, ve) = make_cache(pages, G, page, dh, order, 1, -9, -9), make_cache(pages, G, page, dh, order, 2, -9, -9)
    first_k, first_ke = kc.view(torch.uint8).clone(), ke.clone()
    wv, wve = vc.view(torch.uint8).clone(), ve.clone()
    store_blocks(wv, wve, v.double(), slots, page)
    plan = P.rope_plan(dh, rot, interleaved=inter, base=base)
    q_out = torch.empty(T, H, dh, dtype=F16, device="cuda")
    at = torch.tensor(slots, device="cuda")
    P.pi_rope_store8(plan, P.page8_desc(kc, vc), q, k, v, i32(pos), at, q_out, kc, vc, ke, ve)
    assert P.pi_last_device_status() == 0
    assert torch.equal(ve, wve)
    same_codes(vc, wv)
    place = torch.tensor(pos, device="cuda")
    freq = R16.frequencies(rot, base)
    x, slack = R16.rotate(k, place, freq, inter)
    y, qs = R16.rotate(q, place, freq, inter)
    assert float(((q_out.double() - y).abs() - qs - R16.half_step(F16) * (y.abs() + qs) - 2.0 ** -25).max()) <= 0
    # exponents within what the rotation's rounding can move them, codes under the exponents as they are
    keep = at >= 0
    at, x, slack = at[keep], x[keep], slack[keep]
    e = ke[at // page, :, at % page // 16].double()
    wk, wke = first_k.clone(), first_ke.clone()
    store_blocks(wk, wke, x, [s for s in slots if s >= 0], page)
    near = wke != ke
    assert float((wke - ke).abs().max()) <= 1 and float(near.float().mean()) < 1e-3
    got = R.values(kc, ke)[at // page, :, at % page]
    step = torch.exp2(torch.floor(torch.log2(got.abs().clamp(min=2.0 ** -300))).clamp(min=e[..., None] - 6) - 3)
    assert float(((got - x).abs() - step / 2 - slack).max()) <= 0
    # positions before a block's new ones under the same exponent, and blocks without new ones, are as they were
    new_from = torch.full((pages, page // 16), 16, device="cuda")
    new_from.view(-1).scatter_reduce_(0, at // 16, at % 16, "amin")
    stays = torch.arange(16, device="cuda") < new_from[..., None]                                   # [pages, blocks, 16]
    stays = (stays[:, None] & (ke == first_ke)[..., None]).flatten(2)[..., None].expand(-1, -1, -1, dh)
    assert torch.equal(kc.view(torch.uint8)[stays], first_k[stays])


def store_blocks(codes, exps, x, slots, page):
    """R.store with all heads of a block of positions at once (finite values, kept codes without NaN)."""
    i, T, table = 0, len(slots), R.VALUES.cuda()
    while i < T:
        s = slots[i]
        if s < 0:
            i += 1
            continue
        n = 1
        while i + n < T and slots[i + n] == s + n and (s + n) % R.BLOCK != 0:
            n += 1
        p, r = s // page, s % R.BLOCK
        first = s % page - r
        new = x[i:i + n]                                            # [n, heads, dh]
        most = new.abs().amax((0, 2)).tolist()
        e = torch.tensor([R.exponent(m) for m in most], device="cuda")
        if r > 0:
            old = exps[p, :, first // R.BLOCK].long()
            e = torch.maximum(e, old)
            kept = codes[p, :, first:first + r]
            codes[p, :, first:first + r] = R.encode(table[kept.long()] * torch.exp2((old - e).double())[:, None, None])
        exps[p, :, first // R.BLOCK] = e.to(torch.int8)
        codes[p, :, first + r:first + r + n] = R.encode(new / torch.exp2(e.double())[None, :, None]).transpose(0, 1)
        i += n


def test_store_of_single_tokens_in_wide_windows(P):
    """So many decoding rows that a block of threads looks at 16 of them: each begins its block of positions."""
    T, G, dh, page = 9000, 4, 64, 16
    kc, ke = make_cache(T, G, page, dh, "nhd", 1)
    vc, ve = make_cache(T, G, page, dh, "nhd", 2)
    rng = random.Random(T)
    ids = list(range(T))
    rng.shuffle(ids)
    slots = [i * page + rng.randrange(16) if rng.random() < 0.95 else -1 for i in ids]
    kv = torch.randn(T, 2 * G, dh, device="cuda").to(BF16) * 8
    k, v = kv[:, :G].contiguous(), kv[:, G:].contiguous()
    wk, wv = (kc.view(torch.uint8).clone(), ke.clone()), (vc.view(torch.uint8).clone(), ve.clone())
    P.pi_rope_store8(P.rope_plan(dh, 0), P.page8_desc(kc, vc), None, k, v, i32([0] * T), torch.tensor(slots, device="cuda"),
                     None, kc, vc, ke, ve)
    for (c, e), x in ((wk, k), (wv, v)):
        store_each(c, e, x.double(), slots, page)
    assert torch.equal(ke, wk[1]) and torch.equal(ve, wv[1]) and P.pi_last_device_status() == 0
    same_codes(kc, wk[0])
    same_codes(vc, wv[0])


@pytest.mark.parametrize("inp,out,inter", [(F16, F16, False), (BF16, BF16, True), (F32, F16, True)])
def test_store_whose_queries_take_a_launch_of_their_own(P, inp, out, inter):
    """More than 4096 blocks of queries: the same queries as pi_rope_store's, the same cache as without queries; with
    keys and values, rotated alone, and in place."""
    H, G, dh, page, T = 64, 2, 128, 16, 4203
    pages = -(-T // page)
    torch.manual_seed(1)
    qkv = torch.randn(T, (H + 2 * G) * dh, device="cuda").to(inp)
    q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv.split([H * dh, G * dh, G * dh], dim=1))
    plan, pos = P.rope_plan(dh, 64, interleaved=inter), i32(list(range(T)))
    slots = torch.arange(T, device="cuda")
    other = torch.zeros(1, G, page, dh, dtype=out, device="cuda")
    want = torch.empty(T, H, dh, dtype=out, device="cuda")
    P.pi_rope_store(plan, P.page_desc(other, other), q, None, None, pos, None, want, None, None)
    res = []
    for mine in (None, q):
        kc, ke = make_cache(pages, G, page, dh, "hnd", 1)
        vc, ve = make_cache(pages, G, page, dh, "hnd", 2)
        got = None if mine is None else torch.zeros(T, H, dh, dtype=out, device="cuda")
        P.pi_rope_store8(plan, P.page8_desc(kc, vc), mine, k, v, pos, slots, got, kc, vc, ke, ve)
        res.append((kc.view(torch.uint8), ke, vc.view(torch.uint8), ve))
    assert torch.equal(got, want)
    for a, b in zip(*res):
        assert torch.equal(a, b)
    alone = torch.zeros_like(want)
    d = P.page8_desc(kc, vc)
    P.pi_rope_store8(plan, d, q, None, None, pos, None, alone, None, None, None, None)
    assert torch.equal(alone, want)
    if inp is out:
        P.pi_rope_store8(plan, d, q, None, None, pos, None, q, None, None, None, None)
        assert torch.equal(q, want)
    assert P.pi_last_device_status() == 0


# ------------------------------------------------------------------ reads of many rows

@pytest.mark.parametrize("G,dh,page,order,rows", [(8, 128, 32, "nhd", 21003), (12, 64, 16, "hnd", 2011), (32, 128, 64, "hnd", 2605),
                                                  (1, 64, 16, "nhd", 41007), (3, 128, 128, "hnd", 9001)])
@pytest.mark.parametrize("dt", [F16, F32])
@pytest.mark.parametrize("which", ["both", "values"])
def test_read_back_of_many_rows(P, G, dh, page, order, rows, dt, which):
    """Blocks of several rows, threads that go from row to row, threads without a piece and with several: exactly the
    values, and what lies between and behind the rows left alone."""
    r = random.Random(rows)
    n, left = [], rows
    while left > 0:
        n.append(min(left, r.choice((0, 1, 7, 333, 2000))))
        left -= n[-1]
    B, cu = len(n), starts(n)
    start = [r.randint(0, 300) for _ in range(B)]
    M = max(-(-(s + x) // page) for s, x in zip(start, n))
    pages = 97
    table = torch.randint(0, pages, (B, M), generator=torch.Generator().manual_seed(rows), dtype=torch.int32).cuda()
    kc, ke = make_cache(pages, G, page, dh, order, 1)
    vc, ve = make_cache(pages, G, page, dh, order, 2)
    cap = rows + 5
    bufs = [torch.full((cap, G * dh + 8 * (i + 1)), 7.0, dtype=dt, device="cuda") for i in range(2)]
    k_out, v_out = (b[:, :G * dh].unflatten(1, (G, dh)) for b in bufs)
    both = which == "both"
    P.pi_page_read8(P.read8_desc(B, M, cap), P.page8_desc(kc, vc), kc if both else None, vc, ke if both else None, ve, table,
                    i32(start), i32(cu), k_out if both else None, v_out)
    assert P.pi_last_device_status() == 0
    req = torch.repeat_interleave(torch.arange(B), torch.tensor(n)).cuda()
    at = torch.arange(rows, device="cuda") - torch.tensor(cu, device="cuda")[req] + torch.tensor(start, device="cuda")[req]
    ids = table[req, at // page].long()
    for c, e, o, b, used in ((kc, ke, k_out, bufs[0], both), (vc, ve, v_out, bufs[1], True)):
        if used:
            assert torch.equal(o[:rows], R.values(c, e)[ids, :, at % page].to(dt))
        assert bool((b[rows if used else 0:] == 7).all()) and bool((b[:, G * dh:] == 7).all())


# ------------------------------------------------------------------ the ends of fp16

def as_copied(codes, exps):
    """Keys or values as a request of many rows takes them in fp16: rounded to it, magnitudes past 65504 as that."""
    return R.values(codes, exps).clamp(-65504, 65504).half()


@pytest.mark.parametrize("n", [1, 5, 40, 150])
@pytest.mark.parametrize("H,G,dh", [(8, 2, 64), (4, 4, 128)])
def test_attention_past_the_end_of_fp16(P, n, H, G, dh):
    """Values of blocks that lie past 65504: outputs that would round past it are 65504, of either sign."""
    page, kv = 16, 300
    kc, ke = quantised(20, G, page, dh, "hnd", 1)
    vc, ve = make_cache(20, G, page, dh, "hnd", 2, 8, 10)
    vc.view(torch.uint8)[:, :, :, ::2] |= 0x70             # every other column large
    v8 = vc.view(torch.uint8)
    v8[v8 & 127 == 127] -= 1
    v8[:, :, :, 0] &= 0x7f                                 # a column of one sign, and one of the other
    v8[:, :, :, 2] |= 0x80
    torch.manual_seed(n)
    q = torch.randn(n, H, dh, device="cuda").half()
    table = tables([kv], page, 20, 1)
    out, lse = attn(P, q, kc, ke, vc, ve, table, [0, n], [kv])
    few = n <= max(1, 64 // (H // G))                      # all requests of the step short: straight from the codes
    if few:
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, n], [kv])
    else:
        want, wl, tol, ltol = R16.attention(q, R.values(kc, ke), as_copied(vc, ve), i32(table), [0, n], [kv])
    assert bool(torch.isfinite(out).all())
    R16.check(out, want.clamp(-65504, 65504), tol, "out")
    R16.check(lse, wl, ltol, "lse")
    if few:
        assert bool((out[..., 0] == 65504).any()) and bool((out[..., 2] == -65504).any())


@pytest.mark.parametrize("n", [1, 5, 40, 150])
def test_attention_below_the_normal_numbers_of_fp16(P, n):
    """Blocks of values under exponents of -24 .. -16: codes straight from the cache for few rows, rounded to fp16's
    subnormals for many."""
    G, H, dh, page, kv = 2, 8, 64, 16, 300
    kc, ke = quantised(20, G, page, dh, "hnd", 1)
    vc, ve = make_cache(20, G, page, dh, "hnd", 2, -24, -16)
    torch.manual_seed(n)
    q = torch.randn(n, H, dh, device="cuda").half()
    table = tables([kv], page, 20, 1)
    out, lse = attn(P, q, kc, ke, vc, ve, table, [0, n], [kv])
    if n <= 16:
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, n], [kv])
    else:
        want, wl, tol, ltol = R16.attention(q, R.values(kc, ke), as_copied(vc, ve), i32(table), [0, n], [kv])
    R16.check(out, want, tol, "out")
    R16.check(lse, wl, ltol, "lse")


@pytest.mark.parametrize("n", [1, 5, 40, 150])
def test_attention_with_keys_past_the_end_of_fp16(P, n):
    """Keys past 65504 in one block: as they are for few rows, held at 65504 for many."""
    G, H, dh, page, kv, scale = 2, 8, 64, 16, 300, 2.0 ** -16
    kc, ke = make_cache(20, G, page, dh, "hnd", 1, 0, 0)
    ke[3], ke[7] = 10, 8
    vc, ve = quantised(20, G, page, dh, "hnd", 2)
    torch.manual_seed(n)
    q = (0.05 * torch.randn(n, H, dh, device="cuda")).half()
    table = [[i for i in range(19)]]
    out, lse = attn(P, q, kc, ke, vc, ve, table, [0, n], [kv], scale=scale)
    k = R.values(kc, ke) if n <= 16 else as_copied(kc, ke)
    want, wl, tol, ltol = R16.attention(q, k, R.values(vc, ve), i32(table), [0, n], [kv], 0, scale)
    R16.check(out, want, tol, "out")
    R16.check(lse, wl, ltol, "lse")


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("rot,inter", [(64, False), (32, True)])
def test_what_a_cache_holds_after_serving(P, rot, inter):
    """Prompts, chunks, decode steps and rollbacks: keys of a step's new positions read back as the rotated ones, within half
    a step of a code under the largest value that their block can have met."""
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    B, H, G, dh, page = 3, 4, 2, 64, 32
    cache = PagedCache(H, G, dh, B, 900, 600, 1300, page_size=page, rope=P.rope_plan(dh, rot, interleaved=inter), bits=8)
    torch.manual_seed(0)
    have = [0] * B
    for new, keep in (([600, 300, 1], None), ([200, 1, 1], None), ([1, 1, 1], [750, 31, 2]), ([5, 3, 17], None)):
        T = sum(new)
        cache.begin(i32(new), T, max(new), None if keep is None else i32(keep))
        have = [(h if keep is None else min(h, k)) + x for h, k, x in zip(have, keep or have, new)]
        q, k, v = (torch.randn(T, x, dh, device="cuda") for x in (H, G, G))
        cache.attend(0, q, k, v, torch.empty(T, H, dh, dtype=F16, device="cuda"))
        rows = starts(new)
        kr, vr = cache.read(0, i32([h - x for h, x in zip(have, new)]), i32(rows), T, dtype=F32)
        pos = torch.cat([torch.arange(h - x, h) for h, x in zip(have, new)]).cuda()
        assert torch.equal(pos.int(), cache.positions[:T])
        kt, slack = R16.rotate(k, pos, R16.frequencies(rot, 10000.0), inter)
        # codes of a block lie within half a step, 2^-4 of the value or 2^-10 2^e; 448 2^e is at most twice the largest value met
        most = 2 * 6.0
        for got, want, s in ((kr, kt, slack), (vr, v.double(), torch.zeros_like(slack))):
            assert float(want.abs().max()) < most / 2
            assert float(((got.double() - want).abs() - 2.0 ** -4 * want.abs() * 1.0001 - 2.0 ** -10 * most / 448 - s).max()) <= 0
    assert P.pi_last_device_status() == 0
