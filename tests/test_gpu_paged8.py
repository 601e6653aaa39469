"""Parity of the 8-bit paged cache on the GPU: codes and exponents bit for bit where
no rotation is rounded, within half a step of the code else; rows read back exactly;
attention within bounds derived from its roundings."""
import math
import random

import pytest
import torch

from tests import paged8_ref as R
from tests import paged_ref as R16

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


def make_cache(pages, heads, page, dh, order, seed=0, lo=-6, hi=3):
    """Random codes without NaN and exponents lo .. hi."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (pages, heads, page, dh) if order == "hnd" else (pages, page, heads, dh)
    c = torch.randint(0, 127, shape, generator=g, device="cuda") + 128 * torch.randint(0, 2, shape, generator=g, device="cuda")
    c = c.to(torch.uint8).view(R.CODE)
    e = torch.randint(lo, hi + 1, (pages, heads, page // 16), generator=g, device="cuda").to(torch.int8)
    return (c if order == "hnd" else c.transpose(1, 2)), e


def quantised(pages, heads, page, dh, order, seed=0, scale=1.0):
    """Codes and exponents of normal values, a size for each head."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(pages, heads, page // 16, 16, dh, generator=g, device="cuda")
    x *= scale * torch.linspace(0.3, 2.0, heads, device="cuda")[:, None, None, None]
    e = torch.ceil(torch.log2(x.abs().amax((-1, -2)) / 448)).clamp(-32, 32)
    c = (x / torch.exp2(e)[..., None, None]).to(R.CODE).flatten(2, 3)
    if order == "nhd":
        c = c.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(R.CODE)
    return c, e.to(torch.int8)


def same_codes(got, want, what=""):
    """Equal, where a NaN of either sign is one."""
    a, b = got.view(torch.uint8).int(), want.view(torch.uint8).int()
    a, b = torch.where(a & 127 == 127, 127, a), torch.where(b & 127 == 127, 127, b)
    assert torch.equal(a, b), f"{what}: {int((a != b).sum())} of {a.numel()} codes differ"


def slots_of(page, pages, runs, seed=0):
    """Slots and positions of requests that hold c positions and receive n, on pages of their own; pages used."""
    rng = random.Random(seed)
    ids = list(range(pages))
    rng.shuffle(ids)
    slots, pos = [], []
    for c, n in runs:
        own = {}
        for p in range(c, c + n):
            if p // page not in own:
                own[p // page] = ids.pop()
            slots.append(own[p // page] * page + p % page)
            pos.append(p)
    return slots, pos


# ------------------------------------------------------------------ store

RUNS = [[(0, 1)], [(5, 1), (15, 1), (16, 1), (31, 2), (0, 40), (7, 9), (3, 100)], [(1000, 333)], [(c, 1) for c in range(48)]]


@pytest.mark.parametrize("dh,G,page,order,inp", [(64, 1, 16, "hnd", F16), (128, 8, 32, "nhd", BF16), (64, 12, 128, "nhd", F32),
                                                 (128, 5, 16, "hnd", F32), (128, 96, 64, "hnd", F16)])
@pytest.mark.parametrize("runs", range(len(RUNS)))
def test_store_without_rotation(P, dh, G, page, order, inp, runs):
    """Codes and exponents bit for bit: x / 2^e is exact in fp32, so each code has one rounding."""
    runs = RUNS[runs]
    slots, pos = slots_of(page, 64, runs)
    T = len(slots)
    torch.manual_seed(T + dh)
    kv = torch.randn(T, 2 * G * dh + 8, device="cuda") * torch.exp2(torch.randint(-12, 12, (T, 1), device="cuda").float())
    kv = kv.to(inp)
    k, v = kv[:, :G * dh].unflatten(1, (G, dh)), kv[:, G * dh:2 * G * dh].unflatten(1, (G, dh))
    (kc, ke), (vc, ve) = make_cache(64, G, page, dh, order, 1), make_cache(64, G, page, dh, order, 2)
    want = []
    for c, e, x in ((kc, ke, k), (vc, ve, v)):
        wc, we = c.view(torch.uint8).clone(), e.clone()
        R.store(wc, we, x.double(), slots, page)
        want.append((wc, we))
    P.pi_rope_store8(P.rope_plan(dh, 0), P.page8_desc(kc, vc), None, k, v, i32(pos), torch.tensor(slots, device="cuda"), None,
                     kc, vc, ke, ve)
    assert P.pi_last_device_status() == 0
    for (wc, we), c, e in zip(want, (kc, vc), (ke, ve)):
        assert torch.equal(e, we)
        same_codes(c, wc)


@pytest.mark.parametrize("rot,inter,dh", [(128, False, 128), (64, True, 128), (48, False, 128), (16, True, 64), (64, False, 64), (32, False, 64)])
@pytest.mark.parametrize("inp,out", [(F32, F16), (BF16, BF16), (F16, BF16)])
def test_store_with_rotation(P, rot, inter, dh, inp, out):
    """Queries as pi_rope_store leaves them; keys within half a step of their code and what
    fp32 rounds of the rotation; values bit for bit."""
    H, G, page, base = 6, 3, 32, 10000.0
    runs = [(0, 33), (77, 1), (1 << 20, 50), (13, 3)]
    slots, pos = slots_of(page, 16, runs, 3)
    T = len(slots)
    torch.manual_seed(rot)
    qkv = torch.randn(T, (H + 2 * G) * dh, device="cuda").to(inp)
    q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv.split([H * dh, G * dh, G * dh], dim=1))
    (kc, ke), (vc, ve) = make_cache(16, G, page, dh, "hnd", 1, -9, -9), make_cache(16, G, page, dh, "hnd", 2, -9, -9)
    wv, wve = vc.view(torch.uint8).clone(), ve.clone()
    R.store(wv, wve, v.double(), slots, page)
    plan = P.rope_plan(dh, rot, interleaved=inter, base=base)
    q_out, q_16 = torch.empty(T, H, dh, dtype=out, device="cuda"), torch.empty(T, H, dh, dtype=out, device="cuda")
    at = torch.tensor(slots, device="cuda")
    P.pi_rope_store8(plan, P.page8_desc(kc, vc), q, k, v, i32(pos), at, q_out, kc, vc, ke, ve)
    other = torch.zeros(1, G, page, dh, dtype=out, device="cuda")
    P.pi_rope_store(plan, P.page_desc(other, other), q, None, None, i32(pos), None, q_16, None, None)
    assert P.pi_last_device_status() == 0
    assert torch.equal(q_out, q_16) and torch.equal(ve, wve)
    same_codes(vc, wv)
    x, slack = R16.rotate(k, torch.tensor(pos, device="cuda"), R16.frequencies(rot, base), inter)
    got = R.values(kc, ke)[at // page, :, at % page]
    e = ke[at // page, :, at % page // 16].double()
    step = torch.exp2(torch.floor(torch.log2(got.abs().clamp(min=2.0 ** -300))).clamp(min=e[..., None] - 6) - 3)
    # (half a step of the code below or above, whichever is larger: a code at a power of two has a smaller step below)
    assert float(((got - x).abs() - step / 2 - slack).max()) <= 0
    # exponents: the smallest that holds the block's magnitudes
    for i, (c, n) in enumerate(runs):
        t0 = sum(m for _, m in runs[:i])
        for b0 in range(c // 16 * 16, c + n, 16):
            t = slice(t0 + max(b0 - c, 0), t0 + min(b0 + 16 - c, n))
            most = x[t].abs().amax((0, 2))
            mine, kept = e[t][0], (-9 if b0 < c else -32)
            assert bool((most <= 448 * torch.exp2(mine) * (1 + 1e-6)).all())
            assert bool(((most > 224 * torch.exp2(mine) * (1 - 1e-6)) | (mine == kept)).all())


def test_store_token_by_token(P):
    """Blocks grow position by position, and their exponents with them: 50 steps of one token in
    4 rows, magnitudes that rise and fall over 2^-40 .. 2^40 (past both ends of the exponents)."""
    G, dh, page, B = 2, 64, 32, 4
    kc, ke = make_cache(8, G, page, dh, "nhd", 5)
    vc, ve = make_cache(8, G, page, dh, "nhd", 6)
    wk, wv = (kc.view(torch.uint8).clone(), ke.clone()), (vc.view(torch.uint8).clone(), ve.clone())
    plan, d = P.rope_plan(dh, 0), P.page8_desc(kc, vc)
    torch.manual_seed(0)
    for step in range(50):
        slots = [(2 * b + step // page) * page + step % page for b in range(B)]
        size = torch.exp2(torch.tensor([[40.0 * math.sin(step * 0.7 + b)] for b in range(B)], device="cuda"))
        kv = (torch.randn(B, 2 * G * dh, device="cuda") * size).to(BF16)
        k, v = (x.unflatten(1, (G, dh)) for x in kv.split(G * dh, dim=1))
        P.pi_rope_store8(plan, d, None, k, v, i32([step] * B), torch.tensor(slots, device="cuda"), None, kc, vc, ke, ve)
        R.store(*wk, k.double(), slots, page)
        R.store(*wv, v.double(), slots, page)
    assert torch.equal(ke, wk[1]) and torch.equal(ve, wv[1]) and P.pi_last_device_status() == 0
    same_codes(kc, wk[0])
    same_codes(vc, wv[0])


def test_store_values_that_are_not_finite(P):
    """Infinities and NaN become NaN and leave the exponent alone; a block of nothing else, and one of zeros."""
    G, dh, page = 2, 128, 16
    kv = torch.randn(40, 2 * G, dh, device="cuda")
    kv[3, 0, 7], kv[4, 1, 8], kv[5, 2, 9], kv[6, 3, 10] = math.inf, math.nan, -math.inf, 1e38
    kv[16:32, 0] = math.nan
    kv[16:32, 2] = 0.0
    kv[32:, 1] = -0.0
    kc, ke = make_cache(4, G, page, dh, "hnd", 1)
    vc, ve = make_cache(4, G, page, dh, "hnd", 2)
    wk, wv = (kc.view(torch.uint8).clone(), ke.clone()), (vc.view(torch.uint8).clone(), ve.clone())
    slots = list(range(16, 56))
    k, v = kv[:, :G].contiguous(), kv[:, G:].contiguous()
    P.pi_rope_store8(P.rope_plan(dh, 0), P.page8_desc(kc, vc), None, k, v, i32(slots), torch.tensor(slots, device="cuda"), None,
                     kc, vc, ke, ve)
    R.store(*wk, k.double(), slots, page)
    R.store(*wv, v.double(), slots, page)
    assert torch.equal(ke, wk[1]) and torch.equal(ve, wv[1]) and P.pi_last_device_status() == 0
    same_codes(kc, wk[0])
    same_codes(vc, wv[0])
    # a kept NaN stays one when its block's exponent grows
    more = torch.full((1, G, dh), 3e4, device="cuda")
    P.pi_rope_store8(P.rope_plan(dh, 0), P.page8_desc(kc, vc), None, more, more, i32([40]), torch.tensor([56], device="cuda"),
                     None, kc, vc, ke, ve)
    R.store(*wk, more.double(), [56], page)
    R.store(*wv, more.double(), [56], page)
    assert torch.equal(ke, wk[1])
    same_codes(kc, wk[0])
    same_codes(vc, wv[0])


def test_store_slots_outside(P):
    """-1 is passed over, others set the status; nothing else is written; rows without slots between those of one block."""
    G, dh, page = 1, 64, 16
    kc, ke = make_cache(3, G, page, dh, "hnd", 1)
    vc, ve = make_cache(3, G, page, dh, "hnd", 2)
    wk, wv = (kc.view(torch.uint8).clone(), ke.clone()), (vc.view(torch.uint8).clone(), ve.clone())
    x = torch.randn(6, G, dh, device="cuda").half()
    for slots, status in (([-1, 20, 21, -1, 2, -1], 0), ([48, 20, 21, 1 << 40, 2, 3], 1), ([-2, 33, 34, 35, -1, -1], 1)):
        P.pi_rope_store8(P.rope_plan(dh, 0), P.page8_desc(kc, vc), None, x, x, i32([0] * 6), torch.tensor(slots, device="cuda"),
                         None, kc, vc, ke, ve)
        good = [s if 0 <= s < 48 else -1 for s in slots]
        R.store(*wk, x.double(), good, page)
        R.store(*wv, x.double(), good, page)
        assert P.pi_last_device_status() == status
        assert torch.equal(ke, wk[1]) and torch.equal(ve, wv[1])
        same_codes(kc, wk[0])
        same_codes(vc, wv[0])


def test_store_queries_in_place(P):
    q = torch.randn(9, 4, 64, device="cuda").to(BF16)
    plan, pos = P.rope_plan(64), i32(list(range(9)))
    kc, ke = make_cache(1, 2, 16, 64, "hnd")
    out = torch.empty_like(q)
    P.pi_rope_store8(plan, P.page8_desc(kc, kc), q, None, None, pos, None, out, None, None, None, None)
    P.pi_rope_store8(plan, P.page8_desc(kc, kc), q, None, None, pos, None, q, None, None, None, None)
    assert torch.equal(q, out)


# ------------------------------------------------------------------ read back

@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("dh,G,page,order", [(64, 12, 16, "hnd"), (128, 8, 64, "nhd"), (128, 1, 128, "hnd")])
def test_read_back(P, dt, dh, G, page, order):
    kc, ke = make_cache(40, G, page, dh, order, 1)
    vc, ve = make_cache(40, G, page, dh, order, 2)
    start, n = [0, 37, 5, 15, 64], [1, 70, 0, 17, 33]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    M = 8
    perm = torch.randperm(40, generator=torch.Generator().manual_seed(3)).tolist()
    table = [perm[M * b:M * b + M] for b in range(5)]
    rows = cu[-1] + 3
    wide = torch.full((rows, G * dh + 8), 7.0, dtype=dt, device="cuda")
    k_out, v_out = wide[:, :G * dh].unflatten(1, (G, dh)), torch.full((rows, G, dh), 7.0, dtype=dt, device="cuda")
    P.pi_page_read8(P.read8_desc(5, M, rows), P.page8_desc(kc, vc), kc, vc, ke, ve, i32(table), i32(start), i32(cu), k_out, v_out)
    assert P.pi_last_device_status() == 0
    for out, c, e in ((k_out, kc, ke), (v_out, vc, ve)):
        val = R.values(c, e)
        want = torch.full((rows, G, dh), 7.0, dtype=torch.float64, device="cuda")
        for b in range(5):
            for i in range(n[b]):
                p = start[b] + i
                want[cu[b] + i] = val[table[b][p // page], :, p % page]
        assert torch.equal(out, want.to(dt))
    assert bool((wide[:, G * dh:] == 7).all())
    # one array alone, from position 0
    only = torch.full((rows, G, dh), 7.0, dtype=dt, device="cuda")
    P.pi_page_read8(P.read8_desc(5, M, rows), P.page8_desc(kc, vc), None, vc, None, ve, i32(table), None, i32(cu), None, only)
    assert torch.equal(only[cu[1]], R.values(vc, ve)[table[1][0], :, 0].to(dt)) and bool((only[cu[-1]:] == 7).all())


def test_read_back_many_requests(P):
    """4096 requests of 0 to 3 rows."""
    G, dh, page = 1, 64, 16
    kc, ke = make_cache(64, G, page, dh, "hnd", 1)
    n = [(b * 7) % 4 for b in range(4096)]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    table = [[(b * 5) % 64] for b in range(4096)]
    out = torch.zeros(cu[-1], G, dh, device="cuda")
    P.pi_page_read8(P.read8_desc(4096, 1, cu[-1]), P.page8_desc(kc, kc), kc, None, ke, None, i32(table), i32([2] * 4096), i32(cu),
                    out, None)
    val = R.values(kc, ke).float()
    at = torch.tensor([[t[0], 2 + i] for t, x in zip(table, n) for i in range(x)], device="cuda")
    assert torch.equal(out[:, 0], val[at[:, 0], 0, at[:, 1]]) and P.pi_last_device_status() == 0


def test_read_back_at_the_ends_of_the_types(P):
    """fp16 values that would pass 65504 are 65504; tiny ones round to its subnormals; NaN stays."""
    c = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(16)[:16 * 64 * 4].view(4, 1, 16, 64).view(R.CODE)
    for e in (-128, -32, -20, 7, 8, 9, 32, 100):
        ex = torch.full((4, 1, 1), e, dtype=torch.int8, device="cuda")
        for dt in (F16, BF16, F32):
            out = torch.empty(64, 1, 64, dtype=dt, device="cuda")
            P.pi_page_read8(P.read8_desc(1, 4, 64), P.page8_desc(c, c), c, None, ex, None, i32([[0, 1, 2, 3]]), None, i32([0, 64]),
                            out, None)
            want = R.values(c, ex).reshape(64, 1, 64)
            want = want.clamp(-65504, 65504) if dt is F16 else want
            torch.testing.assert_close(out, want.to(dt), rtol=0, atol=0, equal_nan=True)


def test_read_back_inconsistent(P):
    """Positions and pages that are not there read as zeros and are reported; a request past the rows is not read."""
    G, dh, page = 2, 64, 16
    kc, ke = make_cache(4, G, page, dh, "hnd", 1)
    val = R.values(kc, ke).float()

    def read(table, start, cu, rows):
        out = torch.full((rows, G, dh), 7.0, device="cuda")
        P.pi_page_read8(P.read8_desc(len(table), len(table[0]), rows), P.page8_desc(kc, kc), kc, None, ke, None, i32(table),
                        i32(start), i32(cu), out, None)
        return out, P.pi_last_device_status()
    out, st = read([[0, 4, -1, 3]], [14], [0, 40], 40)
    assert st == 1 and torch.equal(out[:2], val[0, :, 14:].transpose(0, 1)) and bool((out[2:34] == 0).all())
    assert torch.equal(out[34:], val[3, :, :6].transpose(0, 1))
    out, st = read([[1, 2]], [-3], [0, 6], 6)
    assert st == 1 and bool((out[:3] == 0).all()) and torch.equal(out[3:], val[1, :, :3].transpose(0, 1))
    out, st = read([[1, 2]], [30], [0, 6], 6)
    assert st == 1 and bool((out[2:] == 0).all()) and torch.equal(out[:2], val[2, :, 14:].transpose(0, 1))
    out, st = read([[1], [2]], [0, 0], [0, 3, 9], 5)
    assert st == 1 and torch.equal(out[:3], val[1, :, :3].transpose(0, 1)) and bool((out[3:] == 7).all())


# ------------------------------------------------------------------ attention

def attn(P, q, kc, ke, vc, ve, table, cu, kv, window=0, scale=0.0, max_new=None, ws=None, lse=True, q_pad=0):
    T, H, dh = q.shape
    B = len(kv)
    n = [b - a for a, b in zip(cu, cu[1:])]
    cache = P.page8_desc(kc, vc)
    d = P.paged_desc(H, B, T, max(max(n), 1) if max_new is None else max_new, len(table[0]), window=window, scale=scale)
    need = P.pi_paged8_workspace_bytes(d, cache)
    if ws is None:
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    assert ws.numel() >= need
    buf = torch.full((T, H * dh + q_pad), 7.0, dtype=q.dtype, device="cuda")
    out = buf[:, :H * dh].unflatten(1, (H, dh))
    ls = torch.full((T, H), 7.0, device="cuda") if lse else None
    P.pi_paged_attn8(d, cache, q, kc, vc, ke, ve, i32(table), i32(cu), i32(kv), out, ls, ws)
    assert q_pad == 0 or bool((buf[:, H * dh:] == 7).all())
    return out, ls


def tables(kv, page, pages, seed=0):
    ids = list(range(pages))
    random.Random(seed).shuffle(ids)
    M = max(1, max(-(-x // page) for x in kv))
    out = []
    for x in kv:
        u = -(-x // page)
        out.append([ids.pop() for _ in range(u)] + [-1] * (M - u))
    return out


def starts(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def check(P, H, G, dh, dt, page, order, n, kv, window=0, scale=0.0, seed=0, extra=0, q_scale=1.0):
    used = sum(-(-x // page) for x in kv)
    kc, ke = quantised(used + 2, G, page, dh, order, seed + 1)
    vc, ve = quantised(used + 2, G, page, dh, order, seed + 2)
    torch.manual_seed(seed)
    T = sum(n) + extra
    q = (torch.randn(max(T, 1), H, dh, device="cuda") * torch.linspace(0.3, q_scale * 2, H, device="cuda")[:, None]).to(dt)
    table, cu = tables(kv, page, used + 2, seed), starts(n)
    out, lse = attn(P, q, kc, ke, vc, ve, table, cu, kv, window, scale)
    assert P.pi_last_device_status() == 0
    t = torch.tensor(table, device="cuda")
    want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, t, cu, kv, window, scale or None)
    m = sum(n)
    R16.check(out[:m], want[:m], tol[:m], "out")
    R16.check(lse[:m], wl[:m], ltol[:m], "lse")
    assert bool((out[m:] == 7).all()) and bool((lse[m:] == 7).all())


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,G,dh", [(12, 12, 64), (64, 8, 128), (24, 8, 128), (16, 1, 64), (32, 8, 64), (5, 5, 128), (128, 1, 64),
                                    (40, 2, 128)])
@pytest.mark.parametrize("page,order", [(16, "hnd"), (64, "nhd")])
def test_attention_of_single_tokens(P, dt, H, G, dh, page, order):
    """Lengths around blocks, tiles and pages, in one step."""
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 777, 1025]
    check(P, H, G, dh, dt, page, order, [1] * len(kv), kv, seed=H)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,G,dh,n", [(8, 8, 64, 16), (64, 8, 128, 2), (64, 8, 128, 5), (6, 2, 128, 7), (16, 1, 64, 4), (12, 12, 64, 33),
                                      (32, 8, 64, 17), (128, 1, 128, 3)])
@pytest.mark.parametrize("window", [0, 1, 20, 130])
def test_attention_of_a_few_tokens(P, dt, H, G, dh, n, window):
    """Tokens that see one another in part: causal steps and windows inside a tile."""
    kv = [n, n + 1, n + 15, n + 100, n + 333]
    check(P, H, G, dh, dt, 32, "hnd", [n] * len(kv), kv, window, seed=n)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("H,G,dh,window", [(12, 12, 64, 0), (16, 2, 128, 0), (6, 2, 128, 75), (16, 1, 64, 500)])
def test_attention_of_mixed_steps(P, dt, H, G, dh, window):
    """Prompts, chunks behind a cache, single tokens, requests without tokens or keys, one after the other."""
    n = [1, 130, 0, 1, 257, 3, 1, 0, 40, 1, 300]
    kv = [500, 130, 40, 1, 400, 90, 33, 0, 640, 1, 777]
    check(P, H, G, dh, dt, 32, "nhd", n, kv, window, seed=H + window, extra=3)


def test_attention_that_sees_nothing(P):
    """Requests with fewer positions than tokens: the first rows get zeros and -inf."""
    for n, kv in (([5], [3]), ([2, 1], [0, 7]), ([100], [40]), ([300, 1], [0, 0])):
        check(P, 8, 2, 64, F16, 16, "hnd", n, kv, seed=1)


def test_attention_scale_and_large_scores(P):
    check(P, 8, 2, 128, F16, 16, "hnd", [1, 4], [700, 300], scale=0.03, seed=2)
    check(P, 8, 2, 128, BF16, 16, "hnd", [1, 4, 90], [700, 300, 400], scale=1.5, seed=3, q_scale=4.0)


def test_attention_weights_spread_widely(P):
    """A first key far above the others: their weights are tiny, and count together."""
    G, dh, page, kv = 1, 64, 16, 4000
    kc, ke = quantised(251, G, page, dh, "hnd", 1, 0.05)
    vc, ve = quantised(251, G, page, dh, "hnd", 2)
    q = torch.full((1, 4, dh), 1.0, dtype=F16, device="cuda")
    kc.view(torch.uint8)[0, 0, 0] = 0x38   # 1.0
    ke[0] = 0
    vc.view(torch.uint8)[:] &= 0x7f        # values of one sign
    for top in (8.0, 14.0, 19.0):
        table = [list(range(250))]
        out, lse = attn(P, q, kc, ke, vc, ve, table, [0, 1], [kv], scale=top / dh)
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, 1], [kv], 0, top / dh)
        R16.check(out, want, tol, "out")
        R16.check(lse, wl, ltol, "lse")


@pytest.mark.parametrize("n", [1, 3, 90])
def test_attention_exponents_far_apart(P, n):
    """Blocks of keys and values between 2^-32 and 2^32 in one request (bf16 outputs hold them)."""
    G, H, dh, page, kv = 2, 4, 64, 16, 300
    kc, ke = make_cache(20, G, page, dh, "hnd", 1, -9, -7)
    vc, ve = make_cache(20, G, page, dh, "hnd", 2, -32, 32)
    torch.manual_seed(0)
    q = (0.3 * torch.randn(n, H, dh, device="cuda")).to(BF16)
    table = tables([kv], page, 20)
    out, lse = attn(P, q, kc, ke, vc, ve, table, [0, n], [kv])
    want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, n], [kv])
    R16.check(out, want, tol, "out")
    R16.check(lse, wl, ltol, "lse")
    # blocks of zeros under the smallest exponent beside them
    vc.view(torch.uint8)[table[0][3]] = 0
    ve[table[0][3]] = -32
    ve[table[0][4:]] = 5
    out, lse = attn(P, q, kc, ke, vc, ve, table, [0, n], [kv])
    want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, n], [kv])
    R16.check(out, want, tol, "out")
    R16.check(lse, wl, ltol, "lse")


@pytest.mark.parametrize("H,G,dh", [(8, 1, 64), (4, 4, 128)])
@pytest.mark.parametrize("n", [1, 4, 40, 200])
@pytest.mark.parametrize("window", [0, 30])
def test_attention_not_finite(P, H, G, dh, n, window):
    """A NaN in keys or values reaches the tokens that see it, and no others; what lies behind the
    last position, in unseen pages and in rows of no request may be anything."""
    page, kv = 16, 260
    kc, ke = quantised(20, G, page, dh, "hnd", 1)
    vc, ve = quantised(20, G, page, dh, "hnd", 2)
    torch.manual_seed(n)
    q = torch.randn(n, H, dh, device="cuda").half()
    table = tables([kv], page, 20, 4)
    k8, v8 = kc.view(torch.uint8), vc.view(torch.uint8)
    last = table[0][-1]
    k8[last, :, kv % page:], v8[last, :, kv % page:] = 0x7f, 0xff         # behind the last position
    for p in set(range(20)) - set(table[0]):
        k8[p], v8[p], ke[p], ve[p] = 0x7f, 0x7f, 127, -128
    clean = attn(P, q, kc, ke, vc, ve, table, [0, n], [kv], window)
    want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, n], [kv], window)
    R16.check(clean[0], want, tol, "clean")
    for pos, key in ((kv - 1, False), (kv - 1 - n // 2, False), (kv - n, True), (kv - 1 - n // 2, True), (max(0, kv - n - 12), False)):
        k2, v2 = kc.clone(), vc.clone()
        (k2 if key else v2).view(torch.uint8)[table[0][pos // page], 0, pos % page, 5] = 0x7f
        out, lse = attn(P, q, k2, ke, v2, ve, table, [0, n], [kv], window)
        want, wl, tol, ltol = R.attention(q, k2, ke, v2, ve, i32(table), [0, n], [kv], window)
        R16.check(out, want, tol, f"out {pos} {key}")
        R16.check(lse, wl, ltol, f"lse {pos} {key}")
    # a query of NaN, and one that outgrows its type's products
    q2 = q.clone()
    q2[n - 1, 0, 3] = math.nan
    out, lse = attn(P, q2, kc, ke, vc, ve, table, [0, n], [kv], window)
    assert bool(torch.isnan(out[n - 1, 0]).all()) and bool(torch.isnan(lse[n - 1, 0]))
    R16.check(out[n - 1, 1:], clean[0][n - 1, 1:].double(), torch.zeros_like(tol[n - 1, 1:]), "others")


def test_attention_of_tiny_and_huge_queries(P):
    """bf16 queries far outside fp16's range."""
    kc, ke = quantised(20, 2, 16, 64, "hnd", 1)
    vc, ve = quantised(20, 2, 16, 64, "hnd", 2)
    table = tables([300], 16, 20)
    for f, scale in ((1e-30, 1e29), (1e30, 1e-31), (1e-38, 0.1), (3e37, 1e-38)):
        torch.manual_seed(1)
        q = (torch.randn(3, 4, 64, device="cuda") * f).to(BF16)
        out, lse = attn(P, q, kc, ke, vc, ve, table, [0, 3], [300], scale=scale)
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, 3], [300], 0, scale)
        R16.check(out, want, tol, f"{f}")
        R16.check(lse, wl, ltol, f"{f}")


def test_attention_inconsistent_requests(P):
    """As for the 16-bit cache: such a row counts as one without tokens or keys, bad pages read as zeros, all reported."""
    kc, ke = quantised(20, 2, 16, 64, "hnd", 1)
    vc, ve = quantised(20, 2, 16, 64, "hnd", 2)
    q = torch.randn(6, 4, 64, device="cuda").half()
    table = tables([40, 40, 40], 16, 20)
    # (the order of a row's sums goes by all requests of the step, so rows are held to the bound of their own sums)
    good, _, tol, _ = R.attention(q, kc, ke, vc, ve, i32(table), [0, 2, 4, 6], [40, 33, 20])
    out, _ = attn(P, q, kc, ke, vc, ve, table, [0, 2, 4, 6], [40, 33, 20])
    assert P.pi_last_device_status() == 0
    R16.check(out, good, tol)
    out, _ = attn(P, q, kc, ke, vc, ve, table, [0, 2, 4, 6], [40, 49, 20])      # more than a table row holds
    assert P.pi_last_device_status() == 1
    R16.check(out[[0, 1, 4, 5]], good[[0, 1, 4, 5]], tol[[0, 1, 4, 5]])
    assert bool((out[2:4] == 0).all())
    out, _ = attn(P, q, kc, ke, vc, ve, table, [0, 2, 9, 6], [40, 33, 20], max_new=6)   # past the rows, then decreasing
    assert P.pi_last_device_status() == 1
    R16.check(out[:2], good[:2], tol[:2])
    assert bool((out[2:] == 7).all())
    out, _ = attn(P, q, kc, ke, vc, ve, table, [0, 2, 4, 6], [40, -1, 20])
    assert P.pi_last_device_status() == 1
    R16.check(out[4:], good[4:], tol[4:])
    # a page outside the cache: scores of zero and values of zero
    bad = [list(r) for r in table]
    bad[0][1] = 20
    out, _ = attn(P, q, kc, ke, vc, ve, bad, [0, 2, 4, 6], [40, 33, 20])
    assert P.pi_last_device_status() == 1
    R16.check(out[2:], good[2:], tol[2:])
    k2, v2 = kc.clone(), vc.clone()
    k2.view(torch.uint8)[table[0][1]] = 0
    v2.view(torch.uint8)[table[0][1]] = 0
    zeros, _, tol, _ = R.attention(q, k2, ke, v2, ve, i32(table), [0, 2, 4, 6], [40, 33, 20])
    R16.check(out[:2], zeros[:2], tol[:2])


def test_attention_strides_and_no_lse(P):
    kc, ke = quantised(20, 2, 16, 64, "nhd", 1)
    vc, ve = quantised(20, 2, 16, 64, "nhd", 2)
    qkv = torch.randn(5, 8 * 64 + 24, device="cuda").to(BF16)
    q = qkv[:, :4 * 64].unflatten(1, (4, 64))
    table = tables([100], 16, 20)
    out, _ = attn(P, q, kc, ke, vc, ve, table, [0, 5], [100], q_pad=8, lse=False)
    want, _, tol, _ = R.attention(q, kc, ke, vc, ve, i32(table), [0, 5], [100])
    R16.check(out, want, tol)
    # both caches in slices of larger ones, heads apart
    big = torch.zeros(20, 3, 48, 2, 64, dtype=torch.uint8, device="cuda")
    big[:, 1, :16], big[:, 2, :16] = kc.view(torch.uint8).transpose(1, 2), vc.view(torch.uint8).transpose(1, 2)
    k2, v2 = (big[:, i, :16].transpose(1, 2).view(R.CODE) for i in (1, 2))
    again, _ = attn(P, q, k2, ke, v2, ve, table, [0, 5], [100], lse=False)
    assert torch.equal(again, out)


def test_attention_one_workspace_and_repeats(P):
    """Steps of many sizes one after the other on one workspace, each twice: the same bits."""
    G, H, dh, page = 4, 8, 64, 16
    kc, ke = quantised(600, G, page, dh, "hnd", 1)
    vc, ve = quantised(600, G, page, dh, "hnd", 2)
    cache = P.page8_desc(kc, vc)
    ws = torch.zeros(P.pi_paged8_workspace_bytes(P.paged_desc(H, 20, 4000, 1000, 600), cache), dtype=torch.uint8, device="cuda")
    rng = random.Random(1)
    for step in range(12):
        B = rng.choice((1, 2, 7, 20))
        n = [rng.choice((1, 1, 1, 2, 30, 200)) for _ in range(B)]
        kv = [x + rng.randint(0, 200) for x in n]
        q = torch.randn(sum(n), H, dh, device="cuda").half()
        table, cu = tables(kv, page, 600, step), starts(n)
        a = attn(P, q, kc, ke, vc, ve, table, cu, kv, ws=ws)
        b = attn(P, q, kc, ke, vc, ve, table, cu, kv, ws=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), cu, kv)
        R16.check(a[0], want, tol, f"step {step}")
        R16.check(a[1], wl, ltol, f"step {step}")
    assert P.pi_last_device_status() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dt", [F16, BF16])
def test_serving_with_eight_bits(P, dt):
    """PagedCache end to end: prompts in chunks, decode steps, a request that ends and one that rolls back;
    the attention against its definition over what the cache holds, the cache against what was stored."""
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    B, H, G, dh, page = 3, 8, 2, 64, 16
    cache = PagedCache(H, G, dh, B, 200, 70, 160, layers=2, page_size=page, dtype=dt, rope=P.rope_plan(dh, 32), bits=8)
    torch.manual_seed(0)
    steps = [([70, 30, 1], None), ([20, 1, 1], None), ([1, 1, 1], None), ([1, 1, 1], [60, 31, 3]), ([33, 5, 1], [61, 0, 4]), ([1, 1, 1], None)]
    have = [0] * B
    for new, keep in steps:
        T = sum(new)
        cache.begin(i32(new), T, max(new), None if keep is None else i32(keep))
        have = [(h if keep is None else min(h, k)) + n for h, k, n in zip(have, keep or have, new)]
        assert cache.kv_len.tolist() == have
        for layer in range(2):
            q, k, v = (torch.randn(T, x, dh, device="cuda") for x in (H, G, G))
            out = torch.empty(T, H, dh, dtype=dt, device="cuda")
            cache.attend(layer, q, k, v, out)
            pos = cache.positions[:T].long()
            qt, _ = R16.rotate(q, pos, R16.frequencies(32, 10000.0), False)
            turned = cache.q[:T]
            assert float((turned.double() - qt).abs().max()) <= float(qt.abs().max()) * R16.half_step(dt) * 1.01
            want, _, tol, _ = R.attention(turned, cache.kcache[layer], cache.kexp[layer], cache.vcache[layer], cache.vexp[layer],
                                          cache.table, cache.cu.tolist(), have)
            R16.check(out, want, tol, "out")
            # what was stored reads back within half a step of the block's largest value
            rows = starts(have)
            kr, vr = cache.read(layer, None, i32(rows), rows[-1], dtype=F32)
            at = torch.cat([torch.arange(rows[b + 1] - new[b], rows[b + 1]) for b in range(B)]).cuda()
            assert float((vr[at] - v).abs().max()) <= 2.0 ** -4 * float(v.abs().max()) * 1.0001
            assert kr.shape == (rows[-1], G, dh)
    assert P.pi_last_device_status() == 0
    with pytest.raises(ValueError):
        PagedCache(H, G, dh, B, 200, 70, 160).read(0, None, i32([0, 1, 1, 1]), 1)


def test_decode_step_captured(P):
    """A captured decode step goes on from where the last replay ended, as eager steps do."""
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    B, H, G, dh = 5, 8, 2, 128
    make = lambda: PagedCache(H, G, dh, B, 300, 40, 200, page_size=16, rope=P.rope_plan(dh), bits=8)  # noqa: E731
    torch.manual_seed(3)
    x = torch.randn(40, 200, (H + 2 * G) * dh, device="cuda").half()
    cur = torch.empty(B, (H + 2 * G) * dh, dtype=F16, device="cuda")
    split = lambda y: [z.unflatten(1, (-1, dh)) for z in y.split([H * dh, G * dh, G * dh], dim=1)]  # noqa: E731
    ones, res = i32([1] * B), []
    for captured in (False, True):
        c = make()
        c.begin(i32([40, 1, 17, 33, 9]), 100, 40)
        c.attend(0, *split(x[0, :100]), torch.empty(100, H, dh, dtype=F16, device="cuda"))
        out = torch.empty(B, H, dh, dtype=F16, device="cuda")

        def step():
            c.begin(ones, B, 1)
            c.attend(0, *split(cur), out)

        cur.copy_(x[1, :B])
        step()
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph):
                step()
        outs = []
        for t in range(2, 40):
            cur.copy_(x[t, :B])
            graph.replay() if captured else step()
            outs.append(out.clone())
        res.append((torch.stack(outs), c.kv_len.clone(), c.kexp[0].clone(), c.kcache[0].view(torch.uint8).clone()))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_two_streams(P):
    """Calls on two streams with workspaces of their own, at the same time."""
    kc, ke = quantised(300, 8, 16, 128, "hnd", 1)
    vc, ve = quantised(300, 8, 16, 128, "hnd", 2)
    kv = [700, 64, 1500, 300]
    table = i32(tables(kv, 16, 300))
    cache = P.page8_desc(kc, vc)
    d = P.paged_desc(64, 4, 4, 1, table.shape[1])
    q = torch.randn(4, 64, 128, device="cuda").half()
    cu, kvl = i32([0, 1, 2, 3, 4]), i32(kv)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(3)]
    ws = [torch.zeros(P.pi_paged8_workspace_bytes(d, cache), dtype=torch.uint8, device="cuda") for _ in range(3)]
    P.pi_paged_attn8(d, cache, q, kc, vc, ke, ve, table, cu, kvl, outs[2], None, ws[2])
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, w in zip(streams, outs, ws):
            with torch.cuda.stream(s):
                P.pi_paged_attn8(d, cache, q, kc, vc, ke, ve, table, cu, kvl, o, None, w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


def test_the_command_serves_with_eight_bits(P, capsys):
    from activation_sparse_ffn_layer_gb300 import paged
    paged.main(["--config", "c4", "--requests", "3", "--prompt", "50", "--chunk", "20", "--tokens", "4", "--layers", "2", "--bits", "8"])
    assert "decode steps" in capsys.readouterr().out


# ------------------------------------------------------------------ wide batches, layouts, limits

@pytest.mark.parametrize("B,long", [(700, 0), (4096, 0), (600, 5)])
def test_attention_of_many_requests(P, B, long):
    """More requests than threads of a block, most of one token, some without tokens, some (`long`) of 80."""
    rng = random.Random(B)
    H, G, dh, page = 2, 2, 64, 16
    n = [rng.choice((1, 1, 1, 0)) for _ in range(B)]
    for i in range(long):
        n[rng.randrange(B)] = 80
    kv = [x + rng.randint(0, 40) if x else 0 for x in n]
    check(P, H, G, dh, F16, page, "hnd", n, kv, seed=B, extra=1)


@pytest.mark.parametrize("H,G,dh", [(8, 2, 64), (32, 2, 128)])
@pytest.mark.parametrize("gap", [1, 3, 20])
def test_attention_with_empty_requests_between(P, H, G, dh, gap):
    """Requests without keys between others: a warp that ends a cut item goes on through them to items with keys."""
    n, kv = [], []
    for i in range(40):
        n += [1] + [1] * gap
        kv += [37 + 90 * (i * 7 % 23)] + [0] * gap
    check(P, H, G, dh, F16, 16, "hnd", n, kv, seed=gap)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("how", ["keys first", "values first", "one array", "far apart"])
def test_attention_where_the_arrays_lie(P, page, dh, how):
    """Keys below values in memory, above them, the same array for both, and two arrays far from one another."""
    G, H, kv = 2, 8, [300, 45]
    used = sum(-(-x // page) for x in kv)
    a, ea = quantised(used, G, page, dh, "hnd", 1)
    b, eb = quantised(used, G, page, dh, "hnd", 2)
    if how in ("keys first", "values first"):
        both = torch.empty(2, *a.shape, dtype=torch.uint8, device="cuda")
        i = 0 if how == "keys first" else 1
        both[i], both[1 - i] = a.view(torch.uint8), b.view(torch.uint8)
        kc, vc = both[i].view(R.CODE), both[1 - i].view(R.CODE)
        assert (kc.data_ptr() < vc.data_ptr()) == (i == 0)
    elif how == "one array":
        kc, vc = a, a
    else:
        spacer = torch.empty(3 << 30, dtype=torch.uint8, device="cuda")
        kc, vc = a.view(torch.uint8).clone().view(R.CODE), b
        del spacer
    q = torch.randn(2, H, dh, device="cuda").half()
    table = tables(kv, page, used, 1)
    out, lse = attn(P, q, kc, ea, vc, eb, table, [0, 1, 2], kv)
    want, wl, tol, ltol = R.attention(q, kc, ea, vc, eb, i32(table), [0, 1, 2], kv)
    R16.check(out, want, tol, "out")
    R16.check(lse, wl, ltol, "lse")
    assert P.pi_last_device_status() == 0


@pytest.mark.parametrize("page", [16, 32, 128])
def test_attention_behind_a_window_whose_pages_are_gone(P, page):
    """Table entries of positions that no token sees any more are not looked at."""
    G, H, dh, kv, window = 2, 8, 64, 1000, 75
    used = -(-kv // page)
    kc, ke = quantised(used, G, page, dh, "hnd", 1)
    vc, ve = quantised(used, G, page, dh, "hnd", 2)
    table = tables([kv], page, used, 2)
    for n in (1, 4, 90):
        q = torch.randn(n, H, dh, device="cuda").to(BF16)
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), [0, n], [kv], window)
        gone = [list(table[0])]
        for j in range((kv - n - window + 1) // page):
            gone[0][j] = -1
        out, lse = attn(P, q, kc, ke, vc, ve, gone, [0, n], [kv], window)
        assert P.pi_last_device_status() == 0
        R16.check(out, want, tol, f"{n}")
        R16.check(lse, wl, ltol, f"{n}")


@pytest.mark.parametrize("n,kv,H,G", [([1] * 6, [30000, 20000, 300, 25000, 17, 30000], 64, 8), ([4] * 3, [30000, 8000, 30000], 64, 8),
                                      ([300, 1], [4000, 2000], 4, 2)])
def test_attention_whose_waits_run_out(P, n, kv, H, G):
    """With a wait limit of 1 ns a wait that is not satisfied at its first tries gives up: the warps wait for their own
    copies and return, and the status is PI_ERR_TIMEOUT.  The kernel of few rows waits for nothing but copies that it has
    asked for, and a try lasts longer than those, so that its waits end well; the 16-bit kernel's, in a step with a long
    request, run out.  After a zero fill of the workspace the same call gives the bits of a clean run."""
    dh, page = 128, 16
    used = sum(-(-x // page) for x in kv)
    kc, ke = quantised(used, G, page, dh, "hnd", 1)
    vc, ve = quantised(used, G, page, dh, "hnd", 2)
    q = torch.randn(sum(n), H, dh, device="cuda").half()
    table, cu = tables(kv, page, used, 1), starts(n)
    d = P.paged_desc(H, len(kv), sum(n), max(n), len(table[0]))
    ws = torch.zeros(P.pi_paged8_workspace_bytes(d, P.page8_desc(kc, vc)), dtype=torch.uint8, device="cuda")
    want = attn(P, q, kc, ke, vc, ve, table, cu, kv, ws=ws)
    assert P.pi_last_device_status() == 0
    seen = []
    for limit in (1, 1, 1, 1, 3000):
        P.pi_debug_set_wait_timeout(limit)
        try:
            attn(P, q, kc, ke, vc, ve, table, cu, kv, ws=ws)
            torch.cuda.synchronize()
        finally:
            P.pi_debug_set_wait_timeout(0)
        seen.append(P.pi_last_device_status())
        ws.zero_()
        for _ in range(3):
            got = attn(P, q, kc, ke, vc, ve, table, cu, kv, ws=ws)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert P.pi_last_device_status() == 0
    assert set(seen) <= {0, 4} and (4 in seen or max(n) < 64)


@pytest.mark.parametrize("seed", range(6))
def test_steps_of_many_shapes_on_one_workspace(P, seed):
    """Decodes, proposals, chunks and empty rows, cut anywhere by the blocks' and warps' borders, one step after the
    other on one workspace that is filled with zeros only once."""
    r = random.Random(100 + seed)
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(4):
        H, G = r.choice([(4, 4), (8, 2), (16, 1), (64, 8), (24, 8)])
        dh, dt, page, window = r.choice([64, 128]), r.choice([F16, BF16]), r.choice([16, 32, 128]), r.choice([0, 0, 1, 300])
        n, kv = [], []
        for _ in range(r.choice([1, 2, 5, 40])):
            n.append(r.choice([0, 1, 1, 1, r.randint(2, 12), r.randint(30, 200)]))
            kv.append(n[-1] + r.choice([0, r.randint(0, 100), r.randint(100, 1500)]))
        if not any(n):
            n.append(1), kv.append(700)
        used = sum(-(-x // page) for x in kv)
        kc, ke = quantised(used, G, page, dh, r.choice(("hnd", "nhd")), 1)
        vc, ve = quantised(used, G, page, dh, "hnd" if kc.is_contiguous() else "nhd", 2)
        q = torch.randn(sum(n), H, dh, device="cuda").to(dt)
        table, cu = tables(kv, page, used, seed), starts(n)
        out, lse = attn(P, q, kc, ke, vc, ve, table, cu, kv, window, ws=ws)
        want, wl, tol, ltol = R.attention(q, kc, ke, vc, ve, i32(table), cu, kv, window)
        R16.check(out, want, tol, "out")
        R16.check(lse, wl, ltol, "lse")
    assert P.pi_last_device_status() == 0


@pytest.mark.parametrize("T", [600, 3000])
def test_store_of_many_single_tokens(P, T):
    """Steps of many decoding rows (the windows of 1, 4 and 16 tokens): a block each."""
    G, dh, page = 4, 64, 16
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


def store_each(codes, exps, x, slots, page):
    """R.store for tokens in blocks of their own, all at once (pages of one block)."""
    keep = torch.tensor([s >= 0 for s in slots], device="cuda")
    at = torch.tensor(slots, device="cuda")[keep]
    y = x[keep]
    e = torch.tensor([[R.exponent(z) for z in row] for row in y.abs().amax(-1).tolist()], device="cuda")
    p, r = at // page, at % page
    old = exps[p, :, 0].long()
    new = torch.where(r[:, None] > 0, torch.maximum(e, old), e)
    kept = codes[p]                                             # [tokens, heads, page, dh]
    again = R.encode(R.VALUES.cuda()[kept.long()] * torch.exp2((old - new).double())[..., None, None])
    stay = torch.arange(page, device="cuda")[None, :] < r[:, None]
    codes[p] = torch.where(stay[:, None, :, None], again, kept)
    codes[p, :, r] = R.encode(y / torch.exp2(new.double())[..., None])
    exps[p, :, 0] = new.to(torch.int8)


def test_caches_past_32_bits(P):
    """Pages whose codes lie more than 2^32 bytes behind the start: stored, read back and attended to (few rows and many)
    as in a small cache, with the same lengths and so the same bits."""
    G, H, dh, page, pages = 8, 16, 128, 64, 66000
    used, kv, n = 20, [700, 420], [1, 1]
    far = [pages - 1 - 7 * i for i in range(used)]
    assert min(far) * G * page * dh > 1 << 32
    small = [torch.zeros(used, G, page, dh, dtype=torch.uint8, device="cuda").view(R.CODE) for _ in range(2)]
    big = [torch.zeros(pages, G, page, dh, dtype=torch.uint8, device="cuda").view(R.CODE) for _ in range(2)]
    ex = [torch.zeros(used, G, page // 16, dtype=torch.int8, device="cuda") for _ in range(2)]
    bex = [torch.zeros(pages, G, page // 16, dtype=torch.int8, device="cuda") for _ in range(2)]
    table = tables(kv, page, used, 5)
    ftable = [[far[x] if x >= 0 else -1 for x in r] for r in table]
    torch.manual_seed(2)
    T = sum(kv)
    x = torch.randn(T, (H + 2 * G) * dh, device="cuda").to(BF16)
    q, k, v = (y.unflatten(1, (-1, dh)) for y in x.split([H * dh, G * dh, G * dh], dim=1))
    pos = [p for c in kv for p in range(c)]
    res = []
    for (kc, vc), (ke, ve), tb in ((small, ex, table), (big, bex, ftable)):
        slots = torch.tensor([tb[b][p // page] * page + p % page for b, c in enumerate(kv) for p in range(c)], device="cuda")
        qo = torch.empty(T, H, dh, dtype=BF16, device="cuda")
        P.pi_rope_store8(P.rope_plan(dh), P.page8_desc(kc, vc), q, k, v, i32(pos), slots, qo, kc, vc, ke, ve)
        ko, vo = (torch.empty(T, G, dh, dtype=BF16, device="cuda") for _ in range(2))
        P.pi_page_read8(P.read8_desc(2, len(tb[0]), T), P.page8_desc(kc, vc), kc, vc, ke, ve, i32(tb), None, i32(starts(kv)), ko, vo)
        out = [qo, ko, vo]
        for m in (n, [90, 300]):
            out += attn(P, q[:sum(m)], kc, ke, vc, ve, tb, starts(m), kv)
        res.append(out)
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert P.pi_last_device_status() == 0 and float(res[0][2].float().std()) > 0.5


@pytest.mark.parametrize("dh,H,G", [(64, 1, 1), (128, 128, 1), (128, 1024, 8), (64, 1024, 1024)])
def test_the_ends_of_the_head_counts(P, dh, H, G):
    """One head, the largest groups and the most heads, few rows and a long request."""
    check(P, H, G, dh, F16, 16, "nhd", [1, 2], [33, 20], seed=dh)
    check(P, H, G, dh, BF16, 16, "hnd", [70], [75], seed=dh + 1)
