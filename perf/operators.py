"""Cases of the paged-serving operators: block tables and slot maps built on the GPU
(``pi_block_tables``), rotary positions with the store into the paged cache
(``pi_rope_store``) and attention of new tokens over that cache (``pi_paged_attn``).

``listed()`` gives fixed cases, ``draw(rng)`` one more of the same ranges, ``prepare`` the
tensors a serving loop has in hand before the call, ``run`` one pass (plain torch, or the
package's kernels where ``own`` is true), ``work`` the bytes and operations a pass cannot do
without, and ``exact`` the outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}

# (query heads, key/value heads, head width): the repository's attention blocks, then shared
# key/value heads in groups of 3, of 16 and of 4
HEADS = ((12, 12, 64), (32, 32, 128), (56, 56, 128), (64, 8, 128), (96, 96, 128), (24, 8, 128), (16, 1, 64), (32, 8, 64))

# what a drawn case may cost at most: just under the largest listed case of its operator
MOST_TOKENS_TABLES = 60000
MOST_ROPE_BYTES = 650e6
MOST_ATTN_FLOPS = 1.8e12
MOST_ATTN_BYTES = 2.0e9
MOST_SCORES = 4.0e9     # elements of the padded score matrix of the plain form


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # Block tables. A decode step of a small service: eight requests take one token each.
        dict(name="tables_decode_8", op="tables", batch=8, page=16, max_pages=64, fresh=0.0, idle=0.0, chunk=0.0,
             n_hi=1, c_hi=1000, pool=1.5, rs=11),
        # A step of a mid-size service: decodes, prompt chunks, rows that just changed their request.
        dict(name="tables_mixed_200", op="tables", batch=200, page=32, max_pages=128, fresh=0.15, idle=0.1, chunk=0.2,
             n_hi=512, c_hi=4000, pool=1.3, rs=12),
        # The largest step: 2048 rows, some 60 thousand new tokens, a pool that runs out for the last rows.
        dict(name="tables_mixed_2048", op="tables", batch=2048, page=16, max_pages=512, fresh=0.2, idle=0.05, chunk=0.25,
             n_hi=500, c_hi=8000, pool=0.9, rs=13),
        # Rotary positions and store. One decode step of 32 sequences (grouped heads, half layout): a matter of latency.
        dict(name="rope_decode_32", op="rope", tokens=32, each=1, heads=64, kv_heads=8, dh=128, rot=128, inter=False,
             base=10000.0, scaling="none", factor=1.0, p_hi=4000, inp="f16", dt="f16", page=16, pad=0, order="hnd", rs=21),
        # A prompt chunk of odd length from fp32 projections; interleaved pairs on half of the head, positions interpolated.
        dict(name="rope_chunk_1999", op="rope", tokens=1999, each=1999, heads=32, kv_heads=32, dh=128, rot=64, inter=True,
             base=10000.0, scaling="linear", factor=4.0, p_hi=8000, inp="f32", dt="f16", page=32, pad=0, order="hnd", rs=22),
        # Many prompts at once, bfloat16, far positions with frequencies scaled by bands; some padding tokens at the end.
        dict(name="rope_prompts_16384", op="rope", tokens=16384, each=4096, heads=64, kv_heads=8, dh=128, rot=128, inter=False,
             base=500000.0, scaling="ramp", factor=16.0, p_hi=900000, inp="bf16", dt="bf16", page=64, pad=37, order="nhd", rs=23),
        # Attention. One sequence, one token, a short cache: the smallest call.
        dict(name="attn_decode_1", op="attn", batch=1, heads=64, kv_heads=8, dh=128, dt="f16", page=16, n_lo=1, n_hi=1,
             c_lo=1000, c_hi=1000, dec=1.0, window=0, order="hnd", rs=31),
        # A decode step of 32 sequences of very different lengths over grouped heads.
        dict(name="attn_decode_32", op="attn", batch=32, heads=64, kv_heads=8, dh=128, dt="f16", page=16, n_lo=1, n_hi=1,
             c_lo=500, c_hi=8000, dec=1.0, window=0, order="hnd", rs=32),
        # Four sequences with long caches: the most bytes.
        dict(name="attn_decode_long", op="attn", batch=4, heads=64, kv_heads=8, dh=128, dt="bf16", page=64, n_lo=1, n_hi=1,
             c_lo=120000, c_hi=131000, dec=1.0, window=0, order="nhd", rs=33),
        # A step that serves decodes and prompt chunks together, multi-head, with a sliding window.
        dict(name="attn_mixed_16", op="attn", batch=16, heads=32, kv_heads=32, dh=128, dt="bf16", page=32, n_lo=100, n_hi=700,
             c_lo=1, c_hi=4000, dec=0.7, window=2000, order="hnd", rs=34),
        # A whole prompt of odd length in the small multi-head block (64-wide heads).
        dict(name="attn_prompt_1999", op="attn", batch=1, heads=12, kv_heads=12, dh=64, dt="f16", page=16, n_lo=1999, n_hi=1999,
             c_lo=0, c_hi=0, dec=0.0, window=0, order="hnd", rs=35),
        # A chunk of 4096 tokens behind 12288 cached ones over grouped heads: the most operations.
        dict(name="attn_chunk_4096", op="attn", batch=1, heads=64, kv_heads=8, dh=128, dt="bf16", page=16, n_lo=4096, n_hi=4096,
             c_lo=12288, c_hi=12288, dec=0.0, window=0, order="hnd", rs=36),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1) + 0.49)))))))


def draw(rng):
    op = rng.choice(("tables", "rope", "rope", "attn", "attn", "attn"))
    rs = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 64, 128))
    if op == "tables":
        batch = _log(rng, 1, 2048)
        c = dict(op=op, batch=batch, page=page, max_pages=_log(rng, 64, 512), fresh=rng.uniform(0, 0.4),
                 idle=rng.uniform(0, 0.3), chunk=rng.uniform(0, 0.5), n_hi=_log(rng, 1, 1000), c_hi=0,
                 pool=rng.uniform(0.8, 2.0), rs=rs)
        c["c_hi"] = _log(rng, 1, min(8000, page * c["max_pages"] - c["n_hi"] - 1)) if page * c["max_pages"] > c["n_hi"] + 2 else 1
        c["n_hi"] = min(c["n_hi"], page * c["max_pages"] - c["c_hi"])
        while sum(_table_lengths(c)[1]) > MOST_TOKENS_TABLES:
            c["n_hi"] = max(1, c["n_hi"] // 2)
        return c
    heads, kv_heads, dh = rng.choice(HEADS)
    dt, order = rng.choice(("f16", "bf16")), rng.choice(("hnd", "nhd"))
    if op == "rope":
        inp = rng.choice((dt, dt, "f32"))
        per = (heads + 2 * kv_heads) * dh * (SIZE[inp] + 2)
        tokens = _log(rng, 1, min(16384, int(MOST_ROPE_BYTES / per)))
        scaling = rng.choice(("none", "linear", "blend", "ramp"))
        return dict(op=op, tokens=tokens, each=_log(rng, 1, tokens), heads=heads, kv_heads=kv_heads, dh=dh,
                    rot=rng.choice((dh, dh, dh // 2, 16, 48)), inter=rng.random() < 0.5, base=rng.choice((10000.0, 500000.0)),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 4.0, 16.0)),
                    p_hi=_log(rng, 1, 1000000), inp=inp, dt=dt, page=page, pad=rng.choice((0, 0, 3)) if tokens > 3 else 0,
                    order=order, rs=rs)
    kind = rng.choice(("decode", "chunk", "mixed"))
    c = dict(op=op, batch=_log(rng, 1, 32), heads=heads, kv_heads=kv_heads, dh=dh, dt=dt, page=page, n_lo=1, n_hi=1,
             c_lo=0, c_hi=_log(rng, 1, 131000), dec=1.0, window=rng.choice((0, 0, _log(rng, 1, 5000))), order=order, rs=rs)
    if kind != "decode":
        c["n_hi"], c["dec"], c["c_hi"] = _log(rng, 2, 4096), 0.0 if kind == "chunk" else rng.uniform(0.3, 0.9), _log(rng, 1, 16000)
        c["n_lo"] = _log(rng, 1, c["n_hi"])
    else:
        c["c_lo"] = rng.randrange(c["c_hi"])
    while True:
        n, k = _attn_lengths(c)
        w = work(c)
        scores = c["batch"] * heads * max(n) * max(k)
        if w["flops"] <= MOST_ATTN_FLOPS and w["bytes"] <= MOST_ATTN_BYTES and scores <= MOST_SCORES \
                and 4 * c["batch"] * kv_heads * max(k) * dh * 2 <= 20e9:
            return c
        if c["batch"] > 1:
            c["batch"] = max(1, c["batch"] * 2 // 3)
        elif c["n_hi"] > 64:
            c["n_hi"] = c["n_hi"] * 2 // 3
            c["n_lo"] = min(c["n_lo"], c["n_hi"])
        else:
            c["c_hi"] = c["c_hi"] * 2 // 3
            c["c_lo"] = min(c["c_lo"], c["c_hi"])


# --------------------------------------------------- lengths (whole numbers, from the case alone)

def _table_lengths(case):
    """Per row: tokens kept, tokens to come, pages held."""
    r, page, most = random.Random(case["rs"]), case["page"], case["page"] * case["max_pages"]
    cached, new, held = [], [], []
    for _ in range(case["batch"]):
        what = r.random()
        before = r.randint(1, max(1, min(case["c_hi"], most)))
        n = _log(r, 1, case["n_hi"]) if r.random() < case["chunk"] else 1
        if what < case["fresh"]:            # a new request in a row whose last one has ended
            c = 0
        elif what < case["fresh"] + case["idle"]:   # the row's request has ended and none follows
            c, n = 0, 0
        else:
            c = before
        cached.append(c)
        new.append(min(n, most - c))
        held.append(-(-before // page))
    return cached, new, held


def _attn_lengths(case):
    """Per request: new tokens, keys in the cache with them."""
    r = random.Random(case["rs"])
    n, k = [], []
    for _ in range(case["batch"]):
        one = r.random() < case["dec"]
        n.append(1 if one else _log(r, case["n_lo"], case["n_hi"]))
        k.append(n[-1] + (r.randint(case["c_lo"], case["c_hi"]) if case["c_hi"] > case["c_lo"] else case["c_lo"]))
    return n, k


def _visible(n, k, window):
    """Keys that the n newest of k positions see together, and the oldest key that any of them sees."""
    if window <= 0:
        return n * k - n * (n - 1) // 2, 0
    first = k - n                      # position p sees min(p + 1, window) keys
    ramp = max(0, min(n, window - 1 - first))
    return ramp * (first + 1) + ramp * (ramp - 1) // 2 + (n - ramp) * window, max(0, first - window + 1)


# ----------------------------------------------------------------------------- inputs

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _cache(pages, kv_heads, page, dh, order, dt, g, dev):
    """A cache tensor [pages, kv_heads, page, dh], stored heads first ("hnd") or tokens first ("nhd")."""
    if order == "hnd":
        return torch.randn(pages, kv_heads, page, dh, generator=g, device=dev, dtype=TYPES[dt])
    return torch.randn(pages, page, kv_heads, dh, generator=g, device=dev, dtype=TYPES[dt]).transpose(1, 2)


def _inputs(case, seed):
    """The tensors of a case, from the seed alone (the lengths are the case's)."""
    dev = _device()
    g = _gen(seed, dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] == "tables":
        cached, new, held = _table_lengths(case)
        need = sum(max(0, -(-(c + n) // case["page"]) - h) for c, n, h in zip(cached, new, held))
        free = max(1, int(need * case["pool"]))
        pages = sum(held) + free
        perm = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
        B, M = case["batch"], case["max_pages"]
        table = torch.full((B, M), -1, dtype=torch.int32, device=dev)
        h = i32(held)
        col = torch.arange(M, device=dev)
        table[col[None, :] < h[:, None]] = perm[:sum(held)]
        stack = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        stack[:free] = perm[sum(held):]
        return dict(cached=i32(cached), new=i32(new), held=h, table=table, stack=stack, count=i32([free]),
                    pages=pages, tokens=sum(new))
    heads, kv_heads, dh, page = case["heads"], case["kv_heads"], case["dh"], case["page"]
    if case["op"] == "rope":
        T, each, pad = case["tokens"], case["each"], case["pad"]
        r = random.Random(case["rs"] + 7919 * int(seed))
        starts = [r.randint(0, case["p_hi"]) for _ in range(-(-T // each))]
        t = torch.arange(T, device=dev)
        req, off = t // each, t % each
        first = torch.tensor(starts, device=dev)[req]
        pos = first + off
        per = -(-(page + each) // page)        # pages that one run of tokens may touch
        perm = torch.randperm(per * len(starts), generator=g, device=dev)
        at = first % page + off
        slots = perm[req * per + at // page] * page + at % page
        slots[T - pad:] = -1
        qkv = torch.randn(T, (heads + 2 * kv_heads) * dh, generator=g, device=dev, dtype=TYPES[case["inp"]])
        q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv.split([heads * dh, kv_heads * dh, kv_heads * dh], dim=1))
        n = per * len(starts)
        return dict(q=q, k=k, v=v, pos=pos.to(torch.int32), slots=slots,
                    kc=_cache(n, kv_heads, page, dh, case["order"], case["dt"], g, dev),
                    vc=_cache(n, kv_heads, page, dh, case["order"], case["dt"], g, dev))
    n, k = _attn_lengths(case)
    used = [-(-x // page) for x in k]
    pages, M = sum(used) + 3, max(used)
    perm = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((case["batch"], M), -1, dtype=torch.int32, device=dev)
    table[torch.arange(M, device=dev)[None, :] < i32(used)[:, None]] = perm[:sum(used)]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    # queries of some heads are larger, so that their weights rest on few keys
    q = torch.randn(cu[-1], heads, dh, generator=g, device=dev)
    q *= torch.linspace(0.5, 3.0, heads, device=dev)[:, None]
    return dict(q=q.to(TYPES[case["dt"]]), kc=_cache(pages, kv_heads, page, dh, case["order"], case["dt"], g, dev),
                vc=_cache(pages, kv_heads, page, dh, case["order"], case["dt"], g, dev), table=table, cu=i32(cu),
                kv=i32(k), n=n, k=k)


# what the scaled frequencies of a rope case go by: the length the model was made for, and the
# borders of the bands ("blend" in wavelengths per length, "ramp" in turns per length)
ORIGINAL = 8192
BLEND = (1.0, 4.0)
RAMP = (1.0, 32.0)


def _mscale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dev = s["table"].device if "table" in s else s["q"].device
    new = lambda *shape, dt: torch.empty(*shape, dtype=dt, device=dev)  # noqa: E731
    # the buffers that a serving loop keeps from step to step
    if case["op"] == "tables":
        B, T = case["batch"], s["tokens"]
        s["held_out"], s["count_out"] = new(B, dt=torch.int32), new(1, dt=torch.int32)
        s["cu"], s["kv"] = new(B + 1, dt=torch.int32), new(B, dt=torch.int32)
        s["slots"], s["pos"] = new(T, dt=torch.int64), new(T, dt=torch.int32)
    elif case["op"] == "rope":
        s["q_out"] = new(*s["q"].shape, dt=TYPES[case["dt"]])
    else:
        s["out"], s["lse"] = torch.empty_like(s["q"]), new(*s["q"].shape[:2], dt=torch.float32)
    if own:   # ... and the descriptors, the rotary plan and the workspace that belong to them
        import activation_sparse_ffn_layer_gb300 as P
        if case["op"] == "tables":
            s["desc"] = P.tables_desc(case["batch"], case["page"], s["pages"], case["max_pages"], s["tokens"])
        elif case["op"] == "rope":
            lo, hi = RAMP if case["scaling"] == "ramp" else BLEND
            s["plan"] = P.rope_plan(case["dh"], case["rot"], interleaved=case["inter"], base=case["base"],
                                    scaling=case["scaling"], factor=case["factor"], original_max=ORIGINAL, low=lo, high=hi,
                                    mscale=_mscale(case))
            s["cache"] = P.page_desc(s["kc"], s["vc"])
        else:
            s["cache"] = P.page_desc(s["kc"], s["vc"])
            s["desc"] = P.paged_desc(case["heads"], case["batch"], s["q"].shape[0], max(s["n"]), s["table"].shape[1],
                                     window=case["window"])
            s["ws"] = torch.zeros(P.pi_paged_workspace_bytes(s["desc"], s["cache"]), dtype=torch.uint8, device=dev)
        s["P"] = P
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _tables(s) if op == "tables" else _rope(s) if op == "rope" else _attn(s)


def _own(s):
    P, op = s["P"], s["case"]["op"]
    if op == "tables":
        P.pi_block_tables(s["desc"], s["cached"], s["new"], s["held"], s["held_out"], s["table"], s["stack"], s["count"],
                          s["count_out"], s["cu"], s["kv"], s["slots"], s["pos"])
        return [s["held_out"], s["table"], s["stack"], s["count_out"], s["cu"], s["kv"], s["slots"], s["pos"]]
    if op == "rope":
        P.pi_rope_store(s["plan"], s["cache"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["q_out"], s["kc"], s["vc"])
        return [s["q_out"], s["kc"], s["vc"]]
    P.pi_paged_attn(s["desc"], s["cache"], s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], s["out"], s["lse"], s["ws"])
    return [s["out"], s["lse"]]


def _tables(s):
    """Each row's page list is cut or extended to hold cached + new tokens; pages given back go on the stack in row
    order, pages taken come off its top in row order, and a row that the stack cannot serve takes none."""
    case = s["case"]
    page, T = case["page"], s["tokens"]
    cached, new, held = s["cached"].long(), s["new"].long(), s["held"].long()
    table, stack, f = s["table"], s["stack"], s["count"].long()
    dev = table.device
    need = (cached + new + page - 1) // page
    give, want = (held - need).clamp(min=0), (need - held).clamp(min=0)
    give_end, want_end = give.cumsum(0), want.cumsum(0)
    give_all = give_end[-1]
    served = (want == 0) | (want_end <= f + give_all)
    take = want * served
    row = torch.arange(case["batch"], device=dev)
    col = torch.arange(case["max_pages"], device=dev)[None, :]
    # pages given back
    back = (col >= need[:, None]) & (col < held[:, None])
    where = f + (give_end - give)[:, None] + col - need[:, None]
    stack = torch.cat([stack, stack.new_zeros(1)]).scatter(0, torch.where(back, where, len(stack)).flatten(), table.flatten())[:-1]
    # pages taken
    got = served[:, None] & (col >= held[:, None]) & (col < need[:, None])
    top = f + give_all - 1 - ((want_end - want)[:, None] + col - held[:, None])
    table = torch.where(got, stack[top.clamp(0, len(stack) - 1)], table)
    held_out = torch.where(give > 0, need, held + take)
    end = new.cumsum(0)
    cu = torch.cat([end.new_zeros(1), end])
    i = torch.arange(T, device=dev)
    req = (i[:, None] >= end[None, :]).sum(1) if T * case["batch"] <= 1 << 28 else torch.searchsorted(end, i, right=True)
    pos = cached[req] + i - cu[req]
    slots = torch.where(served[req], table[row[req], pos // page].long() * page + pos % page, -1)
    kv = torch.where(served, cached + new, 0)
    i32 = torch.int32
    return [held_out.to(i32), table, stack, (f + give_all - take.sum()).to(i32), cu.to(i32), kv.to(i32), slots, pos.to(i32)]


def _frequencies(case, dev):
    rot, base, s = case["rot"], case["base"], case["factor"]
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    f = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return f / s
    if case["scaling"] == "blend":
        g = ((ORIGINAL * f / (2 * math.pi) - BLEND[0]) / (BLEND[1] - BLEND[0])).clamp(0, 1)
        return (1 - g) * f / s + g * f
    if case["scaling"] == "ramp":
        at = lambda turns: rot * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        a, z = max(math.floor(at(RAMP[1])), 0), min(math.ceil(at(RAMP[0])), rot - 1)
        g = ((i - a) / max(z - a, 0.001)).clamp(0, 1)
        return f / s * g + f * (1 - g)
    return f


def _rotate(x, cos, sin, rot, inter):
    a = x[..., 0:rot:2] if inter else x[..., :rot // 2]
    b = x[..., 1:rot:2] if inter else x[..., rot // 2:rot]
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _rope(s):
    case = s["case"]
    dt, page = TYPES[case["dt"]], case["page"]
    angle = s["pos"].double()[:, None] * _frequencies(case, s["pos"].device)[None, :]
    cos, sin = ((x * _mscale(case)).float()[:, None, :] for x in (angle.cos(), angle.sin()))
    q = _rotate(s["q"].float(), cos, sin, case["rot"], case["inter"]).to(dt)
    k = _rotate(s["k"].float(), cos, sin, case["rot"], case["inter"]).to(dt)
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    s["kc"][slot // page, :, slot % page] = k[keep]
    s["vc"][slot // page, :, slot % page] = s["v"].float().to(dt)[keep]
    return [q, s["kc"], s["vc"]]


def _attn(s):
    """Every request padded to the longest: scores, masked softmax and weighted values as 32-bit products."""
    case = s["case"]
    H, G, dh, page, window = case["heads"], case["kv_heads"], case["dh"], case["page"], case["window"]
    B, nmax, kmax = case["batch"], max(s["n"]), max(s["k"])
    dev = s["q"].device
    cu, kv = s["cu"].long(), s["kv"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(nmax, device=dev)
    at = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)                  # [B, nmax]
    q = s["q"][at].float().view(B, nmax, G, H // G, dh).permute(0, 2, 3, 1, 4).reshape(B, G, H // G * nmax, dh)
    ids = s["table"].clamp(min=0).long()
    k = s["kc"][ids].permute(0, 2, 1, 3, 4).reshape(B, G, -1, dh)[:, :, :kmax].float()
    v = s["vc"][ids].permute(0, 2, 1, 3, 4).reshape(B, G, -1, dh)[:, :, :kmax].float()
    t = torch.arange(kmax, device=dev)
    p = (kv - n)[:, None] + i[None, :]                                                  # [B, nmax] positions
    seen = (t[None, None, :] <= p[:, :, None]) & (t[None, None, :] < kv[:, None, None])
    if window > 0:
        seen &= t[None, None, :] > p[:, :, None] - window
    v = torch.where((t[None, :] < kv[:, None])[:, None, :, None], v, 0.0)
    w = (q @ k.transpose(-1, -2)).view(B, G, H // G, nmax, kmax)
    w *= dh ** -0.5
    w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    w -= top
    w.exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.view(B, G, -1, kmax) @ v).view(B, G, H // G, nmax, dh)
    o /= torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, nmax, H, dh)
    lse = lse.permute(0, 3, 1, 2).reshape(B, nmax, H)
    if B == 1:
        return [o[0].to(s["q"].dtype), lse[0]]
    row = torch.arange(s["q"].shape[0], device=dev)
    req = (row[:, None] >= cu[None, 1:]).sum(1)
    return [o[req, row - cu[req]].to(s["q"].dtype), lse[req, row - cu[req]]]


# ----------------------------------------------------------------------------- bytes and operations

def work(case):
    if case["op"] == "tables":
        cached, new, held = _table_lengths(case)
        page = case["page"]
        moved = sum(abs(-(-(c + n) // page) - h) for c, n, h in zip(cached, new, held))
        touched = sum(-(-(c + n) // page) - c // page for c, n in zip(cached, new))   # table entries that slots come from
        # lengths and page counts in, offsets, lengths and counts out; moved pages; slots (8) and positions (4)
        return {"bytes": 24.0 * case["batch"] + 8.0 * moved + 4.0 * touched + 12.0 * sum(new), "flops": 0.0}
    heads, kv_heads, dh = case["heads"], case["kv_heads"], case["dh"]
    if case["op"] == "rope":
        kept = case["tokens"] - case["pad"]
        q, kv = heads * dh, 2 * kv_heads * dh
        size = SIZE[case["inp"]] + 2
        return {"bytes": float(size * (case["tokens"] * q + kept * kv) + 12 * case["tokens"]),
                "flops": 3.0 * case["rot"] * (case["tokens"] * heads + kept * kv_heads)}
    n, k = _attn_lengths(case)
    rows = keys = seen = 0
    for a, b in zip(n, k):
        pairs, lo = _visible(a, b, case["window"])
        rows, keys, seen = rows + a, keys + b - lo, seen + pairs
    # queries in, outputs and log-sums out, every visible key and value once, the table
    return {"bytes": 2.0 * 2 * rows * heads * dh + 4.0 * rows * heads + 2.0 * 2 * keys * kv_heads * dh + 4.0 * keys / case["page"],
            "flops": 4.0 * seen * heads * dh}


# ----------------------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = _inputs(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](case, s)


def _exact_tables(case, s):
    page = case["page"]
    cached, new, held = (s[x].tolist() for x in ("cached", "new", "held"))
    table, stack, count = s["table"].cpu().numpy().copy(), s["stack"].cpu().numpy().copy(), int(s["count"])
    B = case["batch"]
    need = [-(-(cached[b] + new[b]) // page) for b in range(B)]
    pile = count
    for b in range(B):
        for j in range(need[b], held[b]):
            stack[pile] = table[b, j]
            pile += 1
    out, kv, spent, served = list(held), [0] * B, False, [True] * B
    for b in range(B):
        more = need[b] - held[b]
        if more > 0:
            spent = spent or more > pile
            served[b] = not spent
            if not spent:
                for j in range(held[b], need[b]):
                    pile -= 1
                    table[b, j] = stack[pile]
        if served[b]:
            out[b], kv[b] = need[b], cached[b] + new[b]
    cu, slots, pos = [0], [], []
    for b in range(B):
        cu.append(cu[-1] + new[b])
        for p in range(cached[b], cached[b] + new[b]):
            pos.append(p)
            slots.append(int(table[b, p // page]) * page + p % page if served[b] else -1)
    as32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return [as32(out), torch.from_numpy(table), torch.from_numpy(stack), as32([pile]), as32(cu), as32(kv),
            torch.tensor(slots, dtype=torch.int64), as32(pos)]


def _exact_rope(case, s):
    dev, rot, page, L = s["pos"].device, case["rot"], case["page"], ORIGINAL
    turn = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(case["base"]))
        slow = f / case["factor"]
        if case["scaling"] == "linear":
            f = slow
        elif case["scaling"] == "blend":
            ratio = L / (2.0 * math.pi / f)
            share = min(1.0, max(0.0, (ratio - BLEND[0]) / (BLEND[1] - BLEND[0])))
            f = slow + (f - slow) * share
        elif case["scaling"] == "ramp":
            border = [rot / 2.0 * math.log(L / (2.0 * math.pi * t), case["base"]) for t in (RAMP[1], RAMP[0])]
            first, last = max(math.floor(border[0]), 0), min(math.ceil(border[1]), rot - 1)
            share = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            f = f + (slow - f) * share
        turn.append(f)
    a = torch.outer(s["pos"].double(), torch.tensor(turn, dtype=torch.float64, device=dev))
    unit = torch.polar(torch.full_like(a, _mscale(case)), a)[:, None, :]
    pairs = torch.arange(rot // 2, device=dev)
    first, second = (2 * pairs, 2 * pairs + 1) if case["inter"] else (pairs, pairs + rot // 2)

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k, v = turned(s["k"]), s["v"].double()
    kc, vc = s["kc"].double().contiguous(), s["vc"].double().contiguous()
    live = torch.nonzero(s["slots"] >= 0).flatten()
    pg, off = s["slots"][live] // page, s["slots"][live] % page
    for h in range(case["kv_heads"]):
        kc[pg, h, off] = k[live, h]
        vc[pg, h, off] = v[live, h]
    return [turned(s["q"]), kc, vc]


def _exact_attn(case, s):
    H, G, dh, page, window = case["heads"], case["kv_heads"], case["dh"], case["page"], case["window"]
    if sum(_visible(a, b, 0)[0] for a, b in zip(s["n"], s["k"])) * H * dh * 4 > 6e12:
        return None
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b in range(case["batch"]):
        n, kv = s["n"][b], s["k"][b]
        ids = s["table"][b, :-(-kv // page)].long()
        for g in range(G):
            k = s["kc"][ids, g].reshape(-1, dh)[:kv].double()
            v = s["vc"][ids, g].reshape(-1, dh)[:kv].double()
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                p = torch.arange(kv - n + i0, kv - n + i1, device=dev)
                hi = kv - n + i1                                   # no key from here on is seen
                lo = max(0, kv - n + i0 - window + 1) if window > 0 else 0
                t = torch.arange(lo, hi, device=dev)
                hide = t[None, :] > p[:, None]
                if window > 0:
                    hide |= t[None, :] <= p[:, None] - window
                x = torch.einsum("ihd,td->hit", s["q"][at + i0:at + i1, g * (H // G):(g + 1) * (H // G)].double(), k[lo:hi])
                x = (x / math.sqrt(dh)).masked_fill(hide[None], -math.inf)
                y = torch.logsumexp(x, -1)
                lse[at + i0:at + i1, g * (H // G):(g + 1) * (H // G)] = y.t()
                out[at + i0:at + i1, g * (H // G):(g + 1) * (H // G)] = torch.einsum(
                    "hit,td->ihd", torch.exp(x - y[..., None]), v[lo:hi])
        at += n
    return [out, lse]
