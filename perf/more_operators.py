"""Cases of the paged cache in 8 bits: keys and values quantised as they are stored
(``pi_rope_store8``), read back as 16-bit rows (``pi_page_read8``), and attention of new
tokens over the cache (``pi_paged_attn8``).

A page holds e4m3 codes; each block of 16 positions and each key/value head has an exponent e
of its own, and a code c stands for c 2^e.  The exponent of a block is the smallest with which
its largest magnitude is at most 448 2^e, within -32 .. 32.  Tokens that join a block whose
exponent is too small for them raise it, and the codes there are rounded again.

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
CODE = torch.float8_e4m3fn
BLOCK = 16              # positions that share an exponent
E_MIN, E_MAX = -32, 32

# (query heads, key/value heads, head width): the repository's attention blocks, then shared
# key/value heads in groups of 3, of 16 and of 4
HEADS = ((12, 12, 64), (32, 32, 128), (56, 56, 128), (64, 8, 128), (96, 96, 128), (24, 8, 128), (16, 1, 64), (32, 8, 64))

# what a drawn case may cost at most: just under the largest listed case of its operator
MOST_STORE_BYTES = 6.0e8
MOST_READ_BYTES = 9.5e8
MOST_ATTN_FLOPS = 1.8e12
MOST_ATTN_BYTES = 1.0e9
MOST_SCORES = 4.0e9     # elements of the padded score matrix of the plain form


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # Store, and what the touched blocks hold then. A decode step of 32 sequences (grouped heads, half layout):
        # each token joins a block that has an exponent, and some raise it. A matter of latency.
        dict(name="store8_decode_32", op="store", batch=32, n_lo=1, n_hi=1, c_lo=0, c_hi=4000, heads=64, kv_heads=8, dh=128,
             rot=128, inter=False, base=10000.0, inp="f16", dt="f16", page=16, order="hnd", rs=21),
        # A prompt chunk of odd length from fp32 projections, multi-head; interleaved pairs on half of the head.
        dict(name="store8_chunk_1999", op="store", batch=1, n_lo=1999, n_hi=1999, c_lo=777, c_hi=777, heads=32, kv_heads=32, dh=128,
             rot=64, inter=True, base=10000.0, inp="f32", dt="f16", page=32, order="hnd", rs=22),
        # Many prompts at once, bfloat16, far positions.
        dict(name="store8_prompts_16384", op="store", batch=4, n_lo=4096, n_hi=4096, c_lo=0, c_hi=100000, heads=64, kv_heads=8, dh=128,
             rot=128, inter=False, base=500000.0, inp="bf16", dt="bf16", page=64, order="nhd", rs=23),
        # Read back. One short request of the small block, whose rows go elsewhere.
        dict(name="read8_1", op="read", batch=1, c_lo=1001, c_hi=1001, heads=12, kv_heads=12, dh=64, dt="f16", page=16, order="hnd", rs=41),
        # The caches of 48 requests leave for another machine.
        dict(name="read8_48", op="read", batch=48, c_lo=100, c_hi=8000, heads=64, kv_heads=8, dh=128, dt="bf16", page=32, order="nhd",
             rs=42),
        # Attention. One sequence, one token, a short cache: the smallest call.
        dict(name="attn8_decode_1", op="attn", batch=1, heads=64, kv_heads=8, dh=128, dt="f16", page=16, n_lo=1, n_hi=1,
             c_lo=1000, c_hi=1000, dec=1.0, window=0, order="hnd", rs=31),
        # A decode step of 32 sequences of very different lengths over grouped heads.
        dict(name="attn8_decode_32", op="attn", batch=32, heads=64, kv_heads=8, dh=128, dt="f16", page=16, n_lo=1, n_hi=1,
             c_lo=500, c_hi=8000, dec=1.0, window=0, order="hnd", rs=32),
        # Four sequences with long caches: the most bytes.
        dict(name="attn8_decode_long", op="attn", batch=4, heads=64, kv_heads=8, dh=128, dt="bf16", page=64, n_lo=1, n_hi=1,
             c_lo=120000, c_hi=131000, dec=1.0, window=0, order="nhd", rs=33),
        # Five proposed tokens of each of 24 sequences are looked at together.
        dict(name="attn8_verify_24", op="attn", batch=24, heads=64, kv_heads=8, dh=128, dt="bf16", page=32, n_lo=5, n_hi=5,
             c_lo=200, c_hi=6000, dec=0.0, window=0, order="hnd", rs=37),
        # A step that serves decodes and prompt chunks together, multi-head, with a sliding window.
        dict(name="attn8_mixed_16", op="attn", batch=16, heads=32, kv_heads=32, dh=128, dt="bf16", page=32, n_lo=100, n_hi=700,
             c_lo=1, c_hi=4000, dec=0.7, window=2000, order="hnd", rs=34),
        # A whole prompt of odd length in the small multi-head block (64-wide heads).
        dict(name="attn8_prompt_1999", op="attn", batch=1, heads=12, kv_heads=12, dh=64, dt="f16", page=16, n_lo=1999, n_hi=1999,
             c_lo=0, c_hi=0, dec=0.0, window=0, order="hnd", rs=35),
        # A chunk of 4096 tokens behind 12288 cached ones over grouped heads: the most operations.
        dict(name="attn8_chunk_4096", op="attn", batch=1, heads=64, kv_heads=8, dh=128, dt="bf16", page=16, n_lo=4096, n_hi=4096,
             c_lo=12288, c_hi=12288, dec=0.0, window=0, order="hnd", rs=36),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1) + 0.49)))))))


def draw(rng):
    op = rng.choice(("store", "store", "read", "attn", "attn", "attn", "attn"))
    heads, kv_heads, dh = rng.choice(HEADS)
    dt, order = rng.choice(("f16", "bf16")), rng.choice(("hnd", "nhd"))
    c = dict(op=op, batch=_log(rng, 1, 64), heads=heads, kv_heads=kv_heads, dh=dh, dt=dt, order=order,
             page=rng.choice((16, 32, 64, 128)), rs=rng.randrange(1 << 30))
    if op == "store":
        c.update(n_lo=1, n_hi=rng.choice((1, _log(rng, 1, 4096))), c_lo=0, c_hi=_log(rng, 1, 100000),
                 rot=rng.choice((dh, dh, dh // 2, 16, 48, 0)), inter=rng.random() < 0.5, base=rng.choice((10000.0, 500000.0)),
                 inp=rng.choice((dt, dt, "f32")))
        c["n_lo"] = _log(rng, 1, c["n_hi"])
        while work(c)["bytes"] > MOST_STORE_BYTES:
            c["batch" if c["batch"] > 1 else "n_hi"] = max(1, c["batch" if c["batch"] > 1 else "n_hi"] * 2 // 3)
            c["n_lo"] = min(c["n_lo"], c["n_hi"])
        return c
    if op == "read":
        c["c_hi"] = _log(rng, 1, 16000)
        c["c_lo"] = rng.randint(1, c["c_hi"])
        while work(c)["bytes"] > MOST_READ_BYTES:
            c["batch"] = max(1, c["batch"] * 2 // 3)
        return c
    kind = rng.choice(("decode", "decode", "verify", "chunk", "mixed"))
    c.update(n_lo=1, n_hi=1, c_lo=0, c_hi=_log(rng, 1, 131000), dec=1.0, window=rng.choice((0, 0, _log(rng, 1, 5000))))
    if kind == "decode":
        c["c_lo"] = rng.randrange(c["c_hi"])
    else:
        c["n_hi"], c["c_hi"] = _log(rng, 2, 12 if kind == "verify" else 4096), _log(rng, 1, 16000)
        c["dec"] = rng.uniform(0.3, 0.9) if kind == "mixed" else 0.0
        c["n_lo"] = _log(rng, 1, c["n_hi"])
    while True:
        n, k = _lengths(c)
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

def _lengths(case):
    """Per request: new tokens, and keys in the cache with them."""
    r = random.Random(case["rs"])
    n, k = [], []
    for _ in range(case["batch"]):
        one = r.random() < case.get("dec", 0.0)
        n.append(0 if case["op"] == "read" else 1 if one else _log(r, case["n_lo"], case["n_hi"]))
        k.append(n[-1] + (r.randint(case["c_lo"], case["c_hi"]) if case["c_hi"] > case["c_lo"] else case["c_lo"]))
    return n, k


def _visible(n, k, window):
    """Keys that the n newest of k positions see together, and the oldest key that any of them sees."""
    if window <= 0:
        return n * k - n * (n - 1) // 2, 0
    first = k - n                      # position p sees min(p + 1, window) keys
    ramp = max(0, min(n, window - 1 - first))
    return ramp * (first + 1) + ramp * (ramp - 1) // 2 + (n - ramp) * window, max(0, first - window + 1)


# ----------------------------------------------------------------------------- codes and exponents

def _exponent(most):
    """The smallest e with most <= 448 2^e (448 = 0.875 2^9), within its range."""
    part, e = torch.frexp(most)
    e = e - torch.where(part <= 0.875, 9, 8)
    return torch.where(most == 0, E_MIN, e).clamp(E_MIN, E_MAX)


def _encode(x, e):
    """Codes of fp32 values under exponents e (broadcast)."""
    return torch.ldexp(x, -e).clamp(-448.0, 448.0).to(CODE)


def _quantised(pages, case, g, dev):
    """A cache of random keys or values: codes [pages, kv_heads, page, dh], stored heads first ("hnd") or tokens first
    ("nhd"), and exponents [pages, kv_heads, page / 16].  Heads differ in size, and a few columns are larger."""
    G, page, dh = case["kv_heads"], case["page"], case["dh"]
    codes = torch.empty((pages, G, page, dh) if case["order"] == "hnd" else (pages, page, G, dh), dtype=CODE, device=dev)
    codes = codes if case["order"] == "hnd" else codes.transpose(1, 2)
    exps = torch.empty(pages, G, page // BLOCK, dtype=torch.int8, device=dev)
    size = _sizes(case, dev)
    step = max(1, (1 << 28) // (G * page * dh))
    for i in range(0, pages, step):
        x = torch.randn(min(step, pages - i), G, page // BLOCK, BLOCK, dh, generator=g, device=dev) * size[:, None, None]
        e = _exponent(x.abs().amax((-1, -2)))
        exps[i:i + step] = e.to(torch.int8)
        codes.view(torch.uint8)[i:i + step] = _encode(x, e[..., None, None]).view(torch.uint8).flatten(2, 3)
    return codes, exps


def _sizes(case, dev):
    """Magnitudes of the heads' columns, [kv_heads, dh]."""
    s = torch.ones(case["kv_heads"], case["dh"], device=dev) * torch.linspace(0.3, 2.0, case["kv_heads"], device=dev)[:, None]
    s[:, 5::37] *= 4.0
    return s


# ----------------------------------------------------------------------------- inputs

def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _starts(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def _inputs(case, seed):
    """The tensors of a case, from the seed alone (the lengths are the case's)."""
    dev = _device()
    g = _gen(seed, dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    heads, kv_heads, dh, page, B = case["heads"], case["kv_heads"], case["dh"], case["page"], case["batch"]
    n, k = _lengths(case)
    # the pages that hold the positions of the case (a store's: from the first touched block on)
    from_ = [(b - a) // BLOCK * BLOCK if case["op"] == "store" else 0 for a, b in zip(n, k)]
    first = [x // page for x in from_]
    used = [-(-x // page) - f for x, f in zip(k, first)]
    pages, M = sum(used) + 3, max(-(-x // page) for x in k)
    perm = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((B, M), -1, dtype=torch.int32, device=dev)
    col, lo = torch.arange(M, device=dev)[None, :], i32(first)[:, None]
    table[(col >= lo) & (col < lo + i32(used)[:, None])] = perm[:sum(used)]
    s = dict(table=table, n=n, k=k, cu=i32(_starts(n)), kv=i32(k))
    s["kc"], s["ke"] = _quantised(pages, case, g, dev)
    s["vc"], s["ve"] = _quantised(pages, case, g, dev)
    T = sum(n)
    if case["op"] == "store":
        row = torch.arange(T, device=dev)
        req = torch.repeat_interleave(torch.arange(B, device=dev), i32(n).long(), output_size=T)
        pos = (s["kv"].long() - i32(n).long())[req] + row - s["cu"].long()[req]
        s["pos"] = pos.to(torch.int32)
        s["slots"] = table[req, pos // page].long() * page + pos % page
        size = torch.cat([torch.ones(heads * dh, device=dev), _sizes(case, dev).flatten(), _sizes(case, dev).flatten()])
        qkv = (torch.randn(T, (heads + 2 * kv_heads) * dh, generator=g, device=dev) * size).to(TYPES[case["inp"]])
        s["q"], s["k_new"], s["v_new"] = (x.unflatten(1, (-1, dh)) for x in
                                          qkv.split([heads * dh, kv_heads * dh, kv_heads * dh], dim=1))
    if case["op"] == "attn":
        # queries of some heads are larger, so that their weights rest on few keys
        s["q"] = (torch.randn(T, heads, dh, generator=g, device=dev) *
                  torch.linspace(0.3, 1.5, heads, device=dev)[:, None]).to(TYPES[case["dt"]])
    else:
        # rows that are read back: a request's positions from `start` on
        s["start"], s["cu_rows"] = i32(from_), i32(_starts([b - a for a, b in zip(from_, k)]))
        s["rows"] = sum(k) - sum(from_)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dev, dt = s["table"].device, TYPES[case["dt"]]
    # the buffers that a serving loop keeps from step to step
    if case["op"] == "attn":
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], dtype=torch.float32, device=dev)
    else:
        s["k_out"] = torch.empty(s["rows"], case["kv_heads"], case["dh"], dtype=dt, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
    if case["op"] == "store":
        s["q_out"] = torch.empty(s["q"].shape, dtype=dt, device=dev)
    if own:   # ... and the descriptors, the rotary plan and the workspace that belong to them
        import activation_sparse_ffn_layer_gb300 as P
        s["cache"] = P.page8_desc(s["kc"], s["vc"])
        if case["op"] == "attn":
            s["desc"] = P.paged_desc(case["heads"], case["batch"], s["q"].shape[0], max(s["n"]), s["table"].shape[1],
                                     window=case["window"])
            s["ws"] = torch.zeros(P.pi_paged8_workspace_bytes(s["desc"], s["cache"]), dtype=torch.uint8, device=dev)
        else:
            s["desc"] = P.read8_desc(case["batch"], s["table"].shape[1], s["rows"])
        if case["op"] == "store":
            s["plan"] = P.rope_plan(case["dh"], case["rot"], interleaved=case["inter"], base=case["base"])
        s["P"] = P
    return s


# ----------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _store(s) if op == "store" else _read(s) if op == "read" else _attn(s)


def _own(s):
    P, op = s["P"], s["case"]["op"]
    if op == "attn":
        P.pi_paged_attn8(s["desc"], s["cache"], s["q"], s["kc"], s["vc"], s["ke"], s["ve"], s["table"], s["cu"], s["kv"],
                         s["out"], s["lse"], s["ws"])
        return [s["out"], s["lse"]]
    if op == "store":
        P.pi_rope_store8(s["plan"], s["cache"], s["q"], s["k_new"], s["v_new"], s["pos"], s["slots"], s["q_out"],
                         s["kc"], s["vc"], s["ke"], s["ve"])
    # the cache as the values it stands for
    P.pi_page_read8(s["desc"], s["cache"], s["kc"], s["vc"], s["ke"], s["ve"], s["table"], s["start"], s["cu_rows"],
                    s["k_out"], s["v_out"])
    return [s["q_out"], s["k_out"], s["v_out"]] if op == "store" else [s["k_out"], s["v_out"]]


def _rotate(x, cos, sin, rot, inter):
    a = x[..., 0:rot:2] if inter else x[..., :rot // 2]
    b = x[..., 1:rot:2] if inter else x[..., rot // 2:rot]
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _into(codes, exps, x, slots, page):
    """Tokens x [T, kv_heads, dh] (fp32) into a cache: the blocks' exponents, the codes that stay, the new codes."""
    P, G, nb = exps.shape
    blk, off = slots // BLOCK, slots % BLOCK                   # block number over all pages, place in it
    at = blk[:, None].expand(-1, G)
    most = torch.zeros(P * nb, G, device=x.device).scatter_reduce(0, at, x.abs().amax(-1), "amax")
    kept = torch.full((P * nb,), BLOCK, dtype=torch.int64, device=x.device).scatter_reduce(0, blk, off, "amin")
    old = exps.transpose(1, 2).reshape(P * nb, G).int()
    e = _exponent(most)
    # an untouched block keeps all 16 positions and its exponent; one with no position kept forgets its old one
    e = torch.where((kept == BLOCK)[:, None], old, torch.where((kept > 0)[:, None], torch.maximum(e, old), e))
    raw = codes.view(torch.uint8)
    c = raw.reshape(P, G, nb, BLOCK, codes.shape[-1])
    by_block = lambda v: v.view(P, nb, G).transpose(1, 2)      # noqa: E731
    again = torch.ldexp(c.view(CODE).float(), by_block(old - e)[..., None, None]).to(CODE).view(torch.uint8)
    stay = torch.arange(BLOCK, device=x.device)[None, :] < kept[:, None]
    stay = stay.view(P, 1, nb, BLOCK, 1)
    raw.copy_(torch.where(stay, again, c).flatten(2, 3))
    exps.copy_(by_block(e).to(torch.int8))
    raw[slots // page, :, slots % page] = _encode(x, e[blk][..., None]).view(torch.uint8)


def _store(s):
    case = s["case"]
    dt, rot = TYPES[case["dt"]], case["rot"]
    f = case["base"] ** (-2 * torch.arange(rot // 2, device=s["pos"].device, dtype=torch.float64) / max(rot, 1))
    angle = s["pos"].double()[:, None] * f[None, :]
    cos, sin = (x.float()[:, None, :] for x in (angle.cos(), angle.sin()))
    q = _rotate(s["q"].float(), cos, sin, rot, case["inter"]).to(dt)
    _into(s["kc"], s["ke"], _rotate(s["k_new"].float(), cos, sin, rot, case["inter"]), s["slots"], case["page"])
    _into(s["vc"], s["ve"], s["v_new"].float(), s["slots"], case["page"])
    return [q] + _read(s)


def _values(codes, exps):
    """What gathered codes [..., kv_heads, page, dh] with exponents [..., kv_heads, page / 16] stand for, fp32."""
    c = codes.view(CODE).float().unflatten(-2, (-1, BLOCK))
    return torch.ldexp(c, exps.int()[..., None, None]).flatten(-3, -2)


def _read(s):
    case, page = s["case"], s["case"]["page"]
    row = torch.arange(s["rows"], device=s["table"].device)
    req = (row[:, None] >= s["cu_rows"][None, 1:]).sum(1)
    pos = s["start"][req] + row - s["cu_rows"][req]
    ids = s["table"][req, pos // page].long()
    off = pos % page
    out = []
    for codes, exps in ((s["kc"], s["ke"]), (s["vc"], s["ve"])):
        c = codes.view(torch.uint8)[ids, :, off].view(CODE).float()
        out.append(torch.ldexp(c, exps[ids, :, off // BLOCK].int()[..., None]).to(TYPES[case["dt"]]))
    return out


def _attn(s):
    """Every request padded to the longest: scores, masked softmax and weighted values as 32-bit products."""
    case = s["case"]
    H, G, dh, window = case["heads"], case["kv_heads"], case["dh"], case["window"]
    B, nmax, kmax = case["batch"], max(s["n"]), max(s["k"])
    dev = s["q"].device
    cu, kv = s["cu"].long(), s["kv"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(nmax, device=dev)
    at = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)                  # [B, nmax]
    q = s["q"][at].float().view(B, nmax, G, H // G, dh).permute(0, 2, 3, 1, 4).reshape(B, G, H // G * nmax, dh)
    ids = s["table"].clamp(min=0).long()
    k, v = (_values(c.view(torch.uint8)[ids], e[ids]).permute(0, 2, 1, 3, 4).reshape(B, G, -1, dh)[:, :, :kmax]
            for c, e in ((s["kc"], s["ke"]), (s["vc"], s["ve"])))
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
    row = torch.arange(s["q"].shape[0], device=dev)
    req = (row[:, None] >= cu[None, 1:]).sum(1)
    return [o[req, row - cu[req]].to(s["q"].dtype), lse[req, row - cu[req]]]


# ----------------------------------------------------------------------------- bytes and operations

def work(case):
    heads, G, dh = case["heads"], case["kv_heads"], case["dh"]
    n, k = _lengths(case)
    if case["op"] == "attn":
        rows = keys = seen = 0
        for a, b in zip(n, k):
            pairs, lo = _visible(a, b, case["window"])
            rows, keys, seen = rows + a, keys + b - lo, seen + pairs
        # queries in, outputs and log-sums out, every visible key and value once, exponents, the table
        return {"bytes": 4.0 * rows * heads * dh + 4.0 * rows * heads + 2.0 * keys * G * (dh + 1.0 / BLOCK) + 4.0 * keys / case["page"],
                "flops": 4.0 * seen * heads * dh}
    T = sum(n)
    first = [(b - a) // BLOCK * BLOCK if case["op"] == "store" else 0 for a, b in zip(n, k)]
    rows = sum(k) - sum(first)
    size = SIZE[case["dt"]]
    # codes in (but for the ones just stored), rows out, exponents and the table
    read = 2.0 * (rows - T) * G * (dh + 1.0 / BLOCK) + 2.0 * size * rows * G * dh + 4.0 * rows / case["page"]
    if case["op"] == "read":
        return {"bytes": read, "flops": 2.0 * rows * G * dh}
    # projections in, queries and codes out, exponents, positions and slots
    store = SIZE[case["inp"]] * T * (heads + 2 * G) * dh + size * T * heads * dh + 2.0 * T * G * (dh + 1.0 / BLOCK) + 12.0 * T
    return {"bytes": read + store, "flops": 3.0 * case["rot"] * T * (heads + G) + 4.0 * rows * G * dh}


# ----------------------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = _inputs(case, seed)
    return {"store": _exact_store, "read": _exact_read, "attn": _exact_attn}[case["op"]](case, s)


# the 256 values of a code: sign, 4 bits of exponent (offset 7), 3 bits of fraction
_VALUES = [(-1.0 if c & 128 else 1.0) * (math.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if c & 120 == 0 else
                                         (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10)) for c in range(256)]


def _nearest(y):
    """y (64 bits) on the grid of the codes: ties to the even one."""
    place = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6) * (1 + 2.0 ** -52))).clamp(-6, 8)
    place = torch.where(torch.exp2(place) > y.abs().clamp(min=2.0 ** -6), place - 1, place)   # exact at powers of two
    step = torch.exp2(place - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _wide(case, s, which, b, lo, hi):
    """Positions lo .. hi - 1 of a request, [positions, kv_heads, dh] in 64 bits."""
    t = torch.arange(lo, hi, device=s["table"].device)
    page = case["page"]
    ids = s["table"][b][t // page].long()
    value = torch.tensor(_VALUES, dtype=torch.float64, device=t.device)
    c = value[s[which + "c"].view(torch.uint8)[ids, :, t % page].long()]
    return c * torch.exp2(s[which + "e"][ids, :, t % page // BLOCK].double())[..., None]


def _exact_read(case, s):
    return [torch.cat([_wide(case, s, which, b, 0, s["k"][b]) for b in range(case["batch"])]) for which in "kv"]


def _exact_store(case, s):
    dev, rot = s["pos"].device, case["rot"]
    f = torch.tensor([math.exp(-2.0 * i / rot * math.log(case["base"])) for i in range(rot // 2)], dtype=torch.float64, device=dev)
    a = torch.outer(s["pos"].double(), f)
    unit = torch.polar(torch.ones_like(a), a)[:, None, :]
    pairs = torch.arange(rot // 2, device=dev)
    first, second = (2 * pairs, 2 * pairs + 1) if case["inter"] else (pairs, pairs + rot // 2)

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    new = {"k": turned(s["k_new"]), "v": s["v_new"].double()}
    out, at = {"k": [], "v": []}, 0
    for b in range(case["batch"]):
        n, k = s["n"][b], s["k"][b]
        head = (k - n) % BLOCK                                   # positions of the first block that are there already
        for which in "kv":
            x = new[which][at:at + n]
            G, dh = x.shape[1:]
            pad = -(head + n) % BLOCK
            y = torch.cat([x.new_zeros(head, G, dh), x, x.new_zeros(pad, G, dh)]).view(-1, BLOCK, G, dh)
            most = y.abs().amax((1, 3))                          # [blocks, kv_heads]
            e = torch.ceil(torch.log2(most.clamp(min=2.0 ** -200) / 448.0) - 1e-13).clamp(E_MIN, E_MAX)
            e = torch.where(most > 448.0 * torch.exp2(e), e + 1, e).clamp(E_MIN, E_MAX)
            if head:
                old = _wide(case, s, which, b, k - n - head, k - n)
                slot = int(s["slots"][at])
                e0 = s[which + "e"][slot // case["page"], :, slot % case["page"] // BLOCK].double()
                e[0] = torch.maximum(e[0], e0)
                y[0, :head] = old
            u = torch.exp2(e)[:, None, :, None]
            out[which].append((_nearest(y / u) * u).view(-1, G, dh)[:head + n])
        at += n
    return [turned(s["q"]), torch.cat(out["k"]), torch.cat(out["v"])]


def _exact_attn(case, s):
    H, G, dh, window = case["heads"], case["kv_heads"], case["dh"], case["window"]
    if sum(_visible(a, b, 0)[0] for a, b in zip(s["n"], s["k"])) * H * dh * 4 > 6e12:
        return None
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b in range(case["batch"]):
        n, kv = s["n"][b], s["k"][b]
        base = max(0, kv - n - window + 1) if window > 0 else 0
        kk, vv = (_wide(case, s, which, b, base, kv) for which in "kv")
        for g in range(G):
            mine = slice(g * (H // G), (g + 1) * (H // G))
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                p = torch.arange(kv - n + i0, kv - n + i1, device=dev)
                t = torch.arange(base, kv - n + i1, device=dev)        # no key behind is seen
                hide = t[None, :] > p[:, None]
                if window > 0:
                    hide |= t[None, :] <= p[:, None] - window
                x = torch.einsum("ihd,td->hit", s["q"][at + i0:at + i1, mine].double(), kk[:len(t), g])
                x = (x / math.sqrt(dh)).masked_fill(hide[None], -math.inf)
                y = torch.logsumexp(x, -1)
                lse[at + i0:at + i1, mine] = y.t()
                out[at + i0:at + i1, mine] = torch.einsum("hit,td->ihd", torch.exp(x - y[..., None]), vv[:len(t), g])
        at += n
    return [out, lse]
