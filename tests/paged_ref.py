"""64-bit references of the paged-serving operators and the error bounds their
results must meet (written apart from the kernels, from the definitions)."""
import math

import torch


def half_step(dtype):
    """Largest relative error of one rounding to this type."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ block tables

def tables(page, max_tokens, cached, new, held, table, stack, count):
    """The step row by row (lists and nested lists; returns new ones and whether
    the device status must report an inconsistent row)."""
    table, stack = [list(r) for r in table], list(stack)
    B, width = len(cached), len(table[0])
    bad = [c < 0 or n < 0 or h < 0 or h > width or c + n > width * page for c, n, h in zip(cached, new, held)]
    status = any(bad)
    if count < 0 or count > len(stack):
        status, count = True, max(0, min(count, len(stack)))
    counted, starts, past = 0, [], []
    for b in range(B):
        n = 0 if bad[b] else new[b]
        starts.append(counted)
        counted += n
        past.append(n > 0 and counted > max_tokens)
    status |= any(past)
    cu = [min(x, max_tokens) for x in starts + [counted]]
    ok = [not x and not y for x, y in zip(bad, past)]
    need = [-(-(cached[b] + new[b]) // page) if ok[b] else held[b] for b in range(B)]
    pile, top = list(stack[:count]), count
    for b in range(B):
        for j in range(need[b], held[b]):
            pile.append(table[b][j])
            if top < len(stack):
                stack[top] = table[b][j]
            else:
                status = True
            top += 1
    out, kv, served, dry = list(held), [0] * B, [False] * B, False
    for b in range(B):
        want = need[b] - held[b]
        if not ok[b]:
            continue
        if want > 0 and (dry or want > len(pile)):
            dry = True
            continue
        for j in range(held[b], need[b]):
            table[b][j] = pile.pop()
        out[b], kv[b], served[b] = need[b], cached[b] + new[b], True
    slots, pos = [-1] * max_tokens, [0] * max_tokens
    for b in range(B):
        for t in range(cu[b], cu[b + 1]):
            p = cached[b] + t - cu[b]
            pos[t] = p
            if served[b]:
                slots[t] = table[b][p // page] * page + p % page
    return dict(held=out, table=table, stack=stack, count=min(len(pile), len(stack)), cu=cu, kv=kv, slots=slots, pos=pos,
                status=status)


# ------------------------------------------------------------------ rotary positions

def frequencies(rot, base, scaling="none", factor=1.0, original_max=0.0, low=1.0, high=4.0):
    out = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(base))
        if scaling == "linear":
            f /= factor
        elif scaling == "blend":
            share = min(1.0, max(0.0, (original_max * f / (2 * math.pi) - low) / (high - low)))
            f = f / factor + (f - f / factor) * share
        elif scaling == "ramp":
            edge = [rot / 2.0 * math.log(original_max / (2 * math.pi * r), base) for r in (high, low)]
            a, z = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            share = min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            f = f + (f / factor - f) * share
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotate(x, pos, freq, interleaved, mscale=1.0):
    """x [T, heads, dh] in fp64 and, per element, the bound of the fp32 evaluation:
    the angle is off by at most 2^-25 half turns (0.94e-7) and the functions by 2 ulp
    (2.4e-7), then two products and a sum (3 roundings of 6e-8): together below
    6e-7 (|x1| + |x2|)."""
    y = x.double().clone()
    rot = 2 * len(freq)
    if rot == 0:
        return y, torch.zeros_like(y)
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    ang = pos.double()[:, None] * freq.to(x.device)[None, :]
    c, s = ang.cos()[:, None, :] * mscale, ang.sin()[:, None, :] * mscale
    x1, x2 = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    slack = torch.zeros_like(y)
    slack[..., a] = slack[..., b] = 6e-7 * abs(mscale) * (x1.abs() + x2.abs())
    return y, slack


# ------------------------------------------------------------------ attention

def attention(q, k, v, table, cu, kv, window=0, scale=None):
    """q [T, H, dh]; k, v [pages, KVH, page, dh]; lists cu, kv.  Returns out, lse (fp64)
    and their bounds, for every row of a request (rows of none: NaN in out).

    Bound of out against the exact value, with A = sum a_t |v_t| and u the half step of
    the type: the weights' rounding u A, the output's rounding u |out|, the scores' fp32
    sums (dh + 16) 2^-24 max_t(scale sum |q k|) and the exponential's 2^-20 on both the
    weights and their sum (2 A), fp32 sums over t (kv 2^-24 of A, twice), and fp16 weights
    below its range (each off by at most 2^-32 of the largest, kv max|v| in all)."""
    T, H, dh = q.shape
    page, G = k.shape[2], H // k.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    u = half_step(q.dtype)
    out = torch.full((T, H, dh), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((T, H), math.nan, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = kv[b] - n + i
            lo = max(0, p - window + 1) if window > 0 else 0
            t = cu[b] + i
            if p < lo:
                out[t], lse[t] = 0.0, -math.inf
                continue
            at = torch.arange(lo, p + 1, device=q.device)
            ids = table[b][at // page].long()
            kk = k[ids, :, at % page].double().repeat_interleave(G, dim=1)      # [keys, H, dh]
            vv = v[ids, :, at % page].double().repeat_interleave(G, dim=1)
            qq = q[t].double()
            s = torch.einsum("hd,thd->ht", qq, kk) * scale
            big = (torch.einsum("hd,thd->ht", qq.abs(), kk.abs()) * scale).amax(1)
            lse[t] = torch.logsumexp(s, 1)
            w = torch.exp(s - lse[t][:, None])
            out[t] = torch.einsum("ht,thd->hd", w, vv)
            A = torch.einsum("ht,thd->hd", w, vv.abs())
            d = ((dh + 16) * 2.0 ** -24 * big + 2.0 ** -20)[:, None]
            keys = p + 1 - lo
            tol[t] = u * (A + out[t].abs()) + 2 * A * (d + keys * 2.0 ** -24) + keys * 2.0 ** -32 * vv.abs().amax(0) \
                + 2.0 ** -25
            ltol[t] = d[:, 0] + keys * 2.0 ** -24 + 2.0 ** -22 * lse[t].abs()
    return out, lse, tol, ltol


def check(got, want, tol, what=""):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(torch.isinf(got), torch.isinf(want)), f"{what}: infinities in other places"
    fine = torch.isfinite(want)
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{what}: {int((over > 0).sum())} of {over.numel()} values off by up to {float(over.max()):.3e} beyond the bound"
