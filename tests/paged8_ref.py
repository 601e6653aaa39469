"""64-bit references of the 8-bit paged cache, from the definitions: the values of
codes by table, rounding by distance, blocks token by token."""
import math

import torch

from tests import paged_ref as R

BLOCK, E_MIN, E_MAX = 16, -32, 32
CODE = torch.float8_e4m3fn

# the value of code c: sign, 4 bits of exponent (offset 7), 3 of fraction, one NaN of each sign
VALUES = torch.tensor([(-1.0 if c & 128 else 1.0) * (math.nan if c & 127 == 127 else (c & 7) / 512 if c & 120 == 0 else
                                                     (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)],
                      dtype=torch.float64)


def encode(y):
    """Codes (uint8) of 64-bit values: the nearest magnitude, ties to the even code; not finite: NaN (0x7f)."""
    grid = VALUES[:127].to(y.device)
    m = y.abs().clamp(max=448.0).nan_to_num(0.0).contiguous()
    hi = torch.searchsorted(grid, m).clamp(1, 126)          # grid[hi - 1] < m <= grid[hi]
    lo = hi - 1
    up, down = grid[hi] - m, m - grid[lo]
    c = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = c + 128 * torch.signbit(y).long()
    return torch.where(torch.isfinite(y), c, 127).to(torch.uint8)


def exponent(most):
    for e in range(E_MIN, E_MAX):
        if most <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def values(codes, exps):
    """Codes [pages, heads, page, dh] and exponents [pages, heads, page / 16] as 64-bit values."""
    c = VALUES.to(codes.device)[codes.view(torch.uint8).long()]
    return c * torch.exp2(exps.double().clamp(E_MIN, E_MAX)).repeat_interleave(BLOCK, 2)[..., None]


def store(codes, exps, x, slots, page):
    """One array's tokens x [T, heads, dh] (64 bits) into codes (uint8) and exponents, in place."""
    i, T = 0, len(slots)
    while i < T:
        s = slots[i]
        if s < 0:
            i += 1
            continue
        n = 1
        while i + n < T and slots[i + n] == s + n and (s + n) % BLOCK != 0:
            n += 1
        p, r = s // page, s % BLOCK
        first = s % page - r
        for h in range(x.shape[1]):
            new = x[i:i + n, h]
            fine = new[torch.isfinite(new)].abs()
            e = exponent(float(fine.max()) if fine.numel() else 0.0)
            if r > 0:
                old = int(exps[p, h, first // BLOCK])
                e = max(e, old)
                kept = codes[p, h, first:first + r]
                codes[p, h, first:first + r] = torch.where(kept & 127 == 127, kept,
                                                           encode(VALUES.to(kept.device)[kept.long()] * 2.0 ** (old - e)))
            exps[p, h, first // BLOCK] = e
            codes[p, h, first + r:first + r + n] = encode(new / 2.0 ** e)
        i += n


def attention(q, kc, ke, vc, ve, table, cu, kv, window=0, scale=None):
    """As the 16-bit cache's reference, with one more term in the bound of out: fp16 weights
    below their range are off by 2^-25 at most, where the largest, of a key in a block of
    exponent e, is 2^7 or more; so by 2^-32 448 2^e each in the output."""
    k, v = values(kc, ke), values(vc, ve)
    out, lse, tol, ltol = R.attention(q, k, v, table, cu, kv, window, scale)
    for b in range(len(kv)):
        pages = [p for p in table[b][:-(-kv[b] // kc.shape[2])].tolist() if 0 <= p < kc.shape[0]]
        if pages and cu[b + 1] > cu[b]:
            most = float(torch.exp2(ve[pages].double()).max())
            tol[cu[b]:cu[b + 1]] += kv[b] * 2.0 ** -32 * 448 * most
    return out, lse, tol, ltol
