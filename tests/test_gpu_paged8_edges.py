"""The 8-bit paged cache at its edges: workspaces that heads of both widths share, rows of no request, reads
beside requests that are not consistent."""
import random

import pytest
import torch

from tests import paged8_ref as R
from tests import paged_ref as R16
from tests.test_gpu_paged8 import BF16, F16, P, attn, i32, make_cache, quantised, starts, tables  # noqa: F401

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
