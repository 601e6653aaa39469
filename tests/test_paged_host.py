"""Paged serving on the host: refused arguments launch nothing, and the rotary
plan holds the frequencies of the formulas."""
import ctypes as C
import math

import pytest
import torch

from tests import paged_ref as R


@pytest.fixture(scope="module")
def P():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_ffn_layer_gb300 as P
    return P


FAKE = 1 << 20   # an aligned address that no refused call touches


def test_tables_refusals(P):
    L = P.lib()
    D = P.binding.pi_tables_desc
    args = [FAKE] * 12 + [None]
    for bad in (D(0, 16, 8, 8, 8), D(4097, 16, 8, 8, 8), D(4, 8, 8, 8, 8), D(4, 24, 8, 8, 8), D(4, 16, 0, 8, 8),
                D(4, 16, 8, 0, 8), D(4, 16, 8, 8, -1), D(4, 128, 8, 1 << 24, 8), D(4, 16, 8, 8, (1 << 24) + 1)):
        assert L.pi_block_tables(C.byref(bad), *args) == 1
    ok = D(4, 16, 8, 8, 8)
    assert L.pi_block_tables(None, *args) == 1
    for i in range(12):
        some = list(args)
        some[i] = None
        assert L.pi_block_tables(C.byref(ok), *some) == 1, i
        some[i] = FAKE + 2
        assert L.pi_block_tables(C.byref(ok), *some) == 1, i


def _page(P, **kw):
    d = dict(kv_heads=2, head_dim=64, page_size=16, num_pages=4, dtype=0, page_stride=2048, head_stride=1024,
             token_stride=64)
    d.update(kw)
    return P.binding.pi_page_desc(*[d[n] for n, _ in P.binding.pi_page_desc._fields_])


BAD_PAGES = [dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=96), dict(page_size=8), dict(page_size=256),
             dict(num_pages=0), dict(dtype=2), dict(dtype=-1), dict(token_stride=60), dict(token_stride=68),
             dict(head_stride=0), dict(head_stride=1032), dict(page_stride=-2048)]


def test_rope_refusals(P):
    L, B = P.lib(), P.binding
    plan = P.rope_plan(64)
    ok = B.pi_qkv_desc(3, 4, 0, 256, 128, 128, 256)
    ptrs = [FAKE] * 8 + [None]   # q k v positions slots q_out kcache vcache stream
    call = lambda pl, pg, d, a: L.pi_rope_store(C.byref(pl), C.byref(pg), C.byref(d), *a)  # noqa: E731
    for kw in BAD_PAGES:
        assert call(plan, _page(P, **kw), ok, ptrs) == 1, kw
    for d in (B.pi_qkv_desc(-1, 4, 0, 256, 128, 128, 256), B.pi_qkv_desc(3, 0, 0, 256, 128, 128, 256),
              B.pi_qkv_desc(3, 4, 3, 256, 128, 128, 256), B.pi_qkv_desc(3, 4, 0, 248, 128, 128, 256),
              B.pi_qkv_desc(3, 4, 0, 260, 128, 128, 256), B.pi_qkv_desc(3, 4, 0, 256, 64, 128, 256),
              B.pi_qkv_desc(3, 4, 0, 256, 128, 0, 256), B.pi_qkv_desc(3, 4, 0, 256, 128, 128, 128)):
        assert call(plan, _page(P), d, ptrs) == 1
    assert call(P.rope_plan(128), _page(P), ok, ptrs) == 1            # another head width
    for i in range(8):
        some = list(ptrs)
        some[i] = None
        assert call(plan, _page(P), ok, some) == 1, i
        some[i] = FAKE + 2
        assert call(plan, _page(P), ok, some) == 1, i
    assert call(plan, _page(P), ok, [None] * 3 + [FAKE] + [None] * 5) == 1   # neither q nor k
    # in place only where the elements lie alike
    same = [FAKE] * 8 + [None]
    assert call(plan, _page(P), B.pi_qkv_desc(3, 4, 2, 256, 128, 128, 256), same) == 1
    assert call(plan, _page(P), B.pi_qkv_desc(3, 4, 0, 512, 128, 128, 256), same) == 1
    assert call(plan, _page(P), B.pi_qkv_desc(0, 4, 0, 256, 128, 128, 256), ptrs) == 0   # no tokens, nothing to do


def test_paged_attention_refusals(P):
    L, B = P.lib(), P.binding
    ok = P.paged_desc(8, 2, 5, 4, 3)
    pg = _page(P)
    need = P.pi_paged_workspace_bytes(ok, pg)
    assert need > 0
    ptr = dict(q=FAKE, qs=512, k=FAKE, v=FAKE, table=FAKE, cu=FAKE, kv=FAKE, out=FAKE, os=512, lse=FAKE, ws=FAKE, n=need)
    call = lambda d, p, **kw: L.pi_paged_attn(C.byref(d), C.byref(p), *{**ptr, **kw}.values(), None)  # noqa: E731
    for kw in BAD_PAGES:
        assert P.pi_paged_workspace_bytes(ok, _page(P, **kw)) == 0 and call(ok, _page(P, **kw)) == 1, kw
    for d in (P.paged_desc(0, 2, 5, 4, 3), P.paged_desc(7, 2, 5, 4, 3), P.paged_desc(8, 0, 5, 4, 3),
              P.paged_desc(8, 4097, 5, 4, 3), P.paged_desc(8, 2, -1, 4, 3), P.paged_desc(8, 2, 5, 0, 3),
              P.paged_desc(8, 2, 5, 6, 3), P.paged_desc(8, 2, 5, 4, 0), P.paged_desc(8, 2, 5, 4, 1 << 27),
              P.paged_desc(8, 2, 5, 4, 3, window=-1), P.paged_desc(8, 2, 5, 4, 3, scale=-1.0),
              P.paged_desc(8, 2, 5, 4, 3, scale=math.nan), P.paged_desc(258, 2, 5, 4, 3)):
        assert P.pi_paged_workspace_bytes(d, pg) == 0 and call(d, pg) == 1
    for name in ("q", "k", "v", "table", "cu", "kv", "out"):
        assert call(ok, pg, **{name: None}) == 1 and call(ok, pg, **{name: FAKE + 2}) == 1, name
    assert call(ok, pg, lse=FAKE + 2) == 1
    assert call(ok, pg, qs=504) == 1 and call(ok, pg, qs=516) == 1 and call(ok, pg, os=256) == 1
    assert call(ok, pg, ws=None) == 5 and call(ok, pg, ws=FAKE + 8) == 5 and call(ok, pg, n=need - 1) == 5
    assert call(P.paged_desc(8, 2, 0, 1, 3), pg) == 0    # no rows, nothing to do
    assert B.lib().pi_paged_attn(None, C.byref(pg), *ptr.values(), None) == 1


def test_rope_plan_refusals(P):
    for kw in (dict(head_dim=96), dict(rot_dim=72), dict(rot_dim=8), dict(rot_dim=-16), dict(base=1.0),
               dict(base=math.inf), dict(mscale=math.nan), dict(scaling="linear", factor=0.0),
               dict(scaling="blend", factor=2.0), dict(scaling="ramp", factor=2.0, original_max=100.0, low=4.0, high=4.0)):
        with pytest.raises(P.PiError):
            P.rope_plan(**{"head_dim": 64, **kw})
    with pytest.raises(ValueError):
        P.rope_plan(64, scaling="other")


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0),
                                dict(scaling="blend", factor=8.0, original_max=8192, low=1.0, high=4.0, base=500000.0),
                                dict(scaling="ramp", factor=16.0, original_max=4096, low=1.0, high=32.0)])
@pytest.mark.parametrize("rot", [0, 16, 48, 128])
def test_rope_plan_holds_the_frequencies(P, rot, kw):
    """turns[i] is f_i / (2 pi) modulo 1 in 64-bit fixed point: fp64 evaluation of
    both sides is off by a few 2^-53 of f_i (pow, log, exp: below 2^-48)."""
    plan = P.rope_plan(128, rot, **kw)
    f = R.frequencies(rot, kw.get("base", 10000.0), *(kw.get(n, d) for n, d in (
        ("scaling", "none"), ("factor", 1.0), ("original_max", 0.0), ("low", 1.0), ("high", 4.0))))
    assert plan.rot_dim == rot and plan.head_dim == 128 and plan.interleaved == 0 and plan.mscale == 1.0
    for i in range(rot // 2):
        assert abs(plan.turns[i] / 2.0 ** 64 - float(f[i]) / (2 * math.pi)) <= 2.0 ** -48 * float(f[i]) + 2.0 ** -53
    assert all(plan.turns[i] == 0 for i in range(rot // 2, 64))


def test_binding_refuses_other_tensors(P):
    """Wrong devices, types, shapes and strides raise before the library is called."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        P.page_desc(k, k[:2])
    with pytest.raises(ValueError):
        P.page_desc(k.float(), k)
    with pytest.raises(ValueError):
        P.page_desc(k, k.transpose(1, 2).contiguous().transpose(1, 2))
    d = P.page_desc(k, k)
    assert (d.kv_heads, d.head_dim, d.page_size, d.num_pages, d.dtype) == (2, 64, 16, 4, 0)
    assert (d.page_stride, d.head_stride, d.token_stride) == (2048, 1024, 64)
    t = k.transpose(1, 2).contiguous().transpose(1, 2)
    d = P.page_desc(t, t)
    assert (d.page_stride, d.head_stride, d.token_stride) == (2048, 64, 128)
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):     # host tensors
        P.pi_block_tables(P.tables_desc(4, 16, 8, 2, 8), i, i, i, i, i, i, i, i, i, i, i.long(), i)
    with pytest.raises(ValueError):
        P.pi_paged_attn(P.paged_desc(2, 1, 1, 1, 1), d, k[0], k, k, i, i, i, k[0], None, i)


def test_reference_tables_by_hand():
    """Pages of 16: row 0 keeps 20 of its positions and takes 20 (needs 3 pages, holds 2),
    row 1 ended (gives back pages 7, 8), row 2 wants two, row 3 three: too many."""
    r = R.tables(16, 100, [20, 0, 0, 0], [20, 0, 30, 40], [2, 2, 0, 0],
                 [[5, 6, -1], [7, 8, -1], [-1] * 3, [-1] * 3], [1, 2, -1, -1, -1], 2)
    assert r["held"] == [3, 0, 2, 0] and r["count"] == 1 and not r["status"]
    assert r["stack"] == [1, 2, 7, 8, -1]
    assert r["table"] == [[5, 6, 8], [7, 8, -1], [7, 2, -1], [-1] * 3]
    assert r["cu"] == [0, 20, 20, 50, 90] and r["kv"] == [40, 0, 30, 0]
    assert r["slots"][:20] == [6 * 16 + 4 + i for i in range(12)] + [8 * 16 + i for i in range(8)]
    assert r["slots"][20:50] == [7 * 16 + i for i in range(16)] + [2 * 16 + i for i in range(14)]
    assert r["slots"][50:] == [-1] * 50 and r["pos"][:21] == list(range(20, 40)) + [0] and r["pos"][90:] == [0] * 10


def test_reference_rotation_by_hand():
    """One pair, a quarter turn per position."""
    x = torch.tensor([[[3.0, 4.0, 5.0]]])
    y, _ = R.rotate(x, torch.tensor([1]), torch.tensor([math.pi / 2], dtype=torch.float64), True)
    assert torch.allclose(y, torch.tensor([[[-4.0, 3.0, 5.0]]], dtype=torch.float64))
    y, _ = R.rotate(x, torch.tensor([2]), torch.tensor([math.pi / 2], dtype=torch.float64), False, mscale=2.0)
    assert torch.allclose(y, torch.tensor([[[-6.0, -8.0, 5.0]]], dtype=torch.float64))


def test_reference_attention_by_hand():
    """Keys 0 and e: the second token's weights are 1 : e^{1} over values 1 and 3."""
    q = torch.zeros(2, 1, 64)
    q[:, 0, 0] = 8.0
    k = torch.zeros(1, 1, 16, 64)
    k[0, 0, 1, 0] = 1.0
    v = torch.zeros(1, 1, 16, 64)
    v[0, 0, 0, 5], v[0, 0, 1, 5] = 1.0, 3.0
    out, lse, _, _ = R.attention(q, k, v, torch.zeros(1, 1, dtype=torch.int32), [0, 2], [2])
    e = math.e
    assert abs(float(out[0, 0, 5]) - 1.0) < 1e-12 and abs(float(out[1, 0, 5]) - (1 + 3 * e) / (1 + e)) < 1e-12
    assert abs(float(lse[1, 0]) - math.log(1 + e)) < 1e-12
