"""The 8-bit paged cache on the host: refused arguments launch nothing, and the
reference's rounding is the type's."""
import ctypes as C
import math

import pytest
import torch

from tests import paged8_ref as R


@pytest.fixture(scope="module")
def P():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_ffn_layer_gb300 as P
    return P


FAKE = 1 << 20   # an aligned address that no refused call touches


def _page(P, **kw):
    d = dict(kv_heads=2, head_dim=64, page_size=16, num_pages=4, page_stride=2048, head_stride=1024, token_stride=64)
    d.update(kw)
    return P.binding.pi_page8_desc(*[d[n] for n, _ in P.binding.pi_page8_desc._fields_])


BAD_PAGES = [dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=96), dict(page_size=8), dict(page_size=256),
             dict(num_pages=0), dict(num_pages=(1 << 26) + 1), dict(token_stride=48), dict(token_stride=72),
             dict(head_stride=0), dict(head_stride=1032), dict(page_stride=-2048), dict(page_stride=(1 << 36) + 16)]


def test_reference_rounds_as_the_type():
    """The table against torch's own type, and the rounding of midpoints and their neighbours."""
    codes = torch.arange(256, dtype=torch.uint8)
    torch.testing.assert_close(R.VALUES, codes.view(R.CODE).double(), rtol=0, atol=0, equal_nan=True)
    g = R.VALUES[:127]
    mid = (g[1:] + g[:-1]) / 2
    y = torch.cat([g, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), torch.linspace(0, 448, 4001, dtype=torch.float64)])
    y = torch.cat([y, -y])
    assert torch.equal(R.encode(y), y.float().to(R.CODE).view(torch.uint8))
    assert R.encode(torch.tensor([math.inf, -math.inf, math.nan, 1e30], dtype=torch.float64)).tolist() == [127, 127, 127, 126]


def test_store8_refusals(P):
    L, B = P.lib(), P.binding
    plan = P.rope_plan(64)
    ok = B.pi_qkv_desc(3, 4, 0, 256, 128, 128, 256)
    ptrs = [FAKE << i for i in range(10)] + [None]   # q k v positions slots q_out kcache vcache kexp vexp stream
    call = lambda pl, pg, d, a, dt=0: L.pi_rope_store8(C.byref(pl), C.byref(pg), C.byref(d), dt, *a)  # noqa: E731
    for kw in BAD_PAGES:
        assert call(plan, _page(P, **kw), ok, ptrs) == 1, kw
    for d in (B.pi_qkv_desc(-1, 4, 0, 256, 128, 128, 256), B.pi_qkv_desc(3, 0, 0, 256, 128, 128, 256),
              B.pi_qkv_desc(3, 4, 3, 256, 128, 128, 256), B.pi_qkv_desc(3, 4, 0, 248, 128, 128, 256),
              B.pi_qkv_desc(3, 4, 0, 260, 128, 128, 256), B.pi_qkv_desc(3, 4, 0, 256, 64, 128, 256),
              B.pi_qkv_desc(3, 4, 0, 256, 128, 0, 256), B.pi_qkv_desc(3, 4, 0, 256, 128, 128, 128)):
        assert call(plan, _page(P), d, ptrs) == 1
    for dt in (-1, 2, 3):                                             # queries come out in 16 bits
        assert call(plan, _page(P), ok, ptrs, dt) == 1
    assert call(P.rope_plan(128), _page(P), ok, ptrs) == 1            # another head width
    for i in range(10):
        some = list(ptrs)
        some[i] = None
        assert call(plan, _page(P), ok, some) == 1, i
        if i < 8:
            some[i] = ptrs[i] + 2
            assert call(plan, _page(P), ok, some) == 1, i
    assert call(plan, _page(P), ok, [None] * 3 + [FAKE] + [None] * 7) == 1   # neither q nor k
    # rotated queries over keys or values, or over queries that lie otherwise
    for i in (1, 2):
        some = list(ptrs)
        some[5] = some[i]
        assert call(plan, _page(P), ok, some) == 1
    same = list(ptrs)
    same[5] = same[0]
    assert call(plan, _page(P), B.pi_qkv_desc(3, 4, 2, 256, 128, 128, 256), same) == 1
    assert call(plan, _page(P), B.pi_qkv_desc(3, 4, 0, 512, 128, 128, 256), same) == 1
    assert call(plan, _page(P), B.pi_qkv_desc(0, 4, 0, 256, 128, 128, 256), ptrs) == 0   # no tokens, nothing to do


def test_read8_refusals(P):
    L, B = P.lib(), P.binding
    ok = (2, 3, 10, 0, 128, 128)
    ptrs = [FAKE << i for i in range(9)] + [None]    # kcache vcache kexp vexp table start cu k_out v_out stream
    call = lambda d, pg, a: L.pi_page_read8(C.byref(B.pi_read8_desc(*d)), C.byref(pg), *a)  # noqa: E731
    for kw in BAD_PAGES:
        assert call(ok, _page(P, **kw), ptrs) == 1, kw
    for i, v in ((0, 0), (0, 4097), (1, 0), (1, 1 << 27), (2, -1), (2, (1 << 30) + 1), (3, 3), (3, -1), (4, 120), (4, 132), (5, 64)):
        d = list(ok)
        d[i] = v
        assert call(d, _page(P), ptrs) == 1, (i, v)
    for i in (0, 1, 2, 3, 4, 6, 7, 8):
        some = list(ptrs)
        some[i] = None
        assert call(ok, _page(P), some) == 1, i
        if i not in (2, 3):
            some[i] = ptrs[i] + 2
            assert call(ok, _page(P), some) == 1, i
    assert call(ok, _page(P), [None, None, None, None] + ptrs[4:7] + [None, None, None]) == 1
    same = list(ptrs)
    same[8] = same[7]
    assert call(ok, _page(P), same) == 1             # both outputs over one another
    assert call((2, 3, 0, 0, 128, 128), _page(P), ptrs) == 0


def test_attention8_refusals(P):
    L, B = P.lib(), P.binding
    ok = P.paged_desc(8, 2, 5, 4, 3)
    pg = _page(P)
    need = P.pi_paged8_workspace_bytes(ok, pg)
    assert need > 0
    ptr = dict(dt=0, q=FAKE, qs=512, k=FAKE << 1, v=FAKE << 2, ke=FAKE << 3, ve=FAKE << 4, table=FAKE << 5, cu=FAKE << 6,
               kv=FAKE << 7, out=FAKE << 8, os=512, lse=FAKE << 9, ws=FAKE << 10, n=need)
    call = lambda d, p, **kw: L.pi_paged_attn8(C.byref(d), C.byref(p), *{**ptr, **kw}.values(), None)  # noqa: E731
    for kw in BAD_PAGES:
        assert P.pi_paged8_workspace_bytes(ok, _page(P, **kw)) == 0 and call(ok, _page(P, **kw)) == 1, kw
    for d in (P.paged_desc(0, 2, 5, 4, 3), P.paged_desc(7, 2, 5, 4, 3), P.paged_desc(8, 0, 5, 4, 3),
              P.paged_desc(8, 4097, 5, 4, 3), P.paged_desc(8, 2, -1, 4, 3), P.paged_desc(8, 2, 5, 0, 3),
              P.paged_desc(8, 2, 5, 6, 3), P.paged_desc(8, 2, 5, 4, 0), P.paged_desc(8, 2, 5, 4, 1 << 27),
              P.paged_desc(8, 2, 5, 4, 3, window=-1), P.paged_desc(8, 2, 5, 4, 3, scale=-1.0),
              P.paged_desc(8, 2, 5, 4, 3, scale=math.nan), P.paged_desc(258, 2, 5, 4, 3)):
        assert P.pi_paged8_workspace_bytes(d, pg) == 0 and call(d, pg) == 1
    for name in ("q", "k", "v", "table", "cu", "kv", "out"):
        assert call(ok, pg, **{name: None}) == 1 and call(ok, pg, **{name: ptr[name] + 2}) == 1, name
    assert call(ok, pg, ke=None) == 1 and call(ok, pg, ve=None) == 1 and call(ok, pg, lse=FAKE + 2) == 1
    assert call(ok, pg, dt=2) == 1 and call(ok, pg, dt=-1) == 1
    assert call(ok, pg, qs=504) == 1 and call(ok, pg, qs=516) == 1 and call(ok, pg, os=256) == 1
    assert call(ok, pg, out=FAKE) == 1                                   # over the queries
    assert call(ok, pg, ws=None) == 5 and call(ok, pg, ws=FAKE + 8) == 5 and call(ok, pg, n=need - 1) == 5
    assert call(P.paged_desc(8, 2, 0, 1, 3), pg) == 0    # no rows, nothing to do
    assert L.pi_paged_attn8(None, C.byref(pg), *ptr.values(), None) == 1


def test_binding_refuses_other_tensors(P):
    codes = torch.zeros(4, 2, 16, 64, dtype=R.CODE)
    with pytest.raises(ValueError):
        P.page8_desc(codes, codes.half())
    with pytest.raises(ValueError):
        P.page8_desc(codes, codes[:2])
    with pytest.raises(ValueError):
        P.page8_desc(codes.half(), codes.half())
    d = P.page8_desc(codes, codes)
    with pytest.raises(ValueError):                       # not on a GPU
        P.binding._cache8(d, codes, torch.zeros(4, 2, 1, dtype=torch.int8), "kcache")
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    with pytest.raises(ValueError):
        PagedCache(2, 2, 64, 1, 16, 1, 1, bits=4, device="cpu")
    for wrong in (torch.zeros(4, 2, 1, dtype=torch.uint8), torch.zeros(4, 2, 2, dtype=torch.int8),
                  torch.zeros(1, 2, 4, dtype=torch.int8).transpose(0, 2)):
        with pytest.raises(ValueError):
            P.binding._cache8(d, codes, wrong, "kcache")
    with pytest.raises(ValueError):                       # other strides than the description's
        P.binding._cache8(d, torch.zeros(4, 16, 2, 64, dtype=R.CODE).transpose(1, 2), torch.zeros(4, 2, 1, dtype=torch.int8), "kcache")
    bare = P.binding.pi_page8_desc(2, 64, 16, 4, 2048, 1024, 64)    # made by hand
    with pytest.raises(ValueError):
        P.binding._cache8(bare, codes, torch.zeros(4, 2, 2, dtype=torch.int8), "kcache")
