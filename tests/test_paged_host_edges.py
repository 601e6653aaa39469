"""Paged serving on the host: outputs that overlap inputs are refused before any launch."""
import ctypes as C

import pytest

from tests.test_paged_host import FAKE, P, _page  # noqa: F401


def test_attention_output_over_its_queries_is_refused(P):
    """Rows whose sums are not finite are read again after outputs are written."""
    L, d, pg = P.lib(), P.paged_desc(8, 2, 5, 4, 3), _page(P)
    need = P.pi_paged_workspace_bytes(d, pg)

    def call(q, qs, out, os):
        return L.pi_paged_attn(C.byref(d), C.byref(pg), q, qs, FAKE, FAKE, FAKE, FAKE, FAKE, out, os, None, FAKE, need, None)

    row = 512 * 2                                    # bytes of a row of 8 heads of 64
    assert call(FAKE, 512, FAKE, 512) == 1           # in place
    assert call(FAKE, 512, FAKE + row, 512) == 1     # a row further
    assert call(FAKE, 512, FAKE - 4 * row, 512) == 1
    assert call(FAKE, 1024, FAKE + row - 16, 1024) == 1 and call(FAKE, 1024, FAKE + 2 * row + 16, 1024) == 1
    assert call(FAKE, 512, FAKE + row, 1024) == 1    # other strides, one inside the other


def test_rotated_queries_over_others_are_refused(P):
    """In place a thread reads what it writes first; a shifted output would overwrite queries not yet read."""
    L, B = P.lib(), P.binding
    plan, pg = P.rope_plan(64), _page(P)

    far = FAKE + (1 << 16)

    def call(d, q, out, k=None, v=None):
        slots, cache = (None, None) if k is None else (far, far)
        return L.pi_rope_store(C.byref(plan), C.byref(pg), C.byref(d), q, k, v, far, slots, out, cache, cache, None)

    d = B.pi_qkv_desc(3, 4, 0, 256, 0, 0, 256)
    for off in (256 * 2, -256 * 2, 16, 2 * 256 * 2):
        assert call(d, FAKE, FAKE + off) == 1, off
    wide = B.pi_qkv_desc(3, 4, 2, 256, 0, 0, 256)    # fp32 queries
    for off in (0, 256 * 4, 2 * 256 * 4, -256 * 2):
        assert call(wide, FAKE, FAKE + off) == 1, off
    # projections in rows of 8 heads: q 4, k 2, v 2; outputs may take q's place and no other
    both = B.pi_qkv_desc(3, 4, 0, 512, 512, 512, 512)
    k, v = FAKE + 512, FAKE + 768
    assert call(both, FAKE, k, k, v) == 1 and call(both, FAKE, FAKE + 128, k, v) == 1
    assert call(B.pi_qkv_desc(3, 4, 0, 512, 512, 512, 256), FAKE, FAKE, k, v) == 1
    assert call(B.pi_qkv_desc(3, 4, 0, 512, 512, 512, 256), FAKE, FAKE + 2 * 1024 + 512, k, v) == 1
