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
