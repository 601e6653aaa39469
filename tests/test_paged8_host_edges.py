"""The 8-bit paged cache on the host: calls of no rows, and types that a cache is not made for."""
import ctypes as C

import pytest
import torch

from tests.test_paged8_host import P, _page  # noqa: F401


def test_calls_of_no_rows_need_no_tensors(P):
    """An empty tensor has no address: with no rows that is not an argument that is missing."""
    L, B = P.lib(), P.binding
    none = B.pi_qkv_desc(0, 4, 0, 256, 128, 128, 256)
    plan, pg = P.rope_plan(64), _page(P)
    other = B.pi_page_desc(2, 64, 16, 4, 0, 2048, 1024, 64)
    assert L.pi_rope_store8(C.byref(plan), C.byref(pg), C.byref(none), 0, *[None] * 11) == 0
    assert L.pi_rope_store(C.byref(plan), C.byref(other), C.byref(none), *[None] * 9) == 0
    codes = [1 << 20, 1 << 21, 1 << 22, 1 << 23]
    read = lambda rows, a: L.pi_page_read8(C.byref(B.pi_read8_desc(2, 3, rows, 0, 128, 128)), C.byref(pg), *a)  # noqa: E731
    assert read(0, codes + [1 << 24, None, 1 << 25, None, None, None]) == 0
    assert read(0, [None] * 10) == 0
    assert read(1, codes + [1 << 24, None, 1 << 25, None, None, None]) == 1     # a row that nothing takes
    # what describes the call is looked at all the same
    assert L.pi_rope_store8(C.byref(P.rope_plan(128)), C.byref(pg), C.byref(none), 0, *[None] * 11) == 1
    assert L.pi_page_read8(C.byref(B.pi_read8_desc(0, 3, 0, 0, 128, 128)), C.byref(pg), *[None] * 10) == 1
    assert L.pi_page_read8(C.byref(B.pi_read8_desc(2, 3, 0, 3, 128, 128)), C.byref(pg), *[None] * 10) == 1


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64, torch.int8])
def test_a_cache_of_other_types_is_refused(P, bits, dtype):
    """Queries and outputs are fp16 or bf16 with either cache: refused when the cache is made, not at the first step."""
    from activation_sparse_ffn_layer_gb300.paged import PagedCache
    with pytest.raises(ValueError):
        PagedCache(2, 2, 64, 1, 16, 1, 1, dtype=dtype, device="cpu", bits=bits)
