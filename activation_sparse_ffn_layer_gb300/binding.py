"""Thin Python binding of ``libpi.so`` (the C ABI declared in ``include/pi.h``).

Argument marshalling only: torch CUDA tensors in, device pointers and the
current CUDA stream out; every step of the decode path runs in the library's
kernels.  The functions carry the C names.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Tuple

import torch

from .build import LIB

PI_OK, PI_ERR_INVALID_ARG, PI_ERR_UNSUPPORTED, PI_ERR_CUDA, PI_ERR_TIMEOUT, PI_ERR_WORKSPACE = range(6)
PI_W_F16, PI_W_INT4_G32 = 0, 1
PI_T_F16, PI_T_BF16, PI_T_F32 = 0, 1, 2


class pi_layer_desc(C.Structure):
    _fields_ = [("d", C.c_int), ("ffn", C.c_int), ("rank", C.c_int), ("batch", C.c_int),
                ("wdtype", C.c_int), ("gated", C.c_int)]


class pi_layer_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("w1", "w1_scales", "b1", "wu", "w2t", "w2t_scales", "b2",
                                          "p1", "p2", "table")]


class pi_workspace_layout_t(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("mask", "idx", "count", "h", "total")]


class pi_cold_tier(C.Structure):
    _fields_ = [("n_hot", C.c_int)] + [(n, C.c_void_p) for n in ("w1", "w1_scales", "wu", "w2t", "w2t_scales")]


class pi_stack_plan_t(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("fused", "ctas", "pred_in_smem", "p2_ring_slots", "fc_row_slots",
                                       "smem_bytes")]


class pi_attn_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("d", "heads", "kv_heads", "head_dim", "rank", "batch", "max_seq")]


class pi_attn_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("wqkv", "bqkv", "wot", "bo", "p1", "p2", "bp")]


class pi_tables_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("batch", "page_size", "num_pages", "max_pages", "max_tokens")]


class pi_page_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("kv_heads", "head_dim", "page_size", "num_pages", "dtype")] + \
        [(n, C.c_longlong) for n in ("page_stride", "head_stride", "token_stride")]


class pi_rope_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("head_dim", "rot_dim", "interleaved", "scaling")] + \
        [(n, C.c_double) for n in ("base", "factor", "original_max", "low", "high", "mscale")]


class pi_rope_plan(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("head_dim", "rot_dim", "interleaved")] + \
        [("mscale", C.c_float), ("turns", C.c_uint64 * 64)]


class pi_qkv_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("tokens", "heads", "dtype")] + \
        [(n, C.c_longlong) for n in ("q_stride", "k_stride", "v_stride", "out_stride")]


class pi_paged_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("heads", "batch", "max_tokens", "max_new", "max_pages", "window")] + \
        [("scale", C.c_float)]


class pi_page8_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("kv_heads", "head_dim", "page_size", "num_pages")] + \
        [(n, C.c_longlong) for n in ("page_stride", "head_stride", "token_stride")]


class pi_read8_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("batch", "max_pages", "max_rows", "dtype")] + \
        [(n, C.c_longlong) for n in ("k_stride", "v_stride")]


class PiError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


_lib = None

EXPORTS = ("pi_workspace_bytes", "pi_workspace_layout", "pi_predict", "pi_compact", "pi_sparse_fc1",
           "pi_sparse_fc2", "pi_ffn_layer", "pi_rmsnorm_half", "pi_status_string",
           "pi_last_device_status", "pi_launches_per_layer", "pi_ffn_stack", "pi_debug_wait_timeout",
           "pi_sparse_fc2_noalloc", "pi_stack_plan", "pi_stack_plan_for", "pi_debug_set_wait_timeout",
           "pi_sparse_fc1_tiered", "pi_sparse_fc2_tiered", "pi_ffn_layer_tiered", "pi_attn_workspace_bytes",
           "pi_attn_heads", "pi_block_tables", "pi_rope_plan_init", "pi_rope_store", "pi_paged_workspace_bytes",
           "pi_paged_attn", "pi_rope_store8", "pi_page_read8", "pi_paged8_workspace_bytes", "pi_paged_attn8")


def library_path() -> str:
    return LIB


def lib(path: Optional[str] = None):
    """Load ``libpi.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB
    if not os.path.exists(p):
        raise RuntimeError(f"libpi.so not built ({p}); run __graft_entry__.build() or "
                           "python -m activation_sparse_ffn_layer_gb300.build")
    L = C.CDLL(p)
    P, I, Fl, S = C.c_void_p, C.c_int, C.c_float, C.c_size_t
    D = C.POINTER(pi_layer_desc)
    Wt = C.POINTER(pi_layer_weights)
    sig = {
        "pi_workspace_bytes": (S, [D]),
        "pi_workspace_layout": (I, [D, C.POINTER(pi_workspace_layout_t)]),
        "pi_predict": (I, [D, P, P, P, P, Fl, P, P, S, P]),
        "pi_compact": (I, [D, P, P, P, P, P, P]),
        "pi_sparse_fc1": (I, [D, P, Wt, P, P, P, P, P, S, P]),
        "pi_sparse_fc2": (I, [D, P, P, P, Wt, P, P, S, P]),
        "pi_ffn_layer": (I, [D, P, Wt, Fl, P, S, P, P]),
        "pi_rmsnorm_half": (I, [I, I, P, Fl, P, P]),
        "pi_status_string": (C.c_char_p, [I]),
        "pi_last_device_status": (I, [P]),
        "pi_launches_per_layer": (I, [D]),
        "pi_ffn_stack": (I, [D, I, C.POINTER(pi_layer_weights), P, P, Fl, Fl, P, S, P, P, P, P]),
        "pi_debug_wait_timeout": (I, [C.c_longlong, P]),
        "pi_sparse_fc2_noalloc": (I, [D, P, P, P, Wt, P, P]),
        "pi_stack_plan": (I, [D, I, P, C.POINTER(pi_stack_plan_t)]),
        "pi_stack_plan_for": (I, [D, I, P, I, C.POINTER(pi_stack_plan_t)]),
        "pi_debug_set_wait_timeout": (I, [C.c_longlong]),
        "pi_sparse_fc1_tiered": (I, [D, P, Wt, C.POINTER(pi_cold_tier), P, P, P, P, P]),
        "pi_sparse_fc2_tiered": (I, [D, P, P, P, Wt, C.POINTER(pi_cold_tier), P, P, S, P]),
        "pi_ffn_layer_tiered": (I, [D, P, Wt, C.POINTER(pi_cold_tier), Fl, P, S, P, P]),
        "pi_attn_workspace_bytes": (S, [C.POINTER(pi_attn_desc)]),
        "pi_attn_heads": (I, [C.POINTER(pi_attn_desc), P, C.POINTER(pi_attn_weights), P, P, P, Fl, P, P, P, S,
                              P]),
        "pi_block_tables": (I, [C.POINTER(pi_tables_desc)] + [P] * 13),
        "pi_rope_plan_init": (I, [C.POINTER(pi_rope_desc), C.POINTER(pi_rope_plan)]),
        "pi_rope_store": (I, [C.POINTER(pi_rope_plan), C.POINTER(pi_page_desc), C.POINTER(pi_qkv_desc)] + [P] * 9),
        "pi_paged_workspace_bytes": (S, [C.POINTER(pi_paged_desc), C.POINTER(pi_page_desc)]),
        "pi_paged_attn": (I, [C.POINTER(pi_paged_desc), C.POINTER(pi_page_desc), P, C.c_longlong, P, P, P, P, P, P,
                              C.c_longlong, P, P, S, P]),
        "pi_rope_store8": (I, [C.POINTER(pi_rope_plan), C.POINTER(pi_page8_desc), C.POINTER(pi_qkv_desc), I] + [P] * 11),
        "pi_page_read8": (I, [C.POINTER(pi_read8_desc), C.POINTER(pi_page8_desc)] + [P] * 10),
        "pi_paged8_workspace_bytes": (S, [C.POINTER(pi_paged_desc), C.POINTER(pi_page8_desc)]),
        "pi_paged_attn8": (I, [C.POINTER(pi_paged_desc), C.POINTER(pi_page8_desc), I, P, C.c_longlong] + [P] * 8 +
                           [C.c_longlong, P, P, S, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = L
    return L


# ------------------------------------------------------------------ marshalling

def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return C.c_void_p(t.data_ptr())


# handle of a device's current stream without a torch.cuda.Stream object around
# it (3 us a call on a Grace core); the public way where torch has no such call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)   # torch.cuda.current_device without its check for a first use


def _stream():
    if _raw_stream is None or _raw_device is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_raw_device())


def _check(fn: str, st: int):
    if st != PI_OK:
        raise PiError(fn, st, lib().pi_status_string(st).decode())


def desc_of(d: int, ffn: int, rank: int, batch: int = 1, int4: bool = False, gated: bool = False) -> pi_layer_desc:
    return pi_layer_desc(d, ffn, rank, batch, PI_W_INT4_G32 if int4 else PI_W_F16, 1 if gated else 0)


def layer_desc(w, batch: int = 1) -> pi_layer_desc:
    return desc_of(w.d, w.F, w.r, batch, w.int4, w.gated)


def weights_struct(w) -> pi_layer_weights:
    """A pi_layer_weights over a layer's device tensors (keep `w` alive)."""
    s = pi_layer_weights()
    if w.int4:
        s.w1, s.w1_scales = _ptr(w.w1_q), _ptr(w.w1_s)
        s.w2t, s.w2t_scales = _ptr(w.w2t_q), _ptr(w.w2t_s)
    else:
        s.w1, s.w2t = _ptr(w.w1), _ptr(w.w2t)
    s.b1, s.b2, s.p1, s.p2, s.table = _ptr(w.b1), _ptr(w.b2), _ptr(w.p1), _ptr(w.p2), _ptr(w.table)
    if w.gated:
        s.wu = _ptr(w.wu)
    return s


# ------------------------------------------------------------- the C entry points

def pi_workspace_bytes(desc: pi_layer_desc) -> int:
    return int(lib().pi_workspace_bytes(C.byref(desc)))


def pi_workspace_layout(desc: pi_layer_desc) -> pi_workspace_layout_t:
    out = pi_workspace_layout_t()
    _check("pi_workspace_layout", lib().pi_workspace_layout(C.byref(desc), C.byref(out)))
    return out


def pi_predict(desc, x, p1, p2, bpred, tau: float, mask, workspace):
    _check("pi_predict", lib().pi_predict(C.byref(desc), _ptr(x), _ptr(p1), _ptr(p2), _ptr(bpred),
                                          float(tau), _ptr(mask), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream()))


def pi_compact(desc, mask, table, idx, orig_idx, d_count):
    _check("pi_compact", lib().pi_compact(C.byref(desc), _ptr(mask), _ptr(table), _ptr(idx), _ptr(orig_idx),
                                          _ptr(d_count), _stream()))


def pi_sparse_fc1(desc, x, wstruct, idx, d_count, mask, h, workspace):
    _check("pi_sparse_fc1", lib().pi_sparse_fc1(C.byref(desc), _ptr(x), C.byref(wstruct), _ptr(idx),
                                                _ptr(d_count), _ptr(mask), _ptr(h), _ptr(workspace),
                                                workspace.numel() * workspace.element_size(), _stream()))


def pi_sparse_fc2(desc, h, idx, d_count, wstruct, y, workspace):
    _check("pi_sparse_fc2", lib().pi_sparse_fc2(C.byref(desc), _ptr(h), _ptr(idx), _ptr(d_count),
                                                C.byref(wstruct), _ptr(y), _ptr(workspace),
                                                workspace.numel() * workspace.element_size(), _stream()))


def pi_sparse_fc2_noalloc(desc, h, idx, d_count, wstruct, y):
    """pi_sparse_fc2 without a workspace: for callers that cannot allocate
    device memory (the partial sums live in a fixed array inside the library;
    calls must not overlap on the GPU)."""
    _check("pi_sparse_fc2_noalloc", lib().pi_sparse_fc2_noalloc(C.byref(desc), _ptr(h), _ptr(idx), _ptr(d_count),
                                                                C.byref(wstruct), _ptr(y), _stream()))


def pi_ffn_layer(desc, x, wstruct, tau: float, workspace, y):
    _check("pi_ffn_layer", lib().pi_ffn_layer(C.byref(desc), _ptr(x), C.byref(wstruct), float(tau),
                                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                                              _ptr(y), _stream()))


def pi_ffn_stack(desc, wstructs, ranks, x, tau: float, eps: float, workspace, y, x_trace=None,
                 layer_counts=None):
    """`wstructs`: a ctypes array of pi_layer_weights (see weights_array);
    `ranks`: a ctypes int array or None; `layer_counts`: int32 [L, 2] or None."""
    n = len(wstructs)
    _check("pi_ffn_stack", lib().pi_ffn_stack(C.byref(desc), n, wstructs, ranks, _ptr(x), float(tau), float(eps),
                                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                                              _ptr(y), _ptr(x_trace), _ptr(layer_counts), _stream()))


def weights_array(layers):
    """A ctypes array of pi_layer_weights over a list of layers (keep them alive)."""
    arr = (pi_layer_weights * len(layers))()
    for i, w in enumerate(layers):
        arr[i] = weights_struct(w)
    return arr


def ranks_array(layers):
    return (C.c_int * len(layers))(*[int(w.r) for w in layers])


def _addr(t):
    """Address of a tensor for the C ABI: device memory, or host memory the
    GPU can address (pinned)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError("expected a CUDA tensor or pinned host memory")
    return C.c_void_p(t.data_ptr())


def cold_tier(n_hot: int, w1=None, w1_scales=None, wu=None, w2t=None, w2t_scales=None) -> pi_cold_tier:
    """A pi_cold_tier over tensors in device or pinned host memory (keep them alive)."""
    s = pi_cold_tier()
    s.n_hot = int(n_hot)
    s.w1, s.w1_scales, s.wu = _addr(w1), _addr(w1_scales), _addr(wu)
    s.w2t, s.w2t_scales = _addr(w2t), _addr(w2t_scales)
    return s


def pi_sparse_fc1_tiered(desc, x, wstruct, cold, idx, d_count, mask, h):
    _check("pi_sparse_fc1_tiered", lib().pi_sparse_fc1_tiered(C.byref(desc), _ptr(x), C.byref(wstruct), C.byref(cold),
                                                              _ptr(idx), _ptr(d_count), _ptr(mask), _ptr(h),
                                                              _stream()))


def pi_sparse_fc2_tiered(desc, h, idx, d_count, wstruct, cold, y, workspace):
    _check("pi_sparse_fc2_tiered", lib().pi_sparse_fc2_tiered(C.byref(desc), _ptr(h), _ptr(idx), _ptr(d_count),
                                                              C.byref(wstruct), C.byref(cold), _ptr(y),
                                                              _ptr(workspace),
                                                              workspace.numel() * workspace.element_size(),
                                                              _stream()))


def pi_ffn_layer_tiered(desc, x, wstruct, cold, tau: float, workspace, y):
    _check("pi_ffn_layer_tiered", lib().pi_ffn_layer_tiered(C.byref(desc), _ptr(x), C.byref(wstruct), C.byref(cold),
                                                            float(tau), _ptr(workspace),
                                                            workspace.numel() * workspace.element_size(), _ptr(y),
                                                            _stream()))


def pi_stack_plan(desc, n_layers: int, ranks=None) -> pi_stack_plan_t:
    """How a pi_ffn_stack step of `n_layers` layers runs on the current device."""
    out = pi_stack_plan_t()
    _check("pi_stack_plan", lib().pi_stack_plan(C.byref(desc), int(n_layers), ranks, C.byref(out)))
    return out


def pi_stack_plan_for(desc, n_layers: int, sm_count: int, ranks=None) -> pi_stack_plan_t:
    """The same plan for a device with `sm_count` SMs (host only, no device)."""
    out = pi_stack_plan_t()
    _check("pi_stack_plan_for", lib().pi_stack_plan_for(C.byref(desc), int(n_layers), ranks, int(sm_count),
                                                        C.byref(out)))
    return out


def pi_debug_set_wait_timeout(timeout_ns: int):
    _check("pi_debug_set_wait_timeout", lib().pi_debug_set_wait_timeout(int(timeout_ns)))


def pi_debug_wait_timeout(timeout_ns: int):
    _check("pi_debug_wait_timeout", lib().pi_debug_wait_timeout(int(timeout_ns), _stream()))


def pi_rmsnorm_half(d: int, batch: int, y, eps: float, x_out):
    _check("pi_rmsnorm_half", lib().pi_rmsnorm_half(int(d), int(batch), _ptr(y), float(eps), _ptr(x_out),
                                                    _stream()))


def pi_status_string(status: int) -> str:
    return lib().pi_status_string(int(status)).decode()


def pi_launches_per_layer(desc) -> int:
    return int(lib().pi_launches_per_layer(C.byref(desc)))


def pi_last_device_status() -> int:
    return int(lib().pi_last_device_status(_stream()))


# ------------------------------------------------------- head-sparse attention

def attn_desc_of(d: int, heads: int, kv_heads: int, head_dim: int, rank: int, batch: int = 1,
                 max_seq: int = 1024) -> pi_attn_desc:
    return pi_attn_desc(d, heads, kv_heads, head_dim, rank, batch, max_seq)


def attn_desc(w, batch: int = 1, max_seq: int = 1024) -> pi_attn_desc:
    return attn_desc_of(w.d, w.H, w.KVH, w.dh, w.r, batch, max_seq)


def attn_weights_struct(w) -> pi_attn_weights:
    """A pi_attn_weights over an attention block's device tensors (keep `w` alive)."""
    s = pi_attn_weights()
    s.wqkv, s.bqkv, s.wot, s.bo = _ptr(w.wqkv), _ptr(w.bqkv), _ptr(w.wot), _ptr(w.bo)
    s.p1, s.p2, s.bp = _ptr(w.p1), _ptr(w.p2), _ptr(w.bp)
    return s


def pi_attn_workspace_bytes(desc: pi_attn_desc) -> int:
    return int(lib().pi_attn_workspace_bytes(C.byref(desc)))


def pi_attn_heads(desc, x, wstruct, kcache, vcache, pos, tau: float, head_mask, y, workspace):
    _check("pi_attn_heads", lib().pi_attn_heads(C.byref(desc), _ptr(x), C.byref(wstruct), _ptr(kcache),
                                                _ptr(vcache), _ptr(pos), float(tau), _ptr(head_mask), _ptr(y),
                                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                _stream()))


# ------------------------------------------------------------------ paged serving

_DTYPES = {torch.float16: PI_T_F16, torch.bfloat16: PI_T_BF16, torch.float32: PI_T_F32}
_SCALINGS = {"none": 0, "linear": 1, "blend": 2, "ramp": 3}


def _flat(t: torch.Tensor, dtype: torch.dtype, least: int, name: str) -> int:
    """Address of a contiguous CUDA tensor of this type with at least this many elements."""
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.numel() < least:
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of {least} or more {dtype} values")
    return t.data_ptr()


def _table(t: torch.Tensor, batch: int, max_pages: int) -> int:
    """Address of a block table; with two dimensions its rows are max_pages apart."""
    if t.dim() == 2 and t.shape[1] != max_pages:
        raise ValueError(f"block_table: expected rows of {max_pages} entries")
    return _flat(t, torch.int32, batch * max_pages, "block_table")


def _rows(t: torch.Tensor, heads: int, head_dim: int, name: str) -> Tuple[int, int]:
    """Checks a [tokens, heads, head_dim] CUDA tensor whose tokens may be apart;
    returns its tokens and the elements between them."""
    shape, stride = t.shape, t.stride()
    if not t.is_cuda or len(shape) != 3 or shape[1] != heads or shape[2] != head_dim or stride[2] != 1 or \
            (stride[1] != head_dim and heads > 1):
        raise ValueError(f"{name}: expected a CUDA tensor [tokens, {heads}, {head_dim}] with its heads one after another")
    n = shape[0]
    return n, (stride[0] if n > 1 else heads * head_dim)


def tables_desc(batch: int, page_size: int, num_pages: int, max_pages: int, max_tokens: int) -> pi_tables_desc:
    return pi_tables_desc(batch, page_size, num_pages, max_pages, max_tokens)


def pi_block_tables(desc, cached_len, new_len, held, held_out, block_table, free_list, free_count, free_count_out,
                    cu_new, kv_len, slots, positions):
    """Page accounting, block tables, slots and positions of one step from the
    request lengths (`held_out` may be `held`, `free_count_out` may be
    `free_count`).  Running out of pages shows as kv_len 0 and slots -1."""
    B, i32 = desc.batch, torch.int32
    _check("pi_block_tables", lib().pi_block_tables(
        C.byref(desc), _flat(cached_len, i32, B, "cached_len"), _flat(new_len, i32, B, "new_len"),
        _flat(held, i32, B, "held"), _flat(held_out, i32, B, "held_out"),
        _table(block_table, B, desc.max_pages), _flat(free_list, i32, desc.num_pages, "free_list"),
        _flat(free_count, i32, 1, "free_count"), _flat(free_count_out, i32, 1, "free_count_out"),
        _flat(cu_new, i32, B + 1, "cu_new"), _flat(kv_len, i32, B, "kv_len"),
        _flat(slots, torch.int64, desc.max_tokens, "slots"), _flat(positions, i32, desc.max_tokens, "positions"),
        _stream()))


def rope_plan(head_dim: int, rot_dim: Optional[int] = None, interleaved: bool = False, base: float = 10000.0,
              scaling: str = "none", factor: float = 1.0, original_max: float = 0.0, low: float = 1.0,
              high: float = 4.0, mscale: float = 1.0) -> pi_rope_plan:
    """The plan pi_rope_store takes (host only).  `scaling`: "none", "linear"
    (positions / factor), "blend" (frequencies between `low` and `high`
    wavelengths per original_max blended) or "ramp" (pair indices between
    `high` and `low` turns per original_max blended)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling: expected one of {sorted(_SCALINGS)}")
    d = pi_rope_desc(head_dim, head_dim if rot_dim is None else rot_dim, 1 if interleaved else 0, _SCALINGS[scaling],
                     float(base), float(factor), float(original_max), float(low), float(high), float(mscale))
    out = pi_rope_plan()
    _check("pi_rope_plan_init", lib().pi_rope_plan_init(C.byref(d), C.byref(out)))
    return out


def page_desc(kcache: torch.Tensor, vcache: torch.Tensor) -> pi_page_desc:
    """The description of two cache tensors [pages, kv_heads, page_size,
    head_dim] of one shape, type and layout; any order of the first three in
    memory (a transposed view of a tokens-first tensor, for instance)."""
    if kcache.dim() != 4 or kcache.shape != vcache.shape or kcache.dtype is not vcache.dtype or \
            kcache.dtype not in _DTYPES or kcache.stride(3) != 1 or vcache.stride(3) != 1:
        raise ValueError("expected two [pages, kv_heads, page_size, head_dim] tensors of one shape and type with "
                         "contiguous heads")
    pages, heads, page, dh = kcache.shape
    # a dimension of one element is never stepped along
    st = [kcache.stride(i) if n > 1 else dh for i, n in enumerate((pages, heads, page))]
    if st != [vcache.stride(i) if n > 1 else dh for i, n in enumerate((pages, heads, page))]:
        raise ValueError("expected key and value caches of the same strides")
    d = pi_page_desc(heads, dh, page, pages, _DTYPES[kcache.dtype], st[0], st[1], st[2])
    d.like = (kcache.dtype, kcache.shape, kcache.stride())   # what _cache compares first
    return d


def _cache(cache: pi_page_desc, t: torch.Tensor, name: str) -> int:
    if t.is_cuda and getattr(cache, "like", None) == (t.dtype, t.shape, t.stride()):
        return t.data_ptr()
    if not t.is_cuda or _DTYPES.get(t.dtype) != cache.dtype or \
            tuple(t.shape) != (cache.num_pages, cache.kv_heads, cache.page_size, cache.head_dim) or \
            (t.shape[0] > 1 and t.stride(0) != cache.page_stride) or \
            (t.shape[1] > 1 and t.stride(1) != cache.head_stride) or t.stride(2) != cache.token_stride or \
            t.stride(3) != 1:
        raise ValueError(f"{name}: not the cache that the page_desc describes")
    return t.data_ptr()


def pi_rope_store(plan, cache, q, k, v, positions, slots, q_out, kcache, vcache):
    """Rotates q [T, heads, dh] into q_out and k [T, kv_heads, dh] into the
    cache at `slots`, and stores v there.  q and q_out may be None (store
    only), or k, v, slots, kcache and vcache (rotate only)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("expected q or k")
    dh, dtype, heads = cache.head_dim, x.dtype, 1
    qs = ks = vs = os_ = 0
    qp = op = kp = vp = sp = kc = vc = None
    if q is not None:
        heads = q.shape[1]
        (T, qs), (n, os_) = _rows(q, heads, dh, "q"), _rows(q_out, heads, dh, "q_out")
        if n < T or _DTYPES.get(q_out.dtype) != cache.dtype:
            raise ValueError("q_out: expected the shape of q and the type of the cache")
        qp, op = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        (n, ks), (m, vs) = _rows(k, cache.kv_heads, dh, "k"), _rows(v, cache.kv_heads, dh, "v")
        if q is None:
            T = n
        if n != T or m != T or k.dtype is not dtype or v.dtype is not dtype:
            raise ValueError("k, v: expected the tokens and the type of q")
        kp, vp, sp = k.data_ptr(), v.data_ptr(), _flat(slots, torch.int64, T, "slots")
        kc, vc = _cache(cache, kcache, "kcache"), _cache(cache, vcache, "vcache")
    d = pi_qkv_desc(T, heads, _DTYPES.get(dtype, -1), qs, ks, vs, os_)
    _check("pi_rope_store", lib().pi_rope_store(C.byref(plan), C.byref(cache), C.byref(d), qp, kp, vp,
                                                _flat(positions, torch.int32, T, "positions"), sp, op, kc, vc,
                                                _stream()))


def paged_desc(heads: int, batch: int, max_tokens: int, max_new: int, max_pages: int, window: int = 0,
               scale: float = 0.0) -> pi_paged_desc:
    """`scale` 0: 1 / sqrt(head_dim); `window` 0: none."""
    return pi_paged_desc(heads, batch, max_tokens, max_new, max_pages, window, scale)


def pi_paged_workspace_bytes(desc: pi_paged_desc, cache: pi_page_desc) -> int:
    return int(lib().pi_paged_workspace_bytes(C.byref(desc), C.byref(cache)))


def pi_paged_attn(desc, cache, q, kcache, vcache, block_table, cu_new, kv_len, out, lse, workspace):
    """Causal attention of the packed new tokens q [max_tokens, heads, dh] over
    the paged cache into out (same shape and type); lse [max_tokens, heads]
    fp32 or None; workspace uint8, zero-filled before its first use."""
    T, H, B, i32 = desc.max_tokens, desc.heads, desc.batch, torch.int32
    (n, qs), (m, os_) = _rows(q, H, cache.head_dim, "q"), _rows(out, H, cache.head_dim, "out")
    if n < T or m < T or _DTYPES.get(q.dtype) != cache.dtype or out.dtype is not q.dtype:
        raise ValueError("q, out: expected max_tokens rows of the cache's type")
    _check("pi_paged_attn", lib().pi_paged_attn(
        C.byref(desc), C.byref(cache), q.data_ptr(), qs, _cache(cache, kcache, "kcache"),
        _cache(cache, vcache, "vcache"), _table(block_table, B, desc.max_pages),
        _flat(cu_new, i32, B + 1, "cu_new"), _flat(kv_len, i32, B, "kv_len"), out.data_ptr(), os_,
        None if lse is None else _flat(lse, torch.float32, T * H, "lse"), _flat(workspace, torch.uint8, 0, "workspace"),
        workspace.numel(), _stream()))


# ------------------------------------------------------- the paged cache in 8 bits

CODE8 = torch.float8_e4m3fn


def page8_desc(kcache: torch.Tensor, vcache: torch.Tensor) -> pi_page8_desc:
    """The description of two code tensors [pages, kv_heads, page_size, head_dim]
    (torch.float8_e4m3fn) of one shape and layout; any order of the first three in
    memory.  Their exponents are int8 tensors [pages, kv_heads, page_size / 16]."""
    if kcache.dim() != 4 or kcache.shape != vcache.shape or kcache.dtype is not CODE8 or vcache.dtype is not CODE8 or \
            kcache.stride(3) != 1 or vcache.stride(3) != 1:
        raise ValueError("expected two [pages, kv_heads, page_size, head_dim] float8_e4m3fn tensors of one shape with "
                         "contiguous heads")
    pages, heads, page, dh = kcache.shape
    # a dimension of one element is never stepped along
    st = [kcache.stride(i) if n > 1 else dh for i, n in enumerate((pages, heads, page))]
    if st != [vcache.stride(i) if n > 1 else dh for i, n in enumerate((pages, heads, page))]:
        raise ValueError("expected key and value codes of the same strides")
    d = pi_page8_desc(heads, dh, page, pages, st[0], st[1], st[2])
    # what _cache8 compares first: codes, and the shape of their exponents
    d.like, d.exps = (CODE8, kcache.shape, kcache.stride()), torch.Size((pages, heads, page // 16))
    return d


def _cache8(cache: pi_page8_desc, codes: torch.Tensor, exps: torch.Tensor, name: str) -> Tuple[int, int]:
    """Addresses of the codes and exponents that a page8_desc describes."""
    like = getattr(cache, "like", None)
    if like is None or (codes.dtype, codes.shape, codes.stride()) != like:
        if codes.dtype is not CODE8 or \
                tuple(codes.shape) != (cache.num_pages, cache.kv_heads, cache.page_size, cache.head_dim) or \
                (codes.shape[0] > 1 and codes.stride(0) != cache.page_stride) or \
                (codes.shape[1] > 1 and codes.stride(1) != cache.head_stride) or \
                codes.stride(2) != cache.token_stride or codes.stride(3) != 1:
            raise ValueError(f"{name}: not the codes that the page8_desc describes")
    shape = cache.exps if like is not None else (cache.num_pages, cache.kv_heads, cache.page_size // 16)
    if exps.dtype is not torch.int8 or exps.shape != shape or not exps.is_contiguous():
        raise ValueError(f"{name}: expected contiguous int8 exponents [pages, kv_heads, page_size / 16]")
    if not codes.is_cuda or not exps.is_cuda:
        raise ValueError(f"{name}: expected CUDA tensors")
    return codes.data_ptr(), exps.data_ptr()


def pi_rope_store8(plan, cache, q, k, v, positions, slots, q_out, kcache, vcache, kexp, vexp):
    """Rotates q [T, heads, dh] into q_out (fp16 or bf16) and k [T, kv_heads, dh],
    and stores k and v as codes at `slots`, raising the exponents of the blocks
    they join where needed.  q and q_out may be None (store only), or k, v, slots,
    the caches and the exponents (rotate only)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("expected q or k")
    dh, dtype, heads, out = cache.head_dim, x.dtype, 1, PI_T_F16
    qs = ks = vs = os_ = 0
    qp = op = kp = vp = sp = kc = vc = ke = ve = None
    if q is not None:
        heads = q.shape[1]
        (T, qs), (n, os_) = _rows(q, heads, dh, "q"), _rows(q_out, heads, dh, "q_out")
        out = _DTYPES.get(q_out.dtype, -1)
        if n < T:
            raise ValueError("q_out: expected the shape of q")
        qp, op = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        (n, ks), (m, vs) = _rows(k, cache.kv_heads, dh, "k"), _rows(v, cache.kv_heads, dh, "v")
        if q is None:
            T = n
        if n != T or m != T or k.dtype is not dtype or v.dtype is not dtype:
            raise ValueError("k, v: expected the tokens and the type of q")
        kp, vp, sp = k.data_ptr(), v.data_ptr(), _flat(slots, torch.int64, T, "slots")
        (kc, ke), (vc, ve) = _cache8(cache, kcache, kexp, "kcache"), _cache8(cache, vcache, vexp, "vcache")
    d = pi_qkv_desc(T, heads, _DTYPES.get(dtype, -1), qs, ks, vs, os_)
    _check("pi_rope_store8", lib().pi_rope_store8(C.byref(plan), C.byref(cache), C.byref(d), out, qp, kp, vp,
                                                  _flat(positions, torch.int32, T, "positions"), sp, op, kc, vc, ke, ve,
                                                  _stream()))


def read8_desc(batch: int, max_pages: int, max_rows: int) -> pi_read8_desc:
    return pi_read8_desc(batch, max_pages, max_rows)


def pi_page_read8(desc, cache, kcache, vcache, kexp, vexp, block_table, start, cu_rows, k_out, v_out):
    """Positions start[b] .. (start None: from 0) of request b as rows cu_rows[b] ..
    cu_rows[b + 1] - 1 of k_out and v_out [max_rows, kv_heads, dh] (fp16, bf16 or
    fp32).  k_out or v_out may be None, with its codes and exponents."""
    B, i32 = desc.batch, torch.int32
    x = k_out if k_out is not None else v_out
    if x is None:
        raise ValueError("expected k_out or v_out")
    at, strides = [], []
    for codes, exps, out, name in ((kcache, kexp, k_out, "k"), (vcache, vexp, v_out, "v")):
        if out is None:
            at.append((None, None, None))
            strides.append(0)
            continue
        n, stride = _rows(out, cache.kv_heads, cache.head_dim, name + "_out")
        if n < desc.max_rows or out.dtype is not x.dtype:
            raise ValueError(f"{name}_out: expected max_rows rows, of one type")
        at.append((*_cache8(cache, codes, exps, name + "cache"), out.data_ptr()))
        strides.append(stride)
    (kc, ke, ko), (vc, ve, vo) = at
    d = pi_read8_desc(B, desc.max_pages, desc.max_rows, _DTYPES.get(x.dtype, -1), *strides)
    _check("pi_page_read8", lib().pi_page_read8(
        C.byref(d), C.byref(cache), kc, vc, ke, ve, _table(block_table, B, desc.max_pages),
        None if start is None else _flat(start, i32, B, "start"), _flat(cu_rows, i32, B + 1, "cu_rows"), ko, vo, _stream()))


def pi_paged8_workspace_bytes(desc: pi_paged_desc, cache: pi_page8_desc) -> int:
    return int(lib().pi_paged8_workspace_bytes(C.byref(desc), C.byref(cache)))


def pi_paged_attn8(desc, cache, q, kcache, vcache, kexp, vexp, block_table, cu_new, kv_len, out, lse, workspace):
    """pi_paged_attn over an 8-bit cache: q and out [max_tokens, heads, dh] in fp16
    or bf16; workspace uint8, zero-filled before its first use."""
    T, H, B, i32 = desc.max_tokens, desc.heads, desc.batch, torch.int32
    (n, qs), (m, os_) = _rows(q, H, cache.head_dim, "q"), _rows(out, H, cache.head_dim, "out")
    if n < T or m < T or out.dtype is not q.dtype:
        raise ValueError("q, out: expected max_tokens rows of one type")
    (kc, ke), (vc, ve) = _cache8(cache, kcache, kexp, "kcache"), _cache8(cache, vcache, vexp, "vcache")
    _check("pi_paged_attn8", lib().pi_paged_attn8(
        C.byref(desc), C.byref(cache), _DTYPES.get(q.dtype, -1), q.data_ptr(), qs, kc, vc, ke, ve,
        _table(block_table, B, desc.max_pages), _flat(cu_new, i32, B + 1, "cu_new"), _flat(kv_len, i32, B, "kv_len"),
        out.data_ptr(), os_, None if lse is None else _flat(lse, torch.float32, T * H, "lse"),
        _flat(workspace, torch.uint8, 0, "workspace"), workspace.numel(), _stream()))
