"""Paged serving over the C ABI: one set of block tables for all layers of a
decoder, a paged key/value cache per layer, prompt chunks and single tokens in
the same step.

A step is ``begin`` (page accounting, block tables, slots and positions from the
request lengths: ``pi_block_tables``), then per layer ``attend`` (rotary positions
and the store into the cache: ``pi_rope_store``; attention over the cache:
``pi_paged_attn``).  No step synchronises the host; all lengths stay on the device.
With ``bits=8`` the caches hold e4m3 codes with an exponent for each block of 16
positions and head (``pi_rope_store8``, ``pi_paged_attn8``), and ``read`` gives rows of
them back (``pi_page_read8``).

    python -m activation_sparse_ffn_layer_gb300.paged --config c4 --requests 16 --prompt 1000 --tokens 64

serves synthetic projections of an attention block's shape: prompts in chunks,
then decode steps, with the times of each.
"""
from __future__ import annotations

import argparse
import time
from typing import Optional

import torch

from . import binding as B


class PagedCache:
    """Caches, block tables and page pool of ``batch`` request rows.

    ``num_pages`` pages of ``page_size`` positions serve all rows; a row holds at
    most ``max_seq`` positions and receives at most ``max_new`` tokens a step, the
    rows together at most ``max_tokens``.  ``dtype`` is the type of queries and outputs,
    and of the caches where ``bits`` is 16; with 8 they hold codes, and where ``max_new`` is
    above 64 * kv_heads / heads (and 1) the workspace has room for one layer's pages in
    16 bits, which requests of many tokens go over."""

    def __init__(self, heads: int, kv_heads: int, head_dim: int, batch: int, max_seq: int, max_new: int,
                 max_tokens: int, layers: int = 1, page_size: int = 16, num_pages: Optional[int] = None,
                 dtype: torch.dtype = torch.float16, rope: Optional[B.pi_rope_plan] = None, window: int = 0,
                 device="cuda", bits: int = 16):
        if bits not in (8, 16):
            raise ValueError("bits: expected 8 or 16")
        if dtype not in (torch.float16, torch.bfloat16):
            raise ValueError("dtype: expected float16 or bfloat16")
        per_row = -(-max_seq // page_size)
        pages = batch * per_row if num_pages is None else num_pages
        self.batch, self.heads, self.kv_heads, self.head_dim = batch, heads, kv_heads, head_dim
        self.max_new, self.max_tokens, self.window = max_new, max_tokens, window
        self.rope = B.rope_plan(head_dim, 0) if rope is None else rope
        shape = (pages, kv_heads, page_size, head_dim)
        self.bits = bits
        held = dict(dtype=dtype if bits == 16 else B.CODE8, device=device)
        self.kcache = [torch.zeros(shape, **held) for _ in range(layers)]
        self.vcache = [torch.zeros(shape, **held) for _ in range(layers)]
        if bits == 16:
            self.pages = B.page_desc(self.kcache[0], self.vcache[0])
        else:
            exps = dict(size=(pages, kv_heads, page_size // 16), dtype=torch.int8, device=device)
            self.kexp = [torch.zeros(**exps) for _ in range(layers)]
            self.vexp = [torch.zeros(**exps) for _ in range(layers)]
            self.pages = B.page8_desc(self.kcache[0], self.vcache[0])
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((batch, per_row), -1, **i32)
        self.free = torch.arange(pages - 1, -1, -1, **i32)      # lowest page on top
        self.free_count = torch.full((1,), pages, **i32)
        self.held, self.cached = torch.zeros(batch, **i32), torch.zeros(batch, **i32)
        self.cu, self.kv_len = torch.zeros(batch + 1, **i32), torch.zeros(batch, **i32)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
        self.positions = torch.zeros(max_tokens, **i32)
        self.q = torch.empty(max_tokens, heads, head_dim, dtype=dtype, device=device)
        self.tokens = 0
        # sized for the largest step: the partials depend on max_new alone
        size = B.pi_paged_workspace_bytes if bits == 16 else B.pi_paged8_workspace_bytes
        need = size(self._desc(max_tokens, max_new), self.pages)
        if need == 0:
            raise ValueError("heads, cache shape or capacities rejected by the library")
        self.workspace = torch.zeros(need, dtype=torch.uint8, device=device)

    def _desc(self, tokens: int, max_new: int) -> B.pi_paged_desc:
        return B.paged_desc(self.heads, self.batch, tokens, max_new, self.table.shape[1], window=self.window)

    def begin(self, new_len: torch.Tensor, tokens: int, max_new: int, keep: Optional[torch.Tensor] = None):
        """Opens a step in which row b receives new_len[b] tokens (int32, on the
        device), ``tokens`` in all and at most ``max_new`` in a row.  ``keep``: the
        positions rows keep, at most those they have (0: the row's request
        ended, its pages go back).  Rows that cannot be served (the pool ran out,
        the row is full, a negative keep) have kv_len 0 afterwards and hold their
        pages and the positions they kept; the latter two set the device status.
        In 8 bits a position that is given back may leave a mark on those kept: the
        exponent of its block of 16 does not fall again, and the codes under it have
        been rounded to it, so steps with proposals that are taken back need not leave
        the bits of steps without.  All state is updated in place, so a captured step
        goes on from where the last replay ended."""
        if tokens > self.max_tokens or max_new > self.max_new:
            raise ValueError("more tokens than the cache was made for")
        cached = self.cached if keep is None else torch.minimum(keep, self.cached)
        d = B.tables_desc(self.batch, self.pages.page_size, self.pages.num_pages, self.table.shape[1], tokens)
        B.pi_block_tables(d, cached, new_len, self.held, self.held, self.table, self.free, self.free_count,
                          self.free_count, self.cu, self.kv_len, self.slots, self.positions)
        if keep is not None:                      # a negative one changes nothing
            self.cached.copy_(torch.where(cached < 0, self.cached, cached))
        self.cached.copy_(torch.where(self.kv_len > 0, self.kv_len, self.cached))
        self.tokens, self.desc = tokens, self._desc(tokens, max(1, min(max_new, tokens)))

    def attend(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
               lse: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of the step's packed tokens in one layer: q [tokens, heads,
        head_dim], k and v [tokens, kv_heads, head_dim] as projected (fp16, bf16 or
        fp32), out like q in the cache's type.  Rows of another number than the
        step's tokens are refused: the attention would take a former step's."""
        if q.shape[0] != self.tokens:
            raise ValueError(f"expected the {self.tokens} tokens of the step")
        kc, vc, turned = self.kcache[layer], self.vcache[layer], self.q[:self.tokens]
        if self.bits == 8:
            ke, ve = self.kexp[layer], self.vexp[layer]
            B.pi_rope_store8(self.rope, self.pages, q, k, v, self.positions, self.slots, turned, kc, vc, ke, ve)
            B.pi_paged_attn8(self.desc, self.pages, turned, kc, vc, ke, ve, self.table, self.cu, self.kv_len, out, lse,
                             self.workspace)
            return out
        B.pi_rope_store(self.rope, self.pages, q, k, v, self.positions, self.slots, turned, kc, vc)
        B.pi_paged_attn(self.desc, self.pages, turned, kc, vc, self.table, self.cu, self.kv_len, out, lse, self.workspace)
        return out

    def read(self, layer: int, start: Optional[torch.Tensor], cu_rows: torch.Tensor, rows: int,
             dtype: Optional[torch.dtype] = None):
        """Keys and values of one layer of an 8-bit cache as rows [rows, kv_heads, head_dim]
        (``dtype``: that of the queries unless given): request b's positions start[b] .. (None:
        from 0) are rows cu_rows[b] .. cu_rows[b + 1] - 1, for a request that goes elsewhere.
        Rows of no request are zeros, which both tensors are filled with first."""
        if self.bits != 8:
            raise ValueError("read: expected a cache of 8 bits")
        k = torch.zeros(rows, self.kv_heads, self.head_dim, dtype=dtype or self.q.dtype, device=self.q.device)
        v = torch.zeros_like(k)
        d = B.read8_desc(self.batch, self.table.shape[1], rows)
        B.pi_page_read8(d, self.pages, self.kcache[layer], self.vcache[layer], self.kexp[layer], self.vexp[layer],
                        self.table, start, cu_rows, k, v)
        return k, v


def main(argv=None) -> None:
    from synth import ATTN_CONFIGS
    ap = argparse.ArgumentParser(description="serve synthetic projections over a paged cache")
    ap.add_argument("--config", default="c4", choices=sorted(ATTN_CONFIGS), help="attention block whose heads are used")
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000, help="longest prompt; request b has prompt * (b + 1) / requests")
    ap.add_argument("--chunk", type=int, default=512, help="prompt tokens of a request per step")
    ap.add_argument("--tokens", type=int, default=64, help="tokens decoded per request")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--page", type=int, default=16)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--bits", type=int, default=16, choices=(8, 16), help="of the cached keys and values")
    a = ap.parse_args(argv)
    c = ATTN_CONFIGS[a.config]
    H, G, dh, n = c.heads, c.kv_heads, c.head_dim, a.requests
    prompts = [max(1, a.prompt * (b + 1) // n) for b in range(n)]
    most = max(1, min(a.chunk, a.prompt)) * n
    g = torch.Generator(device="cuda").manual_seed(7000 + c.index)
    qkv = torch.randn(most, (H + 2 * G) * dh, generator=g, device="cuda").half()
    out = torch.empty(most, H, dh, dtype=torch.float16, device="cuda")

    def serve():
        cache = PagedCache(H, G, dh, n, a.prompt + a.tokens, a.chunk, a.chunk * n, layers=a.layers, page_size=a.page,
                           rope=B.rope_plan(dh), window=a.window, bits=a.bits)

        def step(new):
            T = sum(new)
            cache.begin(torch.tensor(new, dtype=torch.int32).cuda(non_blocking=True), T, max(new))
            q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv[:T].split([H * dh, G * dh, G * dh], dim=1))
            for layer in range(a.layers):
                cache.attend(layer, q, k, v, out[:T])
            return T

        left, done = list(prompts), 0
        torch.cuda.synchronize()
        t = time.perf_counter()
        while any(left):
            new = [min(x, a.chunk) for x in left]
            done += step(new)
            left = [x - y for x, y in zip(left, new)]
        torch.cuda.synchronize()
        t_prompt = time.perf_counter() - t
        ones = torch.ones(n, dtype=torch.int32, device="cuda")

        def decode():
            cache.begin(ones, n, 1)
            q, k, v = (x.unflatten(1, (-1, dh)) for x in qkv[:n].split([H * dh, G * dh, G * dh], dim=1))
            for layer in range(a.layers):
                cache.attend(layer, q, k, v, out[:n])

        decode()
        graph = torch.cuda.CUDAGraph()            # lengths, tables and slots advance on the device
        with torch.cuda.graph(graph):
            decode()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(a.tokens - 1):
            graph.replay()
        torch.cuda.synchronize()
        return done, t_prompt, time.perf_counter() - t

    serve()                                   # loads the kernels
    done, t_prompt, t_decode = serve()
    if B.pi_last_device_status() != B.PI_OK:
        raise RuntimeError("the device status reports an error")
    each = 1e6 * t_decode / max(1, a.tokens - 1)
    print("%s, %d requests, %d layers: prompts %d tokens in %.2f ms; decode steps (a replayed graph) %.1f us each, "
          "%.1f us a layer" % (c.name, n, a.layers, done, 1e3 * t_prompt, each, each / a.layers))


if __name__ == "__main__":
    main()
