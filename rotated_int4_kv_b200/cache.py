"""A preallocated int4 KV cache over the library's entry points.

The pages put their fused encode kernel behind a cache object of the model runtime
("When Quantization Is Free", gist.science/de/paper/2605.05699, "Methodik" 2): every
new K/V row is compressed on arrival and attention reads the compressed cache. This
class is the torch-level counterpart: it owns the per-layer code and scale buffers,
the (s, lambda) plans and the write position, and every operation is one or two
calls into libkvq (no arithmetic here).
"""
from __future__ import annotations

import numpy as np
import torch

from .api import (Plan, attend_decode, attend_decode_append, decode, encode_batch, make_workspace)
from .paged import (PAGE_SIZES, PagePlan, _new, attend_paged, encode_paged, page_plan, page_release,
                    paged_workspace_size)


class Int4KVCache:
    """Per-layer int4 K and V caches of ``capacity`` tokens for ``batch`` sequences.

    ``k_params`` / ``v_params``: one (signs, lambda) pair for every layer, or a list of
    ``layers`` pairs (K and V get separate transforms); ``transform`` "srft" or "srht";
    ``bits`` 4 (int4 codes) or 8 (int8 codes). All sequences of the batch share the
    write position of a layer.
    """

    def __init__(self, layers: int, batch: int, kv_heads: int, head_dim: int, capacity: int, k_params, v_params,
                 device=None, group: int = 32, transform: str = "srft", bits: int = 4):
        if layers <= 0 or batch <= 0 or kv_heads <= 0 or capacity <= 0:
            raise ValueError("layers, batch, kv_heads and capacity must be positive")
        self.device = torch.device(device) if device is not None else torch.device("cuda")
        self.layers, self.batch, self.kv_heads, self.head_dim, self.group = layers, batch, kv_heads, head_dim, group
        self.bits = bits
        self.capacity = capacity + (capacity & 1)  # the attention kernels fetch scale rows in 16-byte units

        def per_layer(params):
            # one (signs, lambda) pair, or a list of one pair per layer
            first = np.asarray(params[0])
            if first.ndim == 1:
                return [params] * layers
            if len(params) != layers:
                raise ValueError(f"expected one (signs, lambda) pair or {layers} of them")
            return list(params)

        with torch.cuda.device(self.device):
            self.k_plans = [Plan(s, lam, group, transform, bits) for s, lam in per_layer(k_params)]
            self.v_plans = [Plan(s, lam, group, transform, bits) for s, lam in per_layer(v_params)]
        shape_c = (batch, kv_heads, self.capacity, head_dim * bits // 8)
        shape_s = (batch, kv_heads, self.capacity, head_dim // group)
        self.k_codes = [torch.zeros(shape_c, dtype=torch.uint8, device=self.device) for _ in range(layers)]
        self.v_codes = [torch.zeros(shape_c, dtype=torch.uint8, device=self.device) for _ in range(layers)]
        self.k_scales = [torch.zeros(shape_s, dtype=torch.float16, device=self.device) for _ in range(layers)]
        self.v_scales = [torch.zeros(shape_s, dtype=torch.float16, device=self.device) for _ in range(layers)]
        self.pos = [0] * layers
        self._ws = {}

    # -------------------------------------------------------------- bookkeeping
    def seq_length(self, layer: int = 0) -> int:
        return self.pos[layer]

    def reset(self) -> None:
        self.pos = [0] * self.layers

    def memory_bytes(self) -> int:
        """Device bytes of all code and scale buffers."""
        per = sum(t.numel() * t.element_size() for t in (self.k_codes[0], self.v_codes[0], self.k_scales[0],
                                                          self.v_scales[0]))
        return per * self.layers

    @staticmethod
    def compression_ratio(head_dim: int, group: int = 32, bits: int = 4) -> float:
        """fp16 K/V bytes over code + fp16 scale bytes for the same tokens (int4: 3.56 at G = 32)."""
        return (2 * head_dim) / (head_dim * bits // 8 + 2 * (head_dim // group))

    def compression_vs_fp16(self) -> float:
        return self.compression_ratio(self.head_dim, self.group, self.bits)

    def _workspace(self, q_heads: int) -> torch.Tensor:
        ws = self._ws.get(q_heads)
        if ws is None:
            ws = make_workspace(self.batch, q_heads, self.kv_heads, self.head_dim, self.capacity, self.device)
            self._ws[q_heads] = ws
        return ws

    def _room(self, layer: int, n: int) -> None:
        if self.pos[layer] + n > self.capacity:
            raise ValueError(f"layer {layer}: {self.pos[layer]} + {n} tokens exceed the capacity {self.capacity}")

    # -------------------------------------------------------------- operations
    def update(self, layer: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        """Append n tokens: k, v fp16 [batch, kv_heads, n, head_dim] (one grouped encode launch)."""
        n = k.shape[2]
        if tuple(v.shape) != tuple(k.shape):
            raise ValueError("k and v must have the same shape")
        self._room(layer, n)
        p = self.pos[layer]
        encode_batch([(self.k_plans[layer], k, self.k_codes[layer], self.k_scales[layer], p),
                      (self.v_plans[layer], v, self.v_codes[layer], self.v_scales[layer], p)], stream=stream)
        self.pos[layer] = p + n

    def attend(self, layer: int, q: torch.Tensor, out=None, softmax_scale: float = 0.0, stream=None) -> torch.Tensor:
        """One-query attention of q fp16 [batch, q_heads, head_dim] over the cached tokens."""
        return attend_decode(self.k_plans[layer], self.v_plans[layer], q, self.k_codes[layer], self.k_scales[layer],
                             self.v_codes[layer], self.v_scales[layer], T_len=self.pos[layer],
                             softmax_scale=softmax_scale, out=out, workspace=self._workspace(q.shape[1]),
                             stream=stream)

    def step(self, layer: int, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, out=None,
             softmax_scale: float = 0.0, stream=None) -> torch.Tensor:
        """One decode step in one launch: append the token k_new, v_new (fp16 [batch, kv_heads, head_dim]
        or [batch, kv_heads, 1, head_dim]) and attend over the cache including it."""
        self._room(layer, 1)
        p = self.pos[layer]
        o = attend_decode_append(self.k_plans[layer], self.v_plans[layer], q, k_new, v_new, self.k_codes[layer],
                                 self.k_scales[layer], self.v_codes[layer], self.v_scales[layer], p,
                                 softmax_scale=softmax_scale, out=out, workspace=self._workspace(q.shape[1]),
                                 stream=stream)
        self.pos[layer] = p + 1
        return o

    def dequantize(self, layer: int, t0: int = 0, n: int = None, stream=None):
        """(K, V) fp16 [batch, kv_heads, n, head_dim] of cached tokens t0 .. t0 + n - 1 (decode kernel)."""
        if n is None:
            n = self.pos[layer] - t0
        k = decode(self.k_plans[layer], self.k_codes[layer], self.k_scales[layer], t0, n, stream=stream)
        v = decode(self.v_plans[layer], self.v_codes[layer], self.v_scales[layer], t0, n, stream=stream)
        return k, v


class PagedInt4KVCache:
    """Per-layer paged caches of requests of different lengths.

    ``num_pages`` pages of ``page_size`` tokens are shared by up to ``max_requests`` requests of at
    most ``max_pages`` pages each; the block table, the lengths and the free list live on the GPU
    and serve every layer. One serving step: :meth:`begin` (one launch: pages, slots and lengths of
    the step), per layer :meth:`update` and :meth:`attend`, and :meth:`release` for requests that
    have ended. No call waits for the GPU, and all may be captured into a CUDA graph.
    """

    def __init__(self, layers: int, max_requests: int, kv_heads: int, head_dim: int, num_pages: int, page_size: int,
                 max_pages: int, k_params, v_params, device=None, group: int = 32, transform: str = "srft",
                 bits: int = 4):
        if min(layers, max_requests, kv_heads, head_dim, num_pages, max_pages) <= 0:
            raise ValueError("layers, max_requests, kv_heads, num_pages and max_pages must be positive")
        if page_size not in PAGE_SIZES:
            raise ValueError(f"page size must be one of {PAGE_SIZES}, got {page_size}")
        dev = torch.device(device) if device is not None else torch.device("cuda")
        self.device = torch.device("cuda", torch.cuda.current_device()) if dev.index is None else dev
        self.layers, self.requests, self.kv_heads, self.head_dim = layers, max_requests, kv_heads, head_dim
        self.page_size, self.num_pages, self.max_pages = page_size, num_pages, max_pages

        def per_layer(params):
            if np.asarray(params[0]).ndim == 1:
                return [params] * layers
            if len(params) != layers:
                raise ValueError(f"expected one (signs, lambda) pair or {layers} of them")
            return list(params)

        with torch.cuda.device(self.device):
            self.k_plans = [Plan(s, lam, group, transform, bits) for s, lam in per_layer(k_params)]
            self.v_plans = [Plan(s, lam, group, transform, bits) for s, lam in per_layer(v_params)]

        def pages(width, dtype):
            return [torch.zeros((num_pages, kv_heads, page_size, width), dtype=dtype, device=self.device)
                    for _ in range(layers)]
        self.k_codes, self.v_codes = (pages(head_dim * bits // 8, torch.uint8) for _ in range(2))
        self.k_scales, self.v_scales = (pages(head_dim // group, torch.float16) for _ in range(2))
        self.block_table = torch.full((max_requests, max_pages), -1, dtype=torch.int32, device=self.device)
        self.kv_lens = torch.zeros(max_requests, dtype=torch.int32, device=self.device)
        self.free_pages = torch.arange(num_pages, dtype=torch.int32, device=self.device)
        self.free_head = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._ws, self._grown = {}, []

    def begin(self, q_lens: torch.Tensor, n_tokens: int, stream=None) -> PagePlan:
        """Pages, slots and lengths of a step in which request b gets q_lens[b] (int32, device) new
        tokens, ``n_tokens`` of them at most in all; see :func:`page_plan`. ``kv_lens`` moves on, but not
        for requests that get no pages (``info[2]`` of them): their tokens have no place in the cache,
        and what :meth:`attend` gives for them means nothing."""
        step = PagePlan.empty(self.requests, n_tokens, self.device, stream)._replace(kv_lens=self.kv_lens)
        return page_plan(self.kv_lens, q_lens, self.block_table, self.free_pages, self.free_head, self.page_size,
                         out=step, stream=stream)

    def update(self, layer: int, k: torch.Tensor, v: torch.Tensor, step: PagePlan, stream=None) -> None:
        """The step's new rows k, v fp16 [n_tokens, kv_heads, head_dim] into their pages (one launch)."""
        encode_paged([(self.k_plans[layer], k, self.k_codes[layer], self.k_scales[layer]),
                      (self.v_plans[layer], v, self.v_codes[layer], self.v_scales[layer])], step.slots, stream=stream)

    def attend(self, layer: int, q: torch.Tensor, step: PagePlan, max_q_len: int = None, max_kv_len: int = None,
               window: int = 0, softmax_scale: float = 0.0, out=None, stream=None) -> torch.Tensor:
        """Causal attention of the step's tokens q fp16 [n_tokens, q_heads, head_dim] over the cache
        (after :meth:`update`); see :func:`attend_paged`. Rows of padding tokens stay as ``out`` had them.
        Calls on different streams that may overlap need caches of their own (one workspace)."""
        n, q_heads = q.shape[0], q.shape[1]
        longest = max(1, n if max_q_len is None else max_q_len)
        need = paged_workspace_size(self.requests, q_heads, self.kv_heads, self.head_dim, n, longest)
        ws = self._ws.get(q_heads)
        if ws is None or ws.numel() < need:
            if ws is not None:  # a captured graph may hold its address; doubled, so that all kept ones are no more than the new one
                self._grown.append(ws)
                need = max(need, 2 * ws.numel())
            ws = self._ws[q_heads] = _new(torch.empty, max(16, need), torch.uint8, self.device, stream)
        return attend_paged(self.k_plans[layer], self.v_plans[layer], q, self.k_codes[layer], self.k_scales[layer],
                            self.v_codes[layer], self.v_scales[layer], self.block_table, self.kv_lens, step.q_starts,
                            max_q_len=longest, max_kv_len=max_kv_len, window=window, softmax_scale=softmax_scale,
                            out=out, workspace=ws, stream=stream)

    def release(self, done: torch.Tensor, stream=None) -> None:
        """Requests with ``done`` (bool, device) give their pages back and become empty."""
        page_release(done, self.kv_lens, self.block_table, self.free_pages, self.free_head, self.page_size,
                     stream=stream)
