"""Torch-level wrapper of the attention operators: one full-attention layer's
weights, its paged cache and the calls in order.  Allocation, checks and
marshalling only; the compute is entirely in libmoe_b200 (include/attn_b200.h).

Lily pages: "Perplexity built an inference engine for one model, one chip",
second paragraph (10 of the model's 40 layers run full attention, 16 query and
2 key/value heads); "Perplexity's Lily brings fast local AI to Apple silicon
Macs", section "Where the Engine Gains Speed" (packed query heads, a cache of
fixed blocks).
"""
from __future__ import annotations

import torch

from . import (ATTN_CACHE_BF16, ATTN_CACHE_E4M3, ATTN_ROPE_HALF, MoeError, attn_config, attn_decode,
               attn_decode_workspace_size, attn_kv_read, attn_prefill, attn_qkv_prepare)


class AttentionLayer:
    """One layer: head counts and sizes, norm weights (bf16 [head_dim], or
    None for no norm), the table of rotation frequencies (fp32 [rot_dim / 2],
    or None for no rotation) and a paged cache of num_pages pages.

    Token rows come as qkv [T, (q_heads + 2 kv_heads) head_dim] bf16: the
    query heads, the key heads, the value heads.  Calls run on the layer's
    device, on torch's current stream; what a kernel finds out of bounds
    raises from check().
    """

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, num_pages: int, page_size: int = 64,
                 cache_type: int = ATTN_CACHE_BF16, q_weight=None, k_weight=None, eps: float = 1e-6, inv_freq=None,
                 rope_layout: int = ATTN_ROPE_HALF, rope_scale: float = 1.0, scale: float | None = None,
                 device="cuda"):
        self.cfg = attn_config(q_heads, kv_heads, head_dim, page_size, cache_type)
        if attn_decode_workspace_size(self.cfg, 1, 1, 1) == 0:
            raise ValueError("unsupported attention configuration")
        if num_pages < 1:
            raise ValueError("num_pages must be at least 1, got %d" % num_pages)
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("the layer runs on a GPU, not on %s" % self.device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.num_pages, self.eps, self.rope_layout, self.rope_scale = num_pages, eps, rope_layout, rope_scale
        self.scale = head_dim ** -0.5 if scale is None else scale
        self.row = (q_heads + 2 * kv_heads) * head_dim
        self.q_weight = self._vector(q_weight, "q_weight", torch.bfloat16, head_dim)
        self.k_weight = self._vector(k_weight, "k_weight", torch.bfloat16, head_dim)
        self.rot_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
        if self.rot_dim > head_dim or self.rot_dim % 16:
            raise ValueError("inv_freq has %d elements: a multiple of 8, at most head_dim / 2" % (self.rot_dim // 2))
        self.inv_freq = self._vector(inv_freq, "inv_freq", torch.float32, self.rot_dim // 2)
        shape = (num_pages, kv_heads, page_size, head_dim)
        kind = torch.bfloat16 if cache_type == ATTN_CACHE_BF16 else torch.float8_e4m3fn
        self.k_cache = torch.zeros(shape, dtype=torch.uint8 if kind != torch.bfloat16 else kind,
                                   device=self.device).view(kind)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.k_scale = self.v_scale = None
        if cache_type == ATTN_CACHE_E4M3:
            self.k_scale = torch.ones(shape[:3], dtype=torch.float32, device=self.device)
            self.v_scale = torch.ones(shape[:3], dtype=torch.float32, device=self.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)

    def _vector(self, t, name: str, dtype, n: int):
        if t is None:
            return None
        if t.numel() != n:
            raise ValueError("%s must have %d elements, got %d" % (name, n, t.numel()))
        return t.to(device=self.device, dtype=dtype).contiguous()

    def _check(self, t, name: str, dtype, shape: tuple) -> None:
        """Raises unless t is a tensor of this type and shape (None: any size)
        on the layer's device with a contiguous last dimension."""
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor, got %s" % (name, type(t).__name__))
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
            raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
        if t.device != self.device:
            raise ValueError("%s is on %s, the layer on %s" % (name, t.device, self.device))
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError("%s: the last dimension must be contiguous" % name)

    def _prepare(self, qkv, positions, slots, keys: bool):
        self._check(qkv, "qkv", torch.bfloat16, (None, self.row))
        T = qkv.shape[0]
        if T < 1:
            raise ValueError("qkv has no rows")
        if T > 1 and (qkv.stride(0) < self.row or qkv.stride(0) % 8):
            raise ValueError("qkv: rows must be a multiple of 8 elements apart and not overlap, got %d" % qkv.stride(0))
        if self.rot_dim:
            self._check(positions, "positions", torch.int32, (T,))
        self._check(slots, "slots", torch.int32, (T,))
        c = self.cfg
        q = torch.empty(T, c.q_heads, c.head_dim, dtype=torch.bfloat16, device=self.device)
        k = torch.empty(T, c.kv_heads, c.head_dim, dtype=torch.bfloat16, device=self.device) if keys else None
        attn_qkv_prepare(c, T, qkv, qkv.stride(0) if T > 1 else self.row, self.q_weight, self.k_weight, self.eps,
                         self.inv_freq, self.rot_dim, self.rope_layout, self.rope_scale, positions, slots,
                         self.num_pages, self.k_cache, self.v_cache, self.k_scale, self.v_scale, q, k, err=self.err)
        return q, k

    def prefill(self, qkv, positions, slots, cu_q, page_table=None, cu_k=None, total_k: int | None = None,
                causal: bool = True) -> torch.Tensor:
        """Outputs [T, q_heads, head_dim] of packed prompts (rows cu_q[b] ..
        cu_q[b + 1] - 1 of qkv are sequence b), written into the cache at
        `slots` too.  With page_table, cu_k and total_k the queries see all of
        each sequence's total_k = cu_k[B] cached rows (a prefix and the rows of
        this call), read back from the cache; without them the rows of this
        call."""
        with torch.cuda.device(self.device):
            self._check(cu_q, "cu_q", torch.int32, (None,))
            B, c = cu_q.shape[0] - 1, self.cfg
            if B < 1:
                raise ValueError("cu_q must hold at least two boundaries")
            cached = page_table is not None
            if cached:
                self._check(page_table, "page_table", torch.int32, (B, None))
                self._check(cu_k, "cu_k", torch.int32, (B + 1,))
                if total_k is None or total_k < 0:
                    raise ValueError("total_k must be given with page_table")
            elif cu_k is not None or total_k is not None:
                raise ValueError("cu_k and total_k are of the cached rows: page_table must be given with them")
            q, k = self._prepare(qkv, positions, slots, keys=not cached)
            T = qkv.shape[0]
            if cached:
                k = torch.empty(total_k, c.kv_heads, c.head_dim, dtype=torch.bfloat16, device=self.device)
                v = torch.empty_like(k)
                pages = page_table.contiguous()
                attn_kv_read(c, B, total_k, pages, max(1, pages.shape[1]), cu_k, self.num_pages,
                             self.k_cache, self.v_cache, self.k_scale, self.v_scale, k, v, err=self.err)
                v_stride = c.kv_heads * c.head_dim
            else:
                cu_k, total_k = cu_q, T
                v = qkv[:, (c.q_heads + c.kv_heads) * c.head_dim:]
                v_stride = qkv.stride(0) if T > 1 else self.row
            out = torch.zeros(T, c.q_heads, c.head_dim, dtype=torch.bfloat16, device=self.device)
            attn_prefill(c, B, T, total_k, cu_q, cu_k, q, c.q_heads * c.head_dim, k, c.kv_heads * c.head_dim, v,
                         v_stride, self.scale, causal, out, err=self.err)
            return out

    def decode(self, qkv, positions, slots, page_table, seq_lens, max_len: int) -> torch.Tensor:
        """Outputs [B nq, q_heads, head_dim] of nq = T / B new tokens of each
        of B sequences (rows b nq + i), written into the cache at `slots` and
        seen by themselves; seq_lens counts them."""
        with torch.cuda.device(self.device):
            self._check(seq_lens, "seq_lens", torch.int32, (None,))
            B, c = seq_lens.shape[0], self.cfg
            self._check(qkv, "qkv", torch.bfloat16, (None, self.row))
            if B < 1 or qkv.shape[0] % B or not 1 <= qkv.shape[0] // B <= 8:
                raise ValueError("%d rows of qkv for %d sequences: 1 to 8 each" % (qkv.shape[0], B))
            self._check(page_table, "page_table", torch.int32, (B, None))
            if max_len < 1 or page_table.shape[1] * c.page_size < max_len:
                raise ValueError("page_table rows of %d pages for %d tokens" % (page_table.shape[1], max_len))
            if B > 1 and page_table.stride(0) < page_table.shape[1]:
                page_table = page_table.contiguous()         # one row for all sequences, expanded
            nq = qkv.shape[0] // B
            q, _ = self._prepare(qkv, positions, slots, keys=False)
            out = torch.empty_like(q)
            ws = torch.empty(attn_decode_workspace_size(c, B, nq, max_len), dtype=torch.uint8, device=self.device)
            attn_decode(c, B, nq, max_len, q, c.q_heads * c.head_dim, page_table,
                        page_table.stride(0) if B > 1 else page_table.shape[1], seq_lens, self.num_pages,
                        self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.scale, out, None, ws,
                        err=self.err)
            return out

    def check(self) -> None:
        """Raises what a kernel reported since the last check (waits for the device: the layer's calls may be on any
        stream)."""
        torch.cuda.synchronize(self.device)
        status = int(self.err.item())
        if status:
            self.err.zero_()
            raise MoeError(status, "attention")
