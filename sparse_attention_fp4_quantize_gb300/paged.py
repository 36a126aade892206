"""A paged KV cache in 8 or 4 bits with the steps of a serving loop over it.

``PagedCache`` owns the device buffers of a batch of requests: the planes and
scales of every layer, the block tables, the free list and the lengths.  A
step is ``plan`` (which blocks the step's tokens go to), then per layer
``append`` (store the layer's new keys and values) and ``attend``; each is one or
two calls of the C library on the given stream, with fixed buffers and no host
synchronisation, so a whole step can be captured in a CUDA graph and replayed
with new lengths in ``new_len`` and new rows.  With ``rope`` the cache rotates
queries and keys by their positions on the way; ``read`` gives stored rows of the
4-bit cache back.

The module owns no arithmetic: csa2_build_slots, csa2_rope,
csa2_quantize_kv_fp8_paged and csa2_paged_attn_fp8 or csa2_quantize_kv_fp4_paged,
csa2_dequantize_kv_fp4_paged and csa2_paged_attn_fp4 do the work.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (csa2_build_slots, csa2_dequantize_kv_fp4_paged, csa2_paged_attn_fp4, csa2_paged_attn_fp8,
               csa2_quantize_kv_fp4_paged, csa2_quantize_kv_fp8_paged, csa2_rope, workspace_for_paged_attn,
               workspace_for_paged_attn_fp4)
from .rope import Rope


@dataclass
class PagedShape:
    requests: int                    # batch slots (a slot without a request has length 0 and no new tokens)
    tokens: int                      # rows of a step: the token budget that new_len shares out
    max_context: int                 # tokens a request may reach
    n_blocks: int                    # blocks in the pool, shared by the requests
    heads: int
    kv_heads: int
    dim: int = 128
    block_size: int = 64
    layers: int = 1
    max_new: int = 1                 # most new tokens of one request in a step (a hint to the attention)
    dtype: torch.dtype = torch.bfloat16
    bits: int = 8                    # of a stored channel: 8 (a scale per block and head) or 4 (one per 16 channels of a row)
    rope: Rope | None = None         # rotate queries and keys (rows come without positions then)


class PagedCache:
    """Buffers and calls of a paged cache.  Write the step's token counts into
    ``new_len`` (-1 ends a request), call ``plan``, then ``append`` and
    ``attend`` per layer; ``positions`` gives the new rows' positions,
    ``cu_len`` where each request's rows begin."""

    def __init__(self, shape: PagedShape, device="cuda"):
        s = self.shape = shape
        dev = self.device = torch.device(device)
        i32 = torch.int32
        M = -(-s.max_context // s.block_size)
        if s.bits not in (4, 8):
            raise ValueError("bits must be 8 or 4, got %r" % (s.bits,))
        rows = (s.layers, s.n_blocks, s.kv_heads, s.block_size)
        if s.bits == 8:
            codes = dict(size=(*rows, s.dim), dtype=torch.uint8, device=dev)
            self.k_scale = torch.ones(rows[:3], dtype=torch.float32, device=dev)
        else:
            codes = dict(size=(*rows, s.dim // 2), dtype=torch.uint8, device=dev)
            self.k_scale = torch.zeros(*rows, s.dim // 16, dtype=torch.uint8, device=dev)
        self.k_codes, self.v_codes = torch.zeros(**codes), torch.zeros(**codes)
        self.v_scale = self.k_scale.clone()
        self.block_table = torch.full((s.requests, M), -1, dtype=i32, device=dev)
        self.free_list = torch.arange(s.n_blocks - 1, -1, -1, dtype=i32, device=dev)
        self.free_count = torch.full((1,), s.n_blocks, dtype=i32, device=dev)
        self.kv_len = torch.zeros(s.requests, dtype=i32, device=dev)
        self.new_len = torch.zeros(s.requests, dtype=i32, device=dev)
        self.cu_len = torch.zeros(s.requests + 1, dtype=i32, device=dev)
        self.positions = torch.full((s.tokens,), -1, dtype=i32, device=dev)
        self.slots = torch.full((s.tokens,), -1, dtype=torch.int64, device=dev)
        self.out = torch.zeros(s.layers, s.tokens, s.heads, s.dim, dtype=s.dtype, device=dev)
        self.lse = torch.zeros(s.layers, s.tokens, s.heads, dtype=torch.float32, device=dev)
        self.err = torch.zeros(1, dtype=i32, device=dev)
        # one per layer: layers may be attended side by side, on streams of their own or in graphs of their own
        workspace = workspace_for_paged_attn if s.bits == 8 else workspace_for_paged_attn_fp4
        self.ws = [workspace(s.requests, s.tokens, s.heads, s.kv_heads, s.dim, s.max_new, device=dev)
                   for _ in range(s.layers)]
        self.cos_sin = self.q_rot = self.k_rot = None
        if s.rope is not None:
            self.cos_sin = s.rope.table(M * s.block_size, dev)
            self.q_rot = torch.zeros_like(self.out)
            if s.bits == 8:
                self.k_rot = torch.zeros(s.layers, s.tokens, s.kv_heads, s.dim, dtype=s.dtype, device=dev)
        self.sm_scale = 1.0 / float(s.dim) ** 0.5

    def plan(self, stream=None):
        """Give the step's tokens their blocks; lengths and free list move on in place."""
        csa2_build_slots(self.kv_len, self.new_len, self.block_table, self.free_list, self.free_count,
                         self.shape.block_size, self.kv_len, self.free_count, self.cu_len, self.positions, self.slots,
                         err_flag=self.err, stream=stream)

    def _turn(self, x, out, stream):
        csa2_rope(x, self.positions, self.cos_sin, q_out=out, first=self.shape.rope.first, layout=self.shape.rope.layout,
                  err_flag=self.err, stream=stream)
        return out

    def append(self, layer: int, k, v, stream=None, *, k_values=None, v_values=None):
        """Store the layer's new rows k, v [tokens, kv_heads, dim].  k_values, v_values (4 bits): buffers of their shape that
        get what is stored."""
        planes = self.k_codes[layer], self.v_codes[layer], self.k_scale[layer], self.v_scale[layer]
        if self.shape.bits == 4:
            rope = self.shape.rope
            turn = {} if rope is None else dict(pos=self.positions, cos_sin=self.cos_sin, first=rope.first, layout=rope.layout)
            csa2_quantize_kv_fp4_paged(k, v, self.slots, *planes, k_values=k_values, v_values=v_values, err_flag=self.err,
                                       stream=stream, **turn)
            return
        if k_values is not None or v_values is not None:
            raise ValueError("stored values come from the 4-bit cache")
        if self.k_rot is not None:
            k = self._turn(k, self.k_rot[layer], stream)
        csa2_quantize_kv_fp8_paged(k, v, self.slots, *planes, err_flag=self.err, stream=stream)

    def read(self, layer: int, slots, k, v, stream=None):
        """The layer's stored rows at slots int64 [n] into k, v [n, kv_heads, dim] (4 bits)."""
        if self.shape.bits != 4:
            raise ValueError("rows are read back from the 4-bit cache")
        csa2_dequantize_kv_fp4_paged(slots, self.k_codes[layer], self.v_codes[layer], self.k_scale[layer],
                                     self.v_scale[layer], k, v, err_flag=self.err, stream=stream)

    def attend(self, layer: int, q, window: int = 0, stream=None):
        """Attention of q [tokens, heads, dim] over the layer's cache; returns (out, lse), the cache's buffers.  Calls for
        several layers may overlap; calls for one layer, which share its buffers, must follow one another."""
        if self.q_rot is not None:
            q = self._turn(q, self.q_rot[layer], stream)
        call = csa2_paged_attn_fp8 if self.shape.bits == 8 else csa2_paged_attn_fp4
        call(q, self.k_codes[layer], self.v_codes[layer], self.k_scale[layer], self.v_scale[layer], self.block_table,
             self.kv_len, self.cu_len, self.out[layer], self.sm_scale, self.shape.max_new, window=window,
             lse=self.lse[layer], err_flag=self.err, workspace=self.ws[layer], stream=stream)
        return self.out[layer], self.lse[layer]
