"""A paged 8-bit KV cache with the steps of a serving loop over it.

``PagedCache`` owns the device buffers of a batch of requests: the E4M3 planes
and scales of every layer, the block tables, the free list and the lengths.  A
step is ``plan`` (which blocks the step's tokens go to), then per layer
``append`` (store the layer's new keys and values) and ``attend``; each is one
call of the C library on the given stream, with fixed buffers and no host
synchronisation, so a whole step can be captured in a CUDA graph and replayed
with new lengths in ``new_len`` and new rows.

The module owns no arithmetic: csa2_build_slots, csa2_quantize_kv_fp8_paged and
csa2_paged_attn_fp8 do the work.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import csa2_build_slots, csa2_paged_attn_fp8, csa2_quantize_kv_fp8_paged, workspace_for_paged_attn


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


class PagedCache:
    """Buffers and calls of a paged cache.  Write the step's token counts into
    ``new_len`` (-1 ends a request), call ``plan``, then ``append`` and
    ``attend`` per layer; ``positions`` gives the new rows' positions (for
    RoPE), ``cu_len`` where each request's rows begin."""

    def __init__(self, shape: PagedShape, device="cuda"):
        s = self.shape = shape
        dev = self.device = torch.device(device)
        i32 = torch.int32
        M = -(-s.max_context // s.block_size)
        planes = (s.layers, s.n_blocks, s.kv_heads, s.block_size, s.dim)
        self.k_codes = torch.zeros(planes, dtype=torch.uint8, device=dev)
        self.v_codes = torch.zeros(planes, dtype=torch.uint8, device=dev)
        self.k_scale = torch.ones(planes[:3], dtype=torch.float32, device=dev)
        self.v_scale = torch.ones(planes[:3], dtype=torch.float32, device=dev)
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
        self.ws = [workspace_for_paged_attn(s.requests, s.tokens, s.heads, s.kv_heads, s.dim, s.max_new, device=dev)
                   for _ in range(s.layers)]
        self.sm_scale = 1.0 / float(s.dim) ** 0.5

    def plan(self, stream=None):
        """Give the step's tokens their blocks; lengths and free list move on in place."""
        csa2_build_slots(self.kv_len, self.new_len, self.block_table, self.free_list, self.free_count,
                         self.shape.block_size, self.kv_len, self.free_count, self.cu_len, self.positions, self.slots,
                         err_flag=self.err, stream=stream)

    def append(self, layer: int, k, v, stream=None):
        """Store the layer's new rows k, v [tokens, kv_heads, dim]."""
        csa2_quantize_kv_fp8_paged(k, v, self.slots, self.k_codes[layer], self.v_codes[layer], self.k_scale[layer],
                                   self.v_scale[layer], err_flag=self.err, stream=stream)

    def attend(self, layer: int, q, window: int = 0, stream=None):
        """Attention of q [tokens, heads, dim] over the layer's cache; returns (out, lse), the cache's buffers.  Calls for
        several layers may overlap; calls for one layer, which share its buffers, must follow one another."""
        csa2_paged_attn_fp8(q, self.k_codes[layer], self.v_codes[layer], self.k_scale[layer], self.v_scale[layer],
                            self.block_table, self.kv_len, self.cu_len, self.out[layer], self.sm_scale,
                            self.shape.max_new, window=window, lse=self.lse[layer], err_flag=self.err,
                            workspace=self.ws[layer], stream=stream)
        return self.out[layer], self.lse[layer]
