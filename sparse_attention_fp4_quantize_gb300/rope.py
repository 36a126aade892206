"""Frequencies of rotary positions, also stretched for long contexts, and the
table that csa2_rope, csa2_quantize_kv_fp4_paged and csa2_rope_quantize_kv_fp4
read.

Pair i turns by theta^(-2i / dim) radians per position.  A context `factor`
times as long as the `original` one follows YaRN (Peng et al., "YaRN: Efficient
Context Window Extension of Large Language Models", 2023): pairs that make
`fast` turns and more over the original context keep their frequency, those that
make `slow` and fewer are slowed down by the factor, those between in part; cosines
and sines are larger by 0.1 ln(factor) + 1.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import ROPE_HALF, csa2_rope_table


@dataclass
class Rope:
    dim: int                         # rotated channels of a head
    theta: float = 10000.0
    factor: float = 1.0              # the context's length over the original one's
    original: int = 4096             # positions of the context that the model was trained with
    fast: float = 32.0
    slow: float = 1.0
    first: int = 0                   # first rotated channel
    layout: int = ROPE_HALF

    def frequencies(self):
        """(radians per position float64 [dim / 2], amplitude)."""
        f = self.theta ** (-torch.arange(0, self.dim, 2, dtype=torch.float64) / self.dim)
        if self.factor == 1.0:
            return f, 1.0
        turns = self.original * f / (2 * math.pi)
        keep = ((turns - self.slow) / (self.fast - self.slow)).clamp(0.0, 1.0)
        return f * keep + f / self.factor * (1.0 - keep), 0.1 * math.log(self.factor) + 1.0

    def table(self, n_pos: int, device="cuda", start: int = 0):
        """cos_sin fp32 [n_pos, dim / 2, 2] of positions start, start + 1, ..., made on the device's current stream."""
        f, amplitude = self.frequencies()
        out = torch.empty(n_pos, self.dim // 2, 2, dtype=torch.float32, device=device)
        csa2_rope_table(f.to(out.device), out, start=start, amplitude=amplitude)
        return out
