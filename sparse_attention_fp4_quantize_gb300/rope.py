"""Frequencies of rotary positions, also stretched for long contexts, and the
table that csa2_rope, csa2_quantize_kv_fp4_paged and csa2_rope_quantize_kv_fp4
read.

Pair i turns by theta^(-2i / dim) radians per position.  A context `factor`
times as long as the `original` one follows YaRN (Peng et al., "YaRN: Efficient
Context Window Extension of Large Language Models", 2023): pairs that make
`fast` turns and more over the original context keep their frequency, those that
make `slow` and fewer are slowed down by the factor, those between in part; cosines
and sines are larger by 0.1 ln(factor) + 1.

The part of a pair between comes in two forms, whose frequencies differ by up to several
times, so that it has to be the one that the model was trained with.
``ramp="index"``, the form of the models that are served with YaRN, is linear in the
pair's index, from the last pair that makes `fast` turns to the first that makes no
more than `slow`; ``ramp="turns"``, the paper's, in the number of turns.  Frequencies
of any other kind are given in `inv_freq`, with the `amplitude` that goes with them.
"""
from __future__ import annotations

import math
from collections.abc import Sequence
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
    ramp: str = "index"              # of the pairs between `fast` and `slow`: "index" or "turns"
    inv_freq: Sequence[float] | torch.Tensor | None = None         # radians per position [dim / 2], in place of theta's and the factor's
    amplitude: float | None = None   # of cosines and sines, in place of 0.1 ln(factor) + 1

    def __post_init__(self):
        if self.inv_freq is not None:                              # kept as numbers: a Rope can be compared
            self.inv_freq = tuple(torch.as_tensor(self.inv_freq, dtype=torch.float64).tolist())

    def _keep(self, f):
        """Share of its own frequency that each pair keeps in a stretched context."""
        if self.ramp == "turns":
            turns = self.original * f / (2 * math.pi)
            return ((turns - self.slow) / (self.fast - self.slow)).clamp(0.0, 1.0)
        if self.ramp != "index":
            raise ValueError("ramp must be 'index' or 'turns', got %r" % (self.ramp,))

        def pair(turns):             # that makes so many, as a real number
            return self.dim * math.log(self.original / (2 * math.pi * turns)) / (2 * math.log(self.theta))
        low, high = max(math.floor(pair(self.fast)), 0), min(math.ceil(pair(self.slow)), self.dim - 1)
        i = torch.arange(f.numel(), dtype=torch.float64)
        return 1.0 - ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)

    def frequencies(self):
        """(radians per position float64 [dim / 2], amplitude)."""
        if self.inv_freq is not None:
            f, amplitude = torch.tensor(self.inv_freq, dtype=torch.float64), 1.0
            if f.shape != (self.dim // 2,):
                raise ValueError("inv_freq must hold dim / 2 = %d numbers, got %s" % (self.dim // 2, tuple(f.shape)))
            if self.factor != 1.0:
                raise ValueError("a factor stretches theta's frequencies, not those of inv_freq")
        else:
            if not 0.0 < self.theta < math.inf or not 1.0 <= self.factor < math.inf:
                raise ValueError("theta=%r must be above 0, factor=%r at least 1" % (self.theta, self.factor))
            f, amplitude = self.theta ** (-torch.arange(0, self.dim, 2, dtype=torch.float64) / self.dim), 1.0
            if self.factor != 1.0:
                if not (self.theta > 1.0 and self.original > 0 and self.fast > self.slow >= 0.0 and (self.slow > 0.0 or self.ramp == "turns")):
                    raise ValueError("a stretched context wants theta=%r > 1, original=%r > 0 and fast=%r > slow=%r > 0" %
                                     (self.theta, self.original, self.fast, self.slow))
                keep = self._keep(f)
                f, amplitude = f * keep + f / self.factor * (1.0 - keep), 0.1 * math.log(self.factor) + 1.0
        return f, amplitude if self.amplitude is None else float(self.amplitude)

    def table(self, n_pos: int, device="cuda", start: int = 0):
        """cos_sin fp32 [n_pos, dim / 2, 2] of positions start, start + 1, ..., made on the device's current stream."""
        f, amplitude = self.frequencies()
        out = torch.empty(n_pos, self.dim // 2, 2, dtype=torch.float32, device=device)
        csa2_rope_table(f.to(out.device), out, start=start, amplitude=amplitude)
        return out
