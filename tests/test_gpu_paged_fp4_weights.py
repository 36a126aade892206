"""What the rounding of the weights to f16 costs in attention over the paged 4-bit cache, on the GPU: rows whose values are all
in their tail."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32, F16 = torch.int32, torch.float16


@pytest.fixture(scope="module")
def csa2():
    import sparse_attention_fp4_quantize_gb300 as lib
    return lib


def _stored(x, unit):
    """Codes and scales of rows x [n, D] whose every group has one magnitude, `unit` times an E4M3 number: exactly x."""
    top = np.abs(x).reshape(x.shape[0], -1, 16).max(-1)
    s = ref.nearest(top / unit, ref.E4M3).astype(np.uint8)
    c = (np.where(x != 0, int(ref.nearest(np.array(unit), ref.GRID)), 0) + 8 * (x < 0)).astype(np.uint8)
    c = c[:, 0::2] | (c[:, 1::2] << 4)
    assert np.array_equal(ref.values(torch.from_numpy(c), torch.from_numpy(s)), x)
    return c, s


def _tail_case(csa2, D, n, B, H, heavy, tail, up):
    """Requests of `heavy` keys of score 0, `heavy` of score `up`, then keys of score `tail` (base 2), which alone have values,
    6 * 448 each; n new rows on top of 1280 tail keys.  Returns (output, weights float64 [keys], first position)."""
    S, kv = 64, 2 * heavy + 1280 + n
    k = np.zeros((kv, D))
    k[heavy:2 * heavy, 0] = up
    k[2 * heavy:, 0], k[2 * heavy:, 16] = math.ceil(tail), tail - math.ceil(tail)
    v = np.zeros((kv, D))
    v[2 * heavy:] = 6 * 448.0
    pages = -(-kv // S)
    (kc, ks), (vc, vs) = [[torch.from_numpy(p).view(pages, 1, S, -1).expand(pages, H, S, -1).contiguous().to(DEV)
                           for p in _stored(np.concatenate([x, np.zeros((pages * S - kv, D))]), unit)] for x, unit in ((k, 1.0), (v, 6.0))]
    q = torch.zeros(B * n, H, D, dtype=F16, device=DEV)
    q[..., 0] = q[..., 16] = 1.0
    table = torch.arange(pages, dtype=I32, device=DEV).expand(B, pages).contiguous()          # all requests read the same blocks
    cu = torch.arange(0, (B + 1) * n, n, dtype=I32, device=DEV)
    out = torch.zeros_like(q)
    csa2.csa2_paged_attn_fp4(q, kc, vc, ks, vs, table, torch.full((B,), kv, dtype=I32, device=DEV), cu, out, math.log(2.0), n)
    torch.cuda.synchronize()
    w = np.exp2(k[:, 0] + k[:, 16] - max(up, 0.0))
    return out.double().cpu().numpy().reshape(B, n, H, D), w, kv - n


# The tile kernel's units are whole where there are many of them, so that its second tile meets the first one's reference;
# the split kernel takes few rows.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,B,H", [(256, 24, 8), (300, 20, 4), (1, 40, 8), (8, 3, 2)])
@pytest.mark.parametrize("tail", [-10.5, -15.5, -20.5, -22.5])
@pytest.mark.parametrize("up", [0.0, 1.0, 6.0, 12.0])
def test_weights_are_off_by_a_step_of_their_sum_at_most(csa2, D, n, B, H, tail, up):
    """A weight w of a sum W is off by max(2^-11 w, 2^-33 W), half a step of f16's 11 bits or of 2^-32 W.  128 keys just above
    the first tile's reference, whose sum leaves f16, raise that by the sum's exponent, far above the scores."""
    out, w, first = _tail_case(csa2, D, n, B, H, 128, tail, up)
    for i in sorted({0, n // 2, n - 1}):
        x, vals = w[:first + i + 1], np.where(np.arange(first + i + 1) < 256, 0.0, 6 * 448.0)
        W = x.sum()
        exact = (x * vals).sum() / W
        off = (np.maximum(x * 2.0 ** -11, W * 2.0 ** -33) * vals).sum() / W
        # besides: the output's rounding (fp16, 2^-11), sums in fp32 of up to 1836 terms (2^-24 each), exponentials (2^-20); below
        # fp16's normal numbers half its least step
        tol = off + exact * (2.0 ** -11 + 1836 * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -25
        worst = np.abs(out[:, i] - exact).max()
        assert worst <= tol, (i, exact, worst / exact, tol / exact)
