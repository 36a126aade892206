"""Plain references of rotary positions and of the paged 4-bit cache, in numpy,
written row by row and without shared code with the kernels.  The attention's is
paged_ref.attention on the cache's values, with scales of one: the kernels' roundings
are the same (keys and values exact, weights to f16)."""
from __future__ import annotations

import numpy as np
import torch

import paged_ref

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])                 # E2M1 magnitudes by code
E4M3 = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()   # finite magnitudes by code


def nearest(x, grid):
    """Place of the grid's nearest value to each x >= 0 (float64), ties to the even place."""
    i = np.searchsorted((grid[1:] + grid[:-1]) / 2, x)                    # values at a middle go below
    up = np.minimum(i + 1, grid.size - 1)
    tie = (i < up) & (x - grid[i] == grid[up] - x) & (i % 2 == 1)
    return np.where(tie, up, i)


def quantise(x):
    """Rows x float64 [..., D]: codes uint8 [..., D/2], scales uint8 [..., D/16], values float64 [..., D]."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    fin = np.where(np.isfinite(g), np.abs(g), 0.0)
    s = nearest(fin.max(-1) / 6, E4M3)
    sv = E4M3[s][..., None]
    g = np.where(np.isnan(g), 0.0, np.clip(g, -1e300, 1e300))
    c = nearest(np.divide(np.abs(g), sv, out=np.zeros_like(g), where=sv > 0), GRID)
    neg = np.signbit(g)
    val = np.where(neg, -1.0, 1.0) * GRID[c] * sv
    c = (c + 8 * neg).reshape(x.shape).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.astype(np.uint8), val.reshape(x.shape)


def values(codes, scales):
    """What codes [..., D/2] and scales [..., D/16] (uint8 torch tensors) stand for, float64."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).cpu().long().numpy()
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    s = scales.cpu().view(torch.float8_e4m3fn).double().numpy()
    return v * np.repeat(s, 16, -1)


def store(x, slots, codes, scales, S):
    """Rows x [T, H, D] (float64) into numpy planes codes [n, H, S, D/2] and scales [n, H, S, D/16]."""
    n = codes.shape[0]
    for t, slot in enumerate(slots):
        if 0 <= slot < n * S:
            c, s, _ = quantise(x[t])
            codes[slot // S, :, slot % S], scales[slot // S, :, slot % S] = c, s


def rotate(x, pos, table, first, half):
    """Rows x [T, H, D] (a 16-bit torch tensor) turned by table [n_pos, pairs, 2] in fp32, every product and sum rounded."""
    y, x32, t = x.clone(), x.float().cpu().numpy(), table.cpu().numpy()
    n = t.shape[1]
    for i in range(len(pos)):
        if not 0 <= pos[i] < t.shape[0]:
            continue
        c, s = t[pos[i], :, 0], t[pos[i], :, 1]
        z = x32[i, :, first:first + 2 * n]
        a, b = (z[:, :n], z[:, n:]) if half else (z[:, 0::2], z[:, 1::2])
        u, w = a * c - b * s, a * s + b * c                               # numpy rounds each to fp32
        out = np.concatenate([u, w], -1) if half else np.stack([u, w], -1).reshape(z.shape)
        y[i, :, first:first + 2 * n] = torch.from_numpy(out).to(x.dtype).to(x.device)
    return y


def random_planes(gen, n, H, S, D, size=1.0):
    """Codes and scales of normal rows whose sizes spread over a few octaves."""
    x = torch.randn(n, H, S, D, generator=gen) * torch.exp2(torch.randn(n, H, S, 1, generator=gen)) * size
    c, s, _ = quantise(x.double().numpy())
    return torch.from_numpy(c), torch.from_numpy(s)


def attention(q, kc, ks, vc, vs, table, kv_len, cu, sm_scale, window=0):
    one = torch.ones(kc.shape[:2], dtype=torch.float64)
    k, v = torch.from_numpy(values(kc, ks)), torch.from_numpy(values(vc, vs))
    return paged_ref.attention(q.double().cpu(), k, v, one, one, table.cpu(), kv_len, cu, sm_scale, window)
