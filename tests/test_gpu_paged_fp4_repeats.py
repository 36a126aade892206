"""Attention over the paged 4-bit cache gives the same bits every time, whatever its workspace held and whatever ran before, on
the GPU."""
from __future__ import annotations

import pytest
import torch

import paged_fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32, BF, F16 = torch.int32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def csa2():
    import sparse_attention_fp4_quantize_gb300 as lib
    return lib


# Requests as (tokens in the cache, new ones); the last of each kind has empty and ragged ones.
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("D,G,H,S,window,requests", [
    (128, 4, 8, 64, 0, [(1000, 1)]),                                     # tiles of 32 keys
    (64, 4, 8, 16, 0, [(700, 1), (3, 1)]),
    (128, 8, 4, 64, 0, [(9000 - 37 * i, 1) for i in range(24)]),         # tiles of 64, units over several CTAs
    (64, 3, 5, 16, 512, [(2000 + 11 * i, 5) for i in range(16)]),        # 15 rows, a window
    (128, 4, 2, 32, 0, [(4000, 8), (1, 1), (0, 0), (900, 3)]),           # 32 rows
    (128, 4, 2, 64, 0, [(3000, 700), (150, 150), (0, 0)]),               # the tile kernel
    (64, 4, 2, 16, 300, [(2500, 333), (800, 1), (77, 2), (1200, 40)]),   # both kernels, a window
])
def test_attention_repeats_itself(csa2, dtype, D, G, H, S, window, requests):
    gen = torch.Generator().manual_seed(D + G + S)
    kv, new = [torch.tensor(x, dtype=I32) for x in zip(*requests)]
    held = -(-kv // S)
    n, B, T = int(held.sum()), len(requests), int(new.sum())
    table = torch.full((B, int(held.max()) + 1), -1, dtype=I32)
    ids, at = torch.randperm(n, generator=gen).int(), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += int(held[b])
    planes = [t.to(DEV) for x in range(2) for t in ref.random_planes(gen, n, H, S, D)]
    kc, ks, vc, vs = planes
    q = torch.randn(T, G * H, D, generator=gen).to(dtype).to(DEV)
    cu = torch.cat([torch.zeros(1, dtype=I32), new.cumsum(0).to(I32)]).to(DEV)
    kv, table = kv.to(DEV), table.to(DEV)
    most = int(new.max())
    ws = torch.empty(csa2.csa2_paged_attn_fp4_workspace_bytes(B, T, G * H, H, D, most), dtype=torch.uint8, device=DEV)
    first = None
    for i in range(12):
        ws.fill_((0, 0xFF, 0x7F, i)[i % 4])                              # NaN, large numbers, zeros
        out, lse = torch.full_like(q, 9.0), torch.full((T, G * H), 9.0, device=DEV)
        csa2.csa2_paged_attn_fp4(q, kc, vc, ks, vs, table, kv, cu, out, D ** -0.5, most, window=window, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        got = out.view(torch.int16).cpu(), lse.view(I32).cpu()
        if first is None:
            first = got
            assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), i
