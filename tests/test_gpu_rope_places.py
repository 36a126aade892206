"""csa2_rope on rows that lie between one another, on the GPU: the bits of dense rows, and nothing else touched."""
from __future__ import annotations

import pytest
import torch

import paged_fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def csa2():
    import sparse_attention_fp4_quantize_gb300 as lib
    return lib


def _table(gen, n_pos, pairs):
    a = torch.rand(n_pos, pairs, generator=gen) * 7
    return torch.stack([a.cos(), a.sin()], -1).to(DEV)


def _same(a, b):
    assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("T,H,D,dim,first", [(1, 4, 64, 64, 0), (50, 3, 128, 64, 32), (2100, 2, 64, 64, 0)])
def test_rotation_into_other_columns_of_the_same_buffer(csa2, half, T, H, D, dim, first):
    gen = torch.Generator().manual_seed(T + D)
    buf = torch.randn(T, 4 * H, D, generator=gen).to(BF).to(DEV)
    pos, table = torch.randint(0, 40, (T,), generator=gen).int().to(DEV), _table(gen, 40, dim // 2)
    layout = csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED
    for src, dst in ((0, 2), (3, 1), (1, 0)):
        at = lambda x, i: x[:, i * H:(i + 1) * H]  # noqa: E731
        got, want = buf.clone(), buf.clone()
        at(want, dst).copy_(ref.rotate(at(buf, src).cpu(), pos.tolist(), table, first, half))
        csa2.csa2_rope(at(got, src), pos, table, q_out=at(got, dst), first=first, layout=layout)
        torch.cuda.synchronize()
        _same(got, want)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("T,H,D", [(1, 5, 64), (37, 3, 128), (2000, 4, 64)])
def test_projections_side_by_side_in_every_head(csa2, T, H, D, heads_first):
    """q, k and v of a head beside one another: rotated in place, and written there by the reading back."""
    gen = torch.Generator().manual_seed(T + D)
    buf = torch.randn(T, H, 3 * D, generator=gen).to(F16).to(DEV)
    if heads_first:
        buf = buf.transpose(0, 1).contiguous().transpose(0, 1)
    pos, table = torch.randint(0, 40, (T,), generator=gen).int().to(DEV), _table(gen, 40, D // 2)
    q, k, v = buf[..., :D], buf[..., D:2 * D], buf[..., 2 * D:]
    want = [ref.rotate(x.cpu(), pos.tolist(), table, 0, True).to(DEV) for x in (q, k)] + [v.clone()]
    csa2.csa2_rope(q, pos, table, k=k)
    torch.cuda.synchronize()
    for got, w in zip((q, k, v), want):
        _same(got, w)
    n, S = T // 16 + 2, 16
    planes = [t.to(DEV) for _ in range(2) for t in ref.random_planes(gen, n, H, S, D)]
    kc, ks, vc, vs = planes
    at = torch.randperm(n * S, generator=gen)[:T].to(DEV)
    csa2.csa2_dequantize_kv_fp4_paged(at, kc, vc, ks, vs, k, v)
    torch.cuda.synchronize()
    held = [torch.from_numpy(ref.values(c[at // S, :, at % S], s[at // S, :, at % S])).to(F16).to(DEV) for c, s in ((kc, ks), (vc, vs))]
    for got, w in zip((q, k, v), [want[0]] + held):
        _same(got, w)
