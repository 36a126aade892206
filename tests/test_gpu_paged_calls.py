"""Calls of the paged 8-bit cache that follow one another, meet far-apart sizes or
hold nothing where nothing is read, on the GPU."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


@pytest.fixture(scope="module")
def csa2():
    import sparse_attention_fp4_quantize_gb300 as lib
    return lib


# ---------------------------------------------------------------- calls behind one another
def _mixed_steps(sync):
    """Steps of a batch that decodes and takes a prompt chunk, plan and append directly in front of the attention;
    every step's lengths and rows are other ones.  `sync`: the host waits after every call."""
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    B, H, Hq, D, L, T, steps = 8, 2, 16, 128, 2, 160, 24
    cache = PagedCache(PagedShape(requests=B, tokens=T, max_context=1024, n_blocks=B * 16, heads=Hq, kv_heads=H, dim=D,
                                  block_size=64, layers=L, max_new=100))
    gen = torch.Generator(DEV).manual_seed(50)
    rows = [[torch.randn(T, n, D, generator=gen, device=DEV).to(torch.bfloat16) for n in (Hq, H, H)] for _ in range(steps)]
    news = [torch.tensor([100 if b == i % B else 1 for b in range(B)], dtype=I32, device=DEV) for i in range(steps)]
    wait = torch.cuda.synchronize if sync else lambda: None
    wait()
    got = []
    for new, (q, k, v) in zip(news, rows):
        cache.new_len.copy_(new)
        wait()
        cache.plan()
        for layer in range(L):
            wait()
            cache.append(layer, k, v)
            wait()
            out, lse = cache.attend(layer, q, window=0 if layer == 0 else 300)
            wait()
            got += [out[:107].clone(), lse[:107].clone()]
    torch.cuda.synchronize()
    assert int(cache.err) == 0
    return got


def test_mixed_steps_back_to_back_give_the_bits_of_steps_one_by_one(csa2):
    apart = _mixed_steps(True)
    for _ in range(3):
        for a, b in zip(apart, _mixed_steps(False)):
            assert torch.equal(a, b)
