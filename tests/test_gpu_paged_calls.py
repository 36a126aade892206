"""Calls of the paged 8-bit cache that follow one another, meet far-apart sizes or
hold nothing where nothing is read, on the GPU."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_ref as ref

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


def _attend(csa2, inp, sm, max_new, window=0):
    q, kc, vc, ks, vs, table, kv, cu = [t.to(DEV) for t in inp]
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    csa2.csa2_paged_attn_fp8(q, kc, vc, ks, vs, table, kv, cu, out, sm, max_new, window=window, lse=lse, err_flag=err)
    torch.cuda.synchronize()
    return out, lse, int(err)


def _reference(inp, sm, window=0):
    q, kc, vc, ks, vs, table, kv, cu = inp
    return ref.attention(q.double(), ref.values_of(kc), ref.values_of(vc), ks.double(), vs.double(), table, kv, cu, sm,
                         window)


def _inputs(seed, kv, new, Hq, H, D, S, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    table, n = ref.ragged(gen, kv, S)
    kc, ks = ref.random_planes(gen, n, H, S, D)
    vc, vs = ref.random_planes(gen, n, H, S, D)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=I32)
    q = torch.randn(int(cu[-1]), Hq, D, generator=gen).to(dtype)
    return q, kc, vc, ks, vs, table, torch.tensor(kv, dtype=I32), cu


# ---------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("n,at,nats,D,H", [(16384, 0, 17, 128, 320), (16384, 9001, 18, 64, 320), (131072, 0, 18, 64, 160),
                                           (131072, 5, 20, 64, 160)])
def test_a_sink_of_small_value_leaves_the_tail_its_weight(csa2, dtype, new, n, at, nats, D, H):
    """One key has nearly all the weight and no value: what comes out is the sum of many weights e^-nats.  A weight
    is an f16 number of 11 bits whose reference lies 2^8 above 1, so those below 2^-14 2^-8 of the largest, and only
    those, are off by up to half of f16's subnormal step, 2^-25 2^-8: n 2^-33 max|v| in place of the n 2^-25 max|v|
    that ref.attention allows.  So many heads, all alike, that one CTA walks through most of a head's keys."""
    gen = torch.Generator().manual_seed(n + nats)
    S, G = 64, 2
    table, pool = ref.ragged(gen, [n], S)
    kc, vc = torch.zeros(pool, 1, S, D), 1 + torch.randn(pool, 1, S, D, generator=gen) / 8
    kc[..., 1:] = torch.randn(pool, 1, S, D - 1, generator=gen)              # channels that q does not look at
    sink = int(table[0, at // S])
    kc[sink, 0, at % S, 0], vc[sink, 0, at % S] = 16.0, 0.0
    kc, vc = [x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (kc, vc)]
    q = torch.zeros(new, G, D)
    q[:, :, 0] = torch.linspace(1.0, 1.04, G)[None]                         # two query heads, their tails not alike
    ones = torch.ones(pool, 1)
    inp = (q.to(dtype), kc, vc, ones, ones, table, torch.tensor([n], dtype=I32), torch.tensor([0, new], dtype=I32))
    o, l, to, tl = _reference(inp, nats / 16)
    seen = (n - new + 1 + torch.arange(new)).double()[:, None, None]
    to = to - seen * (2.0 ** -25 - 2.0 ** -33) * ref.values_of(vc).abs().amax()
    assert (to > 0).all()
    all_heads = [x.to(DEV).expand(-1, H, *x.shape[2:]).contiguous() for x in inp[1:5]]
    out, lse, err = _attend(csa2, (inp[0].repeat(1, H, 1), *all_heads, *inp[5:]), nats / 16, new)
    assert err == 0
    for h in range(0, H, 7):
        ref.check_attention(out[:, G * h:G * h + G], lse[:, G * h:G * h + G], (o, l, to, tl))


# ---------------------------------------------------------------- behind a window
@pytest.mark.parametrize("new", [1, 3, 40, 200])
@pytest.mark.parametrize("D,S,window", [(64, 16, 100), (128, 16, 1), (128, 32, 77), (64, 64, 300)])
def test_nothing_is_read_before_the_window(csa2, new, D, S, window):
    """Blocks wholly before every row's window: given back (-1, no flag), or another request's, with rows that are not written."""
    inp = list(_inputs(new + S, [2050, 130], [new, min(new, 130)], 8, 2, D, S))
    want = _reference(inp, 0.1, window)
    q, kc, vc, ks, vs, table, kv, cu = inp
    for entry in (-1, kc.shape[0]):
        x = [t.clone() for t in inp]
        for b in range(2):
            x[5][b, :max(0, int(kv[b]) - int(cu[b + 1] - cu[b]) - window + 1) // S] = entry
        x[1], x[2] = [torch.cat([t, torch.full_like(t[:1], 0x7F)]) for t in (kc, vc)]
        x[3], x[4] = torch.cat([ks, torch.full_like(ks[:1], float("nan"))]), torch.cat([vs, torch.full_like(vs[:1], float("inf"))])
        out, lse, err = _attend(csa2, x, 0.1, new, window)
        ref.check_attention(out, lse, want)
        assert err == 0


# ---------------------------------------------------------------- scales at the ends of fp32
@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("exponent", [127, 126, 120, 61, 41, 39, -39, -41, -61, -126, -130])
def test_value_scales_at_the_ends_of_fp32(csa2, new, exponent):
    """V scales that have no fp32 reciprocal or are subnormal, codes that keep the values finite."""
    inp = list(_inputs(200 + exponent, [1500], [new], 4, 2, 64, 16))
    vc = (ref.values_of(inp[2]) / 448).float().clamp(-0.9, 0.9).to(torch.float8_e4m3fn).view(torch.uint8)
    inp[2], inp[4] = vc, torch.full_like(inp[4], 2.0 ** exponent)
    out, lse, err = _attend(csa2, inp, 0.05, new)
    ref.check_attention(out, lse, _reference(inp, 0.05))
    assert err == 0


# ---------------------------------------------------------------- slot maps
def test_slots_with_lengths_in_the_gap_between_table_rows(csa2):
    """Nothing that is written may overlap anything else; a strided table's gaps are nobody's."""
    B, M, S, T = 3, 4, 16, 40
    wide = torch.full((B, M + B), -1, dtype=I32, device=DEV)
    kv, new = wide[0, M:], wide[1, M:]
    kv.copy_(torch.tensor([0, 16, 5])), new.copy_(torch.tensor([20, 1, 0]))
    wide[1, 0], wide[2, 0] = 6, 7
    free, count = torch.arange(6, dtype=I32, device=DEV), torch.tensor([6], dtype=I32, device=DEV)
    kv_out, cu = torch.zeros(B, dtype=I32, device=DEV), torch.zeros(B + 1, dtype=I32, device=DEV)
    slots = torch.zeros(T, dtype=torch.int64, device=DEV)
    csa2.csa2_build_slots(kv, new, wide[:, :M], free, count, S, kv_out, count, cu, None, slots)
    torch.cuda.synchronize()
    assert kv_out.tolist() == [20, 17, 5] and kv.tolist() == [0, 16, 5] and int(count) == 3
    assert wide[:, :M].tolist() == [[5, 4, -1, -1], [6, 3, -1, -1], [7, -1, -1, -1]]
    assert slots.tolist() == [5 * S + i for i in range(16)] + [4 * S + i for i in range(4)] + [3 * S] + [-1] * 19


# ---------------------------------------------------------------- layers side by side
def test_layers_attended_on_streams_of_their_own(csa2):
    """The same bits as one behind the other: long contexts, whose parts are joined through the workspace."""
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    B, H, Hq, D, L, n = 2, 2, 8, 128, 2, 3000
    cache = PagedCache(PagedShape(requests=B, tokens=2 * n, max_context=n + 1, n_blocks=100, heads=Hq, kv_heads=H, dim=D,
                                  layers=L, max_new=1))
    gen = torch.Generator(DEV).manual_seed(3)
    q, k, v = [torch.randn(L, 2 * n, h, D, generator=gen, device=DEV).to(torch.bfloat16) for h in (Hq, H, H)]
    for new in (n, 1):
        cache.new_len.fill_(new)
        cache.plan()
        for layer in range(L):
            cache.append(layer, k[layer], v[layer])
    want = [[t.clone() for t in cache.attend(layer, q[layer])] for layer in range(L)]
    streams = [torch.cuda.Stream() for _ in range(L)]
    torch.cuda.synchronize()
    for _ in range(20):
        for layer in range(L):
            cache.attend(layer, q[layer], stream=streams[layer])
    torch.cuda.synchronize()
    for layer in range(L):
        assert torch.equal(cache.out[layer][:B], want[layer][0][:B]) and torch.equal(cache.lse[layer][:B], want[layer][1][:B])
    assert int(cache.err) == 0


# ---------------------------------------------------------------- scores beyond fp32's whole numbers
@pytest.mark.parametrize("new", [1, 80])
def test_scores_of_any_size_come_to_an_end(csa2, new):
    """Scores of 2^20 to 2^40, whose steps in fp32 are larger than the references' moves: one key has all the weight, or
    keys that fp32 cannot tell apart share it, so a row lies between the values' ends."""
    for seed, exponent in enumerate((20, 24, 26, 28, 30, 40)):
        inp = list(_inputs(90 + seed, [1500], [new], 4, 2, 64, 16))
        inp[4] = torch.full_like(inp[4], 1.75)
        out, lse, err = _attend(csa2, inp, 2.0 ** exponent, new)
        assert err == 0 and torch.isfinite(lse).all()
        v = ref.values_of(inp[2]).abs().amax() * 1.75
        assert (out.double().abs().cpu() <= v * 1.01).all()


# ---------------------------------------------------------------- long segments
def test_units_that_a_cta_works_on_for_long(csa2):
    """Five row tiles and more per CTA against 4 million keys each, some 50 ms: whoever works a segment ahead waits for that
    long.  All keys are alike and all values 1 (one block, over and over): out = 1, lse = log of the keys seen."""
    S, D, kv, T = 128, 64, 1 << 22, 200000
    kc, vc = torch.zeros(1, 1, S, D, dtype=torch.uint8, device=DEV), torch.full((1, 1, S, D), 0x38, dtype=torch.uint8, device=DEV)
    one, table = torch.ones(1, 1, device=DEV), torch.zeros(1, kv // S, dtype=I32, device=DEV)
    q = torch.randn(T, 1, D, generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    out, lse, err = torch.zeros_like(q), torch.zeros(T, 1, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    csa2.csa2_paged_attn_fp8(q, kc, vc, one, one, table, torch.tensor([kv], dtype=I32, device=DEV),
                             torch.tensor([0, T], dtype=I32, device=DEV), out, 0.1, T, lse=lse, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert (out == 1).all()
    want = torch.log((kv - T + 1 + torch.arange(T, device=DEV)).double())
    assert ((lse[:, 0].double() - want).abs() <= 4 * 2.0 ** -24 * want).all()
