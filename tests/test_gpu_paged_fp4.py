"""The paged 4-bit cache on the GPU: the quantising append and the reading back bit for bit, the attention against its
64-bit reference, and a serving loop that runs them together."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_fp4_ref as ref
import paged_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32, U8 = torch.int32, torch.uint8
BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def csa2():
    import sparse_attention_fp4_quantize_gb300 as lib
    return lib


def _planes(seed, n, H, S, D):
    gen = torch.Generator().manual_seed(seed)
    kc, ks = ref.random_planes(gen, n, H, S, D)
    vc, vs = ref.random_planes(gen, n, H, S, D)
    return [t.to(DEV) for t in (kc, vc, ks, vs)]


def _slots(gen, T, n, S, missing=0.1):
    """Rows of a step anywhere in the cache, each slot at most once, some without one."""
    s = torch.randperm(n * S, generator=gen)[:T]
    return torch.where(torch.rand(T, generator=gen) < missing, -1, s).to(DEV)


def _append_both(csa2, k, v, slots, planes, flags=0, rope=None, values=True):
    """Run the call and the reference on copies; all four planes must be equal, and the values what the codes stand for."""
    kc, vc, ks, vs = [p.clone() for p in planes]
    want = [p.cpu().numpy().copy() for p in planes]
    S, T = kc.shape[2], k.shape[0]
    err = torch.zeros(1, dtype=I32, device=DEV)
    vals = [torch.full(k.shape, 9.0, dtype=k.dtype, device=DEV) for _ in range(2)] if values else [None, None]
    args = {} if rope is None else dict(pos=rope[0], cos_sin=rope[1], first=rope[2], layout=csa2.ROPE_HALF if rope[3] else csa2.ROPE_INTERLEAVED)
    csa2.csa2_quantize_kv_fp4_paged(k, v, slots, kc, vc, ks, vs, k_values=vals[0], v_values=vals[1], err_flag=err, **args)
    torch.cuda.synchronize()
    sl = slots.cpu().numpy().copy()
    kr = k.cpu()
    if rope is not None:
        pos = rope[0].cpu().numpy()
        sl[(pos < 0) | (pos >= rope[1].shape[0])] = -1
        kr = ref.rotate(kr, pos.tolist(), rope[1], rope[2], rope[3])
    ref.store(kr.double().numpy(), sl, want[0], want[2], S)
    ref.store(v.double().cpu().numpy(), sl, want[1], want[3], S)
    for got, w in zip((kc, vc, ks, vs), want):
        assert np.array_equal(got.cpu().numpy(), w)
    if values:
        here = (sl >= 0) & (sl < kc.shape[0] * S)
        for got, c, s in ((vals[0], kc, ks), (vals[1], vc, vs)):
            at = torch.from_numpy(sl[here])
            held = ref.values(c.cpu()[at // S, :, at % S], s.cpu()[at // S, :, at % S])
            assert np.array_equal(got.double().cpu().numpy()[here], held)
            assert (got.cpu()[~torch.from_numpy(here)] == 9.0).all()
    assert int(err) == flags
    return kc, vc, ks, vs


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,H,D,S", [(1, 1, 64, 16), (1, 8, 128, 64), (37, 3, 128, 16), (64, 8, 128, 64), (200, 5, 64, 128), (700, 2, 64, 32),
                                     (3000, 9, 128, 32), (5, 33, 64, 16)])
def test_append_is_exact(csa2, dtype, T, H, D, S):
    gen = torch.Generator().manual_seed(T + H)
    n = T // S + 4
    size = torch.exp2(torch.randint(-14, 9, (T, H, 1), generator=gen).float())
    k = (torch.randn(T, H, D, generator=gen) * size).to(dtype).to(DEV)
    v = torch.randn(T, H, D, generator=gen).to(dtype).to(DEV)
    slots = _slots(gen, T, n, S)
    planes = _planes(T, n, H, S, D)
    _append_both(csa2, k, v, slots, planes)
    _append_both(csa2, k, v, slots, planes, values=False)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("D,dim,first", [(64, 64, 0), (64, 16, 40), (64, 48, 8), (128, 128, 0), (128, 64, 64), (128, 80, 24), (128, 32, 0)])
@pytest.mark.parametrize("half", [True, False])
def test_append_rotates_the_keys(csa2, dtype, D, dim, first, half):
    for T, H, S in ((1, 2, 16), (50, 3, 64), (2600, 5, 16)):
        gen = torch.Generator().manual_seed(T + D + dim)
        k, v = [(torch.randn(T, H, D, generator=gen) * 2).to(dtype).to(DEV) for _ in range(2)]
        a = torch.rand(40, dim // 2, generator=gen) * 7
        table = torch.stack([a.cos(), a.sin()], -1).to(DEV)
        pos = torch.randint(0, 40, (T,), generator=gen).int().to(DEV)
        n = T // S + 3
        slots = _slots(gen, T, n, S)
        _append_both(csa2, k, v, slots, _planes(T, n, H, S, D), rope=(pos, table, first, half))


def test_append_skips_tokens_without_a_position(csa2):
    T, H, D, S, n = 30, 2, 64, 16, 4
    gen = torch.Generator().manual_seed(8)
    k, v = [torch.randn(T, H, D, generator=gen).to(BF).to(DEV) for _ in range(2)]
    table = torch.randn(20, 16, 2, generator=gen).to(DEV)
    pos = torch.randint(0, 20, (T,), generator=gen).int().to(DEV)
    slots = _slots(gen, T, n, S, 0.0)
    slots[4] = -1
    pos[4] = -1                                                          # neither: nothing to say
    _append_both(csa2, k, v, slots, _planes(1, n, H, S, D), rope=(pos, table, 0, True))
    pos[7], pos[9] = -1, 20
    _append_both(csa2, k, v, slots, _planes(1, n, H, S, D), rope=(pos, table, 0, True), flags=0x1)


def test_append_reads_slices_of_a_projection(csa2):
    T, H, D, S = 50, 3, 64, 16
    gen = torch.Generator().manual_seed(4)
    qkv = torch.randn(T, 10 * H * D + 8, generator=gen).to(BF).to(DEV)
    k, v = qkv[:, 8 * H * D:9 * H * D].view(T, H, D), qkv[:, 9 * H * D + 8:].view(T, H, D)
    slots, planes = _slots(gen, T, 6, S), _planes(1, 6, H, S, D)
    a = torch.rand(9, 32, generator=gen)
    rope = (torch.randint(0, 9, (T,), generator=gen).int().to(DEV), torch.stack([a.cos(), a.sin()], -1).to(DEV), 0, True)
    _append_both(csa2, k, v, slots, planes, rope=rope)
    heads_first = torch.randn(H, T, D, generator=gen).to(BF).to(DEV).transpose(0, 1)
    _append_both(csa2, heads_first, v, slots, planes, rope=rope)
    _append_both(csa2, qkv[:, :D].view(T, 1, D).expand(T, H, D), v, slots, planes)     # one row for every head


@pytest.mark.parametrize("dtype", [BF, F16])
def test_append_borders(csa2, dtype):
    """Every tie of the codes at every scale, every tie of the scale, and the ends of the types, one group to each."""
    f = torch.finfo(dtype)
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    groups = []
    scales = ref.E4M3[1:]
    for s in scales:                                                     # amax = 6 s, ties and their neighbours below
        m = torch.tensor([6 * s] + [x * s for x in mids], dtype=torch.float64)
        groups.append(torch.cat([m, -m]))
        groups.append(torch.cat([m[:1], m[1:] * (1 + f.eps), -m[1:] * (1 - f.eps)]))
    for a, b in zip(scales[:-1], scales[1:]):
        for x in (3 * (a + b), 3 * (a + b) * (1 + f.eps), 3 * (a + b) * (1 - f.eps)):
            groups.append(torch.tensor([x, x / 7, -x / 3]))
    for x in (0.0, -0.0, f.max, f.tiny, f.tiny * f.eps, 448 * 6, 448 * 6.2, 6 * 2.0 ** -10, 6 * 2.0 ** -10 * (1 + f.eps)):
        groups.append(torch.tensor([x, -x / 2, 0.0, -0.0]))
    x = torch.zeros(-(-len(groups) // 4) * 4, 16, dtype=torch.float64)
    for i, g in enumerate(groups):
        x[i, :g.numel()] = g
    x = x.view(-1, 1, 64).to(dtype).to(DEV)
    x = x[torch.isfinite(x).all(-1)[:, 0]]
    T = x.shape[0]
    _append_both(csa2, x, -x, torch.arange(T, device=DEV), _planes(2, T // 16 + 1, 1, 16, 64))


@pytest.mark.parametrize("dtype", [BF, F16])
def test_append_infinities_and_nan_are_stored_finite_and_flagged(csa2, dtype):
    H, D, S = 2, 128, 32
    k = torch.randn(5, H, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    k[1, 0, 3], k[2, 0, 7], k[3, 0, 9] = math.inf, -math.inf, math.nan
    k[4, 0] = math.inf
    k[:, 1] = math.nan
    v = torch.randn(5, H, D, generator=torch.Generator().manual_seed(2)).to(dtype)
    kc, _, ks, _ = _append_both(csa2, k.to(DEV), v.to(DEV), torch.arange(34, 39, device=DEV), _planes(5, 3, H, S, D), flags=0x20)
    assert np.isfinite(ref.values(kc, ks)).all()


def test_append_bad_slots_are_skipped_and_flagged(csa2):
    H, D, S, n = 2, 64, 16, 4
    x = torch.randn(6, H, D, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    for bad, flag in (([n * S, -1, n * S + 5, 2 ** 40, -2, -2 ** 40], 0x4), ([3, -1, 63, 0, 5, 64], 0x4), ([3, -1, 63, 0, 5, 62], 0)):
        _append_both(csa2, x, x, torch.tensor(bad, device=DEV), _planes(6, n, H, S, D), flags=flag)
    empty = [torch.zeros(0, H, S, D // 2, dtype=U8, device=DEV)] * 2 + [torch.zeros(0, H, S, D // 16, dtype=U8, device=DEV)] * 2
    csa2.csa2_quantize_kv_fp4_paged(x[:0], x[:0], torch.empty(0, dtype=torch.int64, device=DEV), *_planes(6, n, H, S, D))
    csa2.csa2_quantize_kv_fp4_paged(x, x, torch.full((6,), -1, device=DEV), *empty)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- reading back
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,H,D,S", [(1, 1, 64, 16), (64, 8, 128, 64), (333, 5, 64, 128), (4000, 7, 128, 16)])
def test_reading_back_is_exact(csa2, dtype, T, H, D, S):
    """All codes and scales (NaN scales read as NaN), slots more than once, out of range and none."""
    gen = torch.Generator().manual_seed(T)
    n = 30
    kc, vc = [torch.randint(0, 256, (n, H, S, D // 2), generator=gen).byte().to(DEV) for _ in range(2)]
    ks, vs = [(torch.randint(0, 255, (n, H, S, D // 16), generator=gen) | 128 * torch.randint(0, 2, (1,), generator=gen)).byte().to(DEV) for _ in range(2)]
    slots = torch.randint(0, n * S, (T,), generator=gen).to(DEV)
    if T > 10:
        slots[3], slots[5], slots[7] = -1, n * S, -2 ** 50
    k, v = torch.full((T, H, D), 9.0, dtype=dtype, device=DEV), torch.full((H, T, D + 8), 9.0, dtype=dtype, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    csa2.csa2_dequantize_kv_fp4_paged(slots, kc, vc, ks.view(torch.float8_e4m3fn), vs.view(torch.float8_e4m3fn), k,
                                      v.transpose(0, 1)[..., :D], err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == (0x4 if T > 10 else 0) and (v[..., D:] == 9.0).all()
    here = (slots >= 0) & (slots < n * S)
    at = slots[here].cpu()
    for got, c, s in ((k, kc, ks), (v.transpose(0, 1)[..., :D], vc, vs)):
        want = ref.values(c.cpu()[at // S, :, at % S], s.cpu()[at // S, :, at % S])
        assert np.array_equal(got[here].double().cpu().numpy(), want, equal_nan=True)
        assert (got[~here] == 9.0).all()


def test_cache_beyond_32_bit_offsets(csa2):
    """Planes of more than 2^32 bytes: append to, read back from and attend over the last blocks."""
    H, D, S = 8, 128, 128
    n = (1 << 32) // (H * S * D // 2) + 40
    kc = torch.zeros(n, H, S, D // 2, dtype=U8, device=DEV)
    vc = torch.zeros_like(kc)
    ks, vs = [torch.zeros(n, H, S, D // 16, dtype=U8, device=DEV) for _ in range(2)]
    gen = torch.Generator().manual_seed(11)
    T = 200
    k, v = [torch.randn(T, H, D, generator=gen).to(BF).to(DEV) for _ in range(2)]
    ids = torch.tensor([n - 1, n - 3], dtype=I32)
    p = torch.arange(T)
    slots = (ids.long()[p // S] * S + p % S).to(DEV)
    kv, vv = torch.zeros_like(k), torch.zeros_like(v)
    csa2.csa2_quantize_kv_fp4_paged(k, v, slots, kc, vc, ks, vs, k_values=kv, v_values=vv)
    kb, vb = torch.zeros_like(k), torch.zeros_like(v)
    csa2.csa2_dequantize_kv_fp4_paged(slots, kc, vc, ks, vs, kb, vb)
    torch.cuda.synchronize()
    assert np.array_equal(kb.double().cpu().numpy(), ref.quantise(k.double().cpu().numpy())[2])
    assert torch.equal(kb, kv) and torch.equal(vb, vv)
    pick = ids.long().to(DEV)
    for new in (3, 100):
        q = torch.randn(new, 2 * H, D, generator=gen).to(BF).to(DEV)
        out, lse = torch.empty_like(q), torch.empty(new, 2 * H, device=DEV)
        lens, cu = torch.tensor([T], dtype=I32, device=DEV), torch.tensor([0, new], dtype=I32, device=DEV)
        csa2.csa2_paged_attn_fp4(q, kc, vc, ks, vs, ids[None].to(DEV).contiguous(), lens, cu, out, 0.1, new, lse=lse)
        torch.cuda.synchronize()
        small = torch.tensor([[0, 1]], dtype=I32)
        paged_ref.check_attention(out, lse, ref.attention(q, kc[pick], ks[pick], vc[pick], vs[pick], small, [T], [0, new], 0.1))


def test_append_and_reading_back_on_another_stream_and_in_graphs(csa2):
    """A prompt's rows on a stream that is not the current one; then captured and replayed with other rows and slots, and
    eager calls in between."""
    T, H, D, S, n = 150, 4, 128, 32, 12
    gen = torch.Generator().manual_seed(60)
    planes = [p.zero_() for p in _planes(60, n, H, S, D)]
    k, v = [torch.zeros(T, H, D, dtype=BF, device=DEV) for _ in range(2)]
    slots = torch.full((T,), -1, device=DEV)
    back = [torch.zeros_like(k) for _ in range(2)]

    def fill():
        for x in (k, v):
            x.copy_(torch.randn(x.shape, generator=gen).to(BF))
        slots.copy_(_slots(gen, T, n, S, 0.0))

    def calls(stream=None):
        csa2.csa2_quantize_kv_fp4_paged(k, v, slots, *planes, stream=stream)
        csa2.csa2_dequantize_kv_fp4_paged(slots, *planes, *back, stream=stream)

    def right():
        for x, y in zip((k, v), back):
            assert np.array_equal(y.double().cpu().numpy(), ref.quantise(x.double().cpu().numpy())[2])

    fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(side)
    side.synchronize()
    right()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(3):
        fill()
        g.replay()
        torch.cuda.synchronize()
        right()
        fill()
        calls()
        torch.cuda.synchronize()
        right()


@pytest.mark.parametrize("half", [True, False])
def test_append_of_rows_that_heads_and_tokens_share(csa2, half):
    """Strides of 0: one row for all heads, one for all tokens."""
    T, H, D, S = 9, 5, 64, 16
    gen = torch.Generator().manual_seed(61)
    k = torch.randn(T, 1, D, generator=gen).to(BF).to(DEV).expand(T, H, D)
    v = torch.randn(1, H, D, generator=gen).to(BF).to(DEV).expand(T, H, D)
    table = torch.randn(20, 16, 2, generator=gen).to(DEV)
    pos = torch.randint(0, 20, (T,), generator=gen).to(I32).to(DEV)
    _append_both(csa2, k, v, _slots(gen, T, 4, S), _planes(61, 4, H, S, D), rope=(pos, table, 24, half))


# ---------------------------------------------------------------- attention
def _inputs(seed, kv, new, Hq, H, D, S, dtype=BF, q_size=1.0):
    gen = torch.Generator().manual_seed(seed)
    table, n = paged_ref.ragged(gen, kv, S)
    kc, ks = ref.random_planes(gen, n, H, S, D)
    vc, vs = ref.random_planes(gen, n, H, S, D)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=I32)
    q = (torch.randn(int(cu[-1]), Hq, D, generator=gen) * q_size).to(dtype)
    return [q, kc, vc, ks, vs, table, torch.tensor(kv, dtype=I32), cu]


def _attend(csa2, inp, sm, max_new, window=0, pad=0, err=None, **kw):
    q, kc, vc, ks, vs, table, kv, cu = [t.to(DEV) for t in inp]
    out = torch.full((q.shape[0] + pad, *q.shape[1:]), 9.0, dtype=q.dtype, device=DEV)
    lse = torch.full(out.shape[:2], 9.0, device=DEV)
    if pad:
        q = torch.cat([q, torch.full((pad, *q.shape[1:]), float("nan"), dtype=q.dtype, device=DEV)])
    csa2.csa2_paged_attn_fp4(q, kc, vc, ks, vs, table, kv, cu, out, sm, max_new, window=window, lse=lse, err_flag=err, **kw)
    torch.cuda.synchronize()
    if pad:
        assert (out[-pad:] == 9.0).all() and (lse[-pad:] == 9.0).all()
    return out[:out.shape[0] - pad], lse[:lse.shape[0] - pad]


def _reference(inp, sm, window=0):
    q, kc, vc, ks, vs, table, kv, cu = inp
    return ref.attention(q, kc, ks, vc, vs, table, kv, cu, sm, window)


ATTN_CASES = [  # kv, new, Hq, Hkv, D, S, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1, 2, 15, 16, 17, 64, 65], [1] * 7, 8, 2, 128, 16, 0),
    ([1000], [1], 32, 8, 128, 64, 0),
    ([5000, 3, 0, 777], [1, 1, 1, 1], 16, 2, 128, 128, 0),
    ([333, 2050, 129], [5, 2, 3], 15, 5, 64, 32, 0),
    ([333, 2050, 129], [5, 2, 3], 15, 5, 64, 16, 100),
    ([300, 40], [1, 1], 40, 1, 128, 64, 0),
    ([300, 40], [7, 4], 14, 2, 64, 64, 1),
    ([130], [130], 4, 1, 128, 64, 0),
    ([257, 64, 1], [257, 64, 1], 6, 2, 64, 16, 0),
    ([600, 1500, 20], [400, 31, 20], 8, 4, 128, 32, 0),
    ([600, 1500, 20], [400, 31, 20], 8, 4, 128, 32, 64),
    ([700, 900], [300, 0], 7, 7, 128, 128, 250),
    ([900, 33, 1200, 8, 100], [200, 1, 1, 0, 1], 16, 2, 128, 64, 0),
    ([3000], [129], 32, 4, 128, 64, 0),
    ([4100, 4000], [33, 40], 24, 3, 64, 32, 1000),
    ([3000, 17], [1, 1], 16, 1, 128, 32, 0),
    ([2000, 31], [1, 1], 32, 1, 64, 16, 0),
    ([900, 1, 450], [2, 1, 2], 24, 3, 64, 64, 0),
    ([9000], [70], 2, 1, 64, 128, 0),
    ([129, 128, 127, 256, 257], [129, 128, 127, 256, 257], 1, 1, 128, 64, 0),
    ([900, 70, 33], [5, 7, 8], 8, 2, 128, 64, 90),
    ([500, 260, 31], [1, 250, 2], 20, 1, 128, 64, 0),
    ([500, 260, 31], [1, 250, 2], 33, 1, 64, 32, 0),
]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("kv,new,Hq,H,D,S,window", ATTN_CASES)
def test_attention_matches_reference(csa2, dtype, kv, new, Hq, H, D, S, window):
    inp = _inputs(len(kv) * 7 + sum(kv), kv, new, Hq, H, D, S, dtype)
    sm = 1.0 / D ** 0.5 / 2
    err = torch.zeros(1, dtype=I32, device=DEV)
    want = _reference(inp, sm, window)
    out, lse = _attend(csa2, inp, sm, max(new), window, pad=3, err=err)
    paged_ref.check_attention(out, lse, want)
    assert int(err) == 0
    again, lse2 = _attend(csa2, inp, sm, max(new), window)
    assert torch.equal(out, again) and torch.equal(lse, lse2)            # the same bits every time
    for hint in (1, 4 * max(new) + 100):                                 # the hint changes the kernels, not the answer
        o, l = _attend(csa2, inp, sm, hint, window)
        paged_ref.check_attention(o, l, want)


def test_rows_that_see_nothing(csa2):
    """No stored keys; more new rows than tokens (requests that wait): out 0, lse -inf."""
    for new in ([1, 3, 4], [1, 40, 60]):
        inp = _inputs(3, [0, 1, 2], new, 4, 2, 64, 16)
        out, lse = _attend(csa2, inp, 0.2, max(new))
        paged_ref.check_attention(out, lse, _reference(inp, 0.2))
        dead = torch.tensor([0] + list(range(1, new[1])) + list(range(1 + new[1], sum(new) - 2)), device=DEV)
        assert (out[dead] == 0).all() and torch.isneginf(lse[dead]).all()


@pytest.mark.parametrize("new", [1, 60, 300])
@pytest.mark.parametrize("D,S", [(64, 64), (128, 16), (128, 128)])
def test_garbage_behind_the_last_token(csa2, new, D, S):
    """Rows at or beyond kv_len and unused blocks hold any code and NaN scales."""
    kv = [333]
    inp = _inputs(5, kv, [new], 8, 2, D, S, F16)
    want = _reference(inp, 0.1)
    q, kc, vc, ks, vs, table, _, _ = inp
    last = int(table[0, 333 // S])
    held = -(-333 // S)
    for c, s in ((kc, ks), (vc, vs)):
        c[last, :, 333 % S:], s[last, :, 333 % S:] = 0xFF, 0x7F
        for b in set(range(c.shape[0])) - set(table[0, :held].tolist()):
            c[b], s[b] = 0x77, 0xFF
    out, lse = _attend(csa2, inp, 0.1, new)
    paged_ref.check_attention(out, lse, want)


def _widened(inp, tokens=1 << 22):
    """The same call with a table that could hold so many tokens of each request."""
    table, S = inp[5], inp[1].shape[2]
    wide = torch.full((table.shape[0], tokens // S), -1, dtype=I32)
    wide[:, :table.shape[1]] = table
    return [*inp[:5], wide, *inp[6:]]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("S", [16, 32, 64, 128])
@pytest.mark.parametrize("D,Hq", [(64, 8), (128, 8), (64, 14), (128, 24)])
@pytest.mark.parametrize("window", [0, 70])
def test_tables_that_could_hold_long_contexts(csa2, dtype, S, D, Hq, window):
    """The longer tiles that few rows get with them, next to those of the same call with tables that just fit; anything may
    lie behind the last token."""
    kv, new = [1, 2, 63, 64, 65, 700, 2051, 0, 130], [1, 2, 1, 2, 1, 1, 2, 1, 0]
    inp = _inputs(80 + S, kv, new, Hq, 2, D, S, dtype)
    for b, n in enumerate(kv):
        if n % S:
            last = int(inp[5][b, n // S])
            for plane in inp[1:3]:
                plane[last, :, n % S:] = 255
            for plane in inp[3:5]:
                plane[last, :, n % S:] = 127                             # NaN
    want = _reference(inp, 0.2, window)
    for x in (_widened(inp), inp):
        err = torch.zeros(1, dtype=I32, device=DEV)
        out, lse = _attend(csa2, x, 0.2, 2, window, pad=3, err=err)
        paged_ref.check_attention(out, lse, want)
        assert int(err) == 0


@pytest.mark.parametrize("kv,new,Hq,H,D,S,window", ATTN_CASES)
def test_attention_matches_reference_with_wide_tables(csa2, kv, new, Hq, H, D, S, window):
    inp = _inputs(81, kv, new, Hq, H, D, S)
    out, lse = _attend(csa2, _widened(inp), 0.3, max(new), window)
    paged_ref.check_attention(out, lse, _reference(inp, 0.3, window))


@pytest.mark.parametrize("new", [1, 90])
def test_query_rows_do_not_meet(csa2, new):
    """A row of infinities or NaN spoils itself only; magnitudes far from one are exact or nearly."""
    inp = _inputs(6, [400, 200], [new, new], 4, 2, 64, 32)
    want = _reference(inp, 0.125)
    inp[0] = inp[0].clone()
    inp[0][0, 1], inp[0][new, 3] = float("nan"), float("inf")
    out, lse = _attend(csa2, inp, 0.125, new)
    ok = torch.ones(2 * new, 4, dtype=torch.bool)
    ok[0, 1] = ok[new, 3] = False
    paged_ref.check_attention(out, lse, want, ok)
    for size in (1e-20, 1e15):
        x = list(inp)
        x[0] = (torch.randn(2 * new, 4, 64, generator=torch.Generator().manual_seed(1)) * size).to(BF)
        out, lse = _attend(csa2, x, 0.125 / size, new)
        paged_ref.check_attention(out, lse, _reference(x, 0.125 / size))


def test_missing_blocks_hide_their_keys(csa2):
    for new, S in ((1, 64), (70, 64), (1, 16), (70, 16)):
        inp = _inputs(8, [320], [new], 8, 2, 128, S)
        for bad in (-1, -2 ** 31, inp[1].shape[0], 2 ** 31 - 1):
            x = list(inp)
            x[5] = inp[5].clone()
            x[5][0, 1] = bad
            err = torch.zeros(1, dtype=I32, device=DEV)
            out, lse = _attend(csa2, x, 0.1, new, err=err)
            assert int(err) == 0x1
            y = list(inp)                        # the reference: the same request without that block's tokens
            y[5] = torch.cat([inp[5][:, :1], inp[5][:, 2:]], 1)
            y[6] = inp[6] - S
            paged_ref.check_attention(out, lse, _reference(y, 0.1))


def test_lengths_out_of_range_are_bounded(csa2):
    inp = _inputs(9, [100, 90], [2, 3], 4, 2, 64, 16)
    x = list(inp)
    x[6] = torch.tensor([2 ** 31 - 1, -5], dtype=I32)                     # as all of the table's tokens, and none
    x[5] = inp[5][:, :7].contiguous()
    full = list(x)
    full[6] = torch.tensor([112, 0], dtype=I32)
    out, lse = _attend(csa2, x, 0.1, 3)
    assert (out[2:] == 0).all() and torch.isneginf(lse[2:]).all()
    paged_ref.check_attention(out, lse, _reference(full, 0.1))
    x = list(inp)
    x[7] = torch.tensor([-3, 2, 2 ** 30], dtype=I32)                      # first rows clamped to [0, T]
    out, lse = _attend(csa2, x, 0.1, 3)
    paged_ref.check_attention(out, lse, _reference(inp, 0.1))


def test_strided_queries_tables_and_streams(csa2):
    inp = _inputs(10, [500, 77], [3, 40], 8, 2, 128, 32)
    want = _reference(inp, 0.1)
    q, kc, vc, ks, vs, table, kv, cu = [t.to(DEV) for t in inp]
    T = q.shape[0]
    fused = torch.zeros(T, 12, 136, dtype=q.dtype, device=DEV)
    fused[:, 2:10, :128] = q
    wide = torch.full((2, table.shape[1] + 5), -1, dtype=I32, device=DEV)
    wide[:, :table.shape[1]] = table
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(q), torch.empty(T, 8, device=DEV)
    f8 = torch.float8_e4m3fn
    csa2.csa2_paged_attn_fp4(fused[:, 2:10, :128], kc, vc, ks.view(f8), vs.view(f8), wide[:, :table.shape[1]], kv, cu, out, 0.1,
                             40, lse=lse, stream=side)
    side.synchronize()
    paged_ref.check_attention(out, lse, want)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    out2 = torch.empty_like(q)
    csa2.csa2_paged_attn_fp4(heads_first, kc, vc, ks, vs, table, kv, cu, out2, 0.1, 40)       # without lse
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_grow_and_shrink(csa2, new, D):
    """Keys whose size rises or falls block by block: references move often, or never."""
    for step in (0.25, -0.25):
        inp = _inputs(31, [1000], [new], 4, 1, D, 16)
        at = torch.zeros(inp[1].shape[0])
        at[inp[5][0, :63].long()] = torch.arange(63).float()
        gen = torch.Generator().manual_seed(3)
        rows = torch.randn(*inp[1].shape[:3], D, generator=gen) * torch.exp2(step * at - (12 if step > 0 else -4))[:, None, None, None]
        c, s, _ = ref.quantise(rows.double().numpy())
        inp[1], inp[3] = torch.from_numpy(c), torch.from_numpy(s)
        for sm in (0.02, 0.3):
            out, lse = _attend(csa2, inp, sm, new)
            paged_ref.check_attention(out, lse, _reference(inp, sm))


@pytest.mark.parametrize("new", [1, 50])
def test_sign_and_zero_of_the_scale(csa2, new):
    inp = _inputs(32, [700], [new], 4, 2, 64, 64, F16)
    for sm in (-0.2, 0.0):
        out, lse = _attend(csa2, inp, sm, new)
        paged_ref.check_attention(out, lse, _reference(inp, sm))
    inp[3], inp[4] = torch.zeros_like(inp[3]), torch.zeros_like(inp[4])   # a cache of zero scales: every value 0
    out, lse = _attend(csa2, inp, 0.2, new)
    paged_ref.check_attention(out, lse, _reference(inp, 0.2))


def test_many_short_requests(csa2):
    rng = np.random.default_rng(5)
    kv = rng.integers(0, 50, 700)
    new = np.minimum(rng.choice([0, 1, 1, 1, 2, 30], 700), kv)
    inp = _inputs(33, list(kv), list(new), 4, 2, 64, 16)
    for hint in (1, 30):
        out, lse = _attend(csa2, inp, 0.1, hint, pad=1)
        paged_ref.check_attention(out, lse, _reference(inp, 0.1))


def test_a_cache_without_blocks(csa2):
    q = torch.randn(3, 4, 64, device=DEV).to(BF)
    planes = [torch.empty(0, 2, 16, 32, dtype=U8, device=DEV)] * 2 + [torch.empty(0, 2, 16, 4, dtype=U8, device=DEV)] * 2
    table = torch.full((2, 3), -1, dtype=I32, device=DEV)
    for kv, flag in ([0, 0], 0), ([5, 0], 1):
        for hint in (1, 100):
            out, lse = torch.full_like(q, 3.0), torch.full((3, 4), 3.0, device=DEV)
            err = torch.zeros(1, dtype=I32, device=DEV)
            csa2.csa2_paged_attn_fp4(q, *planes, table, torch.tensor(kv, dtype=I32, device=DEV),
                                     torch.tensor([0, 2, 3], dtype=I32, device=DEV), out, 0.1, hint, lse=lse, err_flag=err)
            torch.cuda.synchronize()
            assert (out == 0).all() and torch.isneginf(lse).all() and int(err) == flag


@pytest.mark.parametrize("new", [1, 3, 40, 200])
@pytest.mark.parametrize("D,S,window", [(64, 16, 100), (128, 16, 1), (128, 32, 77), (64, 64, 300), (64, 128, 130)])
def test_nothing_is_read_before_the_window(csa2, new, D, S, window):
    """Blocks wholly before every row's window: given back (-1, no flag), or another request's, with rows that are not written."""
    inp = _inputs(new + S, [2050, 130], [new, min(new, 130)], 8, 2, D, S)
    want = _reference(inp, 0.1, window)
    kc, vc, ks, vs, kv, cu = [inp[i] for i in (1, 2, 3, 4, 6, 7)]
    for entry in (-1, kc.shape[0]):
        x = [t.clone() for t in inp]
        for b in range(2):
            x[5][b, :max(0, int(kv[b]) - int(cu[b + 1] - cu[b]) - window + 1) // S] = entry
        x[1], x[2] = [torch.cat([t, torch.full_like(t[:1], 0x7F)]) for t in (kc, vc)]
        x[3], x[4] = [torch.cat([t, torch.full_like(t[:1], 0x7F)]) for t in (ks, vs)]
        err = torch.zeros(1, dtype=I32, device=DEV)
        out, lse = _attend(csa2, x, 0.1, new, window, err=err)
        paged_ref.check_attention(out, lse, want)
        assert int(err) == 0


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("n,at,nats,D,H", [(16384, 0, 16, 128, 320), (16384, 9001, 17, 64, 320), (131072, 5, 18, 64, 160)])
def test_a_sink_of_small_value_leaves_the_tail_its_weight(csa2, dtype, new, n, at, nats, D, H):
    """One key has nearly all the weight and no value: what comes out is the sum of many weights e^-nats.  A weight is an
    f16 number of 11 bits whose reference lies 2^8 above 1, so those below 2^-14 2^-8 of the largest are off by up to half of
    f16's subnormal step, 2^-25 2^-8: n 2^-33 max|v| in place of the n 2^-25 max|v| that the reference allows."""
    gen = torch.Generator().manual_seed(n + nats)
    S, G = 64, 2
    table, pool = paged_ref.ragged(gen, [n], S)
    k, v = torch.zeros(pool, 1, S, D), 1 + torch.randn(pool, 1, S, D, generator=gen) / 8
    k[..., 16:] = torch.randn(pool, 1, S, D - 16, generator=gen)          # channels that q does not look at
    sink = int(table[0, at // S])
    k[sink, 0, at % S, 0], v[sink, 0, at % S] = 16.0, 0.0
    (kc, ks), (vc, vs) = [[torch.from_numpy(y) for y in ref.quantise(x.double().numpy())[:2]] for x in (k, v)]
    q = torch.zeros(new, G, D)
    q[:, :, 0] = torch.linspace(1.0, 1.04, G)[None]                      # two query heads, their tails not alike
    inp = [q.to(dtype), kc, vc, ks, vs, table, torch.tensor([n], dtype=I32), torch.tensor([0, new], dtype=I32)]
    sm = nats / float(ref.values(kc, ks)[sink, 0, at % S, 0])
    o, l, to, tl = _reference(inp, sm)
    seen = (n - new + 1 + torch.arange(new)).double()[:, None, None]
    to = to - seen * (2.0 ** -25 - 2.0 ** -33) * torch.from_numpy(ref.values(vc, vs)).abs().amax()
    assert (to > 0).all()
    all_heads = [x.to(DEV).expand(-1, H, *x.shape[2:]).contiguous() for x in inp[1:5]]
    out, lse = _attend(csa2, [inp[0].repeat(1, H, 1), *all_heads, *inp[5:]], sm, new)
    for h in range(0, H, 7):
        paged_ref.check_attention(out[:, G * h:G * h + G], lse[:, G * h:G * h + G], (o, l, to, tl))


@pytest.mark.parametrize("new", [1, 80])
def test_scores_of_any_size_come_to_an_end(csa2, new):
    """Scores of 2^20 to 2^40, whose steps in fp32 are larger than the references' moves: a row lies between the values' ends."""
    for seed, exponent in enumerate((20, 24, 26, 28, 30, 40)):
        inp = _inputs(90 + seed, [1500], [new], 4, 2, 64, 16)
        err = torch.zeros(1, dtype=I32, device=DEV)
        out, lse = _attend(csa2, inp, 2.0 ** exponent, new, err=err)
        assert int(err) == 0 and torch.isfinite(lse).all()
        assert (out.double().abs().cpu() <= np.abs(ref.values(inp[2], inp[4])).max() * 1.01).all()


def test_calls_on_two_streams_and_in_two_graphs(csa2):
    """Calls that overlap have a workspace each; a graph replayed between eager calls gives the eager bits."""
    a = _inputs(34, [4000, 300], [1, 1], 8, 1, 128, 64)
    b = _inputs(35, [600, 900], [300, 200], 8, 2, 128, 32)
    want = [_attend(csa2, x, 0.1, n) for x, n in ((a, 1), (b, 300))]
    dev = [[t.to(DEV) for t in x] for x in (a, b)]
    outs = [(torch.zeros_like(w[0]), torch.zeros_like(w[1])) for w in want]
    ws = [csa2.workspace_for_paged_attn_fp4(2, x[0].shape[0], 8, x[1].shape[1], 128, n) for x, n in ((a, 1), (b, 300))]

    def call(i, stream=None):
        q, kc, vc, ks, vs, table, kv, cu = dev[i]
        csa2.csa2_paged_attn_fp4(q, kc, vc, ks, vs, table, kv, cu, outs[i][0], 0.1, (1, 300)[i], lse=outs[i][1],
                                 workspace=ws[i], stream=stream)

    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
        outs[i][0].zero_(), outs[i][1].zero_()
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def test_a_workspace_too_small_is_refused(csa2):
    inp = [t.to(DEV) for t in _inputs(37, [100], [1], 4, 2, 64, 16)]
    need = csa2.csa2_paged_attn_fp4_workspace_bytes(1, 1, 4, 2, 64, 1)
    assert 0 < need <= 64 << 20
    with pytest.raises(csa2.Csa2Error) as e:
        csa2.csa2_paged_attn_fp4(*inp, torch.empty_like(inp[0]), 0.1, 1, workspace=torch.empty(need - 1, dtype=U8, device=DEV))
    assert e.value.status == 3


@pytest.mark.parametrize("D", [64, 128])
def test_row_tiles_that_fill_half_a_unit(csa2, D):
    """Units of 256 rows next to units of at most 128, many per CTA, whose last keys end inside a tile: every run of the call
    gives the same bits, and the first is right."""
    B, new, kv = 24, 96, [1100 + 37 * i for i in range(24)]
    inp = _inputs(40, kv, [new] * B, 32, 8, D, 32)
    dev = [t.to(DEV) for t in inp]
    runs = [(torch.zeros_like(dev[0]), torch.zeros(dev[0].shape[:2], device=DEV)) for _ in range(30)]
    for out, lse in runs:
        csa2.csa2_paged_attn_fp4(*dev, out, 0.1, new, lse=lse)
    torch.cuda.synchronize()
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    some = [0, 7, 23]                                                    # requests, for the reference
    rows = torch.cat([torch.arange(new) + new * b for b in some])
    part = [inp[0][rows], *inp[1:5], inp[5][some], inp[6][some], torch.tensor([0, new, 2 * new, 3 * new], dtype=I32)]
    out, lse = runs[0]
    paged_ref.check_attention(out[rows.to(DEV)], lse[rows.to(DEV)], _reference(part, 0.1))


# ---------------------------------------------------------------- together
def _serve(csa2, bits, S, dtype, graph, steps):
    """A serving loop with rotated rows: prompts, decoding, a request that ends and a new one in its place; every step checked."""
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    from sparse_attention_fp4_quantize_gb300.rope import Rope
    B, H, Hq, D, L, T = 4, 2, 6, 64, 2, 48
    rope = Rope(32, theta=1000.0, factor=2.0, original=64, first=16)
    cache = PagedCache(PagedShape(requests=B, tokens=T, max_context=160, n_blocks=40, heads=Hq, kv_heads=H, dim=D,
                                  block_size=S, layers=L, max_new=T, dtype=dtype, bits=bits, rope=rope))
    k, v = [torch.zeros(L, T, H, D, dtype=dtype, device=DEV) for _ in range(2)]
    q = torch.zeros(L, T, Hq, D, dtype=dtype, device=DEV)

    def step():
        cache.plan()
        for layer in range(L):
            cache.append(layer, k[layer], v[layer])
            cache.attend(layer, q[layer], window=0 if layer == 0 else 33)

    g = None
    if graph:
        step()                                                           # no new tokens yet: a step that changes nothing
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    gen = torch.Generator().manual_seed(S)
    n = cache.shape.n_blocks
    if bits == 4:
        held = [[np.zeros((n, H, S, w), np.uint8) for w in (D // 2, D // 2, D // 16, D // 16)] for _ in range(L)]
    else:
        held = [[f(sh) for f, sh in ((np.zeros, (n, H, S, D)),) * 2 + ((np.ones, (n, H)),) * 2] for _ in range(L)]
    plan = dict(kv_len=np.zeros(B), table=cache.block_table.cpu().numpy(), free_list=cache.free_list.cpu().numpy(),
                free_count=int(cache.free_count))
    news = [[20, 0, 5, 1], [1, 17, 1, 1], [1, 1, 1, 1], [1, 1, 1, 1], [-1, 1, 30, 1], [9, 1, 1, 1]][:steps]
    for new in news:
        cache.new_len.copy_(torch.tensor(new, dtype=I32))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen).to(dtype))
        step() if g is None else g.replay()
        torch.cuda.synchronize()
        plan = paged_ref.build_slots(plan["kv_len"], new, plan["table"], plan["free_list"], plan["free_count"], S, T)
        assert np.array_equal(cache.slots.cpu().numpy(), plan["slots"])
        rows = int(plan["cu"][-1])
        turn = lambda x: ref.rotate(x.cpu(), plan["positions"].tolist(), cache.cos_sin, 16, True)  # noqa: E731
        for layer in range(L):
            kr, vr, ksr, vsr = held[layer]
            qt, tb, win = turn(q[layer]), torch.from_numpy(plan["table"]), 0 if layer == 0 else 33
            if bits == 4:
                ref.store(turn(k[layer]).double().numpy(), plan["slots"], kr, ksr, S)
                ref.store(v[layer].double().cpu().numpy(), plan["slots"], vr, vsr, S)
                assert np.array_equal(cache.k_codes[layer].cpu().numpy(), kr) and np.array_equal(cache.v_scale[layer].cpu().numpy(), vsr)
                t = [torch.from_numpy(x) for x in (kr, ksr, vr, vsr)]
                want = ref.attention(qt, *t, tb, plan["kv_len"], plan["cu"], cache.sm_scale, win)
            else:
                paged_ref.append(turn(k[layer]).double().numpy(), plan["slots"], kr, ksr, S)
                paged_ref.append(v[layer].double().cpu().numpy(), plan["slots"], vr, vsr, S)
                t = [torch.from_numpy(x) for x in (kr, vr, ksr, vsr)]
                want = paged_ref.attention(qt.double(), *t, tb, plan["kv_len"], plan["cu"], cache.sm_scale, win)
            paged_ref.check_attention(cache.out[layer], cache.lse[layer], want, slice(0, rows))
    assert int(cache.err) == 0
    if bits == 4:                                                        # the stored rows of the last step, as they were given
        back, vals = [[torch.zeros(T, H, D, dtype=dtype, device=DEV) for _ in range(2)] for _ in range(2)]
        cache.read(1, cache.slots, *back)
        cache.append(1, k[1], v[1], k_values=vals[0], v_values=vals[1])
        torch.cuda.synchronize()
        assert torch.equal(back[0], vals[0]) and torch.equal(back[1], vals[1]) and back[0][:rows].any() and not back[0][rows:].any()
    return cache.out.clone(), cache.lse.clone()


@pytest.mark.parametrize("bits,S,dtype", [(4, 16, BF), (4, 64, F16), (8, 32, BF)])
def test_serving_loop(csa2, bits, S, dtype):
    out, lse = _serve(csa2, bits, S, dtype, False, 6)
    out2, lse2 = _serve(csa2, bits, S, dtype, True, 6)                    # captured and replayed: the same bits
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_steps_back_to_back_give_the_bits_of_steps_one_by_one(csa2):
    """A batch that decodes and takes a prompt chunk, every call directly behind the one that it reads from."""
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    from sparse_attention_fp4_quantize_gb300.rope import Rope
    B, H, Hq, D, L, T, steps = 8, 2, 16, 128, 2, 160, 24

    def run(sync):
        cache = PagedCache(PagedShape(requests=B, tokens=T, max_context=1024, n_blocks=B * 16, heads=Hq, kv_heads=H, dim=D,
                                      block_size=64, layers=L, max_new=100, bits=4, rope=Rope(128)))
        gen = torch.Generator(DEV).manual_seed(50)
        rows = [[torch.randn(T, n, D, generator=gen, device=DEV).to(BF) for n in (Hq, H, H)] for _ in range(steps)]
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

    apart = run(True)
    for _ in range(3):
        for a, b in zip(apart, run(False)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_request_that_waits_for_blocks_leaves_the_others_alone(csa2, bits):
    """Rows of a request that found no blocks have no position and are not stored; its tokens come again once another request
    has ended."""
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    from sparse_attention_fp4_quantize_gb300.rope import Rope
    H, Hq, D, S, T = 2, 4, 64, 16, 52
    cache = PagedCache(PagedShape(requests=2, tokens=T, max_context=64, n_blocks=3, heads=Hq, kv_heads=H, dim=D, block_size=S,
                                  max_new=32, bits=bits, rope=Rope(D)))
    gen = torch.Generator().manual_seed(62)
    for new, flag, there in (([32, 20], csa2.FLAG_NO_BLOCKS, 0), ([-1, 20], 0, 1)):
        q, k, v = [torch.randn(T, h, D, generator=gen).to(BF).to(DEV) for h in (Hq, H, H)]
        cache.err.zero_()
        cache.new_len.copy_(torch.tensor(new, dtype=I32))
        cache.plan()
        cache.append(0, k, v)
        out, lse = cache.attend(0, q)
        torch.cuda.synchronize()
        assert int(cache.err) == flag
        r0, n = int(cache.cu_len[there]), new[there]
        pos = torch.arange(n)
        assert cache.positions[r0:r0 + n].tolist() == pos.tolist()
        assert cache.slots.ge(0).sum() == n and cache.kv_len.tolist()[there] == n and cache.kv_len.tolist()[1 - there] == 0
        rows = slice(r0, r0 + n)
        turn = lambda x: ref.rotate(x[rows].cpu(), pos.tolist(), cache.cos_sin, 0, True)  # noqa: E731
        table, kv, cu = cache.block_table[there:there + 1].cpu(), torch.tensor([n], dtype=I32), [0, n]
        if bits == 4:
            t = [x[0].cpu() for x in (cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale)]
            want = ref.attention(turn(q), *t, table, kv, cu, cache.sm_scale)
            held = ref.values(t[0], t[1])[table[0, pos // S].long(), :, pos % S]
            assert np.array_equal(held, ref.quantise(turn(k).double().numpy())[2])
        else:
            t = [x[0].cpu().view(torch.float8_e4m3fn).double() for x in (cache.k_codes, cache.v_codes)]
            want = paged_ref.attention(turn(q).double(), *t, cache.k_scale[0].double().cpu(), cache.v_scale[0].double().cpu(), table, kv,
                                       cu, cache.sm_scale)
        paged_ref.check_attention(out[rows], lse[rows], want)


def test_the_extension_makes_the_usual_calls(csa2, monkeypatch):
    """Every call of the loop without the Python way to the library, in the bits of that way; what does not fit is refused there."""
    gen = torch.Generator().manual_seed(70)
    H, Hq, D, S, n, T = 2, 4, 64, 16, 6, 40
    table = torch.randn(T, D // 2, 2, generator=gen).to(DEV)
    q, k, v = [torch.randn(T, h, D, generator=gen).to(BF).to(DEV) for h in (Hq, H, H)]
    pos, slots = torch.arange(T, dtype=I32, device=DEV), torch.randperm(n * S, generator=gen)[:T].to(DEV)
    bt, kv, cu = torch.arange(n, dtype=I32, device=DEV)[None], torch.tensor([n * S], dtype=I32, device=DEV), torch.tensor([0, T], dtype=I32, device=DEV)
    ws = csa2.workspace_for_paged_attn_fp4(1, T, Hq, H, D, T)
    freq = torch.rand(D // 2, generator=gen, dtype=torch.float64).to(DEV)

    def calls():
        planes = [torch.zeros(n, H, S, w, dtype=U8, device=DEV) for w in (D // 2, D // 2, D // 16, D // 16)]
        made, qr, kb, vb, out = torch.empty_like(table), torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(k), torch.empty_like(q)
        csa2.csa2_rope_table(freq, made)
        csa2.csa2_rope(q, pos, made, q_out=qr)
        csa2.csa2_quantize_kv_fp4_paged(k, v, slots, *planes, pos=pos, cos_sin=table)
        csa2.csa2_dequantize_kv_fp4_paged(slots, *planes, kb, vb)
        csa2.csa2_paged_attn_fp4(qr, *planes, bt, kv, cu, out, 0.1, T, workspace=ws)
        torch.cuda.synchronize()
        return [made, qr, *planes, kb, vb, out]

    with monkeypatch.context() as m:
        m.setattr(csa2, "_lib", None)
        quick = calls()
        for bad in (pos[:-1], pos.long(), pos.cpu()):
            with pytest.raises((TypeError, ValueError, AttributeError)):
                csa2.csa2_rope(q, bad, table)
    with monkeypatch.context() as m:
        m.setattr(csa2, "_csa2_bind", type("Nothing", (), {"__getattr__": lambda self, name: lambda *a: None})())
        slow = calls()
    for a, b in zip(quick, slow):
        assert torch.equal(a, b)
    with pytest.raises(csa2.Csa2Error):
        csa2.csa2_rope(q, pos, table, first=8)                           # fits the call, and is refused behind it
