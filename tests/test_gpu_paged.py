"""The paged 8-bit cache on the GPU: slot maps, the quantising append and the
attention, each against its plain 64-bit reference, and a serving loop that
runs them together."""
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


# ---------------------------------------------------------------- slot maps
def _slots_state(rng, B, M, S, new, kv, spare):
    held = [-(-int(x) // S) for x in kv]
    cap = sum(held) + max(spare, 0) + sum(held[b] for b in range(B) if new[b] < 0) + 4
    ids = rng.permutation(sum(held) + max(spare, 0)).astype(np.int32)
    table = rng.integers(-9, -1, (B, M)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(cap, -7, np.int32)
    free[:ids.size - at] = ids[at:]
    return table, free, ids.size - at


def _run_slots(csa2, kv, new, table, free, count, S, T, in_place=False, positions=True, stride=0):
    t = lambda a: torch.tensor(np.asarray(a), dtype=I32, device=DEV)  # noqa: E731
    kv_d, new_d, free_d, count_d = t(kv), t(new), t(free), t([count])
    wide = torch.full((table.shape[0], table.shape[1] + stride), -3, dtype=I32, device=DEV)
    tab_d = wide[:, :table.shape[1]]
    tab_d.copy_(t(table))
    kv_o = kv_d if in_place else torch.full_like(kv_d, 77)
    count_o = count_d if in_place else torch.full_like(count_d, 77)
    cu = torch.full((len(kv) + 1,), 77, dtype=I32, device=DEV)
    pos = torch.full((T,), 77, dtype=I32, device=DEV) if positions else None
    slots = torch.full((T,), 77, dtype=torch.int64, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    csa2.csa2_build_slots(kv_d, new_d, tab_d, free_d, count_d, S, kv_o, count_o, cu, pos, slots, err_flag=err)
    torch.cuda.synchronize()
    assert (wide[:, table.shape[1]:] == -3).all()
    return dict(kv_len=kv_o.cpu().numpy(), cu=cu.cpu().numpy(), slots=slots.cpu().numpy(),
                positions=None if pos is None else pos.cpu().numpy(), table=tab_d.cpu().numpy(),
                free_list=free_d.cpu().numpy(), free_count=int(count_o), flags=int(err))


def _same(got, want):
    for k in want:
        if got[k] is not None:
            assert np.array_equal(got[k], want[k]), "%s differs" % k


SLOT_CASES = [  # B, M, S, T, spare blocks, kind
    (1, 1, 1, 1, 1, "decode"), (1, 4, 16, 70, 0, "prompt"), (1, 9, 7, 40, 9, "prompt"), (33, 17, 64, 33, 40, "decode"),
    (40, 12, 16, 300, 30, "mixed"), (257, 20, 48, 5000, 260, "mixed"), (1000, 33, 128, 20001, 500, "mixed"),
    (8192, 3, 16, 9000, 3000, "mixed"), (5, 6, 32, 3, 50, "prompt"), (64, 8, 16, 0, 64, "decode"),
]


@pytest.mark.parametrize("B,M,S,T,spare,kind", SLOT_CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_slots_match_a_stack(csa2, B, M, S, T, spare, kind, in_place):
    rng = np.random.default_rng(B * 31 + S)
    kv = rng.integers(0, M * S + 1, B)
    if kind == "decode":
        new = np.ones(B, np.int64)
    elif kind == "prompt":
        new = rng.integers(0, max(2, M * S), B)
    else:
        new = rng.choice([-5, -1, 0, 1, 1, 1, 2, 3 * S + 1], B)
    table, free, count = _slots_state(rng, B, M, S, new, kv, spare)
    want = ref.build_slots(kv, new, table, free, count, S, T)
    got = _run_slots(csa2, kv, new, table, free, count, S, T, in_place, positions=not in_place, stride=B % 3)
    _same(got, want)


def test_slots_take_the_blocks_that_end_in_the_same_step(csa2):
    kv, new = np.array([40, 0, 33]), np.array([-1, 64, 20])
    table = np.array([[5, 2, 9, -1], [-1] * 4, [1, 3, 8, -1]], np.int32)
    got = _run_slots(csa2, kv, new, table, np.full(8, -1, np.int32), 0, 16, 128)
    _same(got, ref.build_slots(kv, new, table, np.full(8, -1, np.int32), 0, 16, 128))
    assert got["flags"] == 0x10 and list(got["kv_len"]) == [0, 0, 33]      # three blocks are not enough for four
    new[1] = 40
    got = _run_slots(csa2, kv, new, table, np.full(8, -1, np.int32), 0, 16, 128)
    _same(got, ref.build_slots(kv, new, table, np.full(8, -1, np.int32), 0, 16, 128))
    assert list(got["table"][1, :3]) == [9, 2, 5] and got["free_count"] == 0


def test_slots_out_of_range_lengths_are_bounded_and_flagged(csa2):
    got = _run_slots(csa2, [-4, 999], [3, 1], np.array([[-1, -1], [6, 7]], np.int32), np.array([4, -2, 5, 9], np.int32),
                     99, 16, 8)
    # lengths act as 0 and 32, the count as 4: block 9 for the first, the second is full
    assert got["flags"] == 0x1 | 0x4
    assert list(got["kv_len"]) == [3, 32] and got["table"][0, 0] == 9 and got["free_count"] == 3
    assert list(got["slots"]) == [144, 145, 146] + [-1] * 5
    got = _run_slots(csa2, [0], [17], np.array([[-1, -1]], np.int32), np.array([4, -2], np.int32), 2, 16, 17)
    assert got["flags"] == 0x1 and list(got["slots"][:16]) == [-1] * 16 and got["slots"][16] == 64


def test_slots_feed_the_fp4_append(csa2):
    """The slot map is dst_slot of the FP4 quantiser: block size N on dense planes gives DecoderStep's append slots."""
    B, N, D = 5, 100, 576
    kl = torch.tensor([100, 7, 64, 1, 33], dtype=I32, device=DEV)
    table = torch.arange(B, dtype=I32, device=DEV)[:, None].contiguous()
    slots = torch.empty(B, dtype=torch.int64, device=DEV)
    cu = torch.empty(B + 1, dtype=I32, device=DEV)
    none = torch.zeros(1, dtype=I32, device=DEV)
    csa2.csa2_build_slots(kl - 1, torch.ones_like(kl), table, none, torch.zeros_like(none), N, torch.empty_like(kl),
                          torch.empty_like(none), cu, None, slots)
    want = torch.arange(B, device=DEV) * N + kl.long() - 1
    held = kl > 1                                   # a first token needs a block, and there is none to take
    assert torch.equal(slots[held], want[held]) and (slots[~held] == -1).all()
    rows = torch.randn(B, D, device=DEV).to(torch.bfloat16)
    codes, scales = torch.zeros(B * N, D // 2, dtype=torch.uint8, device=DEV), torch.zeros(B * N, D // 16, dtype=torch.uint8, device=DEV)
    csa2.csa2_quantize_kv_fp4(rows[held], codes, scales, dst_slot=slots[held])
    torch.cuda.synchronize()
    assert (scales.any(1).nonzero()[:, 0] == want[held].sort().values).all()


# ---------------------------------------------------------------- append
def _check_planes(planes, want_k, want_ks, want_v, want_vs):
    kc, vc, ks, vs = planes
    assert np.array_equal(ks.cpu().numpy().astype(np.float64), want_ks)
    assert np.array_equal(vs.cpu().numpy().astype(np.float64), want_vs)
    assert np.array_equal(ref.values_of(kc).numpy(), want_k)
    assert np.array_equal(ref.values_of(vc).numpy(), want_v)


def _append_both(csa2, k, v, slots, planes, S, flags=0):
    """Run the call and the reference on copies; all four tensors must be equal, bit for bit."""
    kc, vc, ks, vs = [p.clone() for p in planes]
    kr, vr = ref.values_of(kc).numpy().copy(), ref.values_of(vc).numpy().copy()
    ksr, vsr = ks.double().cpu().numpy().copy(), vs.double().cpu().numpy().copy()
    err = torch.zeros(1, dtype=I32, device=DEV)
    csa2.csa2_quantize_kv_fp8_paged(k, v, slots, kc, vc, ks, vs, err_flag=err)
    torch.cuda.synchronize()
    sl = slots.cpu().numpy()
    ref.append(k.double().cpu().numpy(), sl, kr, ksr, S)
    ref.append(v.double().cpu().numpy(), sl, vr, vsr, S)
    _check_planes((kc, vc, ks, vs), kr, ksr, vr, vsr)
    assert int(err) == flags
    return kc, vc, ks, vs


def _planes(seed, n, H, S, D):
    gen = torch.Generator().manual_seed(seed)
    kc, ks = ref.random_planes(gen, n, H, S, D)
    vc, vs = ref.random_planes(gen, n, H, S, D)
    return [t.to(DEV) for t in (kc, vc, ks, vs)]


def _request_slots(gen, starts, counts, S):
    """Slots of requests that hold `starts` tokens and bring `counts`, their blocks in random order, and the pool size."""
    held = [-(-(s + c) // S) for s, c in zip(starts, counts)]
    ids = torch.randperm(sum(held) + 2, generator=gen)
    slots, at = [], 0
    for s, c, m in zip(starts, counts, held):
        p = torch.arange(s, s + c)
        slots.append(ids[at + p // S] * S + p % S)
        at += m
    return torch.cat(slots), sum(held) + 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,D,S", [(1, 64, 16), (3, 128, 64), (8, 128, 32), (5, 64, 128), (2, 128, 128)])
def test_append_is_exact(csa2, dtype, H, D, S):
    gen = torch.Generator().manual_seed(H * 100 + S)
    starts, counts = [0, 1, S - 1, S, 3 * S + 5, 2, 0], [1, 1, 1, 2 * S + 3, 5 * S, 0, S]
    slots, n = _request_slots(gen, starts, counts, S)
    T = slots.numel() + 3                                              # padded rows behind the last request
    slots = torch.cat([slots, torch.full((3,), -1)]).to(DEV)
    size = torch.exp2(torch.randint(-12, 8, (T, H, 1), generator=gen).float())
    k = (torch.randn(T, H, D, generator=gen) * size).to(dtype).to(DEV)
    v = torch.randn(T, H, D, generator=gen).to(dtype).to(DEV)
    _append_both(csa2, k, v, slots, _planes(7, n, H, S, D), S)


def test_append_reads_slices_of_a_projection(csa2):
    gen = torch.Generator().manual_seed(4)
    H, D, S, T = 3, 64, 16, 50
    qkv = torch.randn(T, 10 * H * D + 8, generator=gen).to(torch.bfloat16).to(DEV)
    k = qkv[:, 8 * H * D:9 * H * D].view(T, H, D)
    v = qkv[:, 9 * H * D + 8:].view(T, D, H).transpose(1, 2)           # channels not contiguous: refused
    slots, n = _request_slots(gen, [3], [T], S)
    planes = _planes(1, n, H, S, D)
    with pytest.raises(ValueError):
        csa2.csa2_quantize_kv_fp8_paged(k, v, slots.to(DEV), *planes)
    v = qkv[:, 9 * H * D + 8:].view(T, H, D)
    _append_both(csa2, k, v, slots.to(DEV), planes, S)
    heads_first = torch.randn(H, T, D, generator=gen).to(torch.bfloat16).to(DEV).transpose(0, 1)
    _append_both(csa2, heads_first, v, slots.to(DEV), planes, S)
    one = qkv[:, :D].view(T, 1, D).expand(T, H, D)                     # one row for every head
    _append_both(csa2, one, v, slots.to(DEV), planes, S)


def test_append_token_by_token_keeps_what_is_stored(csa2):
    """A decoding request: rows arrive one by one and grow; every stored value stays within half a step of its row."""
    H, D, S = 2, 64, 16
    gen = torch.Generator().manual_seed(9)
    rows = torch.randn(S, H, D, generator=gen) * torch.exp2(torch.arange(S).float() / 2)[:, None, None]
    rows = rows.to(torch.bfloat16).to(DEV)
    planes = _planes(2, 3, H, S, D)
    for i in range(S):
        x = rows[i:i + 1]
        planes = _append_both(csa2, x, x, torch.tensor([S + i], device=DEV), planes, S)
    val = ref.values_of(planes[0])[1].transpose(0, 1) * planes[2][1].double().cpu()[None, :, None]
    step = planes[2][1].double().cpu()[None, :, None] * 2.0 ** -9        # E4M3's subnormal step, in values
    x = rows.double().cpu()
    # one rounding (2^-4), and at most one more per growth below the subnormal step, halving each time
    assert ((val - x).abs() <= 2.0 ** -4 * x.abs() + step).all()


def test_append_borders_of_the_scale(csa2):
    H, D, S = 1, 64, 16
    for dtype in (torch.bfloat16, torch.float16):
        tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
        big = torch.finfo(dtype).max
        for a in (0.0, 7.0, 7.0 * (1 + torch.finfo(dtype).eps), 448.0, 1.75, 3.5, 1.0, tiny, big, -big, 2.0 ** -14):
            x = torch.zeros(1, H, D, dtype=dtype)
            x[0, 0, 5], x[0, 0, 6] = a, a / 3
            x = x.to(DEV)
            _append_both(csa2, x, x, torch.tensor([16], device=DEV), _planes(3, 2, H, S, D), S)
            _append_both(csa2, x, x, torch.tensor([19], device=DEV), _planes(3, 2, H, S, D), S)


def test_append_infinities_and_nan_are_stored_finite_and_flagged(csa2):
    H, D, S = 2, 128, 32
    for dtype in (torch.bfloat16, torch.float16):
        k = torch.randn(5, H, D, generator=torch.Generator().manual_seed(1)).to(dtype)
        k[1, 0, 3], k[2, 0, 7], k[3, 0, 9] = float("inf"), float("-inf"), float("nan")
        k[:, 1] = float("nan")
        v = torch.randn(5, H, D, generator=torch.Generator().manual_seed(2)).to(dtype)
        kc, vc, _, _ = _append_both(csa2, k.to(DEV), v.to(DEV), torch.arange(34, 39, device=DEV), _planes(5, 3, H, S, D),
                                    S, flags=0x20)
        assert torch.isfinite(ref.values_of(kc)).all() and torch.isfinite(ref.values_of(vc)).all()


def test_append_bad_slots_are_skipped_and_flagged(csa2):
    H, D, S, n = 2, 64, 16, 4
    x = torch.randn(6, H, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    planes = _planes(6, n, H, S, D)
    for bad in ([n * S, -1, n * S + 5, 2 ** 40, -2, -2 ** 40], [3, 3, 3, 3, 3, 3], [5, 4, 3, 2, 1, 0], [0, 2, 3, 4, 20, 22]):
        kc, vc, ks, vs = [p.clone() for p in planes]
        err = torch.zeros(1, dtype=I32, device=DEV)
        csa2.csa2_quantize_kv_fp8_paged(x, x, torch.tensor(bad, device=DEV), kc, vc, ks, vs, err_flag=err)
        torch.cuda.synchronize()
        assert int(err) == 0x4
        keep = {3: [3], 5: [5], 0: [0, 20]}.get(bad[0], [])             # the first row of each run is stored
        touched = ((kc != planes[0]).any(-1).any(1).flatten().nonzero()[:, 0]).tolist()
        lead = [t for t in touched if t in keep]
        assert lead == keep
        assert all(any(t // S == k // S and t < k for k in keep) or t in keep for t in touched)   # others: re-encoded
    empty = [torch.zeros(0, H, S, D, dtype=torch.uint8, device=DEV)] * 2 + [torch.zeros(0, H, device=DEV)] * 2
    csa2.csa2_quantize_kv_fp8_paged(x[:0], x[:0], torch.empty(0, dtype=torch.int64, device=DEV), *planes)
    csa2.csa2_quantize_kv_fp8_paged(x, x, torch.full((6,), -1, device=DEV), *empty)
    torch.cuda.synchronize()


def test_cache_beyond_32_bit_offsets(csa2):
    """Planes of more than 2^31 bytes: append to and attend over the last blocks."""
    H, D, S = 8, 128, 128
    n = (1 << 31) // (H * S * D) + 40
    kc = torch.zeros(n, H, S, D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    ks, vs = torch.ones(n, H, device=DEV), torch.ones(n, H, device=DEV)
    gen = torch.Generator().manual_seed(11)
    T = 200
    k, v = [torch.randn(T, H, D, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2)]
    ids = torch.tensor([n - 1, n - 3], dtype=I32)
    p = torch.arange(T)
    slots = ids.long()[p // S] * S + p % S
    csa2.csa2_quantize_kv_fp8_paged(k, v, slots.to(DEV), kc, vc, ks, vs)
    table = ids[None].to(DEV).contiguous()
    q = torch.randn(3, 2 * H, D, generator=gen).to(torch.bfloat16).to(DEV)
    out, lse = torch.empty_like(q), torch.empty(3, 2 * H, device=DEV)
    kv, cu = torch.tensor([T], dtype=I32, device=DEV), torch.tensor([0, 3], dtype=I32, device=DEV)
    csa2.csa2_paged_attn_fp8(q, kc, vc, ks, vs, table, kv, cu, out, 0.1, 3, lse=lse)
    torch.cuda.synchronize()
    small = torch.tensor([[0, 1]], dtype=I32)
    pick = ids.long().to(DEV)
    kr, vr = np.zeros((2, H, S, D)), np.zeros((2, H, S, D))
    ksr, vsr = np.ones((2, H)), np.ones((2, H))
    sl = (p // S * S + p % S).numpy()
    ref.append(k.double().cpu().numpy(), sl, kr, ksr, S)
    ref.append(v.double().cpu().numpy(), sl, vr, vsr, S)
    _check_planes((kc[pick], vc[pick], ks[pick], vs[pick]), kr, ksr, vr, vsr)
    t = torch.from_numpy
    ref.check_attention(out, lse, ref.attention(q.double().cpu(), t(kr), t(vr), t(ksr), t(vsr), small, [T], [0, 3], 0.1))


# ---------------------------------------------------------------- attention
def _attn_inputs(seed, kv, new, Hq, H, D, S, dtype, spread=1.0, q_size=1.0):
    gen = torch.Generator().manual_seed(seed)
    table, n = ref.ragged(gen, kv, S)
    kc, ks = ref.random_planes(gen, n, H, S, D, spread)
    vc, vs = ref.random_planes(gen, n, H, S, D, spread)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=I32)
    q = (torch.randn(int(cu[-1]), Hq, D, generator=gen) * q_size).to(dtype)
    return q, kc, vc, ks, vs, table, torch.tensor(kv, dtype=I32), cu


def _attend(csa2, inp, sm, max_new, window=0, pad=0, err=None, **kw):
    q, kc, vc, ks, vs, table, kv, cu = [t.to(DEV) for t in inp]
    out = torch.full((q.shape[0] + pad, *q.shape[1:]), 9.0, dtype=q.dtype, device=DEV)
    lse = torch.full(out.shape[:2], 9.0, device=DEV)
    if pad:
        q = torch.cat([q, torch.full((pad, *q.shape[1:]), float("nan"), dtype=q.dtype, device=DEV)])
    csa2.csa2_paged_attn_fp8(q, kc, vc, ks, vs, table, kv, cu, out, sm, max_new, window=window, lse=lse, err_flag=err,
                             **kw)
    torch.cuda.synchronize()
    if pad:
        assert (out[-pad:] == 9.0).all() and (lse[-pad:] == 9.0).all()
    return out[:out.shape[0] - pad], lse[:lse.shape[0] - pad]


def _reference(inp, sm, window=0):
    q, kc, vc, ks, vs, table, kv, cu = inp
    return ref.attention(q.double(), ref.values_of(kc), ref.values_of(vc), ks.double(), vs.double(), table, kv, cu, sm,
                         window)


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
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,new,Hq,H,D,S,window", ATTN_CASES)
def test_attention_matches_reference(csa2, dtype, kv, new, Hq, H, D, S, window):
    inp = _attn_inputs(len(kv) * 7 + sum(kv), kv, new, Hq, H, D, S, dtype)
    sm = 1.0 / D ** 0.5 / 4
    err = torch.zeros(1, dtype=I32, device=DEV)
    want = _reference(inp, sm, window)
    out, lse = _attend(csa2, inp, sm, max(new), window, pad=3, err=err)
    ref.check_attention(out, lse, want)
    assert int(err) == 0
    again, lse2 = _attend(csa2, inp, sm, max(new), window)
    assert torch.equal(out, again) and torch.equal(lse, lse2)          # the same bits every time
    for hint in (1, 4 * max(new) + 100):                               # the hint changes the kernels, not the answer
        o, l = _attend(csa2, inp, sm, hint, window)
        ref.check_attention(o, l, want)


def test_rows_that_see_nothing(csa2):
    """No stored keys; more new rows than tokens (requests that wait): out 0, lse -inf."""
    for new in ([1, 3, 4], [1, 40, 60]):
        inp = _attn_inputs(3, [0, 1, 2], new, 4, 2, 64, 16, torch.bfloat16)
        out, lse = _attend(csa2, inp, 0.2, max(new))
        ref.check_attention(out, lse, _reference(inp, 0.2))
        dead = torch.tensor([0] + list(range(1, new[1])) + list(range(1 + new[1], sum(new) - 2)), device=DEV)
        assert (out[dead] == 0).all() and torch.isneginf(lse[dead]).all()


@pytest.mark.parametrize("new", [1, 50, 200])
def test_scales_far_apart_and_peaked_rows(csa2, new):
    """V scales over 2^+-20: a block that carries the softmax may hold values far below its neighbours'."""
    inp = list(_attn_inputs(21, [900], [new], 8, 2, 128, 64, torch.bfloat16, q_size=3.0))
    inp[4] = torch.exp2(torch.round(20 * torch.sin(torch.arange(inp[4].numel()).float())).reshape(inp[4].shape))
    q, kc, vc, ks, vs, table, kv, cu = inp
    for sm in (0.05, 1.0):
        out, lse = _attend(csa2, inp, sm, new)
        ref.check_attention(out, lse, _reference(inp, sm))
    inp[4] = torch.full_like(inp[4], 2.0 ** -126)
    inp[3] = torch.full_like(inp[3], 2.0 ** -126)
    out, lse = _attend(csa2, inp, 1.0, new)
    ref.check_attention(out, lse, _reference(inp, 1.0))


@pytest.mark.parametrize("new", [1, 60, 300])
def test_garbage_behind_the_last_token(csa2, new):
    """Rows at or beyond kv_len and unused blocks hold NaN codes and NaN scales."""
    S, kv = 64, [333]
    inp = list(_attn_inputs(5, kv, [new], 8, 2, 128, S, torch.float16))
    want = _reference(inp, 0.1)
    q, kc, vc, ks, vs, table, _, _ = inp
    last = int(table[0, 333 // S])
    kc[last, :, 333 % S:], vc[last, :, 333 % S:] = 0x7F, 0xFF
    used = set(table[0, :6].tolist())
    for b in range(kc.shape[0]):
        if b not in used:
            kc[b], vc[b], ks[b], vs[b] = 0x7F, 0x7F, float("nan"), float("inf")
    out, lse = _attend(csa2, inp, 0.1, new)
    ref.check_attention(out, lse, want)


@pytest.mark.parametrize("new", [1, 90])
def test_query_rows_do_not_meet(csa2, new):
    """A row of infinities or NaN spoils itself only; magnitudes far from one are exact or nearly."""
    inp = list(_attn_inputs(6, [400, 200], [new, new], 4, 2, 64, 32, torch.bfloat16))
    want = _reference(inp, 0.125)
    inp[0] = inp[0].clone()
    inp[0][0, 1], inp[0][new, 3] = float("nan"), float("inf")
    out, lse = _attend(csa2, inp, 0.125, new)
    ok = torch.ones(2 * new, 4, dtype=torch.bool)
    ok[0, 1] = ok[new, 3] = False
    ref.check_attention(out, lse, want, ok)
    for size in (1e-20, 1e15):
        x = list(inp)
        x[0] = (torch.randn(2 * new, 4, 64, generator=torch.Generator().manual_seed(1)) * size).to(torch.bfloat16)
        out, lse = _attend(csa2, x, 0.125 / size, new)
        ref.check_attention(out, lse, _reference(x, 0.125 / size))


def test_missing_blocks_hide_their_keys(csa2):
    for new in (1, 70):
        inp = list(_attn_inputs(8, [320], [new], 8, 2, 128, 64, torch.bfloat16))
        for bad in (-1, -2 ** 31, inp[1].shape[0], 2 ** 31 - 1):
            x = list(inp)
            x[5] = inp[5].clone()
            x[5][0, 1] = bad
            err = torch.zeros(1, dtype=I32, device=DEV)
            out, lse = _attend(csa2, x, 0.1, new, err=err)
            assert int(err) == 0x1
            y = list(inp)                      # the reference: the same request without that block's tokens
            y[5] = torch.cat([inp[5][:, :1], inp[5][:, 2:]], 1)
            y[6] = inp[6] - 64
            ref.check_attention(out, lse, _reference(y, 0.1))


def test_lengths_out_of_range_are_bounded(csa2):
    inp = list(_attn_inputs(9, [100, 90], [2, 3], 4, 2, 64, 16, torch.bfloat16))
    x = list(inp)
    x[6] = torch.tensor([2 ** 31 - 1, -5], dtype=I32)                    # as all of the table's tokens, and none
    x[5] = inp[5][:, :7].contiguous()
    full = list(x)
    full[6] = torch.tensor([112, 0], dtype=I32)
    out, lse = _attend(csa2, x, 0.1, 3)
    assert (out[2:] == 0).all() and torch.isneginf(lse[2:]).all()
    ref.check_attention(out, lse, _reference(full, 0.1))
    x = list(inp)
    x[7] = torch.tensor([-3, 2, 2 ** 30], dtype=I32)                     # first rows clamped to [0, T]
    out, lse = _attend(csa2, x, 0.1, 3)
    ref.check_attention(out, lse, _reference(inp, 0.1))


def test_strided_queries_tables_and_streams(csa2):
    inp = _attn_inputs(10, [500, 77], [3, 40], 8, 2, 128, 32, torch.bfloat16)
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
    csa2.csa2_paged_attn_fp8(fused[:, 2:10, :128], kc.view(torch.float8_e4m3fn), vc, ks, vs, wide[:, :table.shape[1]], kv,
                             cu, out, 0.1, 40, lse=lse, stream=side)
    side.synchronize()
    ref.check_attention(out, lse, want)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    out2 = torch.empty_like(q)
    csa2.csa2_paged_attn_fp8(heads_first, kc, vc, ks, vs, table, kv, cu, out2, 0.1, 40)       # without lse
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


# ---------------------------------------------------------------- together
def _serve(csa2, S, dtype, graph, steps):
    """A serving loop: prompts, decoding, a request that ends and a new one in its place; every step checked."""
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    B, H, Hq, D, L, T = 4, 2, 6, 64, 2, 48
    cache = PagedCache(PagedShape(requests=B, tokens=T, max_context=160, n_blocks=40, heads=Hq, kv_heads=H, dim=D,
                                  block_size=S, layers=L, max_new=T, dtype=dtype))
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
    shape = (cache.shape.n_blocks, H, S, D)
    kr = [np.zeros(shape) for _ in range(L)]
    vr = [np.zeros(shape) for _ in range(L)]
    ksr = [np.ones(shape[:2]) for _ in range(L)]
    vsr = [np.ones(shape[:2]) for _ in range(L)]
    plan = dict(kv_len=np.zeros(B), table=cache.block_table.cpu().numpy(), free_list=cache.free_list.cpu().numpy(),
                free_count=int(cache.free_count))
    news = [[20, 0, 5, 1], [1, 17, 1, 1], [1, 1, 1, 1], [1, 1, 1, 1], [-1, 1, 30, 1], [9, 1, 1, 1]][:steps]
    for new in news:
        cache.new_len.copy_(torch.tensor(new, dtype=I32))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen).to(dtype))
        if g is None:
            step()
        else:
            g.replay()
        torch.cuda.synchronize()
        plan = ref.build_slots(plan["kv_len"], new, plan["table"], plan["free_list"], plan["free_count"], S, T)
        assert np.array_equal(cache.block_table.cpu().numpy(), plan["table"])
        assert np.array_equal(cache.slots.cpu().numpy(), plan["slots"])
        assert np.array_equal(cache.positions.cpu().numpy(), plan["positions"])
        assert np.array_equal(cache.kv_len.cpu().numpy(), plan["kv_len"])
        rows = int(plan["cu"][-1])
        for layer in range(L):
            ref.append(k[layer].double().cpu().numpy(), plan["slots"], kr[layer], ksr[layer], S)
            ref.append(v[layer].double().cpu().numpy(), plan["slots"], vr[layer], vsr[layer], S)
            t = torch.from_numpy
            want = ref.attention(q[layer].double().cpu(), t(kr[layer]), t(vr[layer]), t(ksr[layer]), t(vsr[layer]),
                                 t(plan["table"]), plan["kv_len"], plan["cu"], cache.sm_scale, 0 if layer == 0 else 33)
            ref.check_attention(cache.out[layer], cache.lse[layer], want, slice(0, rows))
    assert int(cache.err) == 0
    return cache.out.clone(), cache.lse.clone()


@pytest.mark.parametrize("S,dtype", [(16, torch.bfloat16), (64, torch.float16)])
def test_serving_loop(csa2, S, dtype):
    out, lse = _serve(csa2, S, dtype, False, 6)
    out2, lse2 = _serve(csa2, S, dtype, True, 6)                          # captured and replayed: the same bits
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


# ---------------------------------------------------------------- more of the attention
@pytest.mark.parametrize("kv,new,Hq,H,D,S", [
    ([3000, 17], [1, 1], 16, 1, 128, 32),          # 16 rows per KV head, one token
    ([2000, 31], [1, 1], 32, 1, 64, 16),           # 32 rows: the tile kernel for single tokens
    ([900, 1, 450], [2, 1, 2], 24, 3, 64, 64),     # 8 and 16 rows of one call
    ([9000], [70], 2, 1, 64, 128),                 # a chunk behind a long prefix: parts joined over many CTAs
    ([9000], [33], 8, 1, 128, 64),
    ([129, 128, 127, 256, 257], [129, 128, 127, 256, 257], 1, 1, 128, 64),   # tile borders
    ([5000], [1], 3, 3, 64, 64),
])
def test_more_layouts(csa2, kv, new, Hq, H, D, S):
    for dtype in (torch.bfloat16, torch.float16):
        inp = _attn_inputs(sum(kv) + Hq, kv, new, Hq, H, D, S, dtype)
        out, lse = _attend(csa2, inp, 0.05, max(new))
        ref.check_attention(out, lse, _reference(inp, 0.05))


@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_grow_and_shrink(csa2, new, D):
    """Scores whose scale rises or falls block by block, V scales against them: references move often, or never."""
    for step in (0.5, -0.5, 3.0):
        inp = list(_attn_inputs(31, [1000], [new], 4, 1, D, 16, torch.bfloat16))
        at = torch.zeros(inp[3].shape[0])
        used = inp[5][0, :63].long()
        at[used] = torch.arange(63).float()
        if abs(step) < 1:
            inp[3] = torch.exp2(torch.round(step * at - 8 if step > 0 else step * at + 4)).clamp(2.0 ** -20, 2.0 ** 5)[:, None].contiguous()
        else:
            inp[3] = torch.full_like(inp[3], 2.0 ** -4)
            inp[4] = torch.exp2((step * at) % 41 - 20).round()[:, None].clamp(2.0 ** -20, 2.0 ** 20).contiguous()
        for sm in (0.02, 0.3):
            out, lse = _attend(csa2, inp, sm, new)
            ref.check_attention(out, lse, _reference(inp, sm))


@pytest.mark.parametrize("new", [1, 50])
def test_sign_and_zero_of_the_scale(csa2, new):
    inp = list(_attn_inputs(32, [700], [new], 4, 2, 64, 64, torch.float16))
    for sm in (-0.2, 0.0):
        out, lse = _attend(csa2, inp, sm, new)
        ref.check_attention(out, lse, _reference(inp, sm))
    inp[3], inp[4] = torch.zeros_like(inp[3]), torch.zeros_like(inp[4])       # a cache of zero scales: every value 0
    out, lse = _attend(csa2, inp, 0.2, new)
    ref.check_attention(out, lse, _reference(inp, 0.2))


def test_many_short_requests(csa2):
    rng = np.random.default_rng(5)
    kv = rng.integers(0, 50, 700)
    new = np.minimum(rng.choice([0, 1, 1, 1, 2, 30], 700), kv)
    inp = _attn_inputs(33, list(kv), list(new), 4, 2, 64, 16, torch.bfloat16)
    for hint in (1, 30):
        out, lse = _attend(csa2, inp, 0.1, hint, pad=1)
        ref.check_attention(out, lse, _reference(inp, 0.1))


def test_a_cache_without_blocks(csa2):
    q = torch.randn(3, 4, 64, device=DEV).to(torch.bfloat16)
    planes = [torch.empty(0, 2, 16, 64, dtype=torch.uint8, device=DEV)] * 2 + [torch.empty(0, 2, device=DEV)] * 2
    table = torch.full((2, 3), -1, dtype=I32, device=DEV)
    for kv, flag in ([0, 0], 0), ([5, 0], 1):
        for hint in (1, 100):
            out, lse = torch.full_like(q, 3.0), torch.full((3, 4), 3.0, device=DEV)
            err = torch.zeros(1, dtype=I32, device=DEV)
            csa2.csa2_paged_attn_fp8(q, *planes, table, torch.tensor(kv, dtype=I32, device=DEV),
                                     torch.tensor([0, 2, 3], dtype=I32, device=DEV), out, 0.1, hint, lse=lse, err_flag=err)
            torch.cuda.synchronize()
            assert (out == 0).all() and torch.isneginf(lse).all() and int(err) == flag


def test_calls_on_two_streams_and_in_two_graphs(csa2):
    """Calls that overlap have a workspace each; a graph replayed between eager calls gives the eager bits."""
    a = _attn_inputs(34, [4000, 300], [1, 1], 8, 1, 128, 64, torch.bfloat16)
    b = _attn_inputs(35, [600, 900], [300, 200], 8, 2, 128, 32, torch.bfloat16)
    want = [_attend(csa2, x, 0.1, n) for x, n in ((a, 1), (b, 300))]
    dev = [[t.to(DEV) for t in x] for x in (a, b)]
    outs = [(torch.zeros_like(w[0]), torch.zeros_like(w[1])) for w in want]
    ws = [csa2.workspace_for_paged_attn(2, x[0].shape[0], 8, x[1].shape[1], 128, n) for x, n in ((a, 1), (b, 300))]

    def call(i, stream=None):
        q, kc, vc, ks, vs, table, kv, cu = dev[i]
        csa2.csa2_paged_attn_fp8(q, kc, vc, ks, vs, table, kv, cu, outs[i][0], 0.1, (1, 300)[i], lse=outs[i][1],
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


def test_append_in_windows_of_many_rows(csa2):
    """Enough rows that a warp looks at a window of them: runs that begin inside, end behind and span windows."""
    H, D, S, T = 4, 64, 16, 9000
    gen = torch.Generator().manual_seed(12)
    counts = [1] * 40 + [5] * 30 + [S] * 20 + [S + 1] * 20 + [7000]
    starts = [(7 * i) % (2 * S) for i in range(len(counts))]
    slots, n = _request_slots(gen, starts, counts, S)
    slots = torch.cat([slots, torch.full((T - slots.numel(),), -1)]).to(DEV)
    k = torch.randn(T, H, D, generator=gen).to(torch.bfloat16).to(DEV)
    v = torch.randn(T, H, D, generator=gen).to(torch.bfloat16).to(DEV)
    _append_both(csa2, k, v, slots, _planes(13, n, H, S, D), S)


@pytest.mark.parametrize("D,S", [(128, 16), (128, 32), (128, 128), (64, 64), (64, 128)])
def test_append_runs_taken_together_and_dealt_out(csa2, D, S):
    """Calls of so many rows that a window holds 64: whole blocks, which the warps take together, next to short
    runs, which they share out; longer than a warp's and a window's loads; with infinities and NaN in both."""
    H, T = 8, 5000
    gen = torch.Generator().manual_seed(D + S)
    counts = [1] * 70 + [3 * S + 1] + [S] * 6 + [2, S - 1] * 6
    starts = [(5 * i) % S for i in range(len(counts))]
    starts[-1] = 0
    slots, n = _request_slots(gen, starts + [0], counts + [T - sum(counts)], S)
    k = torch.randn(T, H, D, generator=gen).to(torch.bfloat16)
    v = torch.randn(T, H, D, generator=gen).to(torch.bfloat16) * 2.0 ** 5
    planes = _planes(21, n, H, S, D)
    _append_both(csa2, k.to(DEV), v.to(DEV), slots.to(DEV), planes, S)
    for r in (3, 75, 75 + S, T - 1):
        k[r, 1, 5], v[r, 2, 7], v[r, 2, 9] = float("nan"), float("inf"), float("-inf")
    _append_both(csa2, k.to(DEV), v.to(DEV), slots.to(DEV), planes, S, flags=0x20)


def test_workspace_belongs_to_the_stream_that_uses_it(csa2, monkeypatch):
    inp = _attn_inputs(36, [900, 40], [1, 1], 8, 2, 128, 64, torch.bfloat16)
    want, _ = _attend(csa2, inp, 0.1, 1)
    dev, side, made = [t.to(DEV) for t in inp], torch.cuda.Stream(), []
    real = csa2.workspace_for_paged_attn
    monkeypatch.setattr(csa2, "workspace_for_paged_attn", lambda *a, **k: made.append(torch.cuda.current_stream()) or real(*a, **k))
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, None):
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        q, kc, vc, ks, vs, table, kv, cu = dev
        csa2.csa2_paged_attn_fp8(q, kc, vc, ks, vs, table, kv, cu, out, 0.1, 1, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert [s.cuda_stream for s in made] == [side.cuda_stream, side.cuda_stream, torch.cuda.current_stream().cuda_stream]


@pytest.mark.parametrize("D", [64, 128])
def test_row_tiles_that_fill_half_a_unit(csa2, D):
    """Units of 256 rows next to units of at most 128, many per CTA, whose last keys end inside a tile: every run
    of the call gives the same bits, and the first is right."""
    B, new, kv = 24, 96, [1100 + 37 * i for i in range(24)]
    inp = _attn_inputs(40, kv, [new] * B, 32, 8, D, 32, torch.bfloat16)
    q, kc, vc, ks, vs, table, kvl, cu = dev = [t.to(DEV) for t in inp]
    runs = [(torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)) for _ in range(30)]
    for out, lse in runs:
        csa2.csa2_paged_attn_fp8(*dev, out, 0.1, new, lse=lse)
    torch.cuda.synchronize()
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    some = [0, 7, 23]                                                  # requests, for the reference
    rows = torch.cat([torch.arange(new) + new * b for b in some])
    part = (inp[0][rows], kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), table.cpu()[some], kvl.cpu()[some],
            torch.tensor([0, new, 2 * new, 3 * new], dtype=I32))
    for out, lse in (runs[0], runs[-1]):
        ref.check_attention(out[rows.to(DEV)], lse[rows.to(DEV)], _reference(part, 0.1))


@pytest.mark.parametrize("kv,new,Hq,H,D,S,window", [
    ([900, 70, 33], [5, 7, 8], 8, 2, 64, 16, 0),                       # 20, 28 and 32 rows per KV head: several row tiles
    ([900, 70, 33], [5, 7, 8], 8, 2, 128, 64, 90),
    ([4000, 1], [1, 1], 17, 1, 128, 32, 0),
    ([500, 31, 200], [1, 1, 1], 64, 2, 64, 64, 0),                     # 32 heads of a group
    ([500, 260, 31], [1, 250, 2], 20, 1, 128, 64, 0),                  # next to a prompt and to 40 rows
    ([500, 260, 31], [1, 250, 2], 33, 1, 64, 32, 0),                   # one token's rows are too many already
])
def test_rows_of_several_row_tiles(csa2, kv, new, Hq, H, D, S, window):
    inp = _attn_inputs(41, kv, new, Hq, H, D, S, torch.bfloat16)
    out, lse = _attend(csa2, inp, 0.08, max(new), window, pad=2)
    ref.check_attention(out, lse, _reference(inp, 0.08, window))
