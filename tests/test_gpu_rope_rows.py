"""Rotary positions on the GPU: the table against arithmetic of more than 64 bits, the rotation bit for bit."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32
BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def csa2():
    import sparse_attention_fp4_quantize_gb300 as lib
    return lib


# ---------------------------------------------------------------- the table
def _turns(freq, p):
    """p * freq / (2 pi) modulo 1, in whole numbers: freq is a fraction of two, 1 / (2 pi) has 200 bits."""
    inv = (1 << 200) * 10 ** 60 // 6283185307179586476925286766559005768394338798750211641949889
    n, d = float(freq).as_integer_ratio()
    x = p * n * inv // d                                                 # in 2^-200 turns
    return (x % (1 << 200)) / (1 << 200) if x >= 0 else 1 - (-x % (1 << 200)) / (1 << 200)


def _check_table(got, freq, start, amp, rows):
    """|error| <= amp (6 2^-24 |v| + 2^-50 + 2 pi (start + n) 2^-64): the reduced angle's rounding to fp32 and its share of
    the value (2^-24), the two functions' 2 units in the last place (2 2^-23), the amplitude's product (2^-24), their
    sum rounded up; the fixed-point frequency's rounding times the position; double's own cosine here."""
    got = got.double().cpu().numpy()
    for n in rows:
        for i in range(len(freq)):
            t = _turns(freq[i], start + n)
            q = round(4 * t)
            a = 2 * math.pi * (t - q / 4)                               # |a| <= pi / 4, so both functions keep their leading bits
            c, s = math.cos(a), math.sin(a)
            c, s = [(c, s), (-s, c), (-c, -s), (s, -c)][q % 4]
            for g, v in zip(got[n, i], (amp * c, amp * s)):
                tol = 6 * 2.0 ** -24 * abs(v) + abs(amp) * (2.0 ** -50 + 2 * math.pi * (start + n) * 2.0 ** -64)
                assert abs(g - v) <= tol, (n, i, g, v)


@pytest.mark.parametrize("half,n_pos,start,amp", [(1, 1, 0, 1.0), (32, 300, 0, 1.0), (64, 100, 1 << 20, 1.25), (5, 1000, 12345, -0.5),
                                                  (200, 40, (1 << 31) - 40, 1.0), (512, 3, 77, 2.0), (300, 20, 5, 1.0)])
def test_table_matches_exact_angles(csa2, half, n_pos, start, amp):
    f = 1e6 ** (-np.arange(half) / half) * 1.0000001
    out = torch.full((n_pos + 1, half, 2), 9.0, device=DEV)
    csa2.csa2_rope_table(torch.from_numpy(f).to(DEV), out[:n_pos], start=start, amplitude=amp)
    torch.cuda.synchronize()
    assert (out[n_pos] == 9.0).all()
    _check_table(out, f, start, amp, sorted({0, n_pos // 3, n_pos // 2, n_pos - 1}))


def test_table_of_odd_frequencies(csa2):
    """Whole turns, quarter turns, negative, tiny, large; those that are none give NaN and leave the others alone."""
    f = np.array([0.0, math.pi, math.pi / 2, -0.37, 1e-12, -3e-15, 1e-300, 1048576.0, 777777.7, 2 * math.pi, 1e-9, 2.0 ** -31])
    x = np.concatenate([f, [math.nan, math.inf, -math.inf, 1048577.0, -1e300]])
    out = torch.empty(200, x.size, 2, device=DEV)
    csa2.csa2_rope_table(torch.from_numpy(x).to(DEV), out, start=1000)
    torch.cuda.synchronize()
    _check_table(out[:, :f.size], f, 1000, 1.0, (0, 1, 2, 3, 199))
    assert torch.isnan(out[:, f.size:]).all()


def test_stretched_table_of_the_class(csa2):
    from sparse_attention_fp4_quantize_gb300.rope import Rope
    rope = Rope(128, theta=5e5, factor=16.0, original=8192)
    f, amp = rope.frequencies()
    t = rope.table(131072)
    assert t.shape == (131072, 64, 2)
    _check_table(t, f.numpy(), 0, amp, (0, 1, 4095, 77777, 131071))
    assert torch.equal(rope.table(1000, start=70000), t[70000:71000])    # a part of it, bit for bit


# ---------------------------------------------------------------- the rotation
def _case(seed, T, Hq, Hk, D, dim, dtype, n_pos=50):
    gen = torch.Generator().manual_seed(seed)
    q, k = [(torch.randn(T, H, D, generator=gen) * 3).to(dtype).to(DEV) for H in (Hq, Hk)]
    a = torch.rand(n_pos, dim // 2, generator=gen) * 7
    table = torch.stack([a.cos(), a.sin()], -1).to(DEV)
    return q, k, torch.randint(0, n_pos, (T,), generator=gen).int().to(DEV), table


def _same(a, b):
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("T,Hq,Hk,D,dim,first", [
    (1, 1, 0, 64, 64, 0), (1, 64, 8, 128, 128, 0), (7, 3, 1, 64, 16, 48), (33, 5, 2, 80, 32, 8), (130, 8, 8, 96, 96, 0),
    (5, 32, 4, 128, 64, 64), (1000, 6, 2, 128, 48, 16), (9, 1, 1, 1024, 1024, 0), (3, 2, 1, 1016, 16, 1000), (4096, 20, 5, 128, 128, 0),
    (2, 300, 100, 16, 16, 0),
])
def test_rotation_is_exact(csa2, dtype, half, T, Hq, Hk, D, dim, first):
    q, k, pos, table = _case(T + D, T, Hq, Hk, D, dim, dtype)
    layout = csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED
    pc = pos.tolist()
    want_q, want_k = ref.rotate(q.cpu(), pc, table, first, half).to(DEV), ref.rotate(k.cpu(), pc, table, first, half).to(DEV)
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    err = torch.zeros(1, dtype=I32, device=DEV)
    csa2.csa2_rope(q, pos, table, k=k if Hk else None, q_out=qo, k_out=ko if Hk else None, first=first, layout=layout, err_flag=err)
    torch.cuda.synchronize()
    _same(qo, want_q)
    _same(ko, want_k)
    csa2.csa2_rope(q, pos, table, k=k if Hk else None, first=first, layout=layout, err_flag=err)      # in place
    torch.cuda.synchronize()
    _same(q, want_q)
    _same(k, want_k)
    assert int(err) == 0


def test_rows_without_a_position_are_left_as_they_were(csa2):
    q, k, pos, table = _case(1, 40, 4, 2, 64, 64, BF)
    pos[3], pos[17], pos[39] = -1, -1, -1
    for bad, flag in ((None, 0), (50, 1), (-2, 1), (2 ** 31 - 1, 1), (-2 ** 31, 1)):
        x = pos.clone()
        if bad is not None:
            x[8] = bad
        qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
        err = torch.zeros(1, dtype=I32, device=DEV)
        csa2.csa2_rope(q, x, table, k=k, q_out=qo, k_out=ko, err_flag=err)
        torch.cuda.synchronize()
        out = ((x < 0) | (x >= 50)).nonzero()[:, 0]
        assert int(err) == flag and (qo[out] == 9.0).all() and (ko[out] == 9.0).all()
        some = ((x >= 0) & (x < 50)).nonzero()[:, 0].cpu()
        _same(qo[some.to(DEV)], ref.rotate(q[some.to(DEV)].cpu(), x.cpu()[some].tolist(), table, 0, True).to(DEV))


def test_slices_of_a_projection_and_other_strides(csa2):
    T, Hq, Hk, D = 77, 6, 2, 64
    q, k, pos, table = _case(2, T, Hq, Hk, D, 32, F16)
    pc = pos.tolist()
    want_q, want_k = [ref.rotate(x.cpu(), pc, table, 8, True).to(DEV) for x in (q, k)]
    qkv = torch.zeros(T, Hq + 2 * Hk, D, dtype=F16, device=DEV)
    qkv[:, :Hq], qkv[:, Hq:Hq + Hk] = q, k
    qo = torch.zeros(Hq, T, D + 8, dtype=F16, device=DEV)                # heads first, gaps between rows
    csa2.csa2_rope(qkv[:, :Hq], pos, table, k=qkv[:, Hq:Hq + Hk], q_out=qo.transpose(0, 1)[..., :D], first=8)
    torch.cuda.synchronize()
    _same(qo.transpose(0, 1)[..., :D].contiguous(), want_q)
    assert (qo[..., D:] == 0).all() and (qkv[:, Hq + Hk:] == 0).all()
    _same(qkv[:, Hq:Hq + Hk].contiguous(), want_k)                       # in place, between the others
    _same(qkv[:, :Hq].contiguous(), q)
    csa2.csa2_rope(qkv[:, :Hq], pos, table, first=8)
    _same(qkv[:, :Hq].contiguous(), want_q)
    one = q[:, :1].expand(T, Hq, D)                                      # one head for all, written out
    out = torch.zeros_like(q)
    csa2.csa2_rope(one, pos, table, q_out=out, first=8)
    for h in range(Hq):
        _same(out[:, h].contiguous(), want_q[:, 0].contiguous())
    with pytest.raises(csa2.Csa2Error):
        csa2.csa2_rope(one, pos, table, first=8)                         # in place it would turn six times


def test_infinities_nan_and_ends_of_the_type(csa2):
    for dtype in (BF, F16):
        q, _, pos, table = _case(3, 4, 2, 1, 64, 64, dtype)
        big = torch.finfo(dtype).max
        q[0, 0, 3], q[0, 0, 40], q[1, 1, 5], q[2, 0, 1], q[2, 0, 33] = math.inf, math.nan, -math.inf, big, big
        q[3, 0] = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
        want = ref.rotate(q.cpu(), pos.tolist(), table, 0, True)
        csa2.csa2_rope(q, pos, table)
        torch.cuda.synchronize()
        got = q.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(got[fine], want[fine])


def test_the_fp4_entries_take_the_table(csa2):
    """csa2_rope_quantize_kv_fp4 on a table made here = csa2_rope, then csa2_quantize_kv_fp4: the same bytes."""
    R, D = 300, 576
    gen = torch.Generator().manual_seed(5)
    rows = torch.randn(R, D, generator=gen).to(BF).to(DEV)
    from sparse_attention_fp4_quantize_gb300.rope import Rope
    table = Rope(64, factor=4.0).table(5000)
    pos = torch.randint(0, 5000, (R,), generator=gen).int().to(DEV)
    planes = [[torch.zeros(R, D // 2, dtype=torch.uint8, device=DEV), torch.zeros(R, D // 16, dtype=torch.uint8, device=DEV)] for _ in range(2)]
    csa2.csa2_rope_quantize_kv_fp4(rows, pos, table, *planes[0])
    turned = torch.empty_like(rows)
    csa2.csa2_rope(rows[:, None], pos, table, q_out=turned[:, None], first=D - 64, layout=csa2.ROPE_INTERLEAVED)
    csa2.csa2_quantize_kv_fp4(turned, *planes[1])
    torch.cuda.synchronize()
    assert torch.equal(planes[0][0], planes[1][0]) and torch.equal(planes[0][1], planes[1][1])


def test_rotation_in_a_graph_and_on_another_stream(csa2):
    q, k, pos, table = _case(6, 64, 8, 2, 128, 128, BF)
    want = ref.rotate(q.cpu(), pos.tolist(), table, 0, True).to(DEV)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    csa2.csa2_rope(q, pos, table, q_out=out, stream=side)
    side.synchronize()
    _same(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa2.csa2_rope(q, pos, table, q_out=out)
    q2 = torch.randn_like(q)
    q.copy_(q2)
    pos.copy_((pos + 1) % 50)
    g.replay()
    torch.cuda.synchronize()
    _same(out, ref.rotate(q2.cpu(), pos.tolist(), table, 0, True).to(DEV))


def test_table_in_parts_on_another_stream_and_in_a_graph(csa2):
    """A table filled in two parts has the bits of one filled at once; captured and replayed with other frequencies."""
    n, half = 700, 48
    f = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(DEV)
    whole, parts = [torch.zeros(n, half, 2, device=DEV) for _ in range(2)]
    csa2.csa2_rope_table(f, whole, start=1 << 30, amplitude=1.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    csa2.csa2_rope_table(f, parts[:333], start=1 << 30, amplitude=1.5, stream=side)
    csa2.csa2_rope_table(f, parts[333:], start=(1 << 30) + 333, amplitude=1.5, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(whole, parts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa2.csa2_rope_table(f, parts)
    f.copy_(f.flip(0).clone())
    g.replay()
    csa2.csa2_rope_table(f, whole)
    torch.cuda.synchronize()
    assert torch.equal(whole, parts) and (parts[0] == torch.tensor([1.0, 0.0], device=DEV)).all()


def test_rows_beyond_32_bit_offsets(csa2):
    """Token strides that put the last row past 2^32 bytes."""
    T, D, step = 3, 64, (1 << 30) + 8
    buf = torch.zeros(2 * step + D, dtype=BF, device=DEV)
    q = buf.as_strided((T, 1, D), (step, D, 1))
    x, _, pos, table = _case(7, T, 1, 1, D, D, BF)
    q.copy_(x)
    csa2.csa2_rope(q, pos, table)
    torch.cuda.synchronize()
    _same(q.contiguous(), ref.rotate(x.cpu(), pos.tolist(), table, 0, True).to(DEV))
