"""Plain references of the paged 8-bit cache, in Python integers and 64-bit
floats, written request by request and block by block (no prefix sums, no
shared code with the kernels), and the error bounds of the GPU results.

Bounds.  A rounding is off by at most half a step of its type, eps / 2
relative.  For one output element out = sum_j w_j v_j / sum_j w_j with
A = sum_j w_j |v_j| / sum_j w_j:
  * the weights are rounded to f16 before the product: 2^-11 A, and weights
    in f16's subnormal range by at most 2^-25 of the largest: n 2^-25 max|v|
  * a logit is a sum of D products accumulated in fp32, then scaled (three
    more roundings): |dz| <= (D + 8) 2^-24 Z with Z = sm_scale sum_d |q_d k_d|;
    numerator and denominator each move by a factor e^|dz|, and the exponential
    itself by 2^-21: 2 (|dz| + 2^-21) A
  * sums over n keys in fp32: 2 (n + 64) 2^-24 A
  * the result is rounded to q's type: eps / 2 of |out| and of its error.
The log-sum-exp moves by |dz| + 2^-21 + (n + 64) 2^-24 and two roundings of its
own size.
"""
from __future__ import annotations

import math

import numpy as np
import torch

MIN_SCALE = 2.0 ** -126


# ---------------------------------------------------------------- slot maps
def build_slots(kv_len, new_len, table, free_list, free_count, S, T):
    """One step, request by request on a real stack.  Lists and numpy arrays in, a dict out."""
    B, M = table.shape
    table, free = table.copy(), free_list.copy()
    kv_len, new_len = [int(x) for x in kv_len], [int(x) for x in new_len]
    stack = [int(x) for x in free_list[:free_count]]
    for b in range(B):
        if new_len[b] < 0:
            stack += [int(x) for x in table[b, : -(-kv_len[b] // S)]]
    kv_out, cu, slots, pos = [], [0], np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    flags, rows, wanted = 0, 0, 0
    total = len(stack)
    for b in range(B):
        n, kv = new_len[b], kv_len[b]
        if n < 0:
            kv_out.append(0)
        elif n == 0:
            kv_out.append(kv)
        else:
            first, rows = rows, rows + n
            need = -(-(kv + n) // S) - -(-kv // S)
            ok = True
            if rows > T or kv + n > M * S:
                ok, flags = False, flags | 0x4
            else:
                wanted += need                       # waiting requests hold their place in the queue
                if need and wanted > total:
                    ok, flags = False, flags | 0x10
            if ok:
                for page in range(-(-kv // S), -(-(kv + n) // S)):
                    table[b, page] = stack.pop()
                for i in range(n):
                    p = kv + i
                    slots[first + i] = int(table[b, p // S]) * S + p % S
                    pos[first + i] = p
            kv_out.append(kv + n if ok else kv)
        cu.append(min(rows, T))
    if len(stack) > free_count:
        free[free_count:len(stack)] = stack[free_count:]
    return dict(kv_len=np.array(kv_out, np.int32), cu=np.array(cu, np.int32), slots=slots, positions=pos, table=table,
                free_list=free, free_count=len(stack), flags=flags)


# ---------------------------------------------------------------- append
def e4m3(x):
    """Nearest E4M3 value (ties to even) of finite |x| <= 448, 64-bit arithmetic."""
    a = np.abs(x)
    _, e = np.frexp(a)
    step = np.exp2(np.clip(e - 1, -6, 8) - 3.0)
    return np.copysign(np.rint(a / step) * step, x)


def need_of(amax):
    if amax == 0:
        return MIN_SCALE
    m, e = math.frexp(amax / 448.0)
    return max(MIN_SCALE, math.ldexp(1.0, e - 1 if m == 0.5 else e))


def append(x, slots, values, scale, S):
    """Rows x [T, H, D] (float64) into values [n, H, S, D] (what the codes stand for) and scale [n, H], in place."""
    i, T = 0, len(slots)
    while i < T:
        if slots[i] < 0:
            i += 1
            continue
        blk, off = divmod(int(slots[i]), S)
        n = 1
        while i + n < T and slots[i + n] == slots[i] + n and (slots[i] + n) // S == blk:
            n += 1
        rows = x[i:i + n].transpose(1, 0, 2)
        for h in range(x.shape[1]):
            fin = np.where(np.isfinite(rows[h]), np.abs(rows[h]), 0.0)
            s = need_of(float(fin.max()))
            if off:
                s = max(s, float(scale[blk, h]))
                if s != scale[blk, h]:
                    values[blk, h, :off] = e4m3(values[blk, h, :off] * (scale[blk, h] / s))
            scale[blk, h] = s
            r = np.where(np.isnan(rows[h]), 0.0, np.clip(rows[h], -448.0 * s, 448.0 * s)) / s
            values[blk, h, off:off + n] = e4m3(r)
        i += n


# ---------------------------------------------------------------- attention
def attention(q, k_val, v_val, k_scale, v_scale, table, kv_len, cu, sm_scale, window=0):
    """out, lse in 64 bits and their bounds (before q's type's own rounding), [T, Hq, D] and [T, Hq].  k_val, v_val:
    the codes' values [n, H, S, D]; all float64 torch tensors on the CPU."""
    T, Hq, D = q.shape
    H, S = k_val.shape[1], k_val.shape[2]
    G = Hq // H
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    for b in range(len(kv_len)):
        kv, c0, c1 = int(kv_len[b]), int(cu[b]), int(cu[b + 1])
        if c1 <= c0 or kv <= 0:
            continue
        pages = table[b, : -(-kv // S)].long()
        k = (k_val[pages] * k_scale[pages][..., None, None]).transpose(0, 1).reshape(H, -1, D)[:, :kv]
        v = (v_val[pages] * v_scale[pages][..., None, None]).transpose(0, 1).reshape(H, -1, D)[:, :kv]
        p = kv - (c1 - c0) + torch.arange(c1 - c0)
        j = torch.arange(kv)
        seen = j <= p[:, None]
        if window > 0:
            seen &= j > p[:, None] - window
        seen = seen[None].expand(G, -1, -1)
        for h in range(H):
            x = q[c0:c1, h * G:(h + 1) * G].transpose(0, 1)                   # [G, n, D]
            z = (x @ k[h].T * sm_scale).masked_fill(~seen, -math.inf)
            zabs = (x.abs() @ k[h].abs().T * abs(sm_scale)).masked_fill(~seen, 0.0).amax(-1)
            some = seen.any(-1)
            w = torch.where(some[..., None], torch.softmax(z, -1), torch.zeros_like(z))
            o, A = w @ v[h], w @ v[h].abs()
            n = seen.sum(-1).double()
            dz = (D + 8) * 2.0 ** -24 * zabs + 2.0 ** -21
            to = A * (2.0 ** -11 + 2 * dz + 2 * (n + 64) * 2.0 ** -24)[..., None]
            to = to + (n * 2.0 ** -25)[..., None] * v[h].abs().amax()
            ls = torch.where(some, torch.logsumexp(z, -1), torch.full_like(n, -math.inf))
            tl = dz + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * torch.where(some, ls.abs(), torch.zeros_like(n))
            out[c0:c1, h * G:(h + 1) * G], tol_o[c0:c1, h * G:(h + 1) * G] = o.transpose(0, 1), to.transpose(0, 1)
            lse[c0:c1, h * G:(h + 1) * G], tol_l[c0:c1, h * G:(h + 1) * G] = ls.T, tl.T
    return out, lse, tol_o, tol_l


def check_attention(out, lse, ref, rows=None):
    """GPU out (bf16 / fp16) and lse (fp32) against attention()'s answer; rows: those that count."""
    o, l, to, tl = ref
    half = torch.finfo(out.dtype).eps / 2
    sel = slice(None) if rows is None else rows
    got = out.double().cpu()[sel]
    o, l, to, tl = o[sel], l[sel], to[sel], tl[sel]
    tiny = torch.finfo(out.dtype).tiny * torch.finfo(out.dtype).eps        # the type's subnormal step
    tol = to + half * (o.abs() + to) + tiny
    err = (got - o).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), "out: worst err / bound %.3g" % float((err / tol).max())
    if lse is not None:
        gl = lse.double().cpu()[sel]
        none = torch.isinf(l)
        assert (torch.isneginf(gl) == none).all()
        el = (gl - l)[~none].abs()
        assert (el <= tl[~none]).all(), "lse: worst err / bound %.3g" % float((el / tl[~none]).max())


# ---------------------------------------------------------------- inputs
def values_of(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def random_planes(gen, n, H, S, D, spread=1.0):
    """Codes (no NaN) and power-of-two scales whose exponents spread over a few steps."""
    x = torch.randn(n, H, S, D, generator=gen)
    codes = (x * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.exp2(torch.round(torch.randn(n, H, generator=gen) * spread) - 5)
    return codes, scale


def ragged(gen, kv, S, extra=2):
    """A block table for the lengths kv, its blocks in random order in a pool with some to spare, and the pool's size."""
    held = [-(-int(x) // S) for x in kv]
    n = sum(held) + extra
    ids = torch.randperm(n, generator=gen).int()
    table, at = torch.full((len(held), max(held + [1]) + 1), -1, dtype=torch.int32), 0
    for b, m in enumerate(held):
        table[b, :m] = ids[at:at + m]
        at += m
    return table, n
