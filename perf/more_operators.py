"""What is measured of the paged 4-bit cache: the rotary positions of its rows, its quantising append, the reading back
of what it holds and the attention over it.

Each case is one call of one operator as a serving loop makes it.  The plain form computes the same from elementary
torch operations; with ``own`` set the framework's operators are called.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

GROUP = 16                       # channels that share a scale
E4M3_MAX = 448.0
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)                    # E2M1 magnitudes by code


def _dt(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def listed():
    return [
        # the table of a small model with half of a head rotated, made when it is loaded
        dict(name="table-4k", op="table", n_pos=4096, half=32, factor=1.0),
        # a context stretched eightfold
        dict(name="table-long-scaled", op="table", n_pos=262144, half=64, factor=8.0),
        # a decode step: one token of each of 64 requests
        dict(name="rope-decode-64", op="rope", dtype="bf16", tokens=64, heads=64, kv_heads=8, dim=128, rope_dim=128, first=0,
             half=True, fused=True),
        # prompts of several requests: q and k are slices of one projection's output
        dict(name="rope-prompt-16k", op="rope", dtype="bf16", tokens=16384, heads=32, kv_heads=8, dim=128, rope_dim=128,
             first=0, half=True, fused=True),
        # a decode step's append with the keys' rotation
        dict(name="append-decode-64", op="append", dtype="bf16", requests=64, tokens=64, heads=8, dim=128, block=64,
             kind="decode", fused=False, rope_dim=128, first=0, half=True),
        # a prompt chunk whose attention reads the values that later steps will see, rotated keys among them
        dict(name="append-prompt-16k", op="append", dtype="bf16", requests=9, tokens=16384, heads=8, dim=128, block=64,
             kind="prompt", fused=True, rope_dim=128, first=0, half=True),
        # the prefix of one request, small heads, an odd number of them, fp16
        dict(name="read-prefix-fp16", op="read", dtype="fp16", requests=1, tokens=1501, heads=5, dim=64, block=16),
        # the caches of many requests moved to another place
        dict(name="read-64k", op="read", dtype="bf16", requests=24, tokens=65536, heads=8, dim=128, block=64),
        # one user, one token, a short context: latency
        dict(name="attn-decode-1", op="attn", dtype="bf16", requests=1, new=1, context=1000, heads=32, kv_heads=8,
             dim=128, block=64, window=0, kind="decode"),
        # the decode step of a served batch with ragged contexts
        dict(name="attn-decode-64", op="attn", dtype="bf16", requests=64, new=1, context=16384, heads=64, kv_heads=8,
             dim=128, block=64, window=0, kind="decode"),
        # several draft tokens per request, sliding window, small heads and blocks, fp16
        dict(name="attn-draft-window-fp16", op="attn", dtype="fp16", requests=48, new=5, context=9001, heads=15,
             kv_heads=5, dim=64, block=16, window=4096, kind="decode"),
        # prompts of a ragged batch on top of cached prefixes
        dict(name="attn-prompt-8k", op="attn", dtype="bf16", requests=3, new=4096, context=8192, heads=32, kv_heads=8,
             dim=128, block=64, window=0, kind="prompt"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng, dim):
    rope_dim = 16 * rng.randint(1, dim // 16)
    return dict(rope_dim=rope_dim, first=8 * rng.randint(0, (dim - rope_dim) // 8), half=rng.choice([True, True, False]))


def draw(rng):
    op = rng.choice(["table", "rope", "append", "read", "attn", "attn", "attn"])
    if op == "table":
        half = 4 * rng.randint(1, 32)
        return dict(op=op, n_pos=_log(rng, 1, 262144 * 64 // max(half, 64)), half=half, factor=rng.choice([1.0, 2.0, 8.0, 32.0]))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    dim, block = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    fused = rng.choice([True, False])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        kv_heads, group = rng.randint(0, 8), rng.choice([1, 2, 3, 4, 5, 7])
        heads = max(1, kv_heads) * group
        most = 16384 * 40 * 128 // ((heads + kv_heads) * dim)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, min(most, 65536)), heads=heads, kv_heads=kv_heads, dim=dim,
                    fused=fused, **_draw_rope(rng, dim))
    heads = rng.randint(1, 8)
    if op == "append":
        kind = rng.choice(["decode", "mixed", "prompt"])
        requests = _log(rng, 1, 256)
        tokens = requests if kind == "decode" else _log(rng, max(requests, 16), 16384)
        rope = _draw_rope(rng, dim) if rng.random() < 0.75 else dict(rope_dim=0, first=0, half=True)
        return dict(op=op, dtype=dtype, requests=requests, tokens=tokens, heads=heads, dim=dim, block=block, kind=kind,
                    fused=fused, **rope)
    if op == "read":
        requests = _log(rng, 1, 64)
        return dict(op=op, dtype=dtype, requests=requests, tokens=_log(rng, requests, 65536), heads=heads, dim=dim, block=block)
    kind = rng.choice(["decode", "decode", "prompt", "mixed"])
    kv_heads, group = heads, rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if kind != "decode":
        group = min(group, 4)
    window = rng.choice([0, 0, 0, _log(rng, 16, 8192)])
    if kind == "decode":
        requests = _log(rng, 1, 64)
        context = _log(rng, 1, min(131072, (64 * 16384) // requests))
        new = rng.choice([1, 1, 1, 2, 5])
    elif kind == "prompt":
        requests = rng.randint(1, 3)
        context = _log(rng, 16, 8192)
        new = max(1, min(4096, int(context * rng.uniform(0.3, 1.0))))
    else:                                  # a prompt's chunk next to requests that decode
        requests = rng.randint(2, 17)
        context = _log(rng, 64, 12000)
        new = max(1, min(512, int(context * rng.uniform(0.1, 1.0))))
    return dict(op=op, dtype=dtype, requests=requests, new=new, context=context, heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, block=block, window=window, kind=kind)


# ---------------------------------------------------------------- the format, in 32 bits
def _unpacked(codes):
    """The codes of bytes [.., n], low nibble first: [.., 2 n]."""
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def _values(codes, scales):
    """What codes [.., D/2] and scales [.., D/16] stand for, fp32 [.., D]."""
    c = _unpacked(codes)
    e, m = (c >> 1) & 3, (c & 1).float()
    mag = torch.where(e > 0, torch.exp2(e.float() - 1) * (1 + 0.5 * m), 0.5 * m)
    mag = torch.where(c >= 8, -mag, mag)
    s = scales.view(torch.float8_e4m3fn).float()
    return (mag.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _quantised(x):
    """Rows x [.., D] fp32: codes [.., D/2], scales [.., D/16], both bytes.  The scale of 16 channels is a sixth of their
    largest magnitude as E4M3, a code the nearest multiple of it, ties to the even code."""
    g = x.unflatten(-1, (-1, GROUP))
    s8 = (g.abs().amax(-1) / 6).clamp_max(E4M3_MAX).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    r = (g / torch.where(s > 0, s, torch.ones_like(s))).abs() * (s > 0)
    c = ((r > 0.25).byte() + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5)) | (torch.signbit(g).byte() << 3)
    c = c.flatten(-2).unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4), s8.view(torch.uint8)


# ---------------------------------------------------------------- inputs
def _frequencies(half, theta, factor, dtype=torch.float64):
    """theta^(-i / half); with a factor, the slow pairs (less than one turn in 4096 positions) slowed down by it, the fast
    ones (32 and more) not, those between in part."""
    f = theta ** (-torch.arange(half, dtype=dtype) / half)
    turns = 4096 * f / (2 * math.pi)
    fast = ((turns - 1) / 31).clamp(0, 1)
    return f * fast + f / factor * (1 - fast)


def _cos_sin(n_pos, half, theta=10000.0):
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * _frequencies(half, theta, 1.0).cuda()
    return torch.stack([a.cos(), a.sin()], -1).float()


def _prepare_table(case, seed):
    rng = np.random.default_rng(seed)
    f = _frequencies(case["half"], float(rng.uniform(1e4, 1e6)), case["factor"]).cuda()
    return dict(inv_freq=f, start=int(rng.integers(0, 1 << 20)), amplitude=0.1 * math.log(case["factor"]) + 1.0,
                n_pos=case["n_pos"], table=torch.zeros(case["n_pos"], case["half"], 2, device="cuda"))


def _positions(rng, tokens, most):
    """Positions of a step's tokens: runs of requests, each behind what it already holds."""
    runs = max(1, min(tokens, 1 + tokens // 64))
    cuts = np.sort(rng.choice(np.arange(1, tokens), runs - 1, replace=False)) if runs > 1 else np.array([], np.int64)
    n = np.diff(np.concatenate([[0], cuts, [tokens]]))
    start = rng.integers(0, most - n.max(), n.size)
    return np.repeat(start, n) + np.arange(tokens) - np.repeat(np.cumsum(n) - n, n)


N_POS = 131072                   # rows of the prepared tables


def _prepare_rope(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    x = torch.randn(T, H + 2 * K, D, generator=gen, device="cuda").to(_dt(case))
    q, k = (x[:, :H], x[:, H:H + K]) if case["fused"] else (x[:, :H].contiguous(), x[:, H:H + K].contiguous())
    pos = torch.tensor(_positions(rng, T, N_POS), dtype=torch.int32, device="cuda")
    k = k if K else None
    return dict(q=q, k=k, pos=pos, cos_sin=_cos_sin(N_POS, case["rope_dim"] // 2), first=case["first"], half=case["half"],
                q_out=torch.zeros(T, H, D, dtype=x.dtype, device="cuda"),
                k_out=torch.zeros(T, K, D, dtype=x.dtype, device="cuda") if K else None)


def _split(rng, total, parts):
    """`total` into `parts` positive whole numbers."""
    cuts = np.sort(rng.choice(np.arange(1, total), parts - 1, replace=False)) if parts > 1 else np.array([], np.int64)
    return np.diff(np.concatenate([[0], cuts, [total]])).astype(np.int64)


def _token_counts(case, rng):
    """New tokens per request that fill the case's token budget, by its kind."""
    B, T = case["requests"], case["tokens"]
    if case["kind"] == "decode":
        return np.ones(B, np.int64)
    if case["kind"] == "prompt":
        return _split(rng, max(B, T - T // 16), B)
    n = np.ones(B, np.int64)               # mixed: every eighth request brings a prompt chunk
    many = np.arange(B) % 8 == 0
    room = T - B
    if room > 0:
        n[many] += rng.multinomial(int(room * 0.9), np.full(int(many.sum()), 1.0 / many.sum()))
    return n


def _rows(gen, T, H, D, dtype, fused):
    """Post-projection rows: heads of unequal size, a few large channels."""
    size = torch.exp(0.5 * torch.randn(H, 1, generator=gen, device="cuda"))
    hot = torch.where(torch.rand(H, D, generator=gen, device="cuda") < 0.02, 6.0, 1.0)
    if fused:                              # slices of one projection's output
        x = torch.randn(T, 4 * H, D, generator=gen, device="cuda")
        x[:, 2 * H:3 * H] *= size * hot
        x = x.to(dtype)
        return x[:, 2 * H:3 * H], x[:, 3 * H:]
    k = (torch.randn(T, H, D, generator=gen, device="cuda") * size * hot).to(dtype)
    return k, torch.randn(T, H, D, generator=gen, device="cuda").to(dtype)


def _planes(gen, n, H, S, D):
    """A cache of n blocks with rows in it: codes and scales of the keys, of the values."""
    u8 = dict(dtype=torch.uint8, device="cuda")
    kc, ks = torch.empty(n, H, S, D // 2, **u8), torch.empty(n, H, S, D // GROUP, **u8)
    vc, vs = torch.empty_like(kc), torch.empty_like(ks)
    for at in range(0, n, 2048):           # in pieces: the cache in fp32 would be large
        m = min(2048, n - at)
        for t, c, s in zip(_rows(gen, m * S, H, D, torch.float32, False), (kc, vc), (ks, vs)):
            c[at:at + m], s[at:at + m] = _quantised(t.view(m, S, H, D).transpose(1, 2).contiguous())
    return dict(k_codes=kc, v_codes=vc, k_scales=ks, v_scales=vs)


def _slots(rng, start, n, S, blocks):
    """Slots of requests that hold `start` tokens and bring n, in blocks of any order, and the blocks that they take."""
    held = -(-(start + n) // S)
    ids = rng.permutation(blocks)
    first = np.cumsum(held) - held
    req = np.repeat(np.arange(n.size), n)
    pos = np.arange(int(n.sum())) - np.repeat(np.cumsum(n) - n, n) + start[req]
    return ids[first[req] + pos // S] * S + pos % S, pos


def _prepare_append(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    B, S, H, D, T = case["requests"], case["block"], case["heads"], case["dim"], case["tokens"]
    n = _token_counts(case, rng)
    start = rng.integers(0, 2 * S, B)      # tokens that each request already holds
    if case["kind"] == "prompt":
        start[rng.random(B) < 0.7] = 0
    at, pos = _slots(rng, start, n, S, T // S + 4 * B + 3)
    slots = np.full(T, -1, np.int64)
    slots[: at.size] = at
    where = np.full(T, -1, np.int32)
    where[: at.size] = pos
    dt = _dt(case)
    k, v = _rows(gen, T, H, D, dt, case["fused"])
    return dict(k=k, v=v, slots=torch.tensor(slots, device="cuda"), pos=torch.tensor(where, device="cuda"),
                cos_sin=_cos_sin(N_POS, case["rope_dim"] // 2) if case["rope_dim"] else None, first=case["first"],
                half=case["half"], k_values=torch.zeros(T, H, D, dtype=dt, device="cuda"),
                v_values=torch.zeros(T, H, D, dtype=dt, device="cuda"), **_planes(gen, T // S + 4 * B + 3, H, S, D))


def _prepare_read(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    B, S, H, D, T = case["requests"], case["block"], case["heads"], case["dim"], case["tokens"]
    blocks = T // S + B + 3
    at, _ = _slots(rng, np.zeros(B, np.int64), _split(rng, T, B), S, blocks)
    k = torch.zeros(T, H, D, dtype=_dt(case), device="cuda")
    return dict(slots=torch.tensor(at, device="cuda"), k=k, v=torch.zeros_like(k), **_planes(gen, blocks, H, S, D))


def _new_tokens(case):
    """New tokens per request: by the case alone, as they set the number of rows."""
    B, n = case["requests"], min(case["new"], case["context"])
    if case["kind"] == "decode":
        return np.full(B, n)
    rng = np.random.default_rng(B * 1000003 + n)
    new = rng.integers(max(1, n // 2), n + 1, B)
    new[0] = n
    if case["kind"] == "mixed":            # every sixteenth request brings a prompt chunk
        new[1:] = np.where(np.arange(1, B) % 16 == 0, new[1:], 1)
    return new


def _lengths(case, rng):
    """(tokens in the cache with the new ones, new tokens) per request."""
    B, C, new = case["requests"], case["context"], _new_tokens(case)
    kv = np.maximum(new, rng.integers(max(1, C // (8 if case["kind"] == "decode" else 2)), C + 1, B))
    kv[0] = max(C, int(new[0]))
    return kv, new


def _prepare_attn(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    S, H, D, B = case["block"], case["kv_heads"], case["dim"], case["requests"]
    kv, new = _lengths(case, rng)
    held = -(-kv // S)
    nb = int(held.sum())
    table = np.full((B, int(held.max()) + 2), -1, np.int32)
    row = np.repeat(np.arange(B), held)
    table[row, np.arange(nb) - np.repeat(np.cumsum(held) - held, held)] = rng.permutation(nb)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    q = torch.randn(T, case["heads"], D, generator=gen, device="cuda").to(_dt(case))
    return dict(q=q, table=torch.tensor(table, device="cuda"), kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                cu_len=torch.tensor(cu, dtype=torch.int32, device="cuda"), out=torch.zeros_like(q),
                lse=torch.zeros(T, case["heads"], device="cuda"), sm_scale=1.0 / math.sqrt(D), window=case["window"],
                max_new=int(new.max()), kv_max=int(kv.max()), **_planes(gen, nb, H, S, D),
                workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))   # kept by a serving loop


def prepare(case, seed):
    st = {"table": _prepare_table, "rope": _prepare_rope, "append": _prepare_append, "read": _prepare_read,
          "attn": _prepare_attn}[case["op"]](case, seed)
    st["op"] = case["op"]
    return st


# ---------------------------------------------------------------- plain forms
def _plain_table(st):
    p = st["start"] + torch.arange(st["n_pos"], dtype=torch.float64, device="cuda")
    a = p[:, None] * st["inv_freq"]
    return (st["amplitude"] * torch.stack([a.cos(), a.sin()], -1)).float()


def _rotated(x, pos, cos_sin, first, half):
    """Rows x [T, H, D] with the pairs of their rotated channels turned; every product and sum rounded to 32 bits, the
    result to x's type.  Rows without a position are as they were."""
    n = cos_sin.shape[1]
    c, s = cos_sin[pos.long().clamp_min(0)][:, None].unbind(-1)
    y = x[..., first:first + 2 * n].float()
    a, b = (y[..., :n], y[..., n:]) if half else (y[..., 0::2], y[..., 1::2])
    u, w = a * c - b * s, a * s + b * c
    y = torch.cat([u, w], -1) if half else torch.stack([u, w], -1).flatten(-2)
    y = torch.cat([x[..., :first], y.to(x.dtype), x[..., first + 2 * n:]], -1)
    return torch.where((pos >= 0)[:, None, None], y, x)


def _plain_rope(st):
    turn = lambda x: _rotated(x, st["pos"], st["cos_sin"], st["first"], st["half"])  # noqa: E731
    return dict(q=turn(st["q"]), k=turn(st["k"]) if st["k"] is not None else None)


def _plain_append(st):
    S = st["k_codes"].shape[2]
    at = torch.nonzero(st["slots"] >= 0)[:, 0]
    b, r = st["slots"][at] // S, st["slots"][at] % S
    k = _rotated(st["k"], st["pos"], st["cos_sin"], st["first"], st["half"]) if st["cos_sin"] is not None else st["k"]
    kc, ks = _quantised(k[at].float())
    vc, vs = _quantised(st["v"][at].float())
    st["k_codes"][b, :, r], st["k_scales"][b, :, r] = kc, ks
    st["v_codes"][b, :, r], st["v_scales"][b, :, r] = vc, vs
    st["k_values"][at], st["v_values"][at] = _values(kc, ks).to(k.dtype), _values(vc, vs).to(k.dtype)
    return _append_out(st)


def _append_out(st):
    """The values that the stored rows stand for, and the planes.  Which code and scale a row gets is laid down to the
    bit, so packed codes are compared as the whole numbers that they are."""
    f8 = torch.float8_e4m3fn
    return dict(k_values=st["k_values"], v_values=st["v_values"], k_codes=st["k_codes"], v_codes=st["v_codes"],
                k_scales=st["k_scales"].view(f8), v_scales=st["v_scales"].view(f8))


def _plain_read(st):
    S = st["k_codes"].shape[2]
    b, r = st["slots"] // S, st["slots"] % S
    dt = st["k"].dtype
    return dict(k=_values(st["k_codes"][b, :, r], st["k_scales"][b, :, r]).to(dt),
                v=_values(st["v_codes"][b, :, r], st["v_scales"][b, :, r]).to(dt))


def _gathered(codes, scales, pages):
    """The rows of every request, [B, H, n * S, D] fp32."""
    x = _values(codes[pages], scales[pages])
    B, n, H, S, D = x.shape
    return x.transpose(1, 2).reshape(B, H, n * S, D)


def _plain_attn(st):
    q, S = st["q"], st["k_codes"].shape[2]
    H, D = st["k_codes"].shape[1], q.shape[2]
    G = q.shape[1] // H
    B, n = st["kv_len"].numel(), st["max_new"]
    dev = q.device
    pages = st["table"][:, : -(-st["kv_max"] // S)].long().clamp_min(0)
    k = _gathered(st["k_codes"], st["k_scales"], pages)
    kv, cu = st["kv_len"].long(), st["cu_len"].long()
    i = torch.arange(n, device=dev)
    count = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp_max(q.shape[0] - 1)
    x = q[row].float().view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    z = torch.matmul(x, k.transpose(2, 3)) * st["sm_scale"]
    del k
    p = (kv - count)[:, None] + i                                       # position of each new token
    j = torch.arange(z.shape[-1], device=dev)
    seen = (j <= p[..., None]) & (j < kv[:, None, None]) & (i < count[:, None])[..., None]
    if st["window"] > 0:
        seen &= j > p[..., None] - st["window"]
    z.view(B, H, G, n, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    w = z.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    v = _gathered(st["v_codes"], st["v_scales"], pages)
    v = torch.where((j < kv[:, None])[:, None, :, None], v, torch.zeros_like(v))   # nothing of unwritten rows
    o = torch.matmul(w, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    real = i < count[:, None]
    o = o.view(B, H, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D)[real]
    lse = lse.view(B, H, G, n).permute(0, 3, 1, 2).reshape(B, n, H * G)[real]
    return dict(out=o.to(q.dtype), lse=lse)


# ---------------------------------------------------------------- the framework's operators
def _own_table(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_rope_table(st["inv_freq"], st["table"], start=st["start"], amplitude=st["amplitude"])
    return st["table"]


def _layout(csa2, st):
    return csa2.ROPE_HALF if st["half"] else csa2.ROPE_INTERLEAVED


def _own_rope(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_rope(st["q"], st["pos"], st["cos_sin"], k=st["k"], q_out=st["q_out"], k_out=st["k_out"], first=st["first"],
                   layout=_layout(csa2, st))
    return dict(q=st["q_out"], k=st["k_out"])


def _own_append(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_quantize_kv_fp4_paged(st["k"], st["v"], st["slots"], st["k_codes"], st["v_codes"], st["k_scales"],
                                    st["v_scales"], pos=st["pos"] if st["cos_sin"] is not None else None,
                                    cos_sin=st["cos_sin"], first=st["first"], layout=_layout(csa2, st),
                                    k_values=st["k_values"], v_values=st["v_values"])
    return _append_out(st)


def _own_read(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_dequantize_kv_fp4_paged(st["slots"], st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], st["k"],
                                      st["v"])
    return dict(k=st["k"], v=st["v"])


def _own_attn(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_paged_attn_fp4(st["q"], st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], st["table"],
                             st["kv_len"], st["cu_len"], st["out"], st["sm_scale"], st["max_new"], window=st["window"],
                             lse=st["lse"], workspace=st["workspace"])
    return dict(out=st["out"], lse=st["lse"])


def run(state):
    if own:
        return {"table": _own_table, "rope": _own_rope, "append": _own_append, "read": _own_read,
                "attn": _own_attn}[state["op"]](state)
    return {"table": _plain_table, "rope": _plain_rope, "append": _plain_append, "read": _plain_read,
            "attn": _plain_attn}[state["op"]](state)


# ---------------------------------------------------------------- work
def _seen(kv, new, window):
    """Visible (new token, key) pairs, and the keys that some new token sees, per request."""
    kv, new = kv.astype(np.float64), new.astype(np.float64)
    first = kv - new + 1                   # keys that the first new token sees
    if window <= 0:
        return new * (first + kv) / 2, kv
    full = np.clip(kv - np.maximum(first, window) + 1, 0, None)                   # tokens with a full window
    short = new - full
    return short * first + short * (short - 1) / 2 + full * window, np.minimum(kv, window + new - 1)


def work(case):
    """One pass's bytes and operations; of the attention at the mean of the lengths that `prepare` draws."""
    if case["op"] == "table":
        n = case["n_pos"] * case["half"]
        return {"bytes": 8 * n + 8 * case["half"], "flops": 20 * n}
    D = case["dim"]
    held = 2 * (D / 2 + D / GROUP)         # bytes of a token's keys and values of one head
    if case["op"] == "rope":
        rows = case["tokens"] * (case["heads"] + case["kv_heads"])
        table = min(case["tokens"], N_POS) * case["rope_dim"] * 4
        return {"bytes": 4 * rows * D + 4 * case["tokens"] + table, "flops": 3 * rows * case["rope_dim"]}
    if case["op"] == "append":
        T = float(_token_counts(case, np.random.default_rng(0)).sum())
        table = (4 + 4 * case["rope_dim"]) * T if case["rope_dim"] else 0
        return {"bytes": T * case["heads"] * (8 * D + held) + 8 * case["tokens"] + table,
                "flops": T * case["heads"] * (8 * D + 3 * case["rope_dim"])}
    if case["op"] == "read":
        return {"bytes": case["tokens"] * (case["heads"] * (4 * D + held) + 8), "flops": 2 * case["tokens"] * case["heads"] * D}
    pairs = keys = rows = 0.0
    for seed in range(4):
        kv, new = _lengths(case, np.random.default_rng(seed))
        p, k = _seen(kv, new, case["window"])
        pairs, keys, rows = pairs + p.sum() / 4, keys + k.sum() / 4, rows + new.sum() / 4
    return {"bytes": float(keys * case["kv_heads"] * held + rows * case["heads"] * (4 * D + 4)),
            "flops": float(4.0 * pairs * case["heads"] * D)}


# ---------------------------------------------------------------- in 64 bits
def _exact_values(codes, scales):
    table = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=codes.device)
    lo, hi = table[(codes % 16).int()], table[(codes // 16).int()]
    v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    v[..., 0::2], v[..., 1::2] = lo, hi
    return v * scales.view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, -1)


def _nearest(x, grid):
    """The nearest of the grid's values (ascending, its even places the even codes) to each x >= 0, ties to the even one."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.bucketize(x, mid)                             # x <= mid[i]: place i, or a tie with the next
    tie = (i < mid.numel()) & (x == mid[i.clamp_max(mid.numel() - 1)])
    return grid[torch.where(tie & (i % 2 == 1), i + 1, i)]


def _exact_quantised(x):
    """(values, scales) of rows x [.., D] in 64 bits."""
    dev = x.device
    e4m3 = torch.arange(0, 127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    s = _nearest(g.abs().amax(-1) / 6, e4m3)
    q = torch.where(s[..., None] > 0, g / s[..., None], torch.zeros_like(g))
    v = _nearest(q.abs(), torch.tensor(GRID, dtype=torch.float64, device=dev)) * s[..., None]
    return torch.where(g < 0, -v, v).reshape(x.shape), s


def _exact_rotated(x, pos, cos_sin, first, half):
    """Each product and sum in 64 bits, rounded to 32: their values, as 24 + 24 bits and more fit 53."""
    n = cos_sin.shape[1]
    r = lambda t: t.float().double()  # noqa: E731
    y = x.double().clone()
    for i in range(n):
        ca, cb = (first + i, first + n + i) if half else (first + 2 * i, first + 2 * i + 1)
        c, s = cos_sin[pos.long().clamp_min(0), i].double().unbind(-1)
        a, b = x[..., ca].double(), x[..., cb].double()
        c, s = c[:, None], s[:, None]
        y[..., ca], y[..., cb] = r(r(a * c) - r(b * s)), r(r(a * s) + r(b * c))
    return torch.where((pos >= 0)[:, None, None], y, x.double())


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "table":
        p = torch.arange(st["start"], st["start"] + st["n_pos"], device="cuda", dtype=torch.float64)
        w = torch.polar(torch.full((), st["amplitude"], dtype=torch.float64, device="cuda").expand(p.numel(), case["half"]).contiguous(),
                        torch.outer(p, st["inv_freq"]))
        return torch.view_as_real(w)
    if case["op"] == "rope":
        turn = lambda x: _exact_rotated(x, st["pos"], st["cos_sin"], st["first"], st["half"])  # noqa: E731
        return dict(q=turn(st["q"]), k=turn(st["k"]) if st["k"] is not None else None)
    if case["op"] == "append":
        S, dt = case["block"], st["k"].dtype
        k = st["k"].double()
        if case["rope_dim"]:               # rounded to the rows' type before it is quantised, by definition
            k = _exact_rotated(st["k"], st["pos"], st["cos_sin"], st["first"], st["half"]).to(dt).double()
        real = (st["slots"] >= 0).nonzero()[:, 0]
        at = st["slots"][real]
        out = {}
        for name, x in (("k", k), ("v", st["v"].double())):
            values, scales = _exact_quantised(x[real])
            held = st[name + "_scales"].view(torch.float8_e4m3fn).double()
            held[at // S, :, at % S] = scales
            rows = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
            rows[real] = values
            out[name + "_values"], out[name + "_scales"], out[name + "_codes"] = rows, held, None
        return out
    if case["op"] == "read":
        S, at = case["block"], st["slots"]
        return {x: _exact_values(st[x + "_codes"][at // S, :, at % S], st[x + "_scales"][at // S, :, at % S]) for x in "kv"}
    S = case["block"]
    q, kv, cu = st["q"], st["kv_len"].tolist(), st["cu_len"].tolist()
    H, G, D = st["k_codes"].shape[1], q.shape[1] // st["k_codes"].shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b in range(len(kv)):
        pages = st["table"][b, : -(-kv[b] // S)].long()
        for h in range(H):
            k = _exact_values(st["k_codes"][pages, h], st["k_scales"][pages, h]).reshape(-1, D)[: kv[b]]
            v = _exact_values(st["v_codes"][pages, h], st["v_scales"][pages, h]).reshape(-1, D)[: kv[b]]
            for lo in range(cu[b], cu[b + 1], 512):
                hi = min(lo + 512, cu[b + 1])
                at = kv[b] - cu[b + 1] + torch.arange(lo, hi, device=q.device)
                j = torch.arange(kv[b], device=q.device)
                hide = j > at[:, None]
                if st["window"] > 0:
                    hide |= j <= at[:, None] - st["window"]
                z = torch.einsum("tgd,kd->gtk", q[lo:hi, h * G:(h + 1) * G].double(), k) * st["sm_scale"]
                z = z.masked_fill(hide, -math.inf)
                lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(z, -1).T
                out[lo:hi, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", torch.softmax(z, -1), v)
    return dict(out=out, lse=lse)
