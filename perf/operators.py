"""What is measured of the paged 8-bit cache: its slot maps, its quantising append and the attention that reads it.

Each case is one call of one operator as a serving loop makes it.  The plain form computes the same from elementary
torch operations; with ``own`` set the framework's kernels are called.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126          # the smallest scale a block gets (the smallest normal fp32)


def _dt(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def listed():
    return [
        # a decode step of a small batch: one new token per request (launch latency)
        dict(name="slots-decode-32", op="slots", requests=32, block=64, table=512, tokens=32, kind="decode"),
        # continuous batching: decoding requests, prompt chunks, requests that ended, refilled in one step
        dict(name="slots-mixed-512", op="slots", requests=512, block=16, table=1024, tokens=16384, kind="mixed"),
        # prompts of many requests planned at once, a padded token budget
        dict(name="slots-prompts-2000", op="slots", requests=2000, block=128, table=256, tokens=65536, kind="prompt"),
        # a decode step's append: 64 requests, most of them inside a partly filled block
        dict(name="append-decode-64", op="append", dtype="bf16", requests=64, tokens=64, heads=8, dim=128, block=64,
             kind="decode", fused=False),
        # a prompt chunk of several requests whose K and V are slices of one fused projection
        dict(name="append-prompt-16k", op="append", dtype="bf16", requests=9, tokens=16384, heads=8, dim=128, block=64,
             kind="prompt", fused=True),
        # small heads, odd head count, small blocks, fp16
        dict(name="append-mixed-fp16", op="append", dtype="fp16", requests=37, tokens=1501, heads=5, dim=64, block=16,
             kind="mixed", fused=False),
        # one user, one token, a short context: latency
        dict(name="attn-decode-1", op="attn", dtype="bf16", requests=1, new=1, context=1000, heads=32, kv_heads=8,
             dim=128, block=64, window=0, kind="decode"),
        # the decode step of a served batch with ragged contexts
        dict(name="attn-decode-64", op="attn", dtype="bf16", requests=64, new=1, context=16384, heads=64, kv_heads=8,
             dim=128, block=64, window=0, kind="decode"),
        # few requests with long contexts: one axis has to be split over the machine
        dict(name="attn-decode-long", op="attn", dtype="bf16", requests=3, new=1, context=131071, heads=32, kv_heads=4,
             dim=128, block=128, window=0, kind="decode"),
        # several draft tokens per request, sliding window, small heads and blocks, fp16
        dict(name="attn-draft-window-fp16", op="attn", dtype="fp16", requests=48, new=5, context=9001, heads=15,
             kv_heads=5, dim=64, block=16, window=4096, kind="decode"),
        # prompts of a ragged batch on top of cached prefixes
        dict(name="attn-prompt-8k", op="attn", dtype="bf16", requests=3, new=4096, context=8192, heads=32, kv_heads=8,
             dim=128, block=64, window=0, kind="prompt"),
        # chunked prefill next to decoding requests, in one call
        dict(name="attn-mixed-17", op="attn", dtype="bf16", requests=17, new=512, context=12000, heads=32, kv_heads=8,
             dim=128, block=32, window=0, kind="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "append", "attn", "attn"])
    if op == "slots":
        kind = rng.choice(["decode", "mixed", "prompt"])
        requests = _log(rng, 1, 2000)
        tokens = requests + rng.randint(0, 7) if kind == "decode" else _log(rng, max(requests, 16), 65536)
        return dict(op=op, requests=requests, block=rng.choice([16, 32, 48, 64, 128]), table=_log(rng, 8, 1024),
                    tokens=tokens, kind=kind)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    dim, block = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        kind = rng.choice(["decode", "mixed", "prompt"])
        requests = _log(rng, 1, 256)
        tokens = requests if kind == "decode" else _log(rng, max(requests, 16), 16384)
        return dict(op=op, dtype=dtype, requests=requests, tokens=tokens, heads=rng.randint(1, 8), dim=dim, block=block,
                    kind=kind, fused=rng.choice([True, False]))
    kind = rng.choice(["decode", "decode", "prompt", "mixed"])
    kv_heads, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
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
    else:
        requests = rng.randint(2, 17)
        context = _log(rng, 64, 12000)
        new = max(1, min(512, int(context * rng.uniform(0.1, 1.0))))
    return dict(op=op, dtype=dtype, requests=requests, new=new, context=context, heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, block=block, window=window, kind=kind)


# ---------------------------------------------------------------- inputs
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


def _prepare_slots(case, seed):
    rng = np.random.default_rng(seed)
    B, S, M = case["requests"], case["block"], case["table"]
    new = _token_counts(case, rng)
    if case["kind"] == "mixed":
        new[rng.random(B) < 0.05] = -1     # ended requests
        new[rng.random(B) < 0.05] = 0      # waiting ones
    kv = rng.integers(0, M * S, B)
    if case["kind"] == "prompt":
        kv[rng.random(B) < 0.7] = 0        # most prompts start an empty request
    over = (kv + np.maximum(new, 0)) > M * S
    kv[over] = np.maximum(0, M * S - new[over])
    held, after = -(-kv // S), -(-(kv + np.maximum(new, 0)) // S)
    cap = B * M + 64                       # a pool that every table could be filled from
    ids = rng.permutation(cap).astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    row = np.repeat(np.arange(B), held)
    col = np.arange(int(held.sum())) - np.repeat(np.cumsum(held) - held, held)
    table[row, col] = ids[: int(held.sum())]
    n_free = cap - int(held.sum())
    if case["kind"] == "mixed":            # memory is short: the last requests may have to wait
        n_free = max(0, int(0.97 * (after - held).sum()) - int(held[new < 0].sum()))
    free = np.full(cap, -1, np.int32)
    free[:n_free] = ids[int(held.sum()):int(held.sum()) + n_free]
    d = lambda a, t: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
    i32 = torch.int32
    T = case["tokens"]
    return dict(kv_len=d(kv, i32), new_len=d(new, i32), table=d(table, i32), free_list=d(free, i32),
                free_count=d([n_free], i32), kv_len_out=torch.zeros(B, dtype=i32, device="cuda"),
                free_count_out=torch.zeros(1, dtype=i32, device="cuda"),
                cu_len=torch.zeros(B + 1, dtype=i32, device="cuda"), positions=torch.zeros(T, dtype=i32, device="cuda"),
                slots=torch.zeros(T, dtype=torch.int64, device="cuda"))


def _heads_rows(gen, T, H, D, dtype, fused):
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


def _scale_of(amax):
    """The least power of two s >= MIN_SCALE with amax <= 448 s.  log2 in 64 bits may land a rounding error above a
    whole number, where amax / 448 is a power of two; other ratios of fp32 values are further than 8e-8 from one."""
    s = torch.exp2(torch.ceil(torch.log2(amax.double() / E4M3_MAX) - 1e-9)).float()
    return s.clamp_min(MIN_SCALE)


def _quantise_blocks(x):
    """[n, H, S, D] fp32 -> E4M3 bytes and a power-of-two scale per (block, head)."""
    scale = _scale_of(x.abs().amax(dim=(2, 3)))
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _prepare_append(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    B, S, H, D, T = case["requests"], case["block"], case["heads"], case["dim"], case["tokens"]
    n = _token_counts(case, rng)
    start = rng.integers(0, 4 * S, B)      # tokens that each request already holds
    if case["kind"] == "prompt":
        start[rng.random(B) < 0.7] = 0
    blocks = -(-(start + n) // S)
    nb = T // S + 6 * B + 3
    ids = rng.permutation(nb)
    first = np.cumsum(blocks) - blocks
    req = np.repeat(np.arange(B), n)
    pos = np.arange(int(n.sum())) - np.repeat(np.cumsum(n) - n, n) + start[req]
    slots = np.full(T, -1, np.int64)
    slots[: pos.size] = ids[first[req] + pos // S] * S + pos % S
    k, v = _heads_rows(gen, T, H, D, _dt(case), case["fused"])
    kc, ks = _quantise_blocks(0.7 * torch.randn(nb, H, S, D, generator=gen, device="cuda"))
    vc, vs = _quantise_blocks(0.7 * torch.randn(nb, H, S, D, generator=gen, device="cuda"))
    return dict(k=k, v=v, slots=torch.tensor(slots, device="cuda"), k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs)


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
    kc = torch.empty(nb, H, S, D, dtype=torch.uint8, device="cuda")
    vc, ks = torch.empty_like(kc), torch.empty(nb, H, device="cuda")
    vs = torch.empty_like(ks)
    for at in range(0, nb, 2048):          # in pieces: the cache in fp32 would be large
        m = min(2048, nb - at)
        x, y = _heads_rows(gen, m * S, H, D, torch.float32, False)
        for t, c, s in ((x, kc, ks), (y, vc, vs)):
            c[at:at + m], s[at:at + m] = _quantise_blocks(t.view(m, S, H, D).transpose(1, 2).contiguous())
    table = np.full((B, int(held.max()) + 2), -1, np.int32)
    ids = rng.permutation(nb)
    row = np.repeat(np.arange(B), held)
    table[row, np.arange(nb) - np.repeat(np.cumsum(held) - held, held)] = ids
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    q = torch.randn(T, case["heads"], D, generator=gen, device="cuda").to(_dt(case))
    out = torch.zeros_like(q)
    return dict(q=q, k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs,
                table=torch.tensor(table, device="cuda"), kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"),
                cu_len=torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out,
                lse=torch.zeros(T, case["heads"], device="cuda"), sm_scale=1.0 / math.sqrt(D), window=case["window"],
                max_new=int(new.max()), kv_max=int(kv.max()),
                workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))   # kept by a serving loop


def prepare(case, seed):
    st = {"slots": _prepare_slots, "append": _prepare_append, "attn": _prepare_attn}[case["op"]](case, seed)
    st["op"], st["block"] = case["op"], case["block"]
    return st


# ---------------------------------------------------------------- plain forms
def _plain_slots(st):
    S, table = st["block"], st["table"]
    B, M = table.shape
    T, cap = st["slots"].numel(), st["free_list"].numel()
    dev = table.device
    kv, new = st["kv_len"].long(), st["new_len"].long()
    n_free = st["free_count"].long()
    grow = new.clamp_min(0)
    held, after = (kv + S - 1) // S, (kv + grow + S - 1) // S
    ended = new < 0
    col = torch.arange(M, device=dev)
    freed = table[(col < held[:, None]) & ended[:, None]].long()     # request by request, block by block
    size = n_free + freed.numel()
    end = torch.cumsum(grow, 0)
    fits = (kv + grow <= M * S) & (end <= T)
    need = torch.where(fits, after - held, 0)
    a_end = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (a_end <= size)) & ~ended
    taken = torch.where(ok & (need > 0), a_end, 0).max()
    stack = torch.cat([st["free_list"].long(), freed, freed.new_zeros(1)])
    at = size - 1 - ((a_end - need)[:, None] + col - held[:, None])  # place in the stack, freed blocks on top
    at = torch.where(at < n_free, at, at - n_free + cap).clamp(0, stack.numel() - 1)
    fresh = ok[:, None] & (col >= held[:, None]) & (col < after[:, None])
    table_out = torch.where(fresh, stack[at].int(), table)
    count = size - taken
    place = torch.arange(cap, device=dev)
    back = torch.cat([freed, freed.new_zeros(1)])[(place - n_free).clamp(0, freed.numel())]
    free_out = torch.where((place >= n_free) & (place < count), back.int(), st["free_list"])
    cu = torch.cat([end.new_zeros(1), end]).clamp_max(T)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(end, t, right=True)
    real = b < B
    b = b.clamp_max(B - 1)
    p = kv[b] + t - (end - grow)[b]
    real = real & ok[b]
    page = table_out[b, (p // S).clamp(0, M - 1)].long()
    return dict(table=table_out, free_list=free_out, kv_len=torch.where(ok, kv + grow, torch.where(ended, 0, kv)).int(),
                free_count=count.int(), cu_len=cu.int(), positions=torch.where(real, p, -1).int(),
                slots=torch.where(real, page * S + p % S, -1))


def _plain_append_one(x, slots, codes, scale, S):
    """Rows x [T, H, D] into the blocks of codes [n, H, S, D]; slots of one block stand next to each other."""
    H = x.shape[1]
    at = torch.nonzero(slots >= 0)[:, 0]
    x, s = x[at].float(), slots[at]
    blk, off = s // S, s % S
    lead = torch.ones_like(blk, dtype=torch.bool)
    lead[1:] = blk[1:] != blk[:-1]
    run = torch.cumsum(lead, 0) - 1
    ids, start = blk[lead], off[lead]
    amax = torch.zeros(ids.numel(), H, device=x.device).index_reduce_(0, run, x.abs().amax(-1), "amax")
    need = _scale_of(amax)
    old = scale[ids]
    now = torch.where(start[:, None] == 0, need, torch.maximum(old, need))
    held = codes[ids].view(torch.float8_e4m3fn).float()
    again = (held * (old / now)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = torch.arange(S, device=x.device) < start[:, None]          # rows the block held before
    codes[ids] = torch.where(keep[:, None, :, None], again, codes[ids])
    scale[ids] = now
    codes[blk, :, off] = (x / now[run][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(st):
    _plain_append_one(st["k"], st["slots"], st["k_codes"], st["k_scale"], st["block"])
    _plain_append_one(st["v"], st["slots"], st["v_codes"], st["v_scale"], st["block"])
    return _append_out(st)


def _append_out(st):
    f8 = torch.float8_e4m3fn
    return dict(k_codes=st["k_codes"].view(f8), v_codes=st["v_codes"].view(f8), k_scale=st["k_scale"],
                v_scale=st["v_scale"])


def _dequantised(codes, scale, pages):
    """The rows of every request, [B, H, n * S, D] fp32."""
    x = codes[pages].view(torch.float8_e4m3fn).float() * scale[pages][..., None, None]
    B, n, H, S, D = x.shape
    return x.transpose(1, 2).reshape(B, H, n * S, D)


def _plain_attn(st):
    S, q = st["block"], st["q"]
    H, D = st["k_codes"].shape[1], q.shape[2]
    G = q.shape[1] // H
    B, n = st["kv_len"].numel(), st["max_new"]
    dev = q.device
    pages = st["table"][:, : -(-st["kv_max"] // S)].long().clamp_min(0)
    k = _dequantised(st["k_codes"], st["k_scale"], pages)
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
    v = _dequantised(st["v_codes"], st["v_scale"], pages)
    v = torch.where((j < kv[:, None])[:, None, :, None], v, torch.zeros_like(v))   # nothing of unwritten rows
    o = torch.matmul(w, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    real = i < count[:, None]
    o = o.view(B, H, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H * G, D)[real]
    lse = lse.view(B, H, G, n).permute(0, 3, 1, 2).reshape(B, n, H * G)[real]
    return dict(out=o.to(q.dtype), lse=lse)


# ---------------------------------------------------------------- the framework's operators
def _own_slots(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_build_slots(st["kv_len"], st["new_len"], st["table"], st["free_list"], st["free_count"], st["block"],
                          st["kv_len_out"], st["free_count_out"], st["cu_len"], st["positions"], st["slots"])
    return dict(table=st["table"], free_list=st["free_list"], kv_len=st["kv_len_out"], free_count=st["free_count_out"],
                cu_len=st["cu_len"], positions=st["positions"], slots=st["slots"])


def _own_append(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_quantize_kv_fp8_paged(st["k"], st["v"], st["slots"], st["k_codes"], st["v_codes"], st["k_scale"],
                                    st["v_scale"])
    return _append_out(st)


def _own_attn(st):
    import sparse_attention_fp4_quantize_gb300 as csa2
    csa2.csa2_paged_attn_fp8(st["q"], st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"],
                             st["kv_len"], st["cu_len"], st["out"], st["sm_scale"], st["max_new"], window=st["window"],
                             lse=st["lse"], workspace=st["workspace"])
    return dict(out=st["out"], lse=st["lse"])


def run(state):
    if own:
        return {"slots": _own_slots, "append": _own_append, "attn": _own_attn}[state["op"]](state)
    return {"slots": _plain_slots, "append": _plain_append, "attn": _plain_attn}[state["op"]](state)


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
    """One pass's bytes and operations at the mean of the lengths that `prepare` draws."""
    if case["op"] == "slots":
        B, T, S = case["requests"], case["tokens"], case["block"]
        blocks = T / S + (B / S if case["kind"] == "decode" else 0)
        return {"bytes": 8 * B + 4 * B + 4 * (B + 1) + 12 * T + 4 * B + 8 * blocks, "flops": T}
    H, D = case.get("kv_heads", case.get("heads")), case["dim"]
    if case["op"] == "append":
        rng = np.random.default_rng(0)
        T = float(_token_counts(case, rng).sum())
        return {"bytes": 2 * T * H * D * 3 + 8 * case["tokens"] + 16 * H * T / case["block"], "flops": 4 * T * H * D}
    pairs = keys = rows = 0.0
    for seed in range(4):
        kv, new = _lengths(case, np.random.default_rng(seed))
        p, k = _seen(kv, new, case["window"])
        pairs, keys, rows = pairs + p.sum() / 4, keys + k.sum() / 4, rows + new.sum() / 4
    return {"bytes": float(keys * H * (2 * D + 8 / case["block"]) + rows * case["heads"] * (4 * D + 4)),
            "flops": float(4.0 * pairs * case["heads"] * D)}


# ---------------------------------------------------------------- in 64 bits
def _e4m3_nearest(x):
    """Nearest E4M3 value, ties to the even code, of |x| <= 448, in 64 bits."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    r = torch.round(a / step) * step                       # torch.round: half to even
    return torch.copysign(r, x)


def _exact_append_one(x, slots, codes, scale, S):
    val = codes.view(torch.float8_e4m3fn).double()
    scale, x = scale.double(), x.double()
    s = slots.cpu().numpy()
    at = np.nonzero(s >= 0)[0]
    cut = np.nonzero(np.diff(s[at] // S, prepend=-1))[0].tolist() + [at.size]
    for lo, hi in zip(cut[:-1], cut[1:]):
        b, o = int(s[at[lo]] // S), int(s[at[lo]] % S)
        rows = x[int(at[lo]):int(at[hi - 1]) + 1].transpose(0, 1)         # [H, run, D]
        amax = rows.abs().amax(dim=(1, 2))
        m, e = torch.frexp(amax / E4M3_MAX)
        need = torch.exp2(torch.where(m == 0.5, e - 1, e).double()).float().double()   # a whole power of two
        need = torch.where(amax > 0, need, torch.zeros_like(need)).clamp_min(MIN_SCALE)
        now = torch.maximum(scale[b], need) if o else need
        if o:
            val[b, :, :o] = _e4m3_nearest(val[b, :, :o] * (scale[b] / now)[:, None, None])
        val[b, :, o:o + hi - lo] = _e4m3_nearest(rows / now[:, None, None])
        scale[b] = now
    return val, scale


def exact(case, seed):
    if case["op"] == "slots":
        return None
    st = prepare(case, seed)
    S = st["block"]
    if case["op"] == "append":
        if case["tokens"] / S + case["requests"] > 4000:
            return None
        k, ks = _exact_append_one(st["k"], st["slots"], st["k_codes"], st["k_scale"], S)
        v, vs = _exact_append_one(st["v"], st["slots"], st["v_codes"], st["v_scale"], S)
        return dict(k_codes=k, v_codes=v, k_scale=ks, v_scale=vs)
    q, kv, cu = st["q"], st["kv_len"].tolist(), st["cu_len"].tolist()
    H, G, D = st["k_codes"].shape[1], q.shape[1] // st["k_codes"].shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b in range(len(kv)):
        pages = st["table"][b, : -(-kv[b] // S)].long()
        for h in range(H):
            k = st["k_codes"][pages, h].view(torch.float8_e4m3fn).double() * st["k_scale"][pages, h].double()[:, None, None]
            v = st["v_codes"][pages, h].view(torch.float8_e4m3fn).double() * st["v_scale"][pages, h].double()[:, None, None]
            k, v = k.reshape(-1, D)[: kv[b]], v.reshape(-1, D)[: kv[b]]
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
