"""Calls of the paged 8-bit cache that the C ABI or the class refuse or keep apart, on the CPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_attention_fp4_quantize_gb300 as csa2

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._build_module().build()
    return csa2._lib


def _refused(rc, lib, word):
    assert rc == 1, (rc, lib.csa2_last_error())
    assert word in lib.csa2_last_error().decode()


# ---------------------------------------------------------------- slot maps
B, M, STRIDE, T, CAP = 4, 8, 20, 10, 32
APART = dict(kv=0x10000, new=0x20000, count=0x30000, kv_out=0x40000, count_out=0x50000, cu=0x60000, pos=0x70000, slots=0x80000,
             free=0x90000, table=0xA0000, err=0xB0000)
BYTES = dict(kv=4 * B, new=4 * B, count=4, kv_out=4 * B, count_out=4, cu=4 * B + 4, pos=4 * T, slots=8 * T, free=4 * CAP, err=4)


def _build_slots(lib, **where):
    p = {n: P(x) for n, x in {**APART, **where}.items()}
    return lib.csa2_build_slots(B, M, STRIDE, 8, T, CAP, p["kv"], p["new"], p["table"], p["free"], p["count"], p["kv_out"],
                                p["count_out"], p["cu"], p["pos"], p["slots"], p["err"], None)


WRITTEN = ["kv_out", "count_out", "cu", "pos", "slots", "free", "err"]


@pytest.mark.parametrize("one", WRITTEN)
def test_build_slots_refuses_what_is_written_over_anything_else(lib, one):
    for other, n in BYTES.items():
        if other == one:
            continue
        own = {"kv_out": "kv", "count_out": "count"}.get(one) == other
        for off in (0, n - 4, 4 - BYTES[one]):
            if (own and off == 0) or (one == "slots" and off % 8):
                continue
            _refused(_build_slots(lib, **{one: APART[other] + off}), lib, "overlaps")


@pytest.mark.parametrize("one", list(BYTES))
def test_build_slots_refuses_the_table_over_anything_else(lib, one):
    row, last, step = 4 * STRIDE, (B - 1) * 4 * STRIDE, 8 if one == "slots" else 4
    for begin in (0, row, last):
        for at in (begin, begin + 4 * M - step, begin + step - BYTES[one]):
            _refused(_build_slots(lib, **{one: APART["table"] + at}), lib, "overlaps")


@pytest.mark.parametrize("one", ["kv", "new", "count", "kv_out", "count_out", "cu", "pos", "free", "table", "err"])
def test_build_slots_refuses_misaligned_words(lib, one):
    for off in (1, 2):
        _refused(_build_slots(lib, **{one: APART[one] + 0x4000 + off}), lib, "aligned")


@pytest.mark.parametrize("one", ["k_scale", "v_scale", "table", "kv_len", "cu_len", "lse", "err"])
def test_attention_refuses_misaligned_words(lib, one):
    at = {n: P(0x10000 * i) for i, n in enumerate(["q", "k", "v", "k_scale", "v_scale", "table", "kv_len", "cu_len", "out", "lse",
                                                   "err", "ws"], 1)}
    for off in (1, 2):
        p = {**at, one: P(at[one].value + off)}
        _refused(lib.csa2_paged_attn_fp8(2, 4, 8, 2, 64, 0, p["q"], 512, 64, p["k"], p["v"], p["k_scale"], p["v_scale"], 9, 64,
                                         p["table"], 4, 4, p["kv_len"], p["cu_len"], 1, 0, 0.1, p["out"], p["lse"], p["err"],
                                         p["ws"], 1 << 30, None), lib, "aligned")


def test_append_refuses_a_misaligned_flag(lib):
    _refused(lib.csa2_quantize_kv_fp8_paged(P(0x1000), P(0x2000), 0, 4, 2, 64, 128, 64, 128, 64, P(0x3000), 8, 16, P(0x4000),
                                            P(0x5000), P(0x6000), P(0x7000), P(0x8002), None), lib, "aligned")


# ---------------------------------------------------------------- the class
class _Calls:
    """A stand-in for the library that keeps the calls' arguments."""

    def __init__(self):
        self.calls = []

    def csa2_paged_attn_workspace_bytes(self, *a):
        return 4096

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


def test_layers_of_a_cache_share_no_workspace(monkeypatch):
    """attend takes a stream: layers that run side by side, on two streams or in two graphs, join their own parts."""
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    fake = _Calls()
    monkeypatch.setattr(csa2, "_lib", fake)
    monkeypatch.setattr(csa2, "_on_device", lambda t: True)
    monkeypatch.setattr(csa2, "_stream", lambda s: s)
    cache = PagedCache(PagedShape(requests=2, tokens=4, max_context=64, n_blocks=4, heads=4, kv_heads=2, dim=64, block_size=16,
                                  layers=3), device="cpu")
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    for layer in range(3):
        cache.attend(layer, q, stream=layer + 1)
    used = sorted(a[-3] for name, a in fake.calls if name == "csa2_paged_attn_fp8")
    assert len(used) == 3 and all(y - x >= 4096 for x, y in zip(used, used[1:]))
