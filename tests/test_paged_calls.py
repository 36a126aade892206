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
