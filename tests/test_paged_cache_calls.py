"""Calls of the paged cache's class that its documentation allows, on the CPU with a stand-in for the library."""
from __future__ import annotations

import pytest
import torch

import sparse_attention_fp4_quantize_gb300 as csa2

BF = torch.bfloat16


class _Calls:
    def __init__(self):
        self.calls = []

    def csa2_paged_attn_workspace_bytes(self, *a):
        return 4096

    csa2_paged_attn_fp4_workspace_bytes = csa2_paged_attn_workspace_bytes

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture()
def calls(monkeypatch):
    f = _Calls()
    monkeypatch.setattr(csa2, "_lib", f)
    monkeypatch.setattr(csa2, "_on_device", lambda t: True)
    monkeypatch.setattr(csa2, "_stream", lambda s: s)
    return f


def _cache(bits):
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    return PagedCache(PagedShape(requests=2, tokens=4, max_context=64, n_blocks=4, heads=4, kv_heads=2, dim=64, block_size=16,
                                 layers=2, bits=bits), device="cpu")


@pytest.mark.parametrize("bits,name", [(8, "csa2_quantize_kv_fp8_paged"), (4, "csa2_quantize_kv_fp4_paged")])
def test_append_takes_the_stream_as_its_fourth_argument(calls, bits, name):
    cache = _cache(bits)
    kv = torch.zeros(4, 2, 64, dtype=BF)
    cache.append(1, kv, kv, 77)
    cache.append(1, kv, kv, stream=78)
    assert [n for n, _ in calls.calls] == [name] * 2
    assert [a[-1] for _, a in calls.calls] == [77, 78]


def test_append_gives_the_stored_values_by_name(calls):
    kv, values = torch.zeros(4, 2, 64, dtype=BF), [torch.zeros(4, 2, 64, dtype=BF) for _ in range(2)]
    _cache(4).append(0, kv, kv, 77, k_values=values[0], v_values=values[1])
    (name, args), = calls.calls
    assert list(args[-4:-2]) == [t.data_ptr() for t in values] and args[-1] == 77
    with pytest.raises(TypeError):
        _cache(4).append(0, kv, kv, 77, *values)
