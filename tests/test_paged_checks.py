"""Refusals of the paged cache's calls, on the CPU: host checks of the C ABI,
and the binding's own."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
import sparse_attention_fp4_quantize_gb300 as csa2

P = ctypes.c_void_p
FAKE, NULL = P(0x1000), None


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._build_module().build()
    return csa2._lib


def _refused(rc, lib, status, word):
    assert rc == status, (rc, lib.csa2_last_error())
    assert word in lib.csa2_last_error().decode()


def test_build_slots_rejects_on_host(lib):
    def call(B=4, M=8, stride=8, S=16, T=10, cap=32, kv=FAKE, table=FAKE, free=FAKE, slots=FAKE):
        return lib.csa2_build_slots(B, M, stride, S, T, cap, kv, FAKE, table, free, FAKE, FAKE, FAKE, FAKE, NULL, slots,
                                    NULL, NULL)
    _refused(call(B=0), lib, 1, "B=0")
    _refused(call(B=8193), lib, 1, "B=8193")
    _refused(call(S=0), lib, 1, "S=0")
    _refused(call(M=1 << 28, stride=1 << 28, S=8), lib, 1, "M * S")
    _refused(call(B=8192, M=1 << 18, stride=1 << 18), lib, 1, "B * M")
    _refused(call(stride=7), lib, 1, "table_stride=7")
    _refused(call(T=-1), lib, 1, "T=-1")
    _refused(call(T=(1 << 30) + 1), lib, 1, "T=")
    _refused(call(cap=-1), lib, 1, "free_cap")
    for a in ("kv", "table", "free", "slots"):
        _refused(call(**{a: NULL}), lib, 1, "null")
    _refused(call(slots=P(0x1004)), lib, 1, "8-byte")


def test_build_slots_refuses_outputs_over_inputs(lib):
    B, T = 4, 10
    apart = dict(kv=0x10000, new=0x20000, count=0x30000, kv_out=0x40000, count_out=0x50000, cu=0x60000, pos=0x70000, slots=0x80000)

    def call(**where):
        w = {**apart, **where}
        p = {n: P(x) for n, x in w.items()}
        return lib.csa2_build_slots(B, 8, 8, 16, T, 32, p["kv"], p["new"], FAKE, FAKE, p["count"], p["kv_out"], p["count_out"],
                                    p["cu"], p["pos"], p["slots"], NULL, NULL)
    sizes = dict(kv_out=4 * B, count_out=4, cu=4 * B + 4, pos=4 * T, slots=8 * T)
    for out, n in sizes.items():
        for name, m in (("kv", 4 * B), ("new", 4 * B), ("count", 4)):
            own = {"kv_out": "kv", "count_out": "count"}.get(out) == name
            for off in (0, m - 4, 4 - n):
                if (own and off == 0) or (out == "slots" and off % 8):
                    continue
                _refused(call(**{out: apart[name] + off}), lib, 1, "overlaps")


def test_quantize_paged_rejects_on_host(lib):
    def call(dt=0, T=4, H=2, D=64, kt=128, kh=64, n=8, S=16, k=FAKE, kc=FAKE, slots=FAKE):
        return lib.csa2_quantize_kv_fp8_paged(k, FAKE, dt, T, H, D, kt, kh, 128, 64, slots, n, S, kc, FAKE, FAKE, FAKE, NULL,
                                              NULL)
    _refused(call(dt=2), lib, 1, "bf16 or fp16")
    _refused(call(T=-1), lib, 1, "T=-1")
    _refused(call(H=0), lib, 1, "Hkv=0")
    _refused(call(S=48), lib, 1, "S=48")
    _refused(call(D=96), lib, 2, "D=96")
    _refused(call(kt=100), lib, 1, "strides")
    _refused(call(kh=-64), lib, 1, "strides")
    _refused(call(n=-1), lib, 1, "n_blocks")
    _refused(call(k=P(0x1008)), lib, 1, "16-byte")
    _refused(call(T=1 << 30, H=1 << 16), lib, 1, "rows")
    _refused(call(kc=P(0x1008)), lib, 1, "16-byte")
    _refused(call(k=NULL), lib, 1, "null")
    _refused(call(kc=NULL), lib, 1, "null")
    _refused(call(slots=P(0x1004)), lib, 1, "misaligned")
    assert call(T=0, k=NULL, kc=NULL, slots=NULL) == 0                    # nothing to store


def test_paged_attention_rejects_on_host(lib):
    def call(B=2, T=4, Hq=8, H=2, D=128, dt=0, q=FAKE, qt=1024, S=64, M=4, stride=4, n=9, max_new=1, window=0, kc=FAKE,
             table=FAKE, ws=P(0x10000), wsb=1 << 30):
        return lib.csa2_paged_attn_fp8(B, T, Hq, H, D, dt, q, qt, 128, kc, FAKE, FAKE, FAKE, n, S, table, M, stride, FAKE,
                                       FAKE, max_new, window, 0.1, FAKE, NULL, NULL, ws, wsb, NULL)
    _refused(call(dt=1), lib, 1, "bf16 or fp16")
    _refused(call(B=-1), lib, 1, "B=-1")
    _refused(call(T=-1), lib, 1, "T=-1")
    _refused(call(Hq=7), lib, 1, "Hq=7")
    _refused(call(H=0), lib, 1, "Hkv=0")
    _refused(call(Hq=4096, H=1, T=1 << 20, qt=0), lib, 1, "rows")
    _refused(call(D=96), lib, 2, "D=96")
    _refused(call(S=24), lib, 1, "S=24")
    _refused(call(M=0, stride=0), lib, 1, "M=0")
    _refused(call(stride=3), lib, 1, "table_stride=3")
    _refused(call(n=-1), lib, 1, "n_blocks")
    _refused(call(max_new=0), lib, 1, "max_new=0")
    _refused(call(window=-1), lib, 1, "window=-1")
    _refused(call(qt=1020), lib, 1, "strides")
    _refused(call(q=P(0x1008)), lib, 1, "16-byte")
    _refused(call(table=NULL), lib, 1, "null")
    _refused(call(kc=NULL), lib, 1, "null")
    assert call(B=0, table=NULL) == 0 and call(T=0, q=NULL) == 0          # nothing to do


class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture()
def fake(monkeypatch):
    f = _FakeLib()
    monkeypatch.setattr(csa2, "_lib", f)
    monkeypatch.setattr(csa2, "_on_device", lambda t: True)
    monkeypatch.setattr(csa2, "_stream", lambda s: None)
    return f


def _z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I32, I64, U8, BF = torch.int32, torch.int64, torch.uint8, torch.bfloat16


def _slots_args():
    B, M, T = 3, 4, 10
    return dict(kv_len=_z(B, dtype=I32), new_len=_z(B, dtype=I32), block_table=_z(B, M, dtype=I32),
                free_list=_z(12, dtype=I32), free_count=_z(1, dtype=I32), block_size=16, kv_len_out=_z(B, dtype=I32),
                free_count_out=_z(1, dtype=I32), cu_len=_z(B + 1, dtype=I32), positions=_z(T, dtype=I32),
                slots=_z(T, dtype=I64))


def _append_args(T=5, H=2, D=64, S=16, n=6):
    return dict(k=_z(T, H, D, dtype=BF), v=_z(T, H, D, dtype=BF), slots=_z(T, dtype=I64), k_codes=_z(n, H, S, D, dtype=U8),
                v_codes=_z(n, H, S, D, dtype=U8), k_scale=_z(n, H), v_scale=_z(n, H))


def _attn_args(T=5, B=2, H=2, Hq=6, D=64, S=16, n=6):
    a = _append_args(T, H, D, S, n)
    return dict(q=_z(T, Hq, D, dtype=BF), k_codes=a["k_codes"], v_codes=a["v_codes"], k_scale=a["k_scale"],
                v_scale=a["v_scale"], block_table=_z(B, 4, dtype=I32), kv_len=_z(B, dtype=I32),
                cu_len=_z(B + 1, dtype=I32), out=_z(T, Hq, D, dtype=BF), sm_scale=0.1, max_new=3,
                lse=_z(T, Hq), err_flag=_z(1, dtype=I32), workspace=_z(1 << 20, dtype=U8))


@pytest.mark.parametrize("fn,args,bad", [
    ("csa2_build_slots", _slots_args, dict(kv_len=_z(3, dtype=I64), new_len=_z(2, dtype=I32), block_table=_z(3, 8, dtype=I32)[:, ::2],
                                           free_list=_z(12), free_count=_z(2, dtype=I32), kv_len_out=_z(4, dtype=I32),
                                           free_count_out=_z(1), cu_len=_z(3, dtype=I32), positions=_z(9, dtype=I32),
                                           slots=_z(10, dtype=I32))),
    ("csa2_quantize_kv_fp8_paged", _append_args, dict(k=_z(5, 2, 64), v=_z(5, 2, 64, dtype=torch.float16), slots=_z(4, dtype=I64),
                                                      k_codes=_z(6, 2, 16, 64, dtype=I32), v_codes=_z(6, 2, 16, 32, dtype=U8),
                                                      k_scale=_z(6, 1), v_scale=_z(6, 2, dtype=torch.float64))),
    ("csa2_paged_attn_fp8", _attn_args, dict(q=_z(5, 6, 64), k_codes=_z(6, 4, 16, 64, dtype=U8), v_scale=_z(2, 6).T,
                                             block_table=_z(2, 8, dtype=I32)[:, ::2], kv_len=_z(3, dtype=I32),
                                             cu_len=_z(2, dtype=I32), out=_z(5, 6, 64, dtype=torch.float16),
                                             lse=_z(5, 6, dtype=BF), err_flag=_z(1), workspace=_z(8, 8, dtype=U8).T)),
])
def test_binding_refuses_what_does_not_fit(fake, fn, args, bad):
    getattr(csa2, fn)(**args())
    assert fake.calls == [fn]
    for name, value in bad.items():
        with pytest.raises((TypeError, ValueError)):
            getattr(csa2, fn)(**{**args(), name: value})
    assert fake.calls == [fn]


def test_binding_refuses_heads_that_do_not_divide(fake):
    a = _attn_args(Hq=6)
    a["q"], a["out"], a["lse"] = _z(5, 5, 64, dtype=BF), _z(5, 5, 64, dtype=BF), _z(5, 5)
    with pytest.raises(ValueError):
        csa2.csa2_paged_attn_fp8(**a)
    assert fake.calls == []


def test_binding_refuses_tensors_off_the_gpu():
    with pytest.raises(ValueError):
        csa2.csa2_quantize_kv_fp8_paged(**_append_args())
    with pytest.raises(ValueError):
        csa2.csa2_build_slots(**_slots_args())


# ---------------------------------------------------------------- the references themselves
def test_reference_e4m3_is_torchs_cast():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.randn(20000) * 0.01])
    assert np.array_equal(ref.e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_reference_scale_is_the_least_power_of_two():
    for a in [448.0, 448.5, 1.0, 7.0, 7.03125, 3.5, 1e-30, 3e38, 2.0 ** -140]:
        s = ref.need_of(a)
        assert a <= 448 * s and (a > 224 * s or s == ref.MIN_SCALE)


def test_reference_attention_is_dense_softmax():
    gen = torch.Generator().manual_seed(3)
    table, n = ref.ragged(gen, [37], 16)
    kc, ks = ref.random_planes(gen, n, 2, 16, 64)
    vc, vs = ref.random_planes(gen, n, 2, 16, 64)
    q = torch.randn(37, 4, 64, generator=gen, dtype=torch.float64)
    out, lse, _, _ = ref.attention(q, ref.values_of(kc), ref.values_of(vc), ks.double(), vs.double(), table, [37], [0, 37], 0.1)
    k = (ref.values_of(kc) * ks.double()[..., None, None])[table[0, :3].long()].transpose(0, 1).reshape(2, 48, 64)[:, :37]
    v = (ref.values_of(vc) * vs.double()[..., None, None])[table[0, :3].long()].transpose(0, 1).reshape(2, 48, 64)[:, :37]
    k, v = k.repeat_interleave(2, 0), v.repeat_interleave(2, 0)
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1)[None], k[None], v[None], is_causal=True,
                                                            scale=0.1)[0].transpose(0, 1)
    assert torch.allclose(out, want, rtol=1e-10, atol=1e-10)
