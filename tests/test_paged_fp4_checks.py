"""Refusals of the rotary positions' and the paged 4-bit cache's calls, on the CPU: host checks of the C ABI, the binding's
own, and the references themselves."""
from __future__ import annotations

import ctypes
import inspect
import math
import struct

import numpy as np
import pytest
import torch

import paged_fp4_ref as ref
import sparse_attention_fp4_quantize_gb300 as csa2

P = ctypes.c_void_p
FAKE, NULL = P(0x1000), None
REAL = csa2._lib


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._build_module().build()
    return csa2._lib


def _refused(rc, lib, status, word):
    assert rc == status, (rc, lib.csa2_last_error())
    assert word in lib.csa2_last_error().decode()


def test_rope_table_rejects_on_host(lib):
    def call(f=FAKE, half=32, start=0, n=16, out=P(0x10000)):
        return lib.csa2_rope_table(f, half, start, n, 1.0, out, NULL)
    _refused(call(half=0), lib, 1, "half=0")
    _refused(call(half=513), lib, 1, "half=513")
    _refused(call(start=-1), lib, 1, "start=-1")
    _refused(call(n=-1), lib, 1, "n_pos=-1")
    _refused(call(n=(1 << 31) + 1), lib, 1, "n_pos")
    _refused(call(f=NULL), lib, 1, "null")
    _refused(call(f=P(0x1004)), lib, 1, "8-byte")
    _refused(call(out=P(0x10004)), lib, 1, "8-byte")
    _refused(call(out=P(0x1000 + 8 * 31)), lib, 1, "overlaps")
    assert call(n=0, f=NULL, out=NULL) == 0


ROPE = dict(q=0x100000, qo=0x200000, Hq=4, qs=(512, 128), qos=(512, 128), k=0x300000, ko=0x400000, Hk=2, ks=(256, 128),
            kos=(256, 128), dt=0, T=8, D=128, pos=0x500000, table=0x600000, n=16, dim=64, first=0, layout=1, err=None)


def _rope(lib, **kw):
    a = {**ROPE, **kw}
    p = lambda x: None if x is None else P(x)  # noqa: E731
    return lib.csa2_rope(p(a["q"]), p(a["qo"]), a["Hq"], *a["qs"], *a["qos"], p(a["k"]), p(a["ko"]), a["Hk"], *a["ks"], *a["kos"],
                         a["dt"], a["T"], a["D"], p(a["pos"]), p(a["table"]), a["n"], a["dim"], a["first"], a["layout"],
                         p(a["err"]), NULL)


@pytest.mark.parametrize("bad,word", [
    (dict(dt=2), "bf16 or fp16"), (dict(T=-1), "T=-1"), (dict(T=(1 << 30) + 1), "T="), (dict(Hq=-1), "Hq=-1"),
    (dict(Hk=40000), "Hk=40000"), (dict(D=100), "D=100"), (dict(D=2048), "D=2048"), (dict(layout=2), "layout=2"),
    (dict(dim=24), "rope_dim=24"), (dict(dim=0), "rope_dim=0"), (dict(dim=144), "rope_dim=144"), (dict(first=4), "first=4"),
    (dict(first=72), "first=72"), (dict(first=-8), "first=-8"), (dict(n=0), "n_pos=0"), (dict(q=None), "null"),
    (dict(qo=None), "null"), (dict(k=None), "null"), (dict(pos=None), "null"), (dict(table=None), "null"),
    (dict(table=0x600008), "16-byte"), (dict(pos=0x500002), "4-byte"), (dict(err=0x700002), "4-byte"),
    (dict(q=0x100008), "16-byte"), (dict(ko=0x400008), "16-byte"), (dict(qs=(516, 128)), "strides"),
    (dict(qos=(512, -128)), "strides"), (dict(ks=(1 << 33, 128)), "strides"), (dict(qos=(0, 128)), "share"),
    (dict(qos=(512, 120)), "share"), (dict(qos=(384, 128)), "share"), (dict(qo=0x100010), "overlaps its input"),
    (dict(qo=0x100000, qos=(1024, 128)), "overlaps its input"), (dict(ko=0x200100), "share elements"),
    (dict(qo=0x300000), "overlaps the other input"), (dict(qo=0x500000), "overlaps pos"), (dict(ko=0x600000), "overlaps pos"),
    (dict(err=0x200000), "overlaps pos"),
])
def test_rope_rejects_on_host(lib, bad, word):
    _refused(_rope(lib, **bad), lib, 1, word)


def test_rope_without_rows_does_nothing(lib):
    assert _rope(lib, T=0, q=None, k=None, pos=None) == 0
    assert _rope(lib, Hq=0, Hk=0, q=None, k=None) == 0


def _append(lib, dt=0, T=4, H=2, D=64, kt=128, kh=64, n=8, S=16, k=P(0x10000), kc=P(0x100000), ks=P(0x300000), slots=P(0x20000),
            pos=NULL, table=NULL, n_pos=9, dim=64, first=0, layout=1, kval=NULL, vval=NULL, err=NULL):
    return lib.csa2_quantize_kv_fp4_paged(k, P(0x30000), dt, T, H, D, kt, kh, 128, 64, slots, n, S, kc, P(0x200000), ks,
                                          P(0x400000), pos, table, n_pos, dim, first, layout, kval, vval, err, NULL)


@pytest.mark.parametrize("bad,status,word", [
    (dict(dt=2), 1, "bf16 or fp16"), (dict(T=-1), 1, "T=-1"), (dict(H=0), 1, "Hkv=0"), (dict(H=32768), 1, "Hkv=32768"),
    (dict(S=48), 1, "S=48"), (dict(D=96), 2, "D=96"), (dict(kt=100), 1, "strides"), (dict(kh=-64), 1, "strides"),
    (dict(n=-1), 1, "n_blocks"), (dict(k=P(0x10008)), 1, "16-byte"), (dict(kc=P(0x100008)), 1, "16-byte"),
    (dict(ks=P(0x300008)), 1, "16-byte"), (dict(k=NULL), 1, "null"), (dict(kc=NULL), 1, "null"), (dict(ks=NULL), 1, "null"),
    (dict(slots=P(0x20004)), 1, "misaligned"), (dict(err=P(0x20002)), 1, "misaligned"),
    (dict(pos=FAKE), 1, "go together"), (dict(table=FAKE), 1, "go together"),
    (dict(pos=FAKE, table=P(0x1008)), 1, "16-byte"), (dict(pos=P(0x1002), table=FAKE), 1, "4-byte"),
    (dict(pos=FAKE, table=FAKE, dim=72), 1, "rope_dim=72"), (dict(pos=FAKE, table=FAKE, dim=80), 1, "rope_dim=80"),
    (dict(pos=FAKE, table=FAKE, first=8), 1, "first=8"), (dict(pos=FAKE, table=FAKE, layout=3), 1, "layout=3"),
    (dict(pos=FAKE, table=FAKE, n_pos=0), 1, "n_pos=0"), (dict(kval=P(0x500008)), 1, "16-byte"),
    (dict(kval=P(0x10000)), 1, "overlap"), (dict(vval=P(0x30000)), 1, "overlap"), (dict(vval=P(0x300000)), 1, "overlap"),
    (dict(kval=P(0x500000), vval=P(0x500010)), 1, "overlap"),
    (dict(kc=P(0x200010)), 1, "overlap"), (dict(ks=P(0x400000)), 1, "overlap"), (dict(ks=P(0x101FF0)), 1, "overlap"),
    (dict(kc=P(0x30000)), 1, "overlap"), (dict(kc=P(0x20000)), 1, "overlap"),
    (dict(pos=P(0x600000), table=FAKE, ks=P(0x600000)), 1, "overlap"), (dict(pos=FAKE, table=P(0x600000), kc=P(0x600100)), 1, "overlap"),
])
def test_append_rejects_on_host(lib, bad, status, word):
    _refused(_append(lib, **bad), lib, status, word)


def test_append_of_nothing_is_nothing(lib):
    assert _append(lib, T=0, k=NULL, kc=NULL, ks=NULL, slots=NULL) == 0


def _read(lib, dt=0, T=4, H=2, D=64, kt=128, kh=64, n=8, S=16, k=P(0x10000), kc=P(0x100000), slots=P(0x20000), v=P(0x30000)):
    return lib.csa2_dequantize_kv_fp4_paged(slots, T, n, H, S, D, kc, P(0x200000), P(0x300000), P(0x400000), dt, k, v, kt, kh,
                                            128, 64, NULL, NULL)


@pytest.mark.parametrize("bad,status,word", [
    (dict(dt=1), 1, "bf16 or fp16"), (dict(T=-1), 1, "T=-1"), (dict(H=0), 1, "Hkv=0"), (dict(S=8), 1, "S=8"),
    (dict(D=32), 2, "D=32"), (dict(kt=124), 1, "strides"), (dict(n=1 << 31), 1, "n_blocks"), (dict(k=P(0x10008)), 1, "16-byte"),
    (dict(kc=NULL), 1, "null"), (dict(slots=NULL), 1, "null"), (dict(slots=P(0x20004)), 1, "misaligned"),
    (dict(kt=0), 1, "share"), (dict(kh=56), 1, "share"), (dict(k=P(0x100000)), 1, "overlaps"), (dict(v=P(0x400000)), 1, "overlaps"),
    (dict(v=P(0x20000)), 1, "overlaps"), (dict(v=P(0x10010)), 1, "share"),
])
def test_reading_back_rejects_on_host(lib, bad, status, word):
    _refused(_read(lib, **bad), lib, status, word)


def test_attention_rejects_on_host(lib):
    def call(B=2, T=4, Hq=8, H=2, D=128, dt=0, q=FAKE, qt=1024, S=64, M=4, stride=4, n=9, max_new=1, window=0, kc=FAKE,
             ks=FAKE, table=FAKE, kv=FAKE, lse=NULL, err=NULL, ws=P(0x10000), wsb=1 << 30):
        return lib.csa2_paged_attn_fp4(B, T, Hq, H, D, dt, q, qt, 128, kc, FAKE, ks, FAKE, n, S, table, M, stride, kv,
                                       FAKE, max_new, window, 0.1, FAKE, lse, err, ws, wsb, NULL)
    for bad, status, word in [
            (dict(dt=1), 1, "bf16 or fp16"), (dict(B=-1), 1, "B=-1"), (dict(T=-1), 1, "T=-1"), (dict(Hq=7), 1, "Hq=7"),
            (dict(H=0), 1, "Hkv=0"), (dict(Hq=4096, H=1, T=1 << 20, qt=0), 1, "rows"), (dict(D=96), 2, "D=96"),
            (dict(S=24), 1, "S=24"), (dict(M=0, stride=0), 1, "M=0"), (dict(stride=3), 1, "table_stride=3"),
            (dict(n=-1), 1, "n_blocks"), (dict(max_new=0), 1, "max_new=0"), (dict(window=-1), 1, "window=-1"),
            (dict(qt=1020), 1, "strides"), (dict(q=P(0x1008)), 1, "16-byte"), (dict(ks=P(0x1008)), 1, "16-byte"),
            (dict(table=NULL), 1, "null"), (dict(kc=NULL), 1, "null"), (dict(ks=NULL), 1, "null"),
            (dict(table=P(0x1002)), 1, "4-byte"), (dict(kv=P(0x1002)), 1, "4-byte"), (dict(lse=P(0x1002)), 1, "4-byte"),
            (dict(err=P(0x1002)), 1, "4-byte")]:
        _refused(call(**bad), lib, status, word)
    assert call(B=0, table=NULL) == 0 and call(T=0, q=NULL) == 0          # nothing to do


# ---------------------------------------------------------------- the binding
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


I32, I64, U8, BF, F16, F64 = torch.int32, torch.int64, torch.uint8, torch.bfloat16, torch.float16, torch.float64


def _table_args():
    return dict(inv_freq=_z(32, dtype=F64), cos_sin=_z(10, 32, 2))


def _rope_args():
    return dict(q=_z(5, 4, 128, dtype=BF), pos=_z(5, dtype=I32), cos_sin=_z(10, 32, 2), k=_z(5, 2, 128, dtype=BF),
                q_out=_z(5, 4, 128, dtype=BF), k_out=_z(5, 2, 128, dtype=BF), err_flag=_z(1, dtype=I32))


def _append_args(T=5, H=2, D=64, S=16, n=6):
    return dict(k=_z(T, H, D, dtype=BF), v=_z(T, H, D, dtype=BF), slots=_z(T, dtype=I64), k_codes=_z(n, H, S, D // 2, dtype=U8),
                v_codes=_z(n, H, S, D // 2, dtype=U8), k_scales=_z(n, H, S, D // 16, dtype=U8),
                v_scales=_z(n, H, S, D // 16, dtype=U8), pos=_z(T, dtype=I32), cos_sin=_z(9, 16, 2),
                k_values=_z(T, H, D, dtype=BF), v_values=_z(T, H, D, dtype=BF))


def _read_args():
    a = _append_args()
    return {n: a[n] for n in ("slots", "k_codes", "v_codes", "k_scales", "v_scales", "k", "v")}


def _attn_args(T=5, B=2, H=2, Hq=6, D=64, S=16, n=6):
    a = _append_args(T, H, D, S, n)
    return dict(q=_z(T, Hq, D, dtype=BF), k_codes=a["k_codes"], v_codes=a["v_codes"], k_scales=a["k_scales"],
                v_scales=a["v_scales"], block_table=_z(B, 4, dtype=I32), kv_len=_z(B, dtype=I32),
                cu_len=_z(B + 1, dtype=I32), out=_z(T, Hq, D, dtype=BF), sm_scale=0.1, max_new=3,
                lse=_z(T, Hq), err_flag=_z(1, dtype=I32), workspace=_z(1 << 20, dtype=U8))


PLANES = dict(k_codes=_z(6, 2, 16, 32), v_codes=_z(6, 2, 16, 16, dtype=U8), k_scales=_z(6, 2, 16, 2, dtype=U8),
              v_scales=_z(6, 2, 16, 4))


BAD = [
    ("csa2_rope_table", _table_args, dict(inv_freq=_z(32), cos_sin=_z(10, 31, 2))),
    ("csa2_rope", _rope_args, dict(q=_z(5, 4, 128), pos=_z(4, dtype=I32), cos_sin=_z(10, 64), k=_z(4, 2, 128, dtype=BF),
                                   q_out=_z(5, 4, 128, dtype=F16), k_out=_z(5, 2, 64, dtype=BF), err_flag=_z(1))),
    ("csa2_quantize_kv_fp4_paged", _append_args, dict(k=_z(5, 2, 64), v=_z(5, 2, 64, dtype=F16), slots=_z(4, dtype=I64),
                                                      pos=None, cos_sin=_z(9, 32), k_values=_z(5, 2, 64),
                                                      v_values=_z(5, 64, 2, dtype=BF).transpose(1, 2), **PLANES)),
    ("csa2_dequantize_kv_fp4_paged", _read_args, dict(slots=_z(4, dtype=I64), k=_z(5, 2, 64), v=_z(5, 2, 64, dtype=F16), **PLANES)),
    ("csa2_paged_attn_fp4", _attn_args, dict(q=_z(5, 6, 64), block_table=_z(2, 8, dtype=I32)[:, ::2], kv_len=_z(3, dtype=I32),
                                             cu_len=_z(2, dtype=I32), out=_z(5, 6, 64, dtype=F16), lse=_z(5, 6, dtype=BF),
                                             err_flag=_z(1), workspace=_z(8, 8, dtype=U8).T, **PLANES)),
]


@pytest.mark.parametrize("fn,args,bad", BAD)
def test_binding_refuses_what_does_not_fit(fake, fn, args, bad):
    getattr(csa2, fn)(**args())
    assert fake.calls == [fn]
    for name, value in bad.items():
        with pytest.raises((TypeError, ValueError)):
            getattr(csa2, fn)(**{**args(), name: value})
    assert fake.calls == [fn]


class _Recorder:
    """C functions that keep what they are given."""

    def __init__(self):
        self.calls = []
        self.fns = {}

    def __getattr__(self, name):
        if name not in self.fns:
            real = getattr(REAL, name)
            self.fns[name] = ctypes.CFUNCTYPE(real.restype, *real.argtypes)(lambda *a: self.calls.append((name, a)) or 7)
        return self.fns[name]


@pytest.fixture()
def quick():
    """The extension, bound to recorders; tensors of the CPU pass for ones of the current device."""
    r = _Recorder()
    csa2._bind(r, lambda dev: 0x7700, lambda: -1)
    yield r
    csa2._bind(REAL)


def _positional(fn, args):
    """All arguments of the Python function, in its order."""
    sig = inspect.signature(getattr(csa2, fn))
    b = sig.bind(**args)
    b.apply_defaults()
    assert list(b.arguments) == list(sig.parameters)
    return list(b.arguments.values())


def _as_given(v):
    return None if v in (None, 0) else (struct.unpack("f", struct.pack("f", v))[0] if isinstance(v, float) else int(v))


BINDINGS = [("csa2_rope_table", _table_args), ("csa2_rope", _rope_args), ("csa2_quantize_kv_fp4_paged", _append_args),
            ("csa2_dequantize_kv_fp4_paged", _read_args), ("csa2_paged_attn_fp4", _attn_args)]


def _usual(fn, args):
    """Calls that fit, of every kind."""
    a = args()
    yield a
    if fn == "csa2_rope_table":
        yield {**a, "start": 1 << 30, "amplitude": 1.5, "stream": 0x99}
        yield {**a, "inv_freq": _z(0, dtype=F64), "cos_sin": _z(0, 0, 2)}
        return
    yield {**a, "stream": type("S", (), {"cuda_stream": 0x55})()}
    yield {**a, "err_flag": _z(2, dtype=torch.uint32)}
    if fn == "csa2_rope":
        yield {**a, "k": None, "k_out": None}
        yield {**a, "q_out": None, "k_out": None, "layout": 0, "first": 8}
        qkv = _z(5, 8, 128, dtype=BF)
        yield {**a, "q": qkv[:, :4], "k": qkv[:, 4:6]}
        yield {**a, "q": _z(1, 4, 128, dtype=F16)[:, :1], "k": None, "q_out": _z(1, 1, 200, dtype=F16)[..., :128], "k_out": None, "pos": _z(1, dtype=I32)}
        return
    planes = {n: torch.zeros_like(a[n]).view(torch.float8_e4m3fn) for n in ("k_scales", "v_scales")}
    yield {**a, **planes}
    if fn == "csa2_quantize_kv_fp4_paged":
        yield {**a, "pos": None, "cos_sin": None, "k_values": None}
        yield {**a, "k": _z(2, 5, 64, dtype=BF).transpose(0, 1), "v": _z(5, 1, 64, dtype=BF).expand(5, 2, 64)}
        yield {**a, "k": _z(5, 2, 64, dtype=torch.int16), "v": _z(5, 2, 64, dtype=torch.int16), "k_values": None, "v_values": None}
    if fn == "csa2_paged_attn_fp4":
        yield {**a, "lse": None, "window": 9, "block_table": _z(2, 8, dtype=I32)[:, :3]}
        yield {**a, "q": _z(5, 20, 64, dtype=BF)[:, 4:10]}
        yield {**a, "block_table": _z(2, 2, dtype=I32)[:, ::2]}


@pytest.mark.parametrize("fn,args", BINDINGS)
def test_the_extension_hands_over_what_the_binding_does(quick, monkeypatch, fn, args):
    cases = list(_usual(fn, args))
    for a in cases:
        assert getattr(csa2._csa2_bind, fn)(*_positional(fn, a)) == 7
    given = []
    monkeypatch.setattr(csa2, "_on_device", lambda t: True)
    monkeypatch.setattr(csa2, "_stream", lambda s: 0x7700 if s is None else getattr(s, "cuda_stream", s))
    monkeypatch.setattr(csa2, "_lib", type("L", (), {fn: staticmethod(lambda *a: given.append(a) or 0)}))
    monkeypatch.setattr(csa2, "_csa2_bind", type("B", (), {fn: staticmethod(lambda *a: None)}))
    for a in cases:
        getattr(csa2, fn)(**a)
    assert len(given) == len(quick.calls) == len(cases)
    for (name, took), want in zip(quick.calls, given):
        assert name == fn and [_as_given(v) for v in took] == [_as_given(v) for v in want]


@pytest.mark.parametrize("fn,args,bad", BAD)
def test_the_extension_leaves_what_does_not_fit(quick, fn, args, bad):
    call = getattr(csa2._csa2_bind, fn)
    for name, value in bad.items():
        assert call(*_positional(fn, {**args(), name: value})) is None, name
    good = _positional(fn, args())
    names = list(inspect.signature(getattr(csa2, fn)).parameters)
    for i, v in enumerate(good):                                         # of other kinds altogether
        for x in ("x", 2 ** 70, _z(3), None):
            if (x is None and not isinstance(v, (int, float))) or (names[i] == "workspace" and torch.is_tensor(x)):
                continue
            assert call(*good[:i], x, *good[i + 1:]) is None, (names[i], x)
    assert call(*good[:-1]) is None and call(*good, None) is None and call() is None
    assert quick.calls == []


def test_the_extension_leaves_other_devices_and_classes(quick):
    a = _positional("csa2_rope", _rope_args())
    sub = a[0].as_subclass(type("T", (torch.Tensor,), {}))
    meta = torch.empty(a[0].shape, dtype=BF, device="meta")
    assert csa2._csa2_bind.csa2_rope(sub, *a[1:]) is None and csa2._csa2_bind.csa2_rope(meta, *a[1:]) is None
    csa2._bind(quick, lambda dev: 0, lambda: 0)                          # the current device is another
    assert csa2._csa2_bind.csa2_rope(*a) is None
    b = _positional("csa2_paged_attn_fp4", {**_attn_args(), "workspace": None})
    csa2._bind(quick, lambda dev: 0, lambda: -1)
    assert csa2._csa2_bind.csa2_paged_attn_fp4(*b) is None and quick.calls == []


def test_binding_refuses_the_rest(fake):
    a = _attn_args(Hq=6)
    a["q"], a["out"], a["lse"] = _z(5, 5, 64, dtype=BF), _z(5, 5, 64, dtype=BF), _z(5, 5)
    with pytest.raises(ValueError):
        csa2.csa2_paged_attn_fp4(**a)
    with pytest.raises(ValueError):
        csa2.csa2_rope(**{**_rope_args(), "k": None})
    assert fake.calls == []


def test_binding_refuses_tensors_off_the_gpu():
    for fn, args in ((csa2.csa2_rope_table, _table_args), (csa2.csa2_rope, _rope_args),
                     (csa2.csa2_quantize_kv_fp4_paged, _append_args), (csa2.csa2_dequantize_kv_fp4_paged, _read_args)):
        with pytest.raises(ValueError):
            fn(**args())


# ---------------------------------------------------------------- the class, with a stand-in for the library
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


def _cache(bits, rope=True, **kw):
    from sparse_attention_fp4_quantize_gb300.paged import PagedCache, PagedShape
    from sparse_attention_fp4_quantize_gb300.rope import Rope
    return PagedCache(PagedShape(requests=2, tokens=4, max_context=64, n_blocks=4, heads=4, kv_heads=2, dim=64, block_size=16,
                                 layers=3, bits=bits, rope=Rope(32) if rope else None, **kw), device="cpu")


@pytest.mark.parametrize("bits,append,attend", [(8, ["csa2_rope", "csa2_quantize_kv_fp8_paged"], ["csa2_rope", "csa2_paged_attn_fp8"]),
                                                (4, ["csa2_quantize_kv_fp4_paged"], ["csa2_rope", "csa2_paged_attn_fp4"])])
def test_the_cache_rotates_on_the_way(calls, bits, append, attend):
    cache = _cache(bits)
    assert [n for n, _ in calls.calls] == ["csa2_rope_table"]
    q, kv = _z(4, 4, 64, dtype=BF), _z(4, 2, 64, dtype=BF)
    del calls.calls[:]
    cache.append(0, kv, kv)
    assert [n for n, _ in calls.calls] == append
    del calls.calls[:]
    used = set()
    for layer in range(3):
        cache.attend(layer, q, stream=layer + 1)
        assert [n for n, _ in calls.calls[-len(attend):]] == attend
        used.add(calls.calls[-1][1][-3])
    assert len(used) == 3                                                # a workspace per layer
    plain = _cache(bits, rope=False)
    del calls.calls[:]
    plain.append(0, kv, kv), plain.attend(0, q)
    assert [n for n, _ in calls.calls] == [append[-1], attend[-1]]


def test_the_cache_refuses(calls):
    kv = _z(4, 2, 64, dtype=BF)
    with pytest.raises(ValueError):
        _cache(6)
    with pytest.raises(ValueError):
        _cache(8).read(0, _z(4, dtype=I64), kv, kv)
    with pytest.raises(ValueError):
        _cache(8).append(0, kv, kv, k_values=kv)


# ---------------------------------------------------------------- frequencies
def test_frequencies_of_a_stretched_context():
    from sparse_attention_fp4_quantize_gb300.rope import Rope
    f, amp = Rope(64).frequencies()
    assert amp == 1.0 and f.dtype is F64
    assert np.allclose(f.numpy(), [10000.0 ** (-i / 32) for i in range(32)], rtol=1e-15)
    g, amp = Rope(64, factor=8.0, original=4096).frequencies()
    assert amp == pytest.approx(0.1 * math.log(8) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32])                   # fast pairs as they were
    assert torch.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)   # slow ones by the factor
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((g < f) & (g > f / 8))[mid].all()


# ---------------------------------------------------------------- the references
def test_reference_scale_and_codes():
    assert list(ref.nearest(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 99]), ref.GRID)) == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    x = torch.cat([torch.linspace(0, 448, 20001), torch.randn(20000).abs() * 0.01])
    assert np.array_equal(ref.E4M3[ref.nearest(x.double().numpy(), ref.E4M3)], x.to(torch.float8_e4m3fn).double().numpy())
    g = np.random.default_rng(1).normal(size=(7, 64))
    c, s, v = ref.quantise(g)
    assert np.array_equal(ref.values(torch.from_numpy(c), torch.from_numpy(s)), v)


def test_reference_quantises_as_the_oracle(orc):
    rows = torch.randn(50, 128, generator=torch.Generator().manual_seed(3)).to(BF)
    rows[3, 5], rows[4, :16], rows[5, :16] = 1e30, 0.0, 2.0 ** -12
    oc, os_ = orc.quantize_kv_fp4(rows.view(torch.int16).numpy().view(np.uint16))
    c, s, _ = ref.quantise(rows.double().numpy())
    assert np.array_equal(c, oc) and np.array_equal(s, os_)
