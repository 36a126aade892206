"""Outputs of the paged 4-bit cache's calls that lie on the error flag are refused, on the CPU: host checks of the C ABI."""
from __future__ import annotations

import ctypes

import pytest

import sparse_attention_fp4_quantize_gb300 as csa2
from test_paged_fp4_checks import _append, _refused

P = ctypes.c_void_p


@pytest.mark.parametrize("flag", [0x100000, 0x2003FC, 0x3000F0, 0x400004, 0x500000, 0x6003FC])
def test_append_on_the_flag_is_refused(flag):
    """8 blocks of 2 heads, 16 tokens, 64 channels: codes of 8192 bytes, scales of 1024; values of 1024."""
    _refused(_append(csa2._lib, kval=P(0x500000), vval=P(0x600000), err=P(flag)), csa2._lib, 1, "overlap")


@pytest.mark.parametrize("flag", [0x10000, 0x303FC])
def test_reading_back_on_the_flag_is_refused(flag):
    """k, v [4, 2, 64]: 1024 bytes."""
    rc = csa2._lib.csa2_dequantize_kv_fp4_paged(P(0x20000), 4, 8, 2, 16, 64, P(0x100000), P(0x200000), P(0x300000), P(0x400000), 0,
                                                P(0x10000), P(0x30000), 128, 64, 128, 64, P(flag), None)
    _refused(rc, csa2._lib, 1, "overlaps")
