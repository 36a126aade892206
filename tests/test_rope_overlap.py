"""Where csa2_rope's outputs may lie, on the CPU: host checks of the C ABI.  Every call here is refused, for a reason that is
looked at last, so that what is named before it was accepted."""
from __future__ import annotations

import numpy as np
import pytest

import paged_fp4_ref  # noqa: F401  (the folder of the tests is on the path)
import sparse_attention_fp4_quantize_gb300 as csa2
from test_paged_fp4_checks import ROPE, _refused, _rope

LAST = "overlaps the other input"


def _says(word, **kw):
    """The call with k written into q's rows, which nothing but the last check refuses: no call gets by."""
    a = {**ROPE, **kw}
    _refused(_rope(csa2._lib, **{**kw, "ko": a["q"], "kos": a["qs"]}), csa2._lib, 1, word)


def test_an_output_may_lie_in_other_columns_of_its_inputs_buffer():
    """q [8, 4, 128] in the first 512 columns of a buffer of 2048, q_out in 512 others of it, before or behind."""
    wide = dict(qs=(2048, 128), qos=(2048, 128))
    for column in (512, 1024, 1536, 512 - 2048):
        _says(LAST, **wide, qo=0x100000 + 2 * column)
    _says(LAST, **wide, q=0x100000 + 2 * 1024, qo=0x100000)
    for column in (8, 504, 1544, 2040, 504 - 2048, 520 - 2048 - 512):    # 8 columns too near, or only 8 apart
        _says("overlaps its input", **wide, qo=0x100000 + 2 * column)


@pytest.mark.parametrize("bad", [dict(qo=0x100010), dict(qos=(1024, 128), qo=0x100000),
                                 dict(qs=(2048, 128), qos=(1024, 128), qo=0x100000 + 2 * 504)])
def test_an_output_on_its_input_is_refused(bad):
    _says("overlaps its input", **bad)


# ---- q in place and k_out; k's input is q's rows, so that the last check always refuses
def _places(T, H, D, token, head, step, token2=None, head2=None):
    """What csa2_rope says of q rows at `base` and k_out rows `step` elements on."""
    token2, head2 = token if token2 is None else token2, head if head2 is None else head2
    base = 0x10000000
    rc = _rope(csa2._lib, q=base, qo=base, Hq=H, qs=(token, head), qos=(token, head), k=base, ko=base + 2 * step, Hk=H, ks=(token, head),
               kos=(token2, head2), T=T, D=D, dim=16, pos=0x100, table=0x200, n=1)
    said = csa2._lib.csa2_last_error().decode()
    assert rc == 1, (rc, said)
    return said


@pytest.mark.parametrize("T", [1, 2, 77])
@pytest.mark.parametrize("parts", [2, 3])
def test_slices_of_every_head_are_apart(T, parts):
    """[T, H, parts * D], the projections of a head beside one another, and the same with heads first."""
    H, D = 5, 64
    for i in range(-parts + 1, parts):
        for token, head in ((H * parts * D, parts * D), (parts * D, T * parts * D)):
            assert (LAST in _places(T, H, D, token, head, i * D)) == (i != 0), (i, token)
            if i:
                for near in (8, -8):
                    at = i * D + near
                    fine = abs(at) >= D and abs(at) <= (parts - 1) * D
                    assert (LAST in _places(T, H, D, token, head, at)) == fine, (i, token, near)


def test_halves_of_the_tokens_of_every_head_are_apart():
    """[H, 2 T, D]: the first and the last T tokens of each head."""
    T, H, D = 6, 3, 64
    assert LAST in _places(T, H, D, D, 2 * T * D, T * D) and LAST in _places(T, H, D, D, 2 * T * D, -T * D)
    assert LAST not in _places(T, H, D, D, 2 * T * D, T * D - 8)


def test_rows_that_share_elements_are_never_accepted():
    """Small layouts of any strides against the elements themselves."""
    rng = np.random.default_rng(1)
    seen = [0, 0, 0]
    for _ in range(4000):
        T, H, D = int(rng.integers(1, 5)), int(rng.integers(1, 5)), 16
        strides = [int(8 * rng.integers(1, 24)) for _ in range(4)]
        if rng.random() < 0.5:
            strides[2:] = strides[:2]
        step = int(8 * rng.integers(-60, 61))
        rows = lambda a, b: (np.arange(T)[:, None, None] * a + np.arange(H)[:, None] * b + np.arange(D)).ravel()  # noqa: E731
        x, y = rows(*strides[:2]), rows(*strides[2:]) + step
        if np.unique(x).size < x.size or np.unique(y).size < y.size:
            continue                                                     # refused as such
        said = _places(T, H, D, *strides[:2], step, *strides[2:])
        if "rows of an output" in said:
            continue
        meet = np.intersect1d(x, y).size > 0
        assert not (meet and LAST in said), (T, H, strides, step)
        seen[0 if meet else 1 if LAST in said else 2] += 1
    assert seen[0] > 100 and seen[1] > 100
