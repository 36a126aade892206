"""Where csa2_rope's outputs may lie, on the CPU: host checks of the C ABI.  Every call here is refused, for a reason that is
looked at last, so that what is named before it was accepted."""
from __future__ import annotations

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
                                 dict(qs=(2048, 128), qos=(1024, 128), qo=0x100000 + 1024)])
def test_an_output_on_its_input_is_refused(bad):
    _says("overlaps its input", **bad)
