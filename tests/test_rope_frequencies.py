"""Frequencies of stretched contexts, on the CPU: both ramps pinned at the middle pairs, the caller's own frequencies."""
from __future__ import annotations

import math

import pytest
import torch

from sparse_attention_fp4_quantize_gb300.rope import Rope

F64 = torch.float64


def _plain(dim, theta):
    return torch.tensor([math.exp(-2 * i / dim * math.log(theta)) for i in range(dim // 2)], dtype=F64)


# (dim, theta, factor, original), and the pairs that make 32 turns and 1 turn over the original context, i of
# original theta^(-2 i / dim) = 2 pi n, rounded down and up: worked out by hand from the logarithms below.
#   128 channels: 128 ln(32768 / 64 pi) / (2 ln 10^6) = 128 * 5.0936 / 27.6310 = 23.596; 128 * 8.5593 / 27.6310 = 39.651
#    64 channels:  64 ln(4096 / 64 pi) / (2 ln 10^4) = 64 * 3.0142 / 18.4207 = 10.472;  64 * 6.4799 / 18.4207 = 22.514
STRETCHED = [((128, 1e6, 4.0, 32768), 23, 40), ((64, 1e4, 40.0, 4096), 10, 23)]


@pytest.mark.parametrize("config,low,high", STRETCHED)
def test_stretched_frequencies_go_by_the_pairs_index(config, low, high):
    """Between the two pairs the share of the slowed frequency grows by 1 / (high - low) per pair."""
    dim, theta, factor, original = config
    f, amp = Rope(dim, theta=theta, factor=factor, original=original).frequencies()
    share = [min(max((i - low) / (high - low), 0.0), 1.0) for i in range(dim // 2)]
    want = _plain(dim, theta) * torch.tensor([1 - s + s / factor for s in share], dtype=F64)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-15)
    # rounded: exponent of up to ln(theta) * 2^-53 in the power, and four more operations
    assert torch.allclose(f, want, rtol=64 * 2.0 ** -52, atol=0.0)


@pytest.mark.parametrize("config,low,high", STRETCHED)
def test_stretched_frequencies_by_turns(config, low, high):
    """The other ramp, linear in the turns that a pair makes over the original context."""
    dim, theta, factor, original = config
    f, amp = Rope(dim, theta=theta, factor=factor, original=original, ramp="turns").frequencies()
    plain = _plain(dim, theta)
    keep = [min(max((original * p / (2 * math.pi) - 1) / 31, 0.0), 1.0) for p in plain.tolist()]
    want = plain * torch.tensor([k + (1 - k) / factor for k in keep], dtype=F64)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-15)
    # near the slow end `keep` is a difference of numbers close to 1: 2^-52 of 32 turns' share, of a result of 1 / factor
    assert torch.allclose(f, want, rtol=64 * factor * 2.0 ** -52, atol=0.0)
    g, _ = Rope(dim, theta=theta, factor=factor, original=original).frequencies()
    assert ((f - g).abs() > 0.01 * g).sum() > 10                         # the two are not near one another


def test_ramps_without_a_middle():
    """A context so short that no pair makes `fast` turns begins its ramp at pair 0; `fast` and `slow` within one pair's
    reach still have a pair on either side."""
    f, _ = Rope(32, theta=1000.0, factor=2.0, original=64).frequencies()       # 5.40 pairs make a turn, none 32
    want = _plain(32, 1000.0) * torch.tensor([1 - 0.5 * min(i / 6, 1) for i in range(16)], dtype=F64)
    assert torch.allclose(f, want, rtol=1e-13, atol=0.0)
    f, _ = Rope(32, theta=1000.0, factor=2.0, original=4096, fast=4096 / (2 * math.pi) * 1.01, slow=4096 / (2 * math.pi) * 1.005).frequencies()
    assert torch.allclose(f, _plain(32, 1000.0) * torch.tensor([1.0] + [0.5] * 15, dtype=F64), rtol=1e-13, atol=0.0)


def test_frequencies_of_the_caller():
    own = [1.0, 0.3, -0.02, 0.0, 1e-9, 7.0, 0.25, 0.125]
    for given in (own, torch.tensor(own, dtype=F64), torch.tensor(own, dtype=F64).numpy()):
        rope = Rope(16, inv_freq=given)
        f, amp = rope.frequencies()
        assert f.dtype is F64 and f.tolist() == own and amp == 1.0 and rope == Rope(16, inv_freq=own)
    assert Rope(16, inv_freq=own, amplitude=1.25).frequencies()[1] == 1.25
    f, amp = Rope(64, factor=8.0, amplitude=0.5).frequencies()            # also with a stretched context's
    assert amp == 0.5 and torch.equal(f, Rope(64, factor=8.0).frequencies()[0])
    for bad in (dict(inv_freq=own[:7]), dict(inv_freq=[own]), dict(inv_freq=own, factor=2.0), dict(ramp="linear", factor=2.0)):
        with pytest.raises(ValueError):
            Rope(16, **bad).frequencies()


@pytest.mark.parametrize("bad", [dict(theta=-10000.0), dict(theta=0.0), dict(theta=math.nan), dict(theta=math.inf), dict(factor=0.5), dict(factor=0.0),
                                 dict(factor=-2.0), dict(factor=math.nan), dict(factor=math.inf), dict(factor=2.0, theta=1.0),
                                 dict(factor=2.0, original=0), dict(factor=2.0, original=-4096), dict(factor=2.0, fast=1.0),
                                 dict(factor=2.0, fast=0.5), dict(factor=2.0, slow=-1.0),
                                 dict(factor=2.0, fast=math.nan)])
@pytest.mark.parametrize("ramp", ["index", "turns"])
def test_frequencies_without_a_meaning_are_refused(ramp, bad):
    with pytest.raises(ValueError, match="theta|factor|original|fast"):
        Rope(64, ramp=ramp, **bad).frequencies()


def test_a_ramp_in_turns_may_end_at_none():
    f, _ = Rope(64, factor=2.0, slow=0.0, ramp="turns").frequencies()
    want = [p * (0.5 + 0.5 * min(4096 * p / (2 * math.pi) / 32, 1.0)) for p in _plain(64, 10000.0).tolist()]
    assert torch.allclose(f, torch.tensor(want, dtype=F64), rtol=1e-13, atol=0.0)
    with pytest.raises(ValueError, match="slow"):
        Rope(64, factor=2.0, slow=0.0).frequencies()                     # no pair makes no turns
