"""The turns per position that the rotary kernels multiply positions by, against 80 decimal digits."""
import pytest

import mla_decode_attention_14_b200 as mla
from mla_decode_attention_14_b200 import build as mla_build
from tests import exact_rope


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(base=1.0000001), dict(base=1e6), dict(base=1e300), dict(base=123.456), dict(factor=4.0),
    dict(factor=40.0, original_len=4096), dict(factor=8.0, original_len=8192, beta_fast=16.0, beta_slow=2.0),
    dict(factor=32.0, original_len=131072, base=500000.0), dict(factor=2.0, original_len=1), dict(factor=1e9),
    dict(factor=3.7, original_len=2 ** 31 - 1), dict(factor=1.0, original_len=4096)])
def test_turns_are_exact_to_the_last_places(kw):
    """Every factor of a turn is off by at most an ulp of 2^-63 in the host's extended precision, some six of them in
    all: under 0.16 * 2^64 * 6 * 2^-64 < 1 unit of 2^-64 turns (a turn per position is below 0.16), and half a unit
    for the rounding, so within one of the nearest integer."""
    got, want = mla.rope(**kw).turns, exact_rope.turns(**kw)
    assert max(abs(a - b) for a, b in zip(got, want)) <= 1, [a - b for a, b in zip(got, want)]


def test_the_exact_form():
    """2^64 / (2 pi) by its own digits, and a frequency that is a power of ten."""
    t = exact_rope.turns()
    assert t[0] == 2935890503282001226 and t[16] == round(2935890503282001226 / 100)
    a = exact_rope.angles([1, 0, -1])
    assert abs(a[0][0] - 1.0) < 1e-15 and a[1][5] == 0.0 and abs(a[2][0] + 1.0 - 6.283185307179586) < 1e-14
