"""Frequencies of the caller's own, and YaRN's with a ramp over the pairs' indices."""
from __future__ import annotations

import ctypes
import math

import pytest

from tests.test_attention_host import mx  # noqa: F401


def turns(d, base, length, i):
    return length * base ** (-2 * i / d) / (2 * math.pi)


def index_of(d, base, length, t):
    """Where turns falls to t, by halving."""
    low, high = -4.0 * d, 4.0 * d
    for _ in range(200):
        mid = (low + high) / 2
        low, high = (mid, high) if turns(d, base, length, mid) > t else (low, mid)
    return low


CASES = [(64, 1e4, 16.0, 65536.0), (64, 1.5e5, 32.0, 4096.0), (128, 1e6, 4.0, 32768.0),
         (128, 500000.0, 8.0, 8192.0), (16, 1e4, 2.0, 100.0), (2, 1e4, 4.0, 4096.0)]


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("d,base,factor,length", CASES)
def test_ramp_over_indices(mx, d, base, factor, length, whole):  # noqa: F811
    w = mx.yarn_frequencies(d, base, factor, length, whole=whole)
    low, high = (index_of(d, base, length, t) for t in (32.0, 1.0))
    if whole:
        low, high = math.floor(low + 1e-9), math.ceil(high - 1e-9)
    low, high = max(low, 0), min(high, d - 1)
    assert len(w) == d // 2
    for i, f in enumerate(w):
        plain = base ** (-2 * i / d)
        if i <= low:
            part = 0.0
        elif i >= high:
            part = 1.0
        else:
            part = (i - low) / (high - low)
        want = plain * (1 - part) + plain * part / factor
        assert abs(f - want) <= 1e-9 * want


@pytest.mark.parametrize("case,pair,times", [(CASES[0], 29, 3.28), (CASES[1], 16, 4.28),
                                             (CASES[2], 32, 1.71)])
def test_it_is_not_the_ramp_over_turns(mx, case, pair, times):  # noqa: F811
    d, base, factor, length = case
    plain, t = base ** (-2 * pair / d), turns(d, base, length, pair)
    g = min(1.0, max(0.0, (t - 1.0) / 31.0))
    over_turns = plain * g + plain / factor * (1 - g)
    got = mx.yarn_frequencies(d, base, factor, length)[pair] / over_turns
    assert abs(max(got, 1 / got) - times) < 0.01


def test_refusals(mx):  # noqa: F811
    d, f = mx.make_rope_dims(16), mx.lib()
    good = [0.5 ** i for i in range(8)]

    def prepare(w, table=1024, size=64):
        w = None if w is None else (ctypes.c_double * len(w))(*w)
        return f.moe_rope_prepare_frequencies(ctypes.byref(d), w, table, size, None)

    assert prepare(None) == mx.MOE_ERR_INVALID_ARG
    for bad in (-1e-9, 2 * math.pi, 7.0, math.inf, -math.inf, math.nan):
        for i in (0, 7):
            assert prepare(good[:i] + [bad] + good[i + 1:]) == mx.MOE_ERR_INVALID_ARG
    assert prepare(good, table=None) == mx.MOE_ERR_INVALID_ARG
    assert prepare(good, table=1032) == mx.MOE_ERR_INVALID_ARG
    assert prepare(good, size=63) == mx.MOE_ERR_INVALID_ARG
    d.rotary_dim = 3
    assert prepare(good) == mx.MOE_ERR_INVALID_ARG
    for n in (7, 9):
        with pytest.raises(ValueError):
            mx.moe_rope_prepare_frequencies(mx.make_rope_dims(16), [0.1] * n, 1024)
