"""Rotations by frequencies of the caller's own (tolerances: test_gpu_rope)."""
from __future__ import annotations

import math

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from block_scaled_fp4_pre_gb300 import attention as att
from tests.test_gpu_rope import data

pytestmark = pytest.mark.gpu


def table_of(dims, w=None):
    t = torch.empty(mx.moe_rope_table_size(dims), dtype=torch.uint8, device="cuda")
    if w is None:
        mx.moe_rope_prepare(dims, t)
    else:
        mx.moe_rope_prepare_frequencies(dims, w, t)
    return t


@pytest.mark.parametrize("layout", [mx.MOE_ROPE_HALF, mx.MOE_ROPE_INTERLEAVED])
@pytest.mark.parametrize("D,rotary", [(64, 64), (128, 64), (80, 20)])
def test_frequencies_given(D, rotary, layout):
    dims = mx.make_rope_dims(D, rotary, layout, scaling=mx.MOE_ROPE_YARN, factor=32.0,
                             original_length=4096.0)
    m = 0.1 * math.log(32.0) + 1
    pos = torch.tensor([0, 1, -1, 777, 4095, 131071, 1 << 20, 2 ** 31 - 1], dtype=torch.int32,
                       device="cuda")
    x = data(len(pos), 5, D, seed=4)
    edges = [0.0, 1.0, math.nextafter(2 * math.pi, 0)] + [0.1 ** i for i in range(3, rotary // 2)]
    for w in (mx.yarn_frequencies(rotary, 150000.0, 32.0, 4096.0),
              mx.yarn_frequencies(rotary, 150000.0, 32.0, 4096.0, whole=False), edges):
        out = torch.empty_like(x)
        mx.moe_rope(dims, table_of(dims, w), x, pos, out)
        angle = pos.cpu().double().view(-1, 1, 1) * torch.tensor(w, dtype=torch.float64)
        # a frequency of up to 2 pi has 2^-50 between doubles, and the oracle's product with the
        # position is rounded to 53 bits: together under |angle| 2^-51
        slack = angle.abs() * 2.0 ** -51
        y = x.cpu().double()
        first, second = (slice(0, rotary // 2), slice(rotary // 2, rotary)) \
            if layout == mx.MOE_ROPE_HALF else (slice(0, rotary, 2), slice(1, rotary, 2))
        a, b, got = y[..., first], y[..., second], out.cpu().double()
        tol = (a.abs() + b.abs()) * m * (2.0 ** -21 + slack)
        for part, want in ((first, m * (a * angle.cos() - b * angle.sin())),
                           (second, m * (b * angle.cos() + a * angle.sin()))):
            assert torch.all((got[..., part] - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8)
        assert torch.equal(out[..., rotary:], x[..., rotary:])


def test_the_same_frequencies_give_the_same_table():
    dims = mx.make_rope_dims(128, base=2.0 ** 64)        # powers of two, exact in any order
    assert torch.equal(table_of(dims), table_of(dims, [0.5 ** i for i in range(64)]))


def test_a_layer_with_frequencies():
    rope = mx.make_rope_dims(64)
    dims = mx.make_attention_dims(4, 2, 64, 8, 16, 16)
    w = mx.yarn_frequencies(64, 1e4, 16.0, 65536.0)
    a, b = att.Attention(dims, rope, frequencies=w), att.Attention(dims, rope)
    assert torch.equal(a.table, table_of(rope, w)) and not torch.equal(a.table, b.table)
