"""The operators around the expert layer at the edges of what they take."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests import test_gpu_norm as norm
from tests.test_gpu_linear import F4, F8, Linear, inputs

pytestmark = pytest.mark.gpu


def test_a_single_row_of_a_wider_matrix():
    # its stride is no multiple of 8, and is not used
    x, r, gamma = norm.make(1, 256, 3)
    wide = torch.zeros(5, 260, dtype=torch.bfloat16, device="cuda")
    wide[2:3, :256] = x                     # 1040 bytes in: 16-byte aligned
    row = wide[2:3, :256]
    want = norm.run(x, r, gamma, mx.MOE_SF_PACKED)
    q, sf = torch.empty_like(want[0]), torch.empty_like(want[1])
    mx.moe_rmsnorm_mxfp8(row, gamma, norm.EPS, q, sf, mx.MOE_SF_PACKED, residual=r, y=row)
    assert torch.equal(q, want[0]) and torch.equal(sf, want[1]) and torch.equal(row, want[3])
    wide[2:3, :256] = x
    for mma in (F4, F8):
        lin = Linear(128, 256, 4, mma)
        a, b = (torch.empty(1, 128, device="cuda") for _ in range(2))
        mx.moe_linear_forward(lin.dims, lin.prepared, x, a, lin.ws)
        mx.moe_linear_forward(lin.dims, lin.prepared, row, b, lin.ws)
        assert torch.equal(a, b)
