"""The operators around the expert layer where something goes wrong: waits that run out and
tensors that are not what a call needs."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.test_gpu_block import make as make_block
from tests.test_gpu_linear import F4, F8, Linear, inputs

pytestmark = pytest.mark.gpu


# the product that quantises bf16 rows itself, over eight blocks and in one; the split one on
# quantised rows; whole tiles of 64 and 128 rows
@pytest.mark.parametrize("mma", [F4, F8])
@pytest.mark.parametrize("rows,N,K", [(5, 512, 4096), (32, 5000, 8192), (3, 100, 256),
                                      (48, 256, 4096), (100, 2048, 8192), (300, 2000, 1024),
                                      (20102, 810, 160)])
def test_a_product_whose_waits_run_out_leaves_nothing_behind(rows, N, K, mma):
    lin = Linear(N, K, rows, mma)
    x = inputs(rows, K)
    want = torch.empty(rows, N, dtype=torch.float32, device="cuda")
    mx.moe_linear_forward(lin.dims, lin.prepared, x, want, lin.ws)
    mx.moe_linear_check(lin.ws)
    out = torch.empty_like(want)
    for _ in range(3):
        mx.moe_debug_linear_give_up(lin.ws, True)
        mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
        mx.moe_debug_linear_give_up(lin.ws, False)
        # the next call's blocks take the shared and tensor memory that the last ones left
        mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
        with pytest.raises(mx.MoeError) as e:
            mx.moe_linear_check(lin.ws)
        assert e.value.status == mx.MOE_ERR_TIMEOUT
        assert torch.equal(out, want)
    mx.moe_linear_check(lin.ws)                 # cleared


def test_give_up_refusals():
    for ws, status in ((None, mx.MOE_ERR_INVALID_ARG),
                       (torch.empty(1024, dtype=torch.uint8, device="cuda")[256:],   # no base
                        mx.MOE_ERR_WORKSPACE_MISMATCH)):
        with pytest.raises(mx.MoeError) as e:
            mx.moe_debug_linear_give_up(ws, True)
        assert e.value.status == status


@pytest.mark.parametrize("T", [4, 20])
def test_block_refuses_routing_of_other_types(T):
    b, attn, res = make_block(T)
    g = torch.Generator(device="cuda").manual_seed(2)
    w, ids = torch.topk(torch.rand(T, 16, generator=g, device="cuda"), 4)     # int64 ids
    b.forward(attn, res.clone(), (ids.int(), w))
    b.check()
    for routing in ((ids, w), (ids.int(), w.bfloat16()), (ids.int()[:, :2].contiguous(), w)):
        kept = res.clone()
        with pytest.raises(ValueError):
            b.forward(attn, kept, routing)
        assert torch.equal(kept, res)


@pytest.mark.parametrize("change", [dict(max_rows=7), dict(mma_type=F4), dict(out_features=127),
                                    dict(in_features=224)])
def test_a_workspace_of_other_dims_is_refused(change):
    # dims whose own workspace would fit this one
    lin = Linear(128, 256, 8, F8)
    d = dict(out_features=128, in_features=256, max_rows=8, mma_type=F8) | change
    other = mx.make_linear_dims(**d)
    assert mx.moe_linear_workspace_size(other) <= lin.ws.numel()
    x = inputs(7, d["in_features"])
    out = torch.full((7, d["out_features"]), 3.0, dtype=torch.float32, device="cuda")
    prepared = torch.empty(mx.moe_linear_weights_size(other), dtype=torch.uint8, device="cuda")
    with pytest.raises(mx.MoeError) as e:
        mx.moe_linear_forward(other, prepared, x, out, lin.ws)
    assert e.value.status == mx.MOE_ERR_WORKSPACE_MISMATCH
    torch.cuda.synchronize()
    assert torch.all(out == 3)
