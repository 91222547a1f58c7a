"""Calls that read a workspace's error bits wait for the stream that they are given, and for no
other."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.attention64 import Paged
from tests.test_gpu_linear import F8, Linear, inputs

pytestmark = pytest.mark.gpu


def beside_the_default_stream(check):
    """Calls check(stream) while the default stream is busy for a fifth of a second."""
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    done.record()
    check(side)
    assert not done.query()
    torch.cuda.synchronize()


def test_attention():
    p = Paged(new=[1, 2], old=[40, 9])
    good, _ = p.run()
    beside_the_default_stream(lambda s: mx.moe_attention_check(p.ws, s))
    # reported once, whichever stream asks, and nothing is lost of a call right behind a check
    pages, side = p.batch.tensors[2], torch.cuda.Stream()
    kept, out = int(pages[0, 1]), torch.empty_like(good)
    for _ in range(50):
        pages[0, 1] = -5
        torch.cuda.synchronize()
        for _ in range(2):
            mx.moe_attention(p.dims, p.batch, p.q, p.k, p.v, out, p.ws, stream=side)
            with pytest.raises(mx.MoeError) as e:
                mx.moe_attention_check(p.ws, side)
            assert e.value.status == mx.MOE_ERR_PAGE
        pages[0, 1] = kept
        torch.cuda.synchronize()
        mx.moe_attention(p.dims, p.batch, p.q, p.k, p.v, out, p.ws, stream=side)
        mx.moe_attention_check(p.ws, side)
        assert torch.equal(out, good)


def test_linear():
    lin = Linear(512, 256, 40, F8)
    x = inputs(40, 256)
    want = torch.empty(40, 512, dtype=torch.float32, device="cuda")
    mx.moe_linear_forward(lin.dims, lin.prepared, x, want, lin.ws)
    mx.moe_linear_check(lin.ws)
    beside_the_default_stream(lambda s: mx.moe_linear_check(lin.ws, s))
    lin.ws.view(torch.int32)[0] = 2                     # as a call that gave up leaves it
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with pytest.raises(mx.MoeError) as e:
        mx.moe_linear_check(lin.ws, side)
    assert e.value.status == mx.MOE_ERR_TIMEOUT
    mx.moe_linear_check(lin.ws, side)
    out = torch.empty_like(want)
    mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
    assert torch.equal(out, want)


def test_layer():
    dims = mx.make_dims(256, 128, 8, 2, 16)
    ws = torch.empty(mx.moe_workspace_size(dims), dtype=torch.uint8, device="cuda")
    mx.moe_workspace_init(dims, ws)
    x = torch.randn(16, 256, device="cuda").bfloat16()
    ids = torch.zeros(16, 2, dtype=torch.int32, device="cuda")
    w = torch.full((16, 2), 0.5, device="cuda")
    beside_the_default_stream(lambda s: mx.moe_check(ws, s))
    side = torch.cuda.Stream()
    for _ in range(20):
        for bad in (8, -1):
            ids[3, 1] = bad
            torch.cuda.synchronize()
            mx.moe_pre_dispatch(dims, x, ids, w, 16, ws, side)
            with pytest.raises(mx.MoeError) as e:
                mx.moe_check(ws, side)
            assert e.value.status == mx.MOE_ERR_ROUTING
        ids[3, 1] = 7
        torch.cuda.synchronize()
        mx.moe_pre_dispatch(dims, x, ids, w, 16, ws, side)
        mx.moe_check(ws, side)
