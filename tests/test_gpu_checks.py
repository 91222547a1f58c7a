"""Calls that read a workspace's error bits wait for the stream that they are given, and for no
other."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.attention64 import Paged

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
