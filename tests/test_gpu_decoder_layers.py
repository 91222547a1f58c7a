"""Several layers of attention: one workspace for all of them."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from block_scaled_fp4_pre_gb300 import attention as att

pytestmark = pytest.mark.gpu


def layers(dims, rope, n, share):
    first = att.Attention(dims, rope)
    return [first] + [att.Attention(dims, rope, ws=first.ws if share else None)
                      for _ in range(n - 1)]


def test_layers_share_a_workspace():
    # contexts whose items are cut between blocks, then steps, in turn through three layers
    hq, hk, D, T = 16, 4, 64, 700
    dims = mx.make_attention_dims(hq, hk, D, 2 * 90, 16, T)
    rope = mx.make_rope_dims(D)
    table = torch.randperm(180, generator=torch.Generator().manual_seed(1)).int().cuda().view(2, 90)
    results = []
    for share in (False, True):
        stack = layers(dims, rope, 3, share)
        assert (stack[1].ws is stack[0].ws) == share
        g = torch.Generator(device="cuda").manual_seed(5)
        seq = torch.tensor([600, 100], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, 600, 700], dtype=torch.int32, device="cuda")
        batch = mx.make_kv_batch(seq, table, T, cu_new=cu, max_new=600)
        outs = []
        for step in range(6):
            qkv = torch.randn(T if step == 0 else 2, (hq + 2 * hk) * D, generator=g,
                              device="cuda").bfloat16()
            for a in stack:
                outs.append(a.forward(qkv, batch).clone())
                qkv = torch.cat((outs[-1], qkv[:, hq * D:]), 1)
            seq += 1
            batch = mx.make_kv_batch(seq, table, 2)
        for a in stack:
            a.check()
        results.append(outs)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_a_workspace_of_other_dims_is_refused():
    rope = mx.make_rope_dims(64)
    first = att.Attention(mx.make_attention_dims(4, 2, 64, 8, 16, 16), rope)
    other = att.Attention(mx.make_attention_dims(4, 2, 64, 9, 16, 16), rope, ws=first.ws)
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    batch = mx.make_kv_batch(lens, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    with pytest.raises(mx.MoeError) as e:
        other.forward(torch.zeros(1, 8 * 64, dtype=torch.bfloat16, device="cuda"), batch)
    assert e.value.status == mx.MOE_ERR_WORKSPACE_MISMATCH
