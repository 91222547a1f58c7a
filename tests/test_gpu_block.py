"""The half decoder block: every step against 64 bits on the step's own input, so that no
step's rounding hides another's.  Bars as in the operators' own tests."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from block_scaled_fp4_pre_gb300 import block as blk
from tests import micro64
from tests.test_gpu_few import check_close
from tests.test_gpu_linear import BAR
from tests.test_gpu_norm import DELTA, check_pair

pytestmark = pytest.mark.gpu


def make(T, H=512, I=256, E=16, k=4, feats=384, nxt=520, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 50)
    dims = mx.make_dims(H, I, E, k, T)
    b = blk.random_block(dims, feats, nxt, seed)
    attn = torch.randn(T, feats, generator=g, device="cuda").bfloat16()
    res = (2 * torch.randn(T, H, generator=g, device="cuda")).bfloat16()
    return b, attn, res


def weight64(lin: blk.Linear, codes, scales):
    return micro64.e2m1_decode(codes.cpu().numpy(), scales.cpu().numpy())


def between(got, ref, slack):
    got = got.double().cpu().numpy()
    assert np.all((micro64.bf16(ref - slack) <= got) & (got <= micro64.bf16(ref + slack)))


def norm64(s, gamma, eps):
    s = s.double().cpu().numpy()
    return s / np.sqrt((s ** 2).mean(-1, keepdims=True) + eps) * gamma.double().cpu().numpy()


@pytest.mark.parametrize("T", [1, 5, 16, 40])
def test_steps(T, monkeypatch):
    kept = []
    real = blk.quantised
    monkeypatch.setattr(blk, "quantised", lambda w: kept.append(real(w)) or kept[-1])
    b, attn, res = make(T)
    wo, wn = kept[-2], kept[-1]                     # after the experts' own
    before = res.clone()
    routing = None
    if T > blk.FEW_TOKENS:
        g = torch.Generator(device="cuda").manual_seed(1)
        ids = torch.stack([torch.randperm(16, generator=g, device="cuda")[:4] for _ in range(T)])
        w = torch.softmax(torch.randn(T, 4, generator=g, device="cuda"), -1)
        routing = (ids.int(), w)
        with pytest.raises(ValueError):
            b.forward(attn, res.clone())
    out = b.forward(attn, res, routing)
    b.check()
    o, h, m = b.o[:T], b.h[:T], b.m[:T]
    v, w = micro64.values(attn.float().cpu().numpy(), "e2m1"), weight64(b.wo, *wo)
    between(o, v @ w.T, BAR * (np.abs(v) @ np.abs(w).T))
    mid = before.float() + o.float()
    ref = norm64(mid, b.gamma_in, b.eps)
    between(h, ref, DELTA * np.abs(ref))
    # the expert layer, by its other form on the same rows and routing
    ids, wt = routing or (b.ids, b.weights)
    other = torch.empty_like(m)
    mx.moe_pre_dispatch(b.dims, h, ids, wt, T, b.ws)
    mx.moe_forward(b.dims, b.prepared, b.ws, other, T)
    check_close(m, other)
    end = mid.bfloat16().float() + m.float()
    assert torch.equal(res, end.bfloat16())
    ref = norm64(end, b.gamma_out, b.eps)
    check_pair(b.q[:T], b.sf, ref, T, 512, mx.MOE_SF_128X4)
    e = b.sf.cpu().numpy()[micro64.sf_offsets(T, 16)].astype(np.float64) - 127
    v = micro64.e4m3_decode(b.q[:T].cpu().numpy()) * np.exp2(np.repeat(e, 32, axis=1))
    w = weight64(b.wn, *wn)
    between(out, v @ w.T, BAR * (np.abs(v) @ np.abs(w).T))


def test_graph_replay_and_smaller_batches():
    b, attn, res = make(12)
    want = {}
    for T in (12, 1, 7):
        r = res[:T].clone()
        want[T] = (b.forward(attn[:T], r).clone(), r)
    got = res.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
        out = b.forward(attn, got)
        graph.capture_end()
    for _ in range(3):
        got.copy_(res)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[12][0]) and torch.equal(got, want[12][1])
    b.check()
