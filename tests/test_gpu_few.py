"""The whole expert layer for a few tokens against 64 bits and against the layer's other
form (moe_pre_dispatch and moe_forward, itself held to the oracle).

Bars: the layer's own 2e-3 normwise against the unrounded result, which is bf16's rounding
(1.7e-3) and little else; the two forms differ by fp32 summation order only, so at most by
one bf16 step where a sum lies next to a rounding boundary: 2^-8 of the value plus 1e-5 of
the row's largest.  A logit's fp32 error is at most H terms of 2^-24 each (summed in chains
of H / 128 + 9): 2^-16 of the sum of magnitudes covers every H here, and a weight's relative
error is twice the largest logit error plus 2^-20 for exp and the division."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests import micro64

pytestmark = pytest.mark.gpu
F4, F8, NV = mx.MOE_MMA_MXF4xMXF4, mx.MOE_MMA_FP8xFP4, mx.MOE_MMA_NVF4xNVF4


class Few:
    def __init__(self, H, I, E, k, mma=F4, max_tokens=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims = mx.make_dims(H, I, E, k, max_tokens, mma)
        grp = mx.sf_group(self.dims)
        quantise = mx.moe_quantize_nvfp4 if mma == NV else mx.moe_quantize_mxfp4
        can = []
        for rows, K in ((2 * I, H), (H, I)):
            w = torch.randn(E * rows, K, generator=g, device="cuda") * K ** -0.5
            c = torch.empty(E * rows, K // 2, dtype=torch.uint8, device="cuda")
            s = torch.empty(E * rows, K // grp, dtype=torch.uint8, device="cuda")
            quantise(w, c, s)
            can += [c.view(E, rows, -1), s.view(E, rows, -1)]
        self.can = can
        self.prepared = torch.empty(mx.moe_prepared_weights_size(self.dims), dtype=torch.uint8,
                                    device="cuda")
        mx.moe_prepare_weights(self.dims, *can, self.prepared)
        self.ws = torch.empty(mx.moe_workspace_size(self.dims), dtype=torch.uint8, device="cuda")
        mx.moe_workspace_init(self.dims, self.ws)
        self.router = (torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).bfloat16()

    def x(self, T, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(T, self.dims.hidden, generator=g, device="cuda")
        x[:, ::131] *= 20
        return x.bfloat16()

    def outputs(self, T):
        k = self.dims.topk
        return (torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
                torch.full((T, k), float("nan"), device="cuda"),
                torch.full((T, self.dims.hidden), float("nan"), dtype=torch.bfloat16,
                           device="cuda"))

    def run(self, x, router="own", ids=None, weights=None, check=True):
        T = x.shape[0]
        i, w, out = self.outputs(T)
        i = i if ids is None else ids
        w = w if weights is None else weights
        r = self.router if isinstance(router, str) else router
        mx.moe_few_forward(self.dims, self.prepared, r, x, i, w, T, self.ws, out)
        if check:
            mx.moe_check(self.ws)
        return i, w, out

    def layer(self, x, ids, weights):
        T = x.shape[0]
        out = torch.empty(T, self.dims.hidden, dtype=torch.bfloat16, device="cuda")
        mx.moe_pre_dispatch(self.dims, x, ids, weights, T, self.ws)
        mx.moe_forward(self.dims, self.prepared, self.ws, out, T)
        return out

    def reference(self, x, ids, weights):
        """64-bit layer (MXFP4 and MXFP8 activations)."""
        kind = "e4m3" if self.dims.mma_type == F8 else "e2m1"
        I = self.dims.inter
        x = micro64.values(x.float().cpu().numpy(), kind)
        ids, weights = ids.cpu().numpy(), weights.double().cpu().numpy()
        out = np.zeros((len(x), self.dims.hidden))
        can = [c.cpu().numpy() for c in self.can]
        for e in np.unique(ids[(ids >= 0) & (ids < self.dims.num_experts)]):
            w1 = micro64.e2m1_decode(can[0][e], can[1][e])
            w2 = micro64.e2m1_decode(can[2][e], can[3][e])
            for t, j in zip(*np.nonzero(ids == e)):
                gu = w1 @ x[t]
                h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
                out[t] += weights[t, j] * (w2 @ micro64.values(h, kind))
        return out


def check_routing(few, x, ids, weights):
    xs = x.double().cpu().numpy()
    r = few.router.double().cpu().numpy()
    logits, mag = xs @ r.T, np.abs(xs) @ np.abs(r).T
    err = 2.0 ** -16 * mag.max()
    ids, weights = ids.cpu().numpy(), weights.double().cpu().numpy()
    for t in range(len(xs)):
        order = sorted(range(len(r)), key=lambda e: (-logits[t, e], e))[:few.dims.topk]
        assert len(set(ids[t])) == few.dims.topk
        got, want = logits[t, ids[t]], logits[t, order]
        assert np.all(np.abs(got - want) <= 2 * err)      # equal but for a near tie
        w = np.exp(got - got.max())
        assert np.all(np.abs(weights[t] / (w / w.sum()) - 1) <= 2 * err + 2.0 ** -20)


def check_close(got, want):
    """Two bf16 results that differ in fp32 summation order."""
    assert torch.isfinite(got).all()
    def order(t):                       # bf16 values as consecutive integers
        b = t.view(torch.int16).int()
        return torch.where(b < 0, -32768 - b, b)

    g, w = got.double(), want.double()
    far = ((order(got) - order(want)).abs() > 1) & \
        ((g - w).abs() > 1e-5 * w.abs().amax(-1, keepdim=True))
    far = far.double().mean().item()
    # a one-step change of an intermediate code moves a whole row a little: 0.1% of codes
    # may differ, none is expected
    assert far == 0, far


SHAPES = [(1, 256, 128, 8, 2), (3, 640, 384, 12, 3), (16, 512, 256, 40, 6), (8, 1024, 640, 5, 5),
          (9, 384, 128, 300, 8), (2, 4096, 512, 16, 6), (5, 256, 2048, 7, 1), (16, 256, 128, 1, 1),
          (16, 256, 128, 1024, 32), (3, 4736, 128, 6, 2), (16, 8192, 256, 10, 4), (1, 4480, 256, 9, 3)]


@pytest.mark.parametrize("mma", [F4, F8, NV])
@pytest.mark.parametrize("T,H,I,E,k", SHAPES)
def test_layer(T, H, I, E, k, mma):
    few = Few(H, I, E, k, mma)
    x = few.x(T)
    ids, weights, out = few.run(x)
    check_routing(few, x, ids, weights)
    check_close(out, few.layer(x, ids, weights))
    if mma != NV and E <= 300:
        ref = few.reference(x, ids, weights)
        err = np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert err <= 2e-3, err
    # the same routing given instead of computed: the same bits
    again = few.run(x, None, ids, weights)[2]
    assert torch.equal(out, again)


@pytest.mark.parametrize("mma", [F4, F8, NV])
def test_full_size_layer(mma):
    few = Few(4096, 2048, 64, 6, mma)
    for T in (1, 2, 7, 16):
        x = few.x(T, T)
        ids, weights, out = few.run(x)
        check_routing(few, x, ids, weights)
        check_close(out, few.layer(x, ids, weights))


@pytest.mark.parametrize("mma", [F4, F8])
def test_given_routing_with_invalid_and_repeated_ids(mma):
    T, E, k = 6, 10, 4
    few = Few(384, 256, E, k, mma)
    x = few.x(T)
    ids = torch.tensor([[0, 1, 2, 3], [9, 9, 9, 9], [-1, 4, 10, 5], [-3, 99, 10, -1],
                        [7, 7, 0, 1], [3, -1, 3, 8]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[.4, .3, .2, .1], [.25, .5, .125, .125], [.9, .5, .7, -.5],
                      [1, 1, 1, 1], [0, 2, .5, .25], [1, 1, -1, 1]], device="cuda")
    out = few.run(x, None, ids.clone(), w.clone(), check=False)[2]
    with pytest.raises(mx.MoeError) as e:
        mx.moe_check(few.ws)
    assert e.value.status == mx.MOE_ERR_ROUTING
    mx.moe_check(few.ws)                                    # cleared
    ref = few.reference(x, ids, w)
    got = out.double().cpu().numpy()
    assert not got[3].any()
    rows = [0, 1, 2, 4, 5]
    # row 5: 3 and 3 cancel exactly but for order; what is left is expert 8
    err = np.linalg.norm((got - ref)[rows]) / np.linalg.norm(ref[rows])
    assert err <= 2e-3
    none = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    out = few.run(x, None, none, w, check=False)[2]
    assert not out.any()
    with pytest.raises(mx.MoeError):
        mx.moe_check(few.ws)


def test_equal_logits_go_to_the_lower_expert():
    few = Few(256, 128, 24, 5)
    few.router[7] = few.router[3]
    few.router[15] = few.router[3]
    x = (few.router[3].float() * 50).bfloat16().view(1, -1).repeat(2, 1)
    x[1] = 0                                                # every logit 0
    ids, weights, out = few.run(x)
    assert ids[0, :3].tolist() == [3, 7, 15]
    assert weights[0, 0] == weights[0, 1] == weights[0, 2]
    assert ids[1].tolist() == [0, 1, 2, 3, 4]
    assert torch.all(weights[1] == 0.2) and not out[1].any()


def test_a_token_of_nan_spoils_no_other_token():
    for mma in (F4, F8, NV):
        few = Few(512, 256, 6, 3, mma)
        x = few.x(5)
        ids, w, out = few.run(x)
        y = x.clone()
        y[2] = float("nan")
        got = few.run(y, None, ids, w, check=False)[2]
        keep = [0, 1, 3, 4]
        assert torch.equal(got[keep], out[keep])


def test_same_bits_every_time_and_between_the_layers_own_calls():
    few = Few(2048, 1024, 32, 6)
    x = few.x(11)
    first = few.run(x)
    ids, w = first[0], first[1]
    layer = few.layer(x, ids, w)
    for i in range(10):
        assert all(torch.equal(a, b) for a, b in zip(first, few.run(x)))
    # a few-token call between a dispatch and its forward leaves the dispatch alone
    y = few.x(16, 9)
    out = torch.empty_like(layer)
    mx.moe_pre_dispatch(few.dims, x, ids, w, 11, few.ws)
    few.run(y)
    mx.moe_forward(few.dims, few.prepared, few.ws, out, 11)
    check_close(out, layer)


def test_back_to_back_calls_of_other_sizes_on_another_stream():
    few = Few(1024, 512, 48, 4)
    xs = [few.x(T, T) for T in (1, 16, 3, 8, 9, 2)]
    want = [few.run(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            got = [few.run(x, check=False) for x in xs]
    side.synchronize()
    mx.moe_check(few.ws)
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_graph_replay():
    few = Few(512, 256, 16, 4)
    x = few.x(4)
    want = few.run(x)
    got = few.outputs(4)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.capture_begin()
        mx.moe_few_forward(few.dims, few.prepared, few.router, x, got[0], got[1], 4, few.ws,
                           got[2])
        graph.capture_end()
    for _ in range(3):
        got[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    few = Few(256, 128, 8, 2, max_tokens=20)
    x = few.x(20)
    ids, w, out = few.outputs(20)

    def refused(status, *a):
        with pytest.raises(mx.MoeError) as e:
            mx.moe_few_forward(*a)
        assert e.value.status == status

    d, p, r, ws, inv = few.dims, few.prepared, few.router, few.ws, mx.MOE_ERR_INVALID_ARG
    refused(mx.MOE_ERR_UNSUPPORTED, d, p, r, x, ids, w, 17, ws, out)
    refused(inv, d, p, r, x, ids, w, 21, ws, out)
    refused(inv, d, p, r, x, ids, w, -1, ws, out)
    refused(inv, d, p, r, None, ids, w, 2, ws, out)
    refused(inv, d, p, r, x, None, w, 2, ws, out)
    refused(inv, d, p, r, x, ids, w, 2, ws, None)
    refused(inv, d, p[16:], r, x, ids, w, 2, ws, out)
    refused(inv, d, p, r.view(-1)[4:], x, ids, w, 2, ws, out)
    refused(mx.MOE_ERR_WORKSPACE_TOO_SMALL, d, p, r, x, ids, w, 2, ws[:4096], out)
    refused(mx.MOE_ERR_WORKSPACE_MISMATCH, d, p, r, x, ids, w, 2, torch.empty_like(ws), out)
    mx.moe_few_forward(d, p, r, x, ids, w, 0, ws, out)      # nothing to do
    assert torch.isnan(out).all()
