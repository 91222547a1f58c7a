"""The MXFP4 linear product against 64 bits.

The activations' quantisation of bf16 rows is exact arithmetic on both sides, so both
multiply the same values; what is left is the fp32 accumulation on the tensor cores, held
to the bar of the layer's GEMMs (1e-5 of the sum of the terms' magnitudes); a bf16 output
lies between the roundings of that interval's ends."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests import micro64

pytestmark = pytest.mark.gpu
F4, F8 = mx.MOE_MMA_MXF4xMXF4, mx.MOE_MMA_FP8xFP4
BAR = 1e-5


class Linear:
    def __init__(self, N, K, max_rows, mma, seed=0):
        rng = np.random.default_rng(seed)
        self.codes, self.scales = micro64.mxfp4_weights(rng, N, K)
        self.w = micro64.e2m1_decode(self.codes, self.scales)
        self.dims = mx.make_linear_dims(N, K, max_rows, mma)
        self.kind = "e2m1" if mma == F4 else "e4m3"
        self.prepared = torch.full((mx.moe_linear_weights_size(self.dims),), 0xEE,
                                   dtype=torch.uint8, device="cuda")
        mx.moe_linear_prepare(self.dims, torch.from_numpy(self.codes).cuda(),
                              torch.from_numpy(self.scales).cuda(), self.prepared)
        # stale bytes, NaN patterns among them, where the workspace needs no defined start
        self.ws = torch.full((mx.moe_linear_workspace_size(self.dims),), 0xFF,
                             dtype=torch.uint8, device="cuda")
        mx.moe_linear_workspace_init(self.dims, self.ws)

    def expect(self, x):
        v = micro64.values(x.float().cpu().numpy(), self.kind)
        return v @ self.w.T, np.abs(v) @ np.abs(self.w).T

    def check(self, got, x):
        ref, mag = self.expect(x)
        lo, hi = ref - BAR * mag, ref + BAR * mag
        if got.dtype == torch.bfloat16:
            lo, hi = micro64.bf16(lo), micro64.bf16(hi)
        got = got.double().cpu().numpy()
        assert np.all((lo <= got) & (got <= hi))


def inputs(rows, K, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g)
    x[:, ::61] *= 40
    return x.bfloat16().cuda()


SHAPES = [(1, 128, 128), (1, 1, 32), (3, 100, 96), (1, 4096, 4096), (16, 513, 1056),
          (32, 128, 2048), (33, 256, 384), (64, 130, 640), (65, 1001, 1056), (128, 384, 256),
          (129, 640, 512), (300, 1000, 1184), (700, 2048, 160)]


@pytest.mark.parametrize("mma", [F4, F8])
@pytest.mark.parametrize("rows,N,K", SHAPES)
def test_product(rows, N, K, mma):
    lin = Linear(N, K, rows, mma, seed=N + K)
    x = inputs(rows, K)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((rows, N), float("nan"), dtype=dtype, device="cuda")
        mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
        mx.moe_linear_check(lin.ws)
        lin.check(out, x)


@pytest.mark.parametrize("rows,N,K", [(1, 256, 128), (24, 4096, 1024), (130, 200, 384),
                                      (64, 1001, 640)])
def test_pair_equals_the_product_on_bf16_rows(rows, N, K):
    lin = Linear(N, K, rows, F8)
    x = inputs(rows, K)
    q = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    sf = torch.empty(mx.moe_mxfp8_scale_bytes(rows, K, mx.MOE_SF_128X4), dtype=torch.uint8,
                     device="cuda")
    mx.moe_mxfp8_quantize(x, rows, K, q, sf, mx.MOE_SF_128X4)
    a = torch.empty(rows, N, dtype=torch.float32, device="cuda")
    b = torch.empty_like(a)
    mx.moe_linear_forward(lin.dims, lin.prepared, x, a, lin.ws)
    mx.moe_linear_forward_pair(lin.dims, lin.prepared, q, sf, rows, b, lin.ws)
    mx.moe_linear_check(lin.ws)
    assert torch.equal(a, b)
    lin.check(a, x)


@pytest.mark.parametrize("mma", [F4, F8])
def test_fewer_rows_than_the_workspace_holds_and_strides(mma):
    N, K = 320, 544
    lin = Linear(N, K, 200, mma)
    for rows in (200, 1, 40, 0, 129, 7):
        x = inputs(rows, K, rows)
        wide = torch.full((rows, K + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 16:16 + K] = x
        buf = torch.full((rows, N + 3), 5.0, dtype=torch.bfloat16, device="cuda")
        mx.moe_linear_forward(lin.dims, lin.prepared, wide[:, 16:16 + K], buf[:, 2:2 + N], lin.ws)
        mx.moe_linear_check(lin.ws)
        if rows:
            lin.check(buf[:, 2:2 + N], x)
        assert torch.all(buf[:, :2] == 5) and torch.all(buf[:, 2 + N:] == 5)


@pytest.mark.parametrize("mma", [F4, F8])
def test_rows_do_not_touch_one_another(mma):
    # a row of NaN or infinity spoils itself only; zero rows give zeros
    rows, N, K = 70, 256, 512
    lin = Linear(N, K, rows, mma)
    x = inputs(rows, K)
    want = torch.empty(rows, N, dtype=torch.float32, device="cuda")
    mx.moe_linear_forward(lin.dims, lin.prepared, x, want, lin.ws)
    y = x.clone()
    y[3, 5] = float("nan")
    y[66, 400] = float("inf")
    y[10] = 0
    got = torch.empty_like(want)
    mx.moe_linear_forward(lin.dims, lin.prepared, y, got, lin.ws)
    keep = [i for i in range(rows) if i not in (3, 10, 66)]
    assert torch.equal(got[keep], want[keep])
    assert torch.all(got[10] == 0)


def test_same_bits_every_time_with_the_sum_split():
    lin = Linear(512, 8192, 4, F4)
    x = inputs(4, 8192)
    outs = []
    for _ in range(20):
        out = torch.empty(4, 512, dtype=torch.float32, device="cuda")
        mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    lin.check(outs[0], x)


def test_large_product_on_sampled_rows():
    rows, N, K = 2000, 4096, 4096
    for mma in (F4, F8):
        lin = Linear(N, K, rows, mma)
        x = inputs(rows, K)
        out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
        mx.moe_linear_check(lin.ws)
        pick = [0, 1, 127, 128, 255, 256, 1023, 1999]
        lin.check(out[pick], x[pick])


def test_graph_replay_and_another_stream():
    lin = Linear(768, 1024, 48, F4)
    x = inputs(48, 1024)
    want = torch.empty(48, 768, dtype=torch.bfloat16, device="cuda")
    mx.moe_linear_forward(lin.dims, lin.prepared, x, want, lin.ws)
    torch.cuda.synchronize()
    out = torch.zeros_like(want)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.capture_begin()
        mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
        graph.capture_end()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    lin = Linear(128, 256, 8, F8)
    x = inputs(8, 256)
    out = torch.empty(8, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(8, 256, dtype=torch.uint8, device="cuda")
    sf = torch.empty(mx.moe_mxfp8_scale_bytes(8, 256, mx.MOE_SF_128X4), dtype=torch.uint8,
                     device="cuda")

    def refused(status, f, *a):
        with pytest.raises(mx.MoeError) as e:
            f(*a)
        assert e.value.status == status

    d, inv = lin.dims, mx.MOE_ERR_INVALID_ARG
    other = mx.make_linear_dims(128, 256, 9, F8)
    refused(mx.MOE_ERR_WORKSPACE_MISMATCH, mx.moe_linear_forward, d, lin.prepared, x, out,
            torch.empty_like(lin.ws))
    refused(mx.MOE_ERR_WORKSPACE_TOO_SMALL, mx.moe_linear_forward, d, lin.prepared, x, out,
            lin.ws[:1024])
    if mx.moe_linear_workspace_size(other) <= lin.ws.numel():
        refused(mx.MOE_ERR_WORKSPACE_MISMATCH, mx.moe_linear_forward, other, lin.prepared, x, out,
                lin.ws)
    big = inputs(9, 256)
    refused(inv, mx.moe_linear_forward, d, lin.prepared, big,
            torch.empty(9, 128, dtype=torch.bfloat16, device="cuda"), lin.ws)
    refused(inv, mx.moe_linear_forward, d, lin.prepared[16:], x, out, lin.ws)
    refused(inv, mx.moe_linear_forward, d, lin.prepared, inputs(8, 260)[:, :256], out, lin.ws)
    refused(inv, mx.moe_linear_forward, d, lin.prepared, x[:1].expand(8, 256), out, lin.ws)
    refused(inv, mx.moe_linear_forward, d, lin.prepared, x, out[:1].expand(8, 128), lin.ws)
    refused(inv, mx.moe_linear_prepare, d, q, sf, lin.prepared[:1024])
    f4 = Linear(128, 256, 8, F4)
    refused(mx.MOE_ERR_UNSUPPORTED, mx.moe_linear_forward_pair, f4.dims, f4.prepared, q, sf, 8,
            out, f4.ws)
    k96 = Linear(128, 96, 8, F8)
    refused(mx.MOE_ERR_UNSUPPORTED, mx.moe_linear_forward_pair, k96.dims, k96.prepared, q, sf, 8,
            out, k96.ws)
    with pytest.raises(ValueError):
        mx.moe_linear_forward(d, lin.prepared, x, out.half(), lin.ws)
    with pytest.raises(ValueError):
        mx.moe_linear_forward(d, lin.prepared, x[:, :128], out, lin.ws)
    for bad, status in (((0, 256, 8, F8), inv), ((128, 40, 8, F8), inv), ((128, 256, 0, F8), inv),
                        ((128, 256, 8, mx.MOE_MMA_NVF4xNVF4), mx.MOE_ERR_UNSUPPORTED)):
        dims = mx.make_linear_dims(*bad)
        assert mx.moe_linear_workspace_size(dims) == 0 and mx.moe_linear_weights_size(dims) == 0
        refused(status, mx.moe_linear_workspace_init, dims, lin.ws)


@pytest.mark.parametrize("mma", [F4, F8])
@pytest.mark.parametrize("rows,N,K", [(700, 2048, 416), (1300, 2200, 256), (577, 4100, 768),
                                      (1153, 3201, 1120)])
def test_tiles_over_sm_pairs(rows, N, K, mma):
    # several 192-row tiles that start in the middle of a scale block, an odd number of
    # weight slabs, features past the last whole slab, a last k-block of half width
    lin = Linear(N, K, rows, mma)
    x = inputs(rows, K)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((rows, N), float("nan"), dtype=dtype, device="cuda")
        mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
        mx.moe_linear_check(lin.ws)
        lin.check(out, x)


def test_pair_in_on_sm_pairs_does_not_read_past_its_scales():
    # 577 rows: the last tile's second scale block lies past the end of sf
    rows, N, K = 577, 4096, 512
    lin = Linear(N, K, rows, F8)
    x = inputs(rows, K)
    q = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    n = mx.moe_mxfp8_scale_bytes(rows, K, mx.MOE_SF_128X4)
    buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    mx.moe_mxfp8_quantize(x, rows, K, q, buf[:n], mx.MOE_SF_128X4)
    out = torch.empty(rows, N, dtype=torch.float32, device="cuda")
    mx.moe_linear_forward_pair(lin.dims, lin.prepared, q, buf[:n], rows, out, lin.ws)
    mx.moe_linear_check(lin.ws)
    lin.check(out, x)


@pytest.mark.parametrize("rows,N,K,mma", [(70000, 128, 32768, F4), (270000, 8192, 32, F8)])
def test_offsets_past_32_bits(rows, N, K, mma):
    # 2.3e9 elements of x, and 2.2e9 of out
    lin = Linear(N, K, rows, mma)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(rows // 100, K, generator=g, device="cuda").bfloat16().repeat(100, 1)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
    mx.moe_linear_check(lin.ws)
    n = rows // 100
    assert torch.equal(out[-n:], out[:n])
    pick = [0, n // 2, rows - n // 3, rows - 1]
    lin.check(out[pick], x[pick])


@pytest.mark.parametrize("mma", [F4, F8])
@pytest.mark.parametrize("rows", [4864, 4870, 5000, 5094])
def test_rounds_of_256_row_tiles(rows, mma):
    # three rounds of tiles through accumulators that share columns; a last tile of 6 rows,
    # 136 (the shared columns unused) and 230
    N, K = 2300, 160
    lin = Linear(N, K, rows, mma)
    x = inputs(rows, K)
    out = torch.full((rows, N), float("nan"), dtype=torch.float32, device="cuda")
    again = torch.empty_like(out)
    mx.moe_linear_forward(lin.dims, lin.prepared, x, out, lin.ws)
    mx.moe_linear_forward(lin.dims, lin.prepared, x, again, lin.ws)
    mx.moe_linear_check(lin.ws)
    lin.check(out, x)
    assert torch.equal(out, again)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_weights_written_just_before(rows):
    # the weights change on the same stream between calls, with no wait in between
    N, K = 1024, 2048
    lins = [Linear(N, K, rows, F4, seed=s) for s in (1, 2)]
    src = [(torch.from_numpy(l.codes).cuda(), torch.from_numpy(l.scales).cuda()) for l in lins]
    x = inputs(rows, K)
    want = [torch.empty(rows, N, device="cuda") for _ in lins]
    for l, w in zip(lins, want):
        mx.moe_linear_forward(l.dims, l.prepared, x, w, l.ws)
    a = lins[0]
    outs = [torch.empty_like(want[0]) for _ in range(20)]
    for i, out in enumerate(outs):
        if i % 3:
            mx.moe_linear_prepare(a.dims, *src[i & 1], a.prepared)
        else:
            a.prepared.copy_(lins[1].prepared if i & 1 else want_prepared(a, src[0]))
        mx.moe_linear_forward(a.dims, a.prepared, x, out, a.ws)
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i & 1])


def want_prepared(lin, src):
    p = torch.empty_like(lin.prepared)
    mx.moe_linear_prepare(lin.dims, *src, p)
    return p
