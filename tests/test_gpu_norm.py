"""RMSNorm with the residual's addition and the MXFP8 output, against 64 bits.

Tolerances, derived: r is one fp32 addition (2^-24) and its bf16 copy is exact rounding of
that; the sum of squares adds at most K / threads + 10 terms a chain, each 2^-24, halved by
the square root, and four more roundings follow: under 2^-18 relative for every K here.
y in bf16 lies between the roundings of that interval's ends; a pair's value adds half an
E4M3 step: 2^-4 of the value, or 2^-10 of the scale where the element is subnormal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests import micro64

pytestmark = pytest.mark.gpu
DELTA = 2.0 ** -18
EPS = 1e-6


def make(rows, K, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g)
    x[:, :: 97] *= 30
    r = 3 * torch.randn(rows, K, generator=g)
    gamma = (1 + 0.3 * torch.randn(K, generator=g)).bfloat16()
    return (x.bfloat16().cuda(), r.bfloat16().cuda() if residual else None, gamma.cuda())


def reference(x, r, gamma, eps=EPS):
    s = x.float().cpu() + (r.float().cpu() if r is not None else 0)
    s64 = s.double().numpy()
    y = s64 / np.sqrt((s64 ** 2).mean(-1, keepdims=True) + eps) * gamma.double().cpu().numpy()
    return s, y


def check_pair(q, sf, y, rows, K, layout):
    q, sf = q.cpu().numpy().reshape(-1, K)[:rows], sf.cpu().numpy()
    groups = K // 32
    if layout == mx.MOE_SF_128X4:
        e = sf[micro64.sf_offsets(rows, groups)].astype(np.int64) - 127
    else:
        e = sf.reshape(-1, groups)[:rows].astype(np.int64) - 127
    lo, hi = (micro64.exponents(y * (1 + s * DELTA), "e4m3") for s in (-1, 1))
    assert np.all((e >= lo) & (e <= hi))
    s = np.repeat(np.exp2(e.astype(np.float64)), 32, axis=1)
    got = micro64.e4m3_decode(q) * s
    assert np.all(np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s)
                  + DELTA * np.abs(y))


def run(x, r, gamma, layout, rows_cap=None, eps=EPS):
    rows, K = x.shape
    cap = rows if rows_cap is None else rows_cap
    q = torch.full((cap, K), 0x55, dtype=torch.uint8, device="cuda")
    sf = torch.full((mx.moe_mxfp8_scale_bytes(cap, K, layout),), 0xAA, dtype=torch.uint8,
                    device="cuda")
    ro, y = torch.empty_like(x), torch.empty_like(x)
    mx.moe_rmsnorm_mxfp8(x, gamma, eps, q, sf, layout, residual=r, residual_out=ro, y=y,
                         rows_cap=cap)
    torch.cuda.synchronize()
    return q, sf, ro, y


@pytest.mark.parametrize("layout", [mx.MOE_SF_PACKED, mx.MOE_SF_128X4])
@pytest.mark.parametrize("rows,K", [(1, 128), (1, 4096), (7, 256), (33, 384), (129, 640),
                                    (130, 1024), (5, 1152), (64, 2048), (3, 4224), (257, 4096),
                                    (2, 8192), (3, 16384), (2, 16512), (1, 65536)])
def test_norm(rows, K, layout):
    x, r, gamma = make(rows, K, rows * 7 + K)
    q, sf, ro, y = run(x, r, gamma, layout)
    s, ref = reference(x, r, gamma)
    assert torch.equal(ro.cpu(), s.bfloat16())
    got = y.double().cpu().numpy()
    assert np.all(micro64.bf16(ref - DELTA * np.abs(ref)) <= got)
    assert np.all(got <= micro64.bf16(ref + DELTA * np.abs(ref)))
    check_pair(q, sf, ref, rows, K, layout)


@pytest.mark.parametrize("layout", [mx.MOE_SF_PACKED, mx.MOE_SF_128X4])
@pytest.mark.parametrize("rows,cap", [(0, 5), (1, 1), (5, 130), (127, 129), (128, 128), (129, 400)])
def test_rows_past_the_live_ones_have_zero_scales(rows, cap, layout):
    K = 512
    x, r, gamma = make(max(rows, 1), K, 3)
    q, sf, _, _ = run(x[:rows], r[:rows], gamma, layout, cap)
    s = sf.cpu().numpy()
    if layout == mx.MOE_SF_128X4:
        allrows = (cap + 127) // 128 * 128
        s = s[micro64.sf_offsets(allrows, K // 32)]
    else:
        s = s.reshape(cap, K // 32)
    assert not s[rows:].any()
    assert np.all(q.cpu().numpy()[rows:] == 0x55)       # codes of dead rows are untouched
    if rows:
        check_pair(q, sf, reference(x[:rows], r[:rows], gamma)[1], rows, K, layout)


def test_no_residual_and_single_outputs():
    x, _, gamma = make(9, 768, 1, residual=False)
    _, ref = reference(x, None, gamma)
    y = torch.empty_like(x)
    mx.moe_rmsnorm_mxfp8(x, gamma, EPS, y=y)
    full = run(x, None, gamma, mx.MOE_SF_128X4)
    assert torch.equal(y, full[3]) and torch.equal(full[2], x)
    ro = torch.empty_like(x)
    mx.moe_rmsnorm_mxfp8(x, gamma, EPS, residual=x, residual_out=ro)
    assert torch.equal(ro, (x.float() + x.float()).bfloat16())
    q, sf = torch.empty_like(full[0]), torch.empty_like(full[1])
    mx.moe_rmsnorm_mxfp8(x, gamma, EPS, q, sf)
    assert torch.equal(q, full[0]) and torch.equal(sf, full[1])
    check_pair(q, sf, ref, 9, 768, mx.MOE_SF_128X4)


def test_strides_and_in_place():
    rows, K = 37, 1024
    x, r, gamma = make(rows, K, 5)
    q0, sf0, ro0, y0 = run(x, r, gamma, mx.MOE_SF_PACKED)
    wide = torch.full((rows, K + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + K] = x
    rw = torch.full((rows, 2 * K), -3.0, dtype=torch.bfloat16, device="cuda")
    rw[:, K:] = r
    q, sf = torch.empty_like(q0), torch.empty_like(sf0)
    # the sum replaces the residual, the norm replaces x
    mx.moe_rmsnorm_mxfp8(wide[:, 8:8 + K], gamma, EPS, q, sf, mx.MOE_SF_PACKED,
                         residual=rw[:, K:], residual_out=rw[:, K:], y=wide[:, 8:8 + K])
    torch.cuda.synchronize()
    assert torch.equal(q, q0) and torch.equal(sf, sf0)
    assert torch.equal(rw[:, K:], ro0) and torch.equal(wide[:, 8:8 + K], y0)
    assert torch.all(rw[:, :K] == -3) and torch.all(wide[:, :8] == 7) and torch.all(wide[:, 8 + K:] == 7)


def test_zero_rows_and_rows_that_overflow():
    rows, K = 6, 512
    x, _, gamma = make(rows, K, 11, residual=False)
    x[1] = 0
    x[3, 17] = float("inf")
    x[4, 9] = float("nan")
    q, sf, ro, y = run(x, None, gamma, mx.MOE_SF_PACKED)
    assert not q[1].any() and not y[1].any()
    assert not sf.view(rows, -1)[1].any()               # amax 0: exponent -127
    keep = [0, 2, 5]
    q2, sf2, _, y2 = run(x[keep].contiguous(), None, gamma, mx.MOE_SF_PACKED)
    assert torch.equal(q[keep], q2) and torch.equal(y[keep], y2)
    assert torch.equal(sf.view(rows, -1)[keep].reshape(-1), sf2)
    assert torch.isnan(y[4]).all()


def test_same_bits_every_time_and_on_another_stream():
    x, r, gamma = make(200, 4096, 2)
    first = run(x, r, gamma, mx.MOE_SF_128X4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            again = run(x, r, gamma, mx.MOE_SF_128X4)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_replay():
    x, r, gamma = make(40, 2048, 4)
    want = run(x, r, gamma, mx.MOE_SF_128X4)
    bufs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.capture_begin()
        mx.moe_rmsnorm_mxfp8(x, gamma, EPS, bufs[0], bufs[1], residual=r, residual_out=bufs[2],
                             y=bufs[3])
        graph.capture_end()
    for b in bufs:
        b.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, bufs))


def test_refusals():
    x, r, gamma = make(4, 256, 0)
    q = torch.empty(4, 256, dtype=torch.uint8, device="cuda")
    sf = torch.empty(mx.moe_mxfp8_scale_bytes(4, 256, mx.MOE_SF_128X4), dtype=torch.uint8,
                     device="cuda")

    def refused(*a, **k):
        with pytest.raises(mx.MoeError) as e:
            mx.moe_rmsnorm_mxfp8(*a, **k)
        assert e.value.status == mx.MOE_ERR_INVALID_ARG

    refused(x, gamma, EPS)                                   # no output
    refused(x, gamma, EPS, q)                                # q without sf
    refused(x, gamma, EPS, q, sf, 7)                         # unknown layout
    refused(x, gamma, -1.0, q, sf)
    refused(x, gamma, float("nan"), q, sf)
    refused(x, gamma, EPS, q, sf, rows_cap=3)
    refused(x[:, :96], gamma[:96], EPS, q, sf)               # K not a multiple of 128
    wide = torch.empty(4, 260, dtype=torch.bfloat16, device="cuda")
    refused(wide[:, :256], gamma, EPS, q, sf)                # stride not a multiple of 8
    odd = torch.empty(4 * 256 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(4, 256)
    refused(odd, gamma, EPS, q, sf)                          # not 16-byte aligned
    refused(x[:1].expand(4, 256), gamma, EPS, q, sf)         # rows that overlap
    refused(x, gamma, EPS, q, sf, residual=r[:1].expand(4, 256))
    with pytest.raises(ValueError):
        mx.moe_rmsnorm_mxfp8(x.float(), gamma, EPS, q, sf)
    with pytest.raises(ValueError):
        mx.moe_rmsnorm_mxfp8(x.t().contiguous().t(), gamma, EPS, q, sf)
    with pytest.raises(ValueError):
        mx.moe_rmsnorm_mxfp8(x, gamma, EPS, q, sf, residual=r[:3])
    with pytest.raises(ValueError):
        mx.moe_rmsnorm_mxfp8(x, gamma[:128], EPS, q, sf)


def test_offsets_past_32_bits():
    rows, K = 33000, 65536                                   # 2.16e9 elements
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    x[:-3] = 1
    x[-3:] = torch.randn(3, K, generator=g, device="cuda").bfloat16()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    q, sf, ro, y = run(x, x, gamma, mx.MOE_SF_128X4)
    q1, sf1, ro1, y1 = run(x[-3:].contiguous(), x[-3:].contiguous(), gamma, mx.MOE_SF_128X4)
    assert torch.equal(q[-3:], q1) and torch.equal(y[-3:], y1) and torch.equal(ro[-3:], ro1)
    at, at1 = (torch.from_numpy(micro64.sf_offsets(n, K // 32)[-3:]).cuda() for n in (rows, 3))
    assert torch.equal(sf[at], sf1[at1])
    assert torch.all(y[:-3] == 1)
