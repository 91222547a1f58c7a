"""The operators around the expert layer at the edges of what they take."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests import micro64
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


def device_sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# Rows of +1 and -1 but for one element of 1 + d or 1 - d, eps 0: the mean of the squares lies
# 2 d / K from 1, and y lies d / K from gamma.  Where gamma is halfway between two values of
# E4M3, the side that y is on decides, and d / K is chosen below 2^-25, half a unit of a float's
# last place, so that y rounded to a float first would be the tie itself.  d is as small as
# each form of the kernel (one warp a row; blocks of one, two, four or eight vectors a thread)
# still sums without a rounding: half a unit of its largest single-float sum.
@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("rows,K,dlog", [
    (4, 128, 21), (4, 256, 21), (9, 512, 21), (400, 1024, 21), (100, 1408, 16), (200, 1408, 20),
    (200, 2048, 20), (8, 4096, 16), (200, 4096, 15), (200, 8192, 15), (3, 16384, 14),
    (2, 65536, 13)])
def test_norm_next_to_a_tie_of_e4m3(rows, K, dlog, side):
    d = side * 2.0 ** -dlog
    assert abs(d) / K < 2.0 ** -25
    g = torch.Generator().manual_seed(K)
    sign = torch.where(torch.rand(rows, K, generator=g) < 0.5, -1.0, 1.0)
    at = torch.randint(K, (rows, 1), generator=g)
    add = torch.zeros(rows, K).scatter_(1, at, d) * sign
    # midpoints 1 1/16, 1 3/16 .. 1 15/16 at three exponents; the largest sets the scale
    m = torch.randint(8, (K,), generator=g)
    mid = (1 + (2 * m + 1) / 16) * 2.0 ** torch.randint(-2, 1, (K,), generator=g)
    x, r, gamma = sign.bfloat16().cuda(), add.bfloat16().cuda(), mid.bfloat16().cuda()
    assert torch.equal(gamma.float().cpu(), mid) and torch.equal(r.float().cpu(), add)
    q, sf, _, _ = norm.run(x, r, gamma, mx.MOE_SF_PACKED, eps=0.0)
    e = sf.cpu().numpy().reshape(rows, -1).astype(np.float64) - 127
    got = micro64.e4m3_decode(q.cpu().numpy()) * np.exp2(np.repeat(e, 32, axis=1))
    got, mid, sign = np.abs(got), mid.double().numpy(), sign.numpy()
    step = np.exp2(np.floor(np.log2(mid)) - 3)               # of E4M3 at gamma
    # more than 1 in the mean: y below gamma, the lower neighbour; else the upper one
    want = mid - side * step / 2
    keep = np.ones((rows, K), bool)
    keep[np.arange(rows), at[:, 0].numpy()] = False          # the odd element itself
    assert np.all((got == want)[keep])
    even = np.rint(mid / step) * step                        # what a tie would have given
    assert 0.3 < np.mean(want != even) < 0.7


def test_norm_codes_that_differ_from_64_bits_are_fewer_than_plain_fp32_gives():
    # measured before on 830 million elements of such rows: 0.14 a million against 0.69
    own = plain = 0
    for seed in range(3):
        rows, K = 16384, 1408
        g = torch.Generator(device="cuda").manual_seed(100 + seed)
        ch = 1 + 20 * (torch.rand(K, generator=g, device="cuda") < 0.004)
        x = (torch.randn(rows, K, generator=g, device="cuda") * ch).bfloat16()
        gamma = (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).bfloat16()
        q, sf, _, _ = norm.run(x, None, gamma, mx.MOE_SF_PACKED)
        up = torch.exp2(127 - sf.view(rows, K // 32).double()).repeat_interleave(32, 1)

        def codes(v):                                        # E4M3 of scaled values, ties to even
            ex = torch.frexp(v)[1].double() - 1
            step = torch.exp2(ex.clamp(min=-6) - 3)
            return torch.round(v / step) * step

        d = x.double()
        y = d / torch.sqrt((d * d).mean(1, keepdim=True) + norm.EPS) * gamma.double()
        f = x.float()
        p = f * torch.rsqrt((f * f).mean(1, keepdim=True) + norm.EPS) * gamma.float()
        want = codes(y * up)
        own += int((q.view(torch.float8_e4m3fn).float().double() != want).sum())
        plain += int((codes(p.double() * up) != want).sum())
    assert 2 * own <= plain, (own, plain)


@pytest.mark.parametrize("K", [1152, 4096, 8192])
def test_norm_of_a_row_among_few_and_among_many(K):
    # up to one row an SM and more rows differ in the order of the sums: the last bits of a
    # float at most, a neighbouring code or bf16 value where a boundary lies there
    sms = device_sms()
    x, r, gamma = norm.make(3 * sms, K, K)
    many = norm.run(x, r, gamma, mx.MOE_SF_PACKED)
    few = norm.run(x[:sms], r[:sms], gamma, mx.MOE_SF_PACKED)
    for n in (1, 2, sms // 2):
        for a, b in zip(norm.run(x[:n], r[:n], gamma, mx.MOE_SF_PACKED), few):
            assert torch.equal(a.view(n, -1), b.view(sms, -1)[:n])
    for n in (sms + 1, 2 * sms):
        for a, b in zip(norm.run(x[:n], r[:n], gamma, mx.MOE_SF_PACKED), many):
            assert torch.equal(a.view(n, -1), b.view(3 * sms, -1)[:n])
    assert torch.equal(few[2], many[2][:sms])                # residual_out is exact
    _, ref = norm.reference(x[:sms], r[:sms], gamma)
    for q, sf, _, y in (few, many):
        q, sf, y = q[:sms], sf[:sms * K // 32], y[:sms].double().cpu().numpy()
        norm.check_pair(q, sf, ref, sms, K, mx.MOE_SF_PACKED)
        lo, hi = (micro64.bf16(ref + s * norm.DELTA * np.abs(ref)) for s in (-1, 1))
        assert np.all((lo <= y) & (y <= hi))


def test_layer_workspace_says_its_layout():
    # the regions of the few-token form made it another layout than version 1
    d = mx.make_dims(256, 128, 8, 2, 16)
    ws = torch.zeros(mx.moe_workspace_size(d), dtype=torch.uint8, device="cuda")
    mx.moe_workspace_init(d, ws)
    assert ws[:32].view(torch.int32).tolist() == [0x454F4D58, 2, 256, 128, 8, 2, 16,
                                                  mx.MOE_MMA_MXF4xMXF4]
    assert ws[32:40].view(torch.int64).item() == ws.numel()
