"""Rotary positions and the append to the paged cache, against 64 bits.

A rotated value is two products of fp32 cosines and sines (each off by a few units of the last
place, and by one more for the magnitude) and one addition: under (|a| + |b|) m 2^-21 together,
and then one rounding to bf16, 2^-8 of the value.  What is not rotated is copied."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.attention64 import Paged, rotated64

pytestmark = pytest.mark.gpu

HALF, INTER = mx.MOE_ROPE_HALF, mx.MOE_ROPE_INTERLEAVED


def table_of(dims):
    t = torch.empty(mx.moe_rope_table_size(dims), dtype=torch.uint8, device="cuda")
    mx.moe_rope_prepare(dims, t)
    return t


def close(dims, got, x, positions):
    want, size = rotated64(dims, x, positions)
    got = got.cpu().double()
    m = max(1.0, dims.magnitude, 0.1 * torch.tensor(dims.factor).log().item() + 1)
    tol = size * m * 2.0 ** -21
    tol = tol + (want.abs() + tol) * 2.0 ** -8 * (size > 0)
    assert torch.all((got - want).abs() <= tol)


def data(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).bfloat16().cuda()


@pytest.mark.parametrize("layout", [HALF, INTER])
@pytest.mark.parametrize("D,rotary", [(8, 8), (8, 2), (64, 64), (80, 20), (80, 80), (128, 128),
                                      (128, 64), (128, 30), (192, 96), (256, 256), (512, 512),
                                      (512, 16)])
def test_rope(D, rotary, layout):
    dims = mx.make_rope_dims(D, rotary, layout)
    for T, heads in ((1, 1), (1, 40), (37, 5), (3, 33)):
        x = data(T, heads, D, seed=T + heads)
        pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(T)).int().cuda()
        out = torch.empty_like(x)
        mx.moe_rope(dims, table_of(dims), x, pos, out)
        close(dims, out, x, pos)
        assert torch.equal(out[..., rotary:], x[..., rotary:])


@pytest.mark.parametrize("layout", [HALF, INTER])
@pytest.mark.parametrize("scaling", [mx.MOE_ROPE_UNSCALED, mx.MOE_ROPE_LINEAR, mx.MOE_ROPE_NTK,
                                     mx.MOE_ROPE_YARN])
def test_far_positions(scaling, layout):
    dims = mx.make_rope_dims(128, 128, layout, 500000.0, scaling, 16.0, 8192.0)
    pos = torch.tensor([0, 1, -1, 4095, 100003, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31],
                       dtype=torch.int32, device="cuda")
    x = data(len(pos), 7, 128)
    out = torch.empty_like(x)
    mx.moe_rope(dims, table_of(dims), x, pos, out)
    # (2^31 times a frequency in double is off by up to 2^31 2^-53 radians on either side)
    close(dims, out, x, pos)
    close_to = mx.make_rope_dims(128, 128, layout, 500000.0, scaling, 16.0, 8192.0,
                                 magnitude=0.75)
    mx.moe_rope(close_to, table_of(close_to), x, pos, out)
    close(close_to, out, x, pos)


@pytest.mark.parametrize("layout", [HALF, INTER])
def test_many_tokens_in_place_and_strided(layout):
    # enough for the form that shares an angle between heads; tokens a part of wider rows
    T, heads, D = 4099, 13, 128
    dims = mx.make_rope_dims(D, 64, layout)
    table = table_of(dims)
    rows = data(T, heads * D + 64, seed=3)
    x = rows[:, 32:32 + heads * D].unflatten(1, (heads, D))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 7
    out = torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda")
    mx.moe_rope(dims, table, x, pos, out)
    close(dims, out, x, pos)
    kept = rows.clone()
    mx.moe_rope(dims, table, x, pos)
    assert torch.equal(x, out)
    assert torch.equal(rows[:, :32], kept[:, :32]) and torch.equal(rows[:, -32:], kept[:, -32:])
    few = data(5, heads, D, seed=4)
    want = torch.empty_like(few)
    mx.moe_rope(dims, table, few, pos[:5], want)
    mx.moe_rope(dims, table, few, pos[:5])
    assert torch.equal(few, want)


def test_rotating_back():
    dims = mx.make_rope_dims(128)
    table, x = table_of(dims), data(50, 4, 128)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 1000
    y, z = torch.empty_like(x), torch.empty_like(x)
    mx.moe_rope(dims, table, x, pos, y)
    mx.moe_rope(dims, table, y, -pos, z)
    # two roundings of a pair's values: each at most 2^-8 of sqrt(2) times the larger
    size = x.double().abs()
    size = torch.maximum(size[..., :64], size[..., 64:]).repeat(1, 1, 2)
    assert torch.all((z.double() - x.double()).abs() <= size * 2 * 1.5 * 1.5 * 2.0 ** -8)


def test_values_that_are_copied_may_be_anything():
    dims = mx.make_rope_dims(80, 20, INTER)
    x = data(6, 3, 80)
    x[..., 20:] = float("nan")
    x[1, :, 20:] = float("-inf")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    mx.moe_rope(dims, table_of(dims), x, pos, out)
    assert torch.isfinite(out[..., :20]).all()
    assert torch.equal(out[..., 20:].view(torch.int16), x[..., 20:].view(torch.int16))


def append(p, rope, q=None, q_out=None, positions=None, seed=1):
    """Appends random rows to p's caches; returns the rows and the caches as they were."""
    k, v = data(p.T, p.hk, p.D, seed=seed), data(p.T, p.hk, p.D, seed=seed + 1)
    before = p.k.clone(), p.v.clone()
    mx.moe_kv_append(p.dims, p.batch, k, v, p.k, p.v, p.ws, rope=rope,
                     table=None if rope is None else table_of(rope), q=q, q_out=q_out,
                     positions=positions)
    return k, v, before


def check_append(p, rope, k, v, before, positions=None):
    places = {}
    for b, n in enumerate(p.new):
        for i in range(n):
            at = p.lens[b] - n + i
            if at >= 0:
                places[p.cu[b] + i] = (at,) + p.slot(b, at)
    t = torch.tensor(sorted(places), dtype=torch.long)
    at, page, row = (torch.tensor([places[int(i)][j] for i in t], dtype=torch.long)
                     for j in range(3))
    got_k, got_v = p.k.cpu()[page, :, row], p.v.cpu()[page, :, row]
    assert torch.equal(got_v, v.cpu()[t])
    if rope is None:
        assert torch.equal(got_k, k.cpu()[t])
    else:
        close(rope, got_k, k.cpu()[t], at if positions is None else positions.cpu()[t])
    for now, was in ((p.k, before[0]), (p.v, before[1])):
        now, was = now.cpu().clone(), was.cpu()
        now[page, :, row] = was[page, :, row]
        assert torch.equal(now.view(torch.int16), was.view(torch.int16))   # nothing else
    return t, at


BATCHES = [dict(new=[1] * 7, old=[0, 3, 15, 16, 31, 100, -1], uniform=True),
           dict(new=[5, 0, 33, 1, 64], old=[0, 9, 15, 1000, -10]),
           dict(new=[1, 2, 3], old=[5, 0, 40], shared=32, tail=6),
           dict(new=[300], old=[77], uniform=True)]


@pytest.mark.parametrize("layout,rotary", [(HALF, None), (INTER, None), (HALF, 32), (INTER, 40),
                                           (HALF, 20)])
@pytest.mark.parametrize("D,page,heads", [(64, 16, (4, 1)), (128, 64, (15, 5)), (128, 16, (8, 8))])
@pytest.mark.parametrize("batch", BATCHES)
def test_append(batch, D, page, heads, layout, rotary):
    p = Paged(**batch, D=D, page=page if batch.get("shared", 0) % page == 0 else 16,
              q_heads=heads[0], kv_heads=heads[1], spare=3)
    rope = mx.make_rope_dims(D, rotary, layout, scaling=mx.MOE_ROPE_YARN, factor=4.0,
                             original_length=256.0)
    out = torch.full_like(p.q, 77.0)
    k, v, before = append(p, rope, p.q, out)
    mx.moe_attention_check(p.ws)
    t, at = check_append(p, rope, k, v, before)
    close(rope, out.cpu()[t], p.q.cpu()[t], at)
    left = torch.ones(p.T, dtype=torch.bool)
    left[t] = False
    assert torch.all(out.cpu()[left] == 77.0)


def test_append_many_tokens():
    p = Paged(new=[1500, 700, 1024], old=[0, 100, 31], q_heads=32, kv_heads=8, page=64)
    rope = mx.make_rope_dims(128)
    out = torch.empty_like(p.q)
    k, v, before = append(p, rope, p.q, out)
    t, at = check_append(p, rope, k, v, before)
    close(rope, out.cpu()[t], p.q.cpu()[t], at)


def test_append_alone_unrotated_and_placed():
    p = Paged(new=[3, 20], old=[12, 0])
    k, v, before = append(p, None)
    check_append(p, None, k, v, before)
    p = Paged(new=[3, 20], old=[12, 0])
    pos = torch.arange(23, dtype=torch.int32, device="cuda") * 1000 - 5000
    rope = mx.make_rope_dims(128)
    k, v, before = append(p, rope, positions=pos)
    check_append(p, rope, k, v, before, pos)


def test_append_from_a_projection_and_in_place():
    p = Paged(new=[9, 9], old=[4, 30], uniform=True)
    rope = mx.make_rope_dims(128)
    qkv = data(p.T, p.hq + 2 * p.hk, 128, seed=9)
    q, k, v = qkv.split((p.hq, p.hk, p.hk), 1)
    q0, k0, v0, before = q.clone(), k.clone(), v.clone(), (p.k.clone(), p.v.clone())
    mx.moe_kv_append(p.dims, p.batch, k, v, p.k, p.v, p.ws, rope=rope, table=table_of(rope), q=q)
    t, at = check_append(p, rope, k0, v0, before)
    close(rope, q, q0, at)
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_append_outside_the_pages_is_reported():
    p = Paged(new=[4, 4], old=[30, 30])
    rope = mx.make_rope_dims(128)
    seq, cu, pages = p.batch.tensors
    for bad in (-1, p.dims.num_pages, 2 ** 31 - 1, -2 ** 31):
        kept = int(pages[1, 1])
        pages[1, 1] = bad
        out = torch.full_like(p.q, 77.0)
        k, v, before = append(p, rope, p.q, out)
        with pytest.raises(mx.MoeError) as e:
            mx.moe_attention_check(p.ws)
        assert e.value.status == mx.MOE_ERR_PAGE
        mx.moe_attention_check(p.ws)                # cleared
        pages[1, 1] = kept
    seq[1] = 16 * pages.shape[1] + 2
    append(p, rope)
    with pytest.raises(mx.MoeError):
        mx.moe_attention_check(p.ws)
