"""Host-side checks of rotary positions, the paged cache and attention: sizes and refusals that
need no GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def mx():
    from block_scaled_fp4_pre_gb300 import build

    build.build()
    import block_scaled_fp4_pre_gb300 as m

    m.lib()
    return m


def attn(mx, **change):
    d = dict(q_heads=8, kv_heads=2, head_dim=128, num_pages=10, page_size=16, max_tokens=64,
             max_shared_tokens=0) | change
    return mx.make_attention_dims(**d)


def test_the_cache_has_the_shape_of_the_dims(mx):
    d = mx.AttentionDims(8, 2, 128, 10, 16, 64, 0)
    assert d.cache_shape == (10, 2, 16, 128)
    d.num_pages = 100
    assert d.cache_shape == (100, 2, 16, 128)


def test_table_sizes(mx):
    for D, r in ((8, 2), (128, 128), (128, 30), (512, 512)):
        assert mx.moe_rope_table_size(mx.make_rope_dims(D, r)) == r // 2 * 8


NAN, INF = float("nan"), float("inf")
YARN = dict(scaling=3, factor=4.0, original_length=4096.0)


@pytest.mark.parametrize("change", [
    dict(head_dim=0), dict(head_dim=4), dict(head_dim=132), dict(head_dim=520),
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130), dict(rotary_dim=-2),
    dict(layout=2), dict(layout=-1), dict(scaling=4), dict(scaling=-1), dict(base=1.0),
    dict(base=NAN), dict(base=INF), dict(base=-3.0), dict(magnitude=-1.0), dict(magnitude=NAN),
    dict(magnitude=INF), dict(scaling=1, factor=0.5), dict(scaling=2, factor=NAN),
    dict(scaling=1, factor=INF), dict(scaling=2, factor=2.0, rotary_dim=2),
    YARN | dict(original_length=0.0), YARN | dict(original_length=NAN),
    YARN | dict(beta_fast=1.0, beta_slow=1.0), YARN | dict(beta_slow=-1.0),
    YARN | dict(beta_fast=NAN), YARN | dict(beta_fast=INF)])
def test_rope_dims_out_of_range(mx, change):
    d = mx.make_rope_dims(**(dict(head_dim=128) | change))
    assert mx.moe_rope_table_size(d) == 0
    f = mx.lib()
    assert f.moe_rope_prepare(ctypes.byref(d), 1024, 1 << 20, None) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_rope(ctypes.byref(d), 1024, 1024, 4096, 1024, 1, 1, 2048, 4096, None) \
        == mx.MOE_ERR_INVALID_ARG
    assert mx.moe_last_error()


def test_fields_that_a_scaling_does_not_read(mx):
    assert mx.moe_rope_table_size(mx.make_rope_dims(64, factor=NAN, original_length=-1.0,
                                                    beta_fast=0.0)) == 256
    assert mx.moe_rope_table_size(mx.make_rope_dims(64, scaling=mx.MOE_ROPE_LINEAR, factor=2.0,
                                                    original_length=-1.0)) == 256


@pytest.mark.parametrize("change", [
    dict(table=None), dict(table=1032), dict(x=None), dict(x=1030), dict(out=None),
    dict(out=1026), dict(positions=None), dict(positions=1025), dict(tokens=-1),
    dict(tokens=1 << 31), dict(heads=0), dict(heads=65537), dict(ldx=512 - 8), dict(ldx=516),
    dict(ldo=0), dict(out=4096, ldo=520)])
def test_rope_arguments(mx, change):
    a = dict(table=1024, x=4096, ldx=512, positions=1024, tokens=3, heads=4, out=8192,
             ldo=512) | change
    d = mx.make_rope_dims(128)
    assert mx.lib().moe_rope(ctypes.byref(d), a["table"], a["x"], a["ldx"], a["positions"],
                             a["tokens"], a["heads"], a["out"], a["ldo"], None) \
        == mx.MOE_ERR_INVALID_ARG
    assert mx.lib().moe_rope(None, 1024, 4096, 512, 1024, 3, 4, 8192, 512, None) \
        == mx.MOE_ERR_INVALID_ARG


def test_rope_of_no_tokens_is_a_no_op(mx):
    d = mx.make_rope_dims(128)
    assert mx.lib().moe_rope(ctypes.byref(d), None, None, 0, None, 0, 4, None, 0, None) == mx.MOE_OK
    assert mx.lib().moe_rope_prepare(ctypes.byref(d), 1024, 511, None) == mx.MOE_ERR_INVALID_ARG
    assert mx.lib().moe_rope_prepare(ctypes.byref(d), 1032, 512, None) == mx.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(head_dim=256), 2), (dict(kv_heads=0), 1),
    (dict(kv_heads=3), 1), (dict(q_heads=0), 1), (dict(q_heads=1026), 1),
    (dict(q_heads=514, kv_heads=2), 1),
    (dict(q_heads=1, kv_heads=2), 1), (dict(page_size=8), 1), (dict(page_size=48), 1),
    (dict(page_size=512), 1), (dict(page_size=-16), 1), (dict(num_pages=0), 1),
    (dict(num_pages=1 << 26), 1), (dict(num_pages=(1 << 31) - 1), 1), (dict(max_tokens=0), 1),
    (dict(max_tokens=(1 << 20) + 1), 1), (dict(max_shared_tokens=-1), 1),
    (dict(max_shared_tokens=65), 1)])
def test_attention_dims_out_of_range(mx, change, status):
    d = attn(mx, **change)
    assert mx.moe_attention_workspace_size(d) == 0
    assert mx.lib().moe_attention_workspace_init(ctypes.byref(d), 1024, 1 << 40, None) == status
    assert mx.moe_last_error()


def test_workspace_grows_with_the_shared_tokens(mx):
    sizes = [mx.moe_attention_workspace_size(attn(mx, max_tokens=4096, max_shared_tokens=n))
             for n in (0, 1, 1024, 4096)]
    assert sizes == sorted(sizes)


def test_workspaces(mx):
    d, f = attn(mx), mx.lib()
    ref = ctypes.byref(d)
    assert f.moe_attention_workspace_init(ref, None, 1 << 40, None) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_attention_workspace_init(ref, 1040, 1 << 40, None) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_attention_workspace_init(ref, 1024, 16, None) == mx.MOE_ERR_WORKSPACE_TOO_SMALL
    assert f.moe_attention_workspace_init(None, 1024, 16, None) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_attention_set_shared(None, 0) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_attention_set_shared(1024, 3) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_attention_set_shared(1024, 0) == mx.MOE_ERR_WORKSPACE_MISMATCH
    assert f.moe_attention_check(None, None) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_attention_check(1024, None) == mx.MOE_ERR_WORKSPACE_MISMATCH
    b = mx.KvBatch(1024, None, 1024, 1, 1, 1, 4, 0)
    for ws, size, status in ((None, 1 << 40, mx.MOE_ERR_INVALID_ARG),
                             (1040, 1 << 40, mx.MOE_ERR_INVALID_ARG),
                             (1024, 16, mx.MOE_ERR_WORKSPACE_TOO_SMALL),
                             (1024, 1 << 40, mx.MOE_ERR_WORKSPACE_MISMATCH)):
        assert f.moe_attention(ref, ctypes.byref(b), 4096, 1024, 1024, 1024, 1.0, 8192, 1024, None,
                               ws, size, None) == status
        assert f.moe_kv_append(ref, ctypes.byref(b), None, None, None, None, 0, None, 0, 1024, 256,
                               1024, 256, 1024, 1024, ws, size, None) == status


def test_batches(mx):
    lens, pages = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.make_kv_batch(lens.long(), pages, 3)
    with pytest.raises(ValueError):
        mx.make_kv_batch(lens, pages[:2], 3)
    with pytest.raises(ValueError):
        mx.make_kv_batch(lens, pages.view(-1), 3)
    with pytest.raises(ValueError):
        mx.make_kv_batch(lens, pages, 3, cu_new=torch.zeros(4, dtype=torch.int32))


def test_token_strides(mx):
    t = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    check = mx._heads
    assert check(t, 6, 4, 64, "t") == 256
    assert check(t.view(6, 256), 6, 4, 64, "t") == 256
    assert check(t[:, :2], 6, 2, 64, "t") == 256
    assert check(t[2:3], 1, 4, 64, "t") == 256
    assert check(t[:1].expand(6, 4, 64), 6, 4, 64, "t") == 0       # refused by the C side
    assert check(t[:, 1:2], 6, 1, 64, "t") == 256
    for bad in (t.float(), t.transpose(0, 1), t[:, ::2], t[..., :32], t[:5], t[:, 0]):
        with pytest.raises(ValueError):
            check(bad, 6, 4, 64, "t")


def test_only_tensors_of_the_current_device(mx, monkeypatch):
    monkeypatch.setattr(mx, "_current_device", lambda: 0)
    with pytest.raises(mx.MoeError) as e:
        mx._here(torch.zeros(4), "t")
    assert e.value.status == mx.MOE_ERR_INVALID_ARG
    with pytest.raises(mx.MoeError):
        mx._ints(torch.zeros(4, dtype=torch.int32), 4, "t")
    for bad in (torch.zeros(4), torch.zeros(3, dtype=torch.int32),
                torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            mx._ints(bad, 4, "t")
