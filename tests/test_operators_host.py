"""Host-side checks of the operators around the expert layer: sizes and refusals that need
no GPU."""
from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module")
def mx():
    from block_scaled_fp4_pre_gb300 import build

    build.build()
    import block_scaled_fp4_pre_gb300 as m

    m.lib()
    return m


def linear(mx, n=256, k=512, rows=8, mma=None):
    return mx.make_linear_dims(n, k, rows, mx.MOE_MMA_MXF4xMXF4 if mma is None else mma)


@pytest.mark.parametrize("n,k,slabs,kp", [(1, 32, 1, 128), (128, 128, 1, 128), (129, 160, 2, 256),
                                          (1001, 1056, 8, 1152), (4096, 4096, 32, 4096)])
def test_weight_sizes(mx, n, k, slabs, kp):
    # whole slabs of 128 rows, K in whole k-blocks (256 elements of 4 bits, 128 for MXFP8
    # activations) and a scale byte per 32 elements of K in whole 128-element blocks
    scales = slabs * 128 * kp // 32
    f4 = slabs * 128 * (-(-kp // 256) * 128) + scales
    f8 = slabs * 128 * (kp // 128 * 64) + scales
    assert mx.moe_linear_weights_size(linear(mx, n, k)) == f4
    assert mx.moe_linear_weights_size(linear(mx, n, k, mma=mx.MOE_MMA_FP8xFP4)) == f8


def test_workspace_holds_the_quantised_rows(mx):
    for mma, per in ((mx.MOE_MMA_MXF4xMXF4, 2), (mx.MOE_MMA_FP8xFP4, 1)):
        for rows in (1, 129, 4096):
            size = mx.moe_linear_workspace_size(linear(mx, 64, 4096, rows, mma))
            assert size >= rows * 4096 // per + -(-rows // 128) * 32 * 512
            assert size <= rows * 4096 // per + -(-rows // 128) * 32 * 512 + 4096


@pytest.mark.parametrize("change", [dict(n=0), dict(n=-3), dict(n=(1 << 20) + 1), dict(k=0),
                                    dict(k=48), dict(k=65568), dict(rows=0), dict(rows=(1 << 20) + 1)])
def test_linear_dims_out_of_range(mx, change):
    d = linear(mx, **change)
    assert mx.moe_linear_weights_size(d) == 0 and mx.moe_linear_workspace_size(d) == 0
    assert mx.lib().moe_linear_workspace_init(ctypes.byref(d), 1024, 1 << 30, None) \
        == mx.MOE_ERR_INVALID_ARG
    assert mx.moe_last_error()


def test_linear_types(mx):
    for mma in (mx.MOE_MMA_NVF4xNVF4, 0, 9):
        d = linear(mx, mma=mma)
        assert mx.moe_linear_weights_size(d) == 0
        assert mx.lib().moe_linear_prepare(ctypes.byref(d), 1024, 1024, 1024, 1 << 30, None) \
            == mx.MOE_ERR_UNSUPPORTED


def test_linear_calls_refuse_before_they_launch(mx):
    d = linear(mx, mma=mx.MOE_MMA_FP8xFP4)
    ref, f = ctypes.byref(d), mx.lib()
    big = 1 << 30
    assert f.moe_linear_forward(None, 1024, 1024, 512, 8, 1024, 256, 0, 1024, big, None) \
        == mx.MOE_ERR_INVALID_ARG
    assert f.moe_linear_forward(ref, 1024, 1024, 512, 8, 1024, 256, 0, None, big, None) \
        == mx.MOE_ERR_INVALID_ARG
    assert f.moe_linear_forward(ref, 1024, 1024, 512, 8, 1024, 256, 0, 1028, big, None) \
        == mx.MOE_ERR_INVALID_ARG                            # workspace not aligned
    assert f.moe_linear_forward(ref, 1024, 1024, 512, 8, 1024, 256, 0, 1024, 16, None) \
        == mx.MOE_ERR_WORKSPACE_TOO_SMALL
    assert f.moe_linear_forward(ref, 1024, 1024, 512, 8, 1024, 256, 0, 1024, big, None) \
        == mx.MOE_ERR_WORKSPACE_MISMATCH                     # never initialised
    assert f.moe_linear_check(1024, None) == mx.MOE_ERR_WORKSPACE_MISMATCH
    assert f.moe_linear_workspace_init(ref, None, big, None) == mx.MOE_ERR_INVALID_ARG
    assert f.moe_linear_workspace_init(ref, 1024, 16, None) == mx.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("change", [dict(K=0), dict(K=100), dict(K=65664), dict(rows=-1),
                                    dict(rows=9), dict(cap=(1 << 23) + 1), dict(eps=-1e-6),
                                    dict(eps=float("nan")), dict(eps=float("inf")), dict(sf=None),
                                    dict(layout=2), dict(q=1032), dict(x=None), dict(gamma=None),
                                    dict(x=1030), dict(ldx=120), dict(ldx=250), dict(ldy=100),
                                    dict(q=None, sf=None, y=None, ro=None)])
def test_norm_arguments(mx, change):
    a = dict(x=1024, ldx=256, r=1024, ldr=256, gamma=1024, eps=1e-6, rows=8, K=256, ro=1024,
             ldro=256, y=1024, ldy=256, q=1024, sf=1024, layout=mx.MOE_SF_128X4, cap=8) | change
    status = mx.lib().moe_rmsnorm_mxfp8(a["x"], a["ldx"], a["r"], a["ldr"], a["gamma"], a["eps"],
                                        a["rows"], a["K"], a["ro"], a["ldro"], a["y"], a["ldy"],
                                        a["q"], a["sf"], a["layout"], a["cap"], None)
    assert status == mx.MOE_ERR_INVALID_ARG
    assert mx.moe_last_error()


def test_few_arguments(mx):
    d = mx.make_dims(256, 128, 8, 2, 16)
    f, ref = mx.lib().moe_few_forward, ctypes.byref(d)
    big = 1 << 33
    assert f(None, 1024, 1024, 1024, 1024, 1024, 1, 1024, big, 1024, None) == mx.MOE_ERR_INVALID_ARG
    assert f(ref, 1024, 1024, 1024, 1024, 1024, 1, None, big, 1024, None) == mx.MOE_ERR_INVALID_ARG
    assert f(ref, 1024, 1024, 1024, 1024, 1024, 1, 1024, 16, 1024, None) \
        == mx.MOE_ERR_WORKSPACE_TOO_SMALL
    assert f(ref, 1024, 1024, 1024, 1024, 1024, 1, 1024, big, 1024, None) \
        == mx.MOE_ERR_WORKSPACE_MISMATCH


def test_matrix_strides(mx):
    import torch

    t = torch.zeros(6, 40, dtype=torch.bfloat16)
    check = mx._matrix
    assert check(t, (6, 40), (torch.bfloat16,), "t") == 40
    assert check(t[:, 8:24], (6, 16), (torch.bfloat16,), "t") == 40
    assert check(t[:1, :32].expand(6, 32), (6, 32), (torch.bfloat16,), "t") == 0   # refused by the C side
    assert check(t[2:3], (1, 40), (torch.bfloat16,), "t") == 40
    assert check(t[0].expand(1, 40), (1, 40), (torch.bfloat16,), "t") == 40
    for bad in (t.t(), t.float(), t[0], t[:, :39]):
        with pytest.raises(ValueError):
            check(bad, (6, 40), (torch.bfloat16,), "t")
    with pytest.raises(ValueError):
        check(torch.zeros(40, 6, dtype=torch.bfloat16).t(), (6, 40), (torch.bfloat16,), "t")


def few_args(mx, torch, T=3, H=256, I=128, E=8, k=2):
    """Arguments of moe_few_forward that lack nothing but a GPU."""
    d = mx.make_dims(H, I, E, k, 16)
    bf = torch.bfloat16
    return d, dict(
        prepared=torch.zeros(mx.moe_prepared_weights_size(d), dtype=torch.uint8),
        router=torch.zeros(E, H, dtype=bf), x=torch.zeros(T, H, dtype=bf),
        topk_ids=torch.zeros(T, k, dtype=torch.int32), topk_weights=torch.zeros(T, k),
        num_tokens=T, ws=torch.zeros(1024, dtype=torch.uint8), out=torch.zeros(T, H, dtype=bf))


def refuses(mx, f, d, args, name, change):
    """f refuses `change` of one tensor, and the right tensor where it is on the host."""
    import torch

    class OnGpu(torch.Tensor):      # a host tensor that says it is on the GPU
        is_cuda = True

    gpu = {n: t.as_subclass(OnGpu) if isinstance(t, torch.Tensor) else t for n, t in args.items()}
    gpu["stream"] = 0                            # no current stream without a GPU
    with pytest.raises(mx.MoeError) as e:        # all right, but for an unknown workspace
        f(d, **gpu)
    assert "workspace" in str(e.value)
    for bad in (change(gpu[name]), args[name]):
        with pytest.raises(mx.MoeError) as e:
            f(d, **{**gpu, name: bad})
        assert e.value.status == mx.MOE_ERR_INVALID_ARG and f"{name}:" in str(e.value)


@pytest.mark.parametrize("name,change", [
    ("prepared", lambda t: t[1:]), ("router", lambda t: t.float()), ("router", lambda t: t[1:]),
    ("router", lambda t: t.t().contiguous().t()), ("router", lambda t: t.view(16, 128)),
    ("x", lambda t: t.half()), ("x", lambda t: t[:2]), ("x", lambda t: t.repeat(1, 2)[:, :256]),
    ("x", lambda t: t.repeat(1, 2)), ("topk_ids", lambda t: t.long()),
    ("topk_ids", lambda t: t[:, :1].contiguous()), ("topk_ids", lambda t: t.t().contiguous().t()),
    ("topk_weights", lambda t: t.bfloat16()), ("topk_weights", lambda t: t[:2]),
    ("out", lambda t: t.float()), ("out", lambda t: t[:2]), ("out", lambda t: t.repeat(1, 2)[:, :256])])
def test_few_refuses_tensors_the_library_would_misread(mx, name, change):
    import torch

    d, a = few_args(mx, torch)
    refuses(mx, mx.moe_few_forward, d, a, name, change)


def linear_args(mx, torch, pair, rows=5, N=256, K=512):
    d = mx.make_linear_dims(N, K, 8, mx.MOE_MMA_FP8xFP4)
    u8 = torch.uint8
    a = dict(prepared=torch.zeros(mx.moe_linear_weights_size(d), dtype=u8),
             out=torch.zeros(rows, N), ws=torch.zeros(mx.moe_linear_workspace_size(d), dtype=u8))
    if pair:
        return d, a | dict(q=torch.zeros(rows, K, dtype=u8), rows=rows,
                           sf=torch.zeros(mx.moe_mxfp8_scale_bytes(rows, K, mx.MOE_SF_128X4), dtype=u8))
    return d, a | dict(x=torch.zeros(rows, K, dtype=torch.bfloat16))


@pytest.mark.parametrize("name,change", [
    ("prepared", lambda t: t[1:]), ("prepared", lambda t: t.repeat(2)[::2]),
    ("q", lambda t: t[:4]), ("q", lambda t: t.t().contiguous().t()), ("q", lambda t: t[:, :256]),
    ("sf", lambda t: t[:-4]), ("sf", lambda t: t.repeat(2)[::2])])
def test_linear_refuses_buffers_it_would_run_past(mx, name, change):
    import torch

    d, a = linear_args(mx, torch, True)
    refuses(mx, mx.moe_linear_forward_pair, d, a, name, change)
    d, a = linear_args(mx, torch, False)
    if name in a:
        refuses(mx, mx.moe_linear_forward, d, a, name, change)


@pytest.mark.parametrize("name,change", [
    ("codes", lambda t: t[1:]), ("codes", lambda t: t.t().contiguous().t()),
    ("scales", lambda t: t[1:]), ("scales", lambda t: t.repeat(1, 2)[:, :16])])
def test_linear_prepare_refuses_buffers_it_would_run_past(mx, name, change):
    import torch

    d, u8 = linear(mx), torch.uint8
    # prepared too small to be written, so that the right buffers go no further either
    a = dict(codes=torch.zeros(256, 256, dtype=u8), scales=torch.zeros(256, 16, dtype=u8),
             prepared=torch.zeros(512, dtype=u8))

    def prepare(d, **kw):
        try:
            mx.moe_linear_prepare(d, **kw)
        except mx.MoeError as e:
            if "prepared has 512 bytes" in str(e) or "aligned" in str(e):
                raise mx.MoeError(e.status, "the call itself, like an unknown workspace") from e
            raise

    refuses(mx, prepare, d, a, name, change)


@pytest.mark.parametrize("name", ["x", "out"])
def test_linear_refuses_host_rows(mx, name):
    import torch

    d, a = linear_args(mx, torch, False)
    refuses(mx, mx.moe_linear_forward, d, a, name, lambda t: t.as_subclass(torch.Tensor))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("name,change", [
    ("q", lambda t: t[:4]), ("q", lambda t: t.t().contiguous().t()), ("sf", lambda t: t[:-4]),
    ("sf", lambda t: t.repeat(2)[::2]), ("x", None), ("gamma", None), ("residual", None),
    ("residual_out", None), ("y", None)])
def test_norm_refuses_buffers_it_would_run_past(mx, layout, name, change):
    import torch

    rows, cap, K = 5, 200, 256
    bf, u8 = torch.bfloat16, torch.uint8
    # eps below 0, so that the right buffers go no further either
    a = dict(x=torch.zeros(rows, K, dtype=bf), gamma=torch.zeros(K, dtype=bf), eps=-1.0,
             q=torch.zeros(rows, K, dtype=u8), layout=layout, rows_cap=cap,
             sf=torch.zeros(mx.moe_mxfp8_scale_bytes(cap, K, layout), dtype=u8),
             **{n: torch.zeros(rows, K, dtype=bf) for n in ("residual", "residual_out", "y")})

    def norm(d, **kw):
        try:
            mx.moe_rmsnorm_mxfp8(**kw)
        except mx.MoeError as e:
            if "eps must be" in str(e):
                raise mx.MoeError(e.status, "the call itself, like an unknown workspace") from e
            raise

    refuses(mx, norm, None, a, name,
            change or (lambda t: t.as_subclass(torch.Tensor)))


def test_what_a_launcher_keeps_belongs_to_a_device(tmp_path):
    import os
    import shutil
    import subprocess

    from block_scaled_fp4_pre_gb300 import build

    cc = shutil.which("g++") or pytest.skip("no g++")
    src = tmp_path / "t.cc"
    src.write_text(r"""
#include "per_device.h"
#include <cstdio>
#define REQUIRE(c) if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; }
using namespace mxmoe;
int main() {
  static PerDevice<int> fit;
  REQUIRE(fit.get(0) == 0 && fit.get(1) == 0);
  fit.set(0, 36);
  REQUIRE(fit.get(0) == 36 && fit.get(1) == 0 && fit.get(63) == 0);
  fit.set(63, 7);
  fit.set(64, 8); fit.set(-1, 9);              // kept nowhere, and nothing written past the end
  REQUIRE(fit.get(63) == 7 && fit.get(64) == 0 && fit.get(-1) == 0 && fit.get(0) == 36);
  static PerDevice<bool> done;
  enum Err { kOk = 0, kBad = 3 };
  int calls = 0;
  Err answer = kOk;
  auto raise = [&] { ++calls; return answer; };
  REQUIRE(once_a_device(done, 0, raise) == kOk && calls == 1);
  REQUIRE(once_a_device(done, 0, raise) == kOk && calls == 1);
  answer = kBad;                               // a second device is asked for itself
  REQUIRE(once_a_device(done, 1, raise) == kBad && calls == 2);
  answer = kOk;                                // and again after a failure
  REQUIRE(once_a_device(done, 1, raise) == kOk && calls == 3);
  REQUIRE(once_a_device(done, 1, raise) == kOk && calls == 3);
  REQUIRE(once_a_device(done, 64, raise) == kOk && calls == 4);
  REQUIRE(once_a_device(done, 64, raise) == kOk && calls == 5);
  return 0;
}
""")
    exe = str(tmp_path / "t")
    subprocess.run([cc, "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, str(src), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    # and the operators' launchers keep nothing in any other way
    for name in ("linear.cu", "few.cu", "norm.cu"):
        with open(os.path.join(build.CSRC, name)) as f:
            kept = [l for l in f if l.lstrip().startswith("static ") and "PerDevice<" not in l
                    and "constexpr" not in l and "static __device__" not in l]
        assert not kept, kept


def test_a_single_row_may_have_any_stride(mx):
    import torch

    t = torch.zeros(6, 44, dtype=torch.bfloat16)
    for row in (t[2:3, :40], t[2:3, :40].expand(1, 40), t[2, :40].view(1, 40),
                torch.as_strided(t, (1, 40), (7, 1)), torch.as_strided(t, (1, 40), (0, 1))):
        assert mx._matrix(row, (1, 40), (torch.bfloat16,), "t") == 40
    assert mx._matrix(t[:2, :40], (2, 40), (torch.bfloat16,), "t") == 44    # refused by the library
    assert mx._matrix(t[:0, :40], (0, 40), (torch.bfloat16,), "t") >= 0
    assert mx._matrix(t[:, :1], (6, 1), (torch.bfloat16,), "t") == 44
