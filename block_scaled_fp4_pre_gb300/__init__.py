"""Python binding of libmxmoe, a GB300 (sm_103a) W4A4 MXFP4 mixture-of-experts layer.

Argument marshalling only: every step of the layer runs in the CUDA kernels of
libmxmoe.so, whose C ABI is include/mxmoe.h.  Function names match the C entry
points.  Device buffers are torch tensors (or raw integer addresses); PyTorch is
used for device memory and streams only.  There is no CPU fallback: if the
library is missing, importing the functions raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import numpy as np
import torch  # loads the CUDA runtime libmxmoe links against

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxmoe.so")

MOE_MMA_MXF4xMXF4 = 1
MOE_MMA_FP8xFP4 = 2
MOE_MMA_NVF4xNVF4 = 3
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE_TOO_SMALL = 3
MOE_ERR_WORKSPACE_MISMATCH = 4
MOE_ERR_CUDA = 5
MOE_ERR_ROUTING = 6
MOE_ERR_TIMEOUT = 7
MOE_ERR_PAGE = 8


class MoeDims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("mma_type", ctypes.c_int32)]

    def __repr__(self):
        return (f"MoeDims(hidden={self.hidden}, inter={self.inter}, num_experts={self.num_experts}, "
                f"topk={self.topk}, max_tokens={self.max_tokens}, mma_type={self.mma_type})")


def make_dims(hidden: int, inter: int, num_experts: int, topk: int, max_tokens: int,
              mma_type: int = MOE_MMA_MXF4xMXF4) -> MoeDims:
    return MoeDims(hidden, inter, num_experts, topk, max_tokens, mma_type)


class LinearDims(ctypes.Structure):
    _fields_ = [("out_features", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("mma_type", ctypes.c_int32)]

    def __repr__(self):
        return (f"LinearDims(out_features={self.out_features}, in_features={self.in_features}, "
                f"max_rows={self.max_rows}, mma_type={self.mma_type})")


def make_linear_dims(out_features: int, in_features: int, max_rows: int,
                     mma_type: int = MOE_MMA_MXF4xMXF4) -> LinearDims:
    return LinearDims(out_features, in_features, max_rows, mma_type)


class RopeDims(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("magnitude", ctypes.c_double)]

    def __repr__(self):
        return "RopeDims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


MOE_ROPE_HALF = 0
MOE_ROPE_INTERLEAVED = 1
MOE_ROPE_UNSCALED = 0
MOE_ROPE_LINEAR = 1
MOE_ROPE_NTK = 2
MOE_ROPE_YARN = 3


def make_rope_dims(head_dim: int, rotary_dim: int | None = None, layout: int = MOE_ROPE_HALF,
                   base: float = 10000.0, scaling: int = MOE_ROPE_UNSCALED, factor: float = 1.0,
                   original_length: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                   magnitude: float = 0.0) -> RopeDims:
    return RopeDims(head_dim, head_dim if rotary_dim is None else rotary_dim, layout, scaling,
                    base, factor, original_length, beta_fast, beta_slow, magnitude)


class AttentionDims(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("max_shared_tokens", ctypes.c_int32)]

    @property
    def cache_shape(self) -> tuple[int, int, int, int]:
        """Of each cache."""
        return self.num_pages, self.kv_heads, self.page_size, self.head_dim

    def __repr__(self):
        return ("AttentionDims("
                + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")")


def make_attention_dims(q_heads: int, kv_heads: int, head_dim: int, num_pages: int,
                        page_size: int, max_tokens: int, max_shared_tokens: int = 0
                        ) -> AttentionDims:
    return AttentionDims(q_heads, kv_heads, head_dim, num_pages, page_size, max_tokens,
                         max_shared_tokens)


class KvBatch(ctypes.Structure):
    """A step's batch (make_kv_batch).  It holds the addresses of its tensors and keeps them
    alive; their contents may change between calls."""
    _fields_ = [("seq_lens_dev", ctypes.c_void_p), ("cu_new_dev", ctypes.c_void_p),
                ("pages_dev", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("tokens", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("pages_ld", ctypes.c_int32), ("shared_len", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_string(status)}: {message}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmxmoe.so (built by __graft_entry__.build() / build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        l = ctypes.CDLL(LIB_PATH)
        D, LD = ctypes.POINTER(MoeDims), ctypes.POINTER(LinearDims)
        RD, AD, KB = (ctypes.POINTER(t) for t in (RopeDims, AttentionDims, KvBatch))
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sigs = {
            "moe_last_error": ([], ctypes.c_char_p),
            "moe_status_string": ([i32], ctypes.c_char_p),
            "moe_validate_dims": ([D], i32),
            "moe_prepared_weights_size": ([D], sz),
            "moe_workspace_size": ([D], sz),
            "moe_workspace_init": ([D, vp, sz, vp], i32),
            "moe_quantize_mxfp4": ([vp, i64, i32, vp, vp, vp], i32),
            "moe_quantize_nvfp4": ([vp, i64, i32, vp, vp, vp], i32),
            "moe_prepare_weights": ([D, vp, vp, vp, vp, vp, sz, vp], i32),
            "moe_pre_dispatch": ([D, vp, vp, vp, i32, vp, sz, vp], i32),
            "moe_forward": ([D, vp, vp, sz, vp, i32, vp], i32),
            "moe_run_host": ([D, vp, vp, sz, vp, vp, vp, vp, i32, vp], i32),
            "moe_few_forward": ([D, vp, vp, vp, vp, vp, i32, vp, sz, vp, vp], i32),
            "moe_check": ([vp, vp], i32),
            "moe_read_dispatch": ([D, vp, i32, vp, vp, vp, vp, vp], i32),
            "moe_read_intermediate": ([D, vp, i32, vp, vp], i32),
            "moe_debug_gate_up": ([D, vp, vp, sz, vp, i32, vp], i32),
            "moe_profile_enable": ([i32], i32),
            "moe_profile_read": ([ctypes.POINTER(ctypes.c_char_p), vp, vp, i32], i32),
            "moe_profile_reset": ([], None),
            "moe_device_sm_count": ([], i32),
            "moe_bucket_noalloc": ([D, vp, vp, i32, vp, vp, vp], i32),
            "moe_debug_wait_probe": ([vp, i64, vp], i32),
            "moe_fp4_mma_probe": ([vp, i32, i32, i32, i64, vp], i32),
            "moe_fp4_mma_probe_pair": ([vp, i32, i32, i64, vp], i32),
            "moe_mxfp8_scale_bytes": ([i64, i64, i32], ctypes.c_size_t),
            "moe_workspace_set_dispatch": ([vp, i32], i32),
            "moe_workspace_set_tiles": ([vp, i32], i32),
            "moe_mxfp8_quantize": ([vp, i64, i64, vp, vp, i32, i64, vp], i32),
            "moe_rmsnorm_mxfp8": ([vp, i64, vp, i64, vp, ctypes.c_float, i64, i64, vp, i64, vp,
                                   i64, vp, vp, i32, i64, vp], i32),
            "moe_linear_weights_size": ([LD], sz),
            "moe_linear_workspace_size": ([LD], sz),
            "moe_linear_prepare": ([LD, vp, vp, vp, sz, vp], i32),
            "moe_linear_workspace_init": ([LD, vp, sz, vp], i32),
            "moe_linear_forward": ([LD, vp, vp, i64, i64, vp, i64, i32, vp, sz, vp], i32),
            "moe_linear_forward_pair": ([LD, vp, vp, vp, i64, vp, i64, i32, vp, sz, vp], i32),
            "moe_linear_check": ([vp, vp], i32),
            "moe_debug_linear_give_up": ([vp, i32], i32),
            "moe_rope_table_size": ([RD], sz),
            "moe_rope_prepare": ([RD, vp, sz, vp], i32),
            "moe_rope_prepare_frequencies": ([RD, vp, vp, sz, vp], i32),
            "moe_rope": ([RD, vp, vp, i64, vp, i64, i32, vp, i64, vp], i32),
            "moe_attention_workspace_size": ([AD], sz),
            "moe_attention_workspace_init": ([AD, vp, sz, vp], i32),
            "moe_attention_set_shared": ([vp, i32], i32),
            "moe_kv_append": ([AD, KB, RD, vp, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp,
                               vp, sz, vp], i32),
            "moe_attention": ([AD, KB, vp, i64, vp, vp, ctypes.c_float, vp, i64, vp, vp, sz, vp],
                              i32),
            "moe_attention_check": ([vp, vp], i32),
        }
        for name, (args, res) in sigs.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = res
        _lib = l
    return _lib


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


status_string = moe_status_string


def moe_last_error() -> str:
    return lib().moe_last_error().decode()


def _check(status: int) -> int:
    if status != MOE_OK:
        raise MoeError(status, moe_last_error())
    return status


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return int(t)


def _nbytes(t) -> int:
    if isinstance(t, torch.Tensor):
        return t.numel() * t.element_size()
    if isinstance(t, np.ndarray):
        return t.nbytes
    raise TypeError("need a tensor or array to know its size")


_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream(stream) -> int | None:
    if stream is None:
        # the current stream's handle without building a Stream object (3 us a call)
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _elements(t, dtype, n: int, name: str, last: int | None = None) -> int | None:
    """Address of a contiguous CUDA tensor of this dtype that holds n elements, rows of `last`.

    The library sees addresses only: it would read another type as this one, and run past a
    tensor that is too small.  None and raw addresses pass."""
    if not isinstance(t, torch.Tensor):
        return None if t is None else int(t)
    if (t.dtype is dtype and t.numel() >= n and t.is_cuda and t.is_contiguous()
            and (last is None or t.size(-1) == last or t.dim() == 1)):
        return t.data_ptr()
    raise MoeError(MOE_ERR_INVALID_ARG,
                   f"{name}: need a contiguous CUDA tensor of {dtype}, {n} elements or more"
                   f"{f' in rows of {last}' if last is not None else ''}; got {t.dtype} "
                   f"{list(t.shape)}, strides {t.stride()}, on {t.device}")


def _bytes(t, n: int, name: str) -> int | None:
    """The same of n bytes, whatever the dtype."""
    try:
        if t.nbytes >= n and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        return None if t is None else int(t)
    raise MoeError(MOE_ERR_INVALID_ARG,
                   f"{name}: need {n} contiguous bytes on the GPU; got {t.dtype} "
                   f"{list(t.shape)}, strides {t.stride()}, on {t.device}")


@functools.lru_cache(maxsize=None)
def _prepared_bytes(hidden: int, inter: int, num_experts: int, mma_type: int) -> int:
    return moe_prepared_weights_size(make_dims(hidden, inter, num_experts, 1, 1, mma_type))


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)

def moe_validate_dims(dims: MoeDims) -> None:
    _check(lib().moe_validate_dims(ctypes.byref(dims)))


def moe_prepared_weights_size(dims: MoeDims) -> int:
    return int(lib().moe_prepared_weights_size(ctypes.byref(dims)))


def moe_workspace_size(dims: MoeDims) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(dims)))


def moe_workspace_init(dims: MoeDims, ws, stream=None) -> None:
    _check(lib().moe_workspace_init(ctypes.byref(dims), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_quantize_mxfp4(src, codes, scales, stream=None) -> None:
    rows, K = src.shape
    _check(lib().moe_quantize_mxfp4(_ptr(src), rows, K, _ptr(codes), _ptr(scales), _stream(stream)))


def moe_quantize_nvfp4(src, codes, scales, stream=None) -> None:
    rows, K = src.shape
    _check(lib().moe_quantize_nvfp4(_ptr(src), rows, K, _ptr(codes), _ptr(scales), _stream(stream)))


def sf_group(dims: MoeDims) -> int:
    """Elements per scale: 16 for nvf4xnvf4, 32 otherwise."""
    return 16 if dims.mma_type == MOE_MMA_NVF4xNVF4 else 32


def moe_prepare_weights(dims: MoeDims, w1_codes, w1_scales, w2_codes, w2_scales, prepared,
                        stream=None) -> None:
    _check(lib().moe_prepare_weights(ctypes.byref(dims), _ptr(w1_codes), _ptr(w1_scales),
                                     _ptr(w2_codes), _ptr(w2_scales), _ptr(prepared),
                                     _nbytes(prepared), _stream(stream)))


def moe_pre_dispatch(dims: MoeDims, x, topk_ids, topk_weights, num_tokens: int, ws,
                     stream=None) -> None:
    _check(lib().moe_pre_dispatch(ctypes.byref(dims), _ptr(x), _ptr(topk_ids), _ptr(topk_weights),
                                  int(num_tokens), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_forward(dims: MoeDims, prepared, ws, out, num_tokens: int, stream=None) -> None:
    _check(lib().moe_forward(ctypes.byref(dims), _ptr(prepared), _ptr(ws), _nbytes(ws), _ptr(out),
                             int(num_tokens), _stream(stream)))


def moe_run_host(dims: MoeDims, prepared, ws, x_host, topk_ids_host, topk_weights_host, out_host,
                 num_tokens: int, stream=None) -> None:
    _check(lib().moe_run_host(ctypes.byref(dims), _ptr(prepared), _ptr(ws), _nbytes(ws),
                              _ptr(x_host), _ptr(topk_ids_host), _ptr(topk_weights_host),
                              _ptr(out_host), int(num_tokens), _stream(stream)))


def moe_few_forward(dims: MoeDims, prepared, router, x, topk_ids, topk_weights, num_tokens: int,
                    ws, out, stream=None) -> None:
    """The whole layer for up to 16 tokens: router (or, with router None, given ids and
    weights), experts and their weighted sum.

    x and out are bf16 [tokens, hidden], router bf16 [experts, hidden], topk_ids int32 and
    topk_weights fp32 [tokens, topk], each contiguous."""
    T, H, E, k = num_tokens, dims.hidden, dims.num_experts, dims.topk
    bf16 = torch.bfloat16
    status = (_lib or lib()).moe_few_forward(
        ctypes.byref(dims),
        _bytes(prepared, _prepared_bytes(H, dims.inter, E, dims.mma_type), "prepared"),
        _elements(router, bf16, E * H, "router", H), _elements(x, bf16, T * H, "x", H),
        _elements(topk_ids, torch.int32, T * k, "topk_ids"),
        _elements(topk_weights, torch.float32, T * k, "topk_weights"), T, ws.data_ptr(), ws.nbytes,
        _elements(out, bf16, T * H, "out", H),
        _raw_stream(_current_device()) if stream is None else _stream(stream))
    if status:
        _check(status)


def moe_check(ws, stream=None) -> None:
    _check(lib().moe_check(_ptr(ws), _stream(stream)))


def _act_row_bytes(dims: MoeDims, K: int) -> int:
    """Bytes of a quantised activation row: E4M3 (fp8xfp4) or packed E2M1."""
    return K if dims.mma_type == MOE_MMA_FP8xFP4 else K // 2


def moe_read_dispatch(dims: MoeDims, ws, num_tokens: int) -> dict:
    T, k, H, E = int(num_tokens), dims.topk, dims.hidden, dims.num_experts
    out = {
        "counts": np.zeros(E, np.int32),
        "assign_slot": np.zeros(T * k, np.int32),
        "x_codes": np.zeros((T * k, _act_row_bytes(dims, H)), np.uint8),
        "x_scales": np.zeros((T * k, H // sf_group(dims)), np.uint8),
        "slot_token": np.zeros(T * k, np.int32),
    }
    _check(lib().moe_read_dispatch(ctypes.byref(dims), _ptr(ws), T, *[_ptr(out[n]) for n in
                                   ("counts", "assign_slot", "x_codes", "x_scales", "slot_token")]))
    return out


def moe_read_intermediate(dims: MoeDims, ws, num_tokens: int) -> dict:
    T, k, I = int(num_tokens), dims.topk, dims.inter
    out = {"h_codes": np.zeros((T * k, _act_row_bytes(dims, I)), np.uint8),
           "h_scales": np.zeros((T * k, I // sf_group(dims)), np.uint8)}
    _check(lib().moe_read_intermediate(ctypes.byref(dims), _ptr(ws), T, _ptr(out["h_codes"]),
                                       _ptr(out["h_scales"])))
    return out


def moe_debug_gate_up(dims: MoeDims, prepared, ws, gate_up, num_tokens: int, stream=None) -> None:
    _check(lib().moe_debug_gate_up(ctypes.byref(dims), _ptr(prepared), _ptr(ws), _nbytes(ws),
                                   _ptr(gate_up), int(num_tokens), _stream(stream)))


def moe_debug_wait_probe(ws, limit_ns: int, stream=None) -> None:
    _check(lib().moe_debug_wait_probe(_ptr(ws), int(limit_ns), _stream(stream)))


MOE_DISPATCH_BUCKETED = 0
MOE_DISPATCH_PULL = 1
MOE_TILES_AUTO = 0
MOE_TILES_WIDE = 1
MOE_TILES_NARROW = 2
MOE_TILES_MEDIUM = 3
MOE_TILES_PAIR = 4


def moe_workspace_set_dispatch(ws, mode: int) -> None:
    """Bucketed token copies (TMA) or per-token rows gathered by the layer kernel."""
    _check(lib().moe_workspace_set_dispatch(_ptr(ws), int(mode)))


def moe_workspace_set_tiles(ws, mode: int) -> None:
    """Token tiles of 128 rows (wide), 64 (medium), 32 (narrow) or chosen per dispatch (auto)."""
    _check(lib().moe_workspace_set_tiles(_ptr(ws), int(mode)))


MOE_SF_PACKED = 0
MOE_SF_128X4 = 1


def moe_mxfp8_scale_bytes(rows_cap: int, K: int, layout: int) -> int:
    return int(lib().moe_mxfp8_scale_bytes(int(rows_cap), int(K), int(layout)))


def moe_mxfp8_quantize(x, rows: int, K: int, q, sf, layout: int, rows_cap: int | None = None,
                       stream=None) -> None:
    """bf16 rows -> E4M3 values and UE8M0 scales (packed int32 or the 4-D 128x4 layout)."""
    _check(lib().moe_mxfp8_quantize(_ptr(x), int(rows), int(K), _ptr(q), _ptr(sf), int(layout),
                                    int(rows if rows_cap is None else rows_cap), _stream(stream)))


def _matrix(t, shape, dtypes, name: str) -> int:
    """Row stride of a 2-D tensor of this shape and one of the dtypes, its rows contiguous."""
    if t.dtype in dtypes and t.shape == shape:
        if t.is_contiguous():   # a single row is, whatever its stride says
            return shape[1]
        ld, step = t.stride()
        if step == 1 or shape[1] == 1:
            return ld           # checked by the library
        raise ValueError(f"{name}: rows must be contiguous")
    raise ValueError(f"{name}: need {list(shape)} of {dtypes}, got {list(t.shape)} of {t.dtype}")


def _on_gpu(**tensors) -> None:
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: need a CUDA tensor, got one on {t.device}")


_BF16 = (torch.bfloat16,)
_OUT = (torch.bfloat16, torch.float32)


def moe_rmsnorm_mxfp8(x, gamma, eps: float, q=None, sf=None, layout: int = MOE_SF_128X4, *,
                      residual=None, residual_out=None, y=None, rows_cap: int | None = None,
                      stream=None) -> None:
    """RMSNorm of x + residual: bf16 sum and norm, and the norm's MXFP8 pair (q, sf).

    x, residual, residual_out and y are bf16 [rows, K] tensors with contiguous rows; q and sf
    as moe_mxfp8_quantize writes them.  Any output may be left out."""
    shape = x.shape
    rows, K = shape
    px, ldx = x.data_ptr(), _matrix(x, shape, _BF16, "x")
    pr = pro = py = None
    ldr = ldro = ldy = 0
    if residual is not None:
        ldr, pr = _matrix(residual, shape, _BF16, "residual"), residual.data_ptr()
    if residual_out is not None:
        ldro, pro = _matrix(residual_out, shape, _BF16, "residual_out"), residual_out.data_ptr()
    if y is not None:
        ldy, py = _matrix(y, shape, _BF16, "y"), y.data_ptr()
    if gamma.dtype is not torch.bfloat16 or gamma.shape != (K,) or not gamma.is_contiguous():
        raise ValueError(f"gamma: need contiguous bf16 [{K}]")
    if not (x.is_cuda and gamma.is_cuda and (pr is None or residual.is_cuda)
            and (pro is None or residual_out.is_cuda) and (py is None or y.is_cuda)):
        _on_gpu(x=x, gamma=gamma, residual=residual, residual_out=residual_out, y=y)
    cap = rows if rows_cap is None else rows_cap
    pq = psf = None
    if q is not None:
        pq = _bytes(q, rows * K, "q")
    if sf is not None:   # (K not in whole scale words: the library refuses it)
        sf_rows = (cap + 127) // 128 * 128 if layout == MOE_SF_128X4 else cap
        psf = _bytes(sf, sf_rows * (K // 128) * 4, "sf")
    status = (_lib or lib()).moe_rmsnorm_mxfp8(px, ldx, pr, ldr, gamma.data_ptr(), eps, rows, K,
                                               pro, ldro, py, ldy, pq, psf, layout, cap,
                                               _raw_stream(_current_device()) if stream is None
                                               else _stream(stream))
    if status:
        _check(status)


def moe_linear_weights_size(dims: LinearDims) -> int:
    return int(lib().moe_linear_weights_size(ctypes.byref(dims)))


def moe_linear_workspace_size(dims: LinearDims) -> int:
    return int(lib().moe_linear_workspace_size(ctypes.byref(dims)))


def moe_linear_prepare(dims: LinearDims, codes, scales, prepared, stream=None) -> None:
    """Canonical MXFP4 codes [N, K/2] and scales [N, K/32] into the product's layout."""
    N, K = dims.out_features, dims.in_features
    _check(lib().moe_linear_prepare(ctypes.byref(dims), _bytes(codes, N * K // 2, "codes"),
                                    _bytes(scales, N * K // 32, "scales"),
                                    _bytes(prepared, 0, "prepared"), _nbytes(prepared),
                                    _stream(stream)))


def moe_linear_workspace_init(dims: LinearDims, ws, stream=None) -> None:
    _check(lib().moe_linear_workspace_init(ctypes.byref(dims), _bytes(ws, 0, "workspace"),
                                           _nbytes(ws), _stream(stream)))


@functools.lru_cache(maxsize=None)
def _linear_bytes(out_features: int, in_features: int, mma_type: int) -> int:
    return moe_linear_weights_size(make_linear_dims(out_features, in_features, 1, mma_type))


def moe_linear_forward(dims: LinearDims, prepared, x, out, ws, stream=None) -> None:
    """out = Q(x) W^T: x bf16 [rows, K], out bf16 or fp32 [rows, N], contiguous rows each."""
    rows, N, K = x.shape[0], dims.out_features, dims.in_features
    ldx = _matrix(x, (rows, K), _BF16, "x")
    ldo = _matrix(out, (rows, N), _OUT, "out")
    if not (x.is_cuda and out.is_cuda):
        _on_gpu(x=x, out=out)
    blob = _bytes(prepared, _linear_bytes(N, K, dims.mma_type), "prepared")
    status = (_lib or lib()).moe_linear_forward(
        ctypes.byref(dims), blob, x.data_ptr(), ldx, rows, out.data_ptr(), ldo,
        out.dtype is torch.float32, ws.data_ptr(), ws.nbytes,
        _raw_stream(_current_device()) if stream is None else _stream(stream))
    if status:
        _check(status)


def moe_linear_forward_pair(dims: LinearDims, prepared, q, sf, rows: int, out, ws,
                            stream=None) -> None:
    """The product on an MXFP8 pair (q [rows, K], sf in MOE_SF_128X4 layout)."""
    N, K = dims.out_features, dims.in_features
    ldo = _matrix(out, (rows, N), _OUT, "out")
    if not out.is_cuda:
        _on_gpu(out=out)
    status = (_lib or lib()).moe_linear_forward_pair(
        ctypes.byref(dims), _bytes(prepared, _linear_bytes(N, K, dims.mma_type), "prepared"),
        _bytes(q, rows * K, "q"),
        # (K not in whole scale blocks: the library refuses it)
        _bytes(sf, (rows + 127) // 128 * (K // 128) * 512, "sf"), rows, out.data_ptr(), ldo,
        out.dtype is torch.float32, ws.data_ptr(), ws.nbytes,
        _raw_stream(_current_device()) if stream is None else _stream(stream))
    if status:
        _check(status)


def moe_linear_check(ws, stream=None) -> None:
    _check(lib().moe_linear_check(_ptr(ws), _stream(stream)))


def moe_debug_linear_give_up(ws, on: bool) -> None:
    """Calls on this linear workspace behave as if a device wait had run out."""
    _check(lib().moe_debug_linear_give_up(_ptr(ws), int(on)))


def moe_rope_table_size(dims: RopeDims) -> int:
    return int(lib().moe_rope_table_size(ctypes.byref(dims)))


def moe_rope_prepare(dims: RopeDims, table, stream=None) -> None:
    """Writes the rotation's table, once for the calls that take it with these dims."""
    _check(lib().moe_rope_prepare(ctypes.byref(dims), _bytes(table, 0, "table"), _nbytes(table),
                                  _stream(stream)))


def moe_rope_prepare_frequencies(dims: RopeDims, frequencies, table, stream=None) -> None:
    """The same with the caller's own frequencies, radians from one position to the next for each
    of the rotary_dim / 2 pairs."""
    w = [float(f) for f in frequencies]
    if len(w) != dims.rotary_dim // 2:
        raise ValueError(f"frequencies: need {dims.rotary_dim // 2}, got {len(w)}")
    _check(lib().moe_rope_prepare_frequencies(
        ctypes.byref(dims), (ctypes.c_double * len(w))(*w), _bytes(table, 0, "table"),
        _nbytes(table), _stream(stream)))


def yarn_frequencies(rotary_dim: int, base: float, factor: float, original_length: float,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, whole: bool = True
                     ) -> list[float]:
    """YaRN's frequencies with a ramp over the pairs' indices, as many models are trained with it
    (MOE_ROPE_YARN's is one over their turns): from base^(-2i / rotary_dim) up to the index at
    which a pair makes beta_fast turns over the trained length, to that over factor from the one
    with beta_slow turns on.  The two indices are rounded outwards to whole ones unless told not to."""
    d = rotary_dim

    def index(turns):                    # original_length base^(-2 index / d) = 2 pi turns
        return d * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))

    low, high = index(beta_fast), index(beta_slow)
    if whole:
        low, high = math.floor(low), math.ceil(high)
    low, high = max(low, 0), min(high, d - 1)
    frequencies = []
    for i in range(d // 2):
        w = base ** (-2 * i / d)
        g = 1 - min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
        frequencies.append(w * g + w / factor * (1 - g))
    return frequencies


def _here(t, name: str, device: int | None = None) -> int:
    """Address of a tensor on the current device."""
    if device is None:
        device = _current_device()
    if t.get_device() == device:
        return t.data_ptr()
    raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: need a tensor on the current CUDA device "
                                        f"{device}, got one on {t.device}")


def _heads(t, tokens: int, heads: int, D: int, name: str) -> int:
    """Token stride of bf16 [tokens, heads, D] or [tokens, heads * D], a token's row contiguous."""
    shape = t.shape
    if t.dtype is torch.bfloat16:
        row = heads * D
        if shape == (tokens, heads, D):
            if t.is_contiguous():
                return row
            strides = t.stride()
            if (strides[2] == 1 or D == 1) and (strides[1] == D or heads == 1):
                return strides[0] if tokens > 1 else row
        elif shape == (tokens, row):
            strides = t.stride()
            if strides[1] == 1 or row == 1:
                return strides[0] if tokens > 1 else row
    raise ValueError(f"{name}: need bf16 [{tokens}, {heads}, {D}] with contiguous tokens, got "
                     f"{t.dtype} {list(shape)}, strides {t.stride()}")


def _ints(t, n: int, name: str, device: int | None = None) -> int:
    if t.dtype is torch.int32 and t.numel() == n and t.is_contiguous():
        return _here(t, name, device)
    raise ValueError(f"{name}: need {n} contiguous int32, got {t.dtype} {list(t.shape)}")


def _table(table, rope: RopeDims, device: int) -> int:
    """Address of the rotation's table; raw addresses pass."""
    if isinstance(table, torch.Tensor):
        _here(table, "table", device)
    return _bytes(table, 4 * rope.rotary_dim, "table")


def moe_rope(dims: RopeDims, table, x, positions, out=None, stream=None) -> None:
    """Rotates x, bf16 [tokens, heads, head_dim] with contiguous tokens, by each token's int32
    position, into out or in place."""
    if x.dim() != 3:
        raise ValueError(f"x: need [tokens, heads, head_dim], got {list(x.shape)}")
    T, heads, D = x.shape
    if D != dims.head_dim:
        raise ValueError(f"x: heads of {D} elements, the rotation's of {dims.head_dim}")
    device = _current_device()
    px, ldx = _here(x, "x", device), _heads(x, T, heads, D, "x")
    po, ldo = px, ldx
    if out is not None and out is not x:
        po, ldo = _here(out, "out", device), _heads(out, T, heads, D, "out")
    status = (_lib or lib()).moe_rope(
        ctypes.byref(dims), _table(table, dims, device), px, ldx,
        _ints(positions, T, "positions", device), T, heads, po, ldo,
        _raw_stream(device) if stream is None else _stream(stream))
    if status:
        _check(status)


def make_kv_batch(seq_lens, pages, tokens: int, cu_new=None, max_new: int | None = None,
                  shared_len: int = 0) -> KvBatch:
    """A step's batch: seq_lens int32 [batch], pages int32 [batch, n], and, unless every sequence
    has tokens / batch new tokens, cu_new int32 [batch + 1] with the most of one, max_new."""
    batch = seq_lens.numel()
    if pages.dim() != 2 or pages.shape[0] != batch:
        raise ValueError(f"pages: need [{batch}, n], got {list(pages.shape)}")
    if cu_new is not None and max_new is None:
        raise ValueError("max_new: needed with cu_new")
    b = KvBatch(_ints(seq_lens, batch, "seq_lens"),
                None if cu_new is None else _ints(cu_new, batch + 1, "cu_new"),
                _ints(pages, pages.numel(), "pages"), batch, tokens,
                1 if max_new is None else max_new, pages.shape[1], shared_len)
    b.tensors, b.device = (seq_lens, cu_new, pages), seq_lens.get_device()
    return b


def moe_attention_workspace_size(dims: AttentionDims) -> int:
    return int(lib().moe_attention_workspace_size(ctypes.byref(dims)))


def moe_attention_workspace_init(dims: AttentionDims, ws, stream=None) -> None:
    _check(lib().moe_attention_workspace_init(ctypes.byref(dims), _bytes(ws, 0, "workspace"),
                                              _nbytes(ws), _stream(stream)))


MOE_SHARED_AUTO = 0
MOE_SHARED_ALWAYS = 1
MOE_SHARED_NEVER = 2


def moe_attention_set_shared(ws, mode: int) -> None:
    """A shared prefix in one pass for the batch, for each sequence, or what pays (auto)."""
    _check(lib().moe_attention_set_shared(_ptr(ws), int(mode)))


def _cache(t, shape: tuple, name: str, device: int) -> int:
    if t.dtype is torch.bfloat16 and t.shape == shape and t.is_contiguous():
        return _here(t, name, device)
    raise ValueError(f"{name}: need contiguous bf16 {list(shape)}, got {t.dtype} "
                     f"{list(t.shape)}")


def _batch_device(batch: KvBatch) -> int:
    device = _current_device()
    if batch.device != device:
        raise MoeError(MOE_ERR_INVALID_ARG, f"batch: its tensors lie on device {batch.device}, "
                                            f"current is {device}")
    return device


def moe_kv_append(dims: AttentionDims, batch: KvBatch, k, v, k_cache, v_cache, ws, *, rope=None,
                  table=None, positions=None, q=None, q_out=None, stream=None) -> None:
    """Appends keys (rotated, given rope and its table) and values to the paged cache, and
    rotates q into q_out (or in place).  q, k and v are bf16 [tokens, heads, head_dim]."""
    device = _batch_device(batch)
    T, shape = batch.tokens, dims.cache_shape
    _, hk, _, D = shape
    pq = pqo = pt = None
    ldq = ldqo = 0
    if q is not None:
        hq = dims.q_heads
        pq, ldq = _here(q, "q", device), _heads(q, T, hq, D, "q")
        pqo, ldqo = pq, ldq
        if q_out is not None and q_out is not q:
            pqo, ldqo = _here(q_out, "q_out", device), _heads(q_out, T, hq, D, "q_out")
    elif q_out is not None:
        raise ValueError("q_out: given without q")
    if rope is not None:
        pt = _table(table, rope, device)
        rope = ctypes.byref(rope)
    elif table is not None:
        raise ValueError("table: given without rope")
    status = (_lib or lib()).moe_kv_append(
        ctypes.byref(dims), ctypes.byref(batch), rope, pt,
        None if positions is None else _ints(positions, T, "positions", device), pq, ldq, pqo,
        ldqo, _here(k, "k", device), _heads(k, T, hk, D, "k"), _here(v, "v", device),
        _heads(v, T, hk, D, "v"), _cache(k_cache, shape, "k_cache", device),
        _cache(v_cache, shape, "v_cache", device), _here(ws, "workspace", device), ws.nbytes,
        _raw_stream(device) if stream is None else _stream(stream))
    if status:
        _check(status)


def moe_attention(dims: AttentionDims, batch: KvBatch, q, k_cache, v_cache, out, ws, *,
                  scale: float | None = None, lse=None, stream=None) -> None:
    """Attention of the batch's new tokens over the paged cache, which holds them already.

    q and out are bf16 [tokens, q_heads, head_dim], lse fp32 [tokens, q_heads] or None; scale is
    head_dim ** -0.5 unless given."""
    device = _batch_device(batch)
    T, shape, hq = batch.tokens, dims.cache_shape, dims.q_heads
    D = shape[3]
    pl = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (T, hq) or not lse.is_contiguous():
            raise ValueError(f"lse: need contiguous fp32 [{T}, {hq}]")
        pl = _here(lse, "lse", device)
    status = (_lib or lib()).moe_attention(
        ctypes.byref(dims), ctypes.byref(batch), _here(q, "q", device),
        _heads(q, T, hq, D, "q"), _cache(k_cache, shape, "k_cache", device),
        _cache(v_cache, shape, "v_cache", device), D ** -0.5 if scale is None else scale,
        _here(out, "out", device), _heads(out, T, hq, D, "out"), pl,
        _here(ws, "workspace", device), ws.nbytes,
        _raw_stream(device) if stream is None else _stream(stream))
    if status:
        _check(status)


def moe_attention_check(ws, stream=None) -> None:
    _check(lib().moe_attention_check(_ptr(ws), _stream(stream)))


def moe_fp4_mma_probe(ws, n: int, blocks_per_sm: int, blocks: int, mma_count: int,
                      stream=None) -> None:
    _check(lib().moe_fp4_mma_probe(_ptr(ws), int(n), int(blocks_per_sm), int(blocks),
                                   int(mma_count), _stream(stream)))


def moe_fp4_mma_probe_pair(ws, n: int, pairs: int, mma_count: int, stream=None) -> None:
    """The probe's M=256 form across SM pairs (tcgen05 cta_group::2)."""
    _check(lib().moe_fp4_mma_probe_pair(_ptr(ws), int(n), int(pairs), int(mma_count),
                                        _stream(stream)))


def moe_profile_enable(on: bool) -> None:
    _check(lib().moe_profile_enable(1 if on else 0))


def moe_profile_read(max_kernels: int = 32) -> dict:
    names = (ctypes.c_char_p * max_kernels)()
    ms = np.zeros(max_kernels, np.float32)
    n_launch = np.zeros(max_kernels, np.int32)
    n = lib().moe_profile_read(names, _ptr(ms), _ptr(n_launch), max_kernels)
    return {names[i].decode(): (float(ms[i]), int(n_launch[i])) for i in range(n)}


def moe_profile_reset() -> None:
    lib().moe_profile_reset()


def moe_device_sm_count() -> int:
    return int(lib().moe_device_sm_count())


def moe_bucket_noalloc(dims: MoeDims, topk_ids, topk_weights, num_tokens: int, counts,
                       assign_slot, stream=None) -> None:
    """Bucketing with the library's own static scratch; allocates nothing on the device."""
    _check(lib().moe_bucket_noalloc(ctypes.byref(dims), _ptr(topk_ids), _ptr(topk_weights),
                                    int(num_tokens), _ptr(counts), _ptr(assign_slot),
                                    _stream(stream)))
