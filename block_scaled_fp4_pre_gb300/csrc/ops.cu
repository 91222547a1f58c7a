// C ABI of the operators around the expert layer (declared in include/mxmoe.h): the
// RMSNorm with an MXFP8 output and the MXFP4 linear product.  Argument checks, layouts
// and the registry of linear workspaces; nothing here allocates device memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>

#include "common.cuh"
#include "mxmoe.h"

using namespace mxmoe;

namespace {

moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

moe_status cuda_fail(cudaError_t e, const char* what) {
  return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t up(size_t v) { return (v + 1023) / 1024 * 1024; }

LinearShape shape_of(const moe_linear_dims& d) {
  return LinearShape{d.out_features, d.in_features, d.mma_type == MOE_MMA_FP8xFP4 ? 1 : 0};
}

struct LinWs {
  size_t flags, q, sf, total;
};

LinWs ws_layout(const moe_linear_dims& d) {
  const LinearShape s = shape_of(d);
  const size_t Kp = (size_t)linear_padded_k(s);
  const size_t rows = (size_t)d.max_rows;
  LinWs L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up(o + bytes);
    return at;
  };
  L.flags = take(256);
  L.q = take(rows * (s.f8 ? Kp : Kp / 2));
  L.sf = take((rows + 127) / 128 * (Kp / 128) * kSFAtomBytes);
  L.total = o;
  return L;
}

struct LinState {
  moe_linear_dims dims;
  bool give_up;   // moe_debug_linear_give_up
};
std::mutex g_mu;
std::map<const void*, LinState> g_linear;

moe_status check_dims(const moe_linear_dims* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARG, "dims is NULL");
  if (d->mma_type != MOE_MMA_MXF4xMXF4 && d->mma_type != MOE_MMA_FP8xFP4)
    return fail(MOE_ERR_UNSUPPORTED,
                "mma_type %d: the linear product is built for MOE_MMA_MXF4xMXF4 and "
                "MOE_MMA_FP8xFP4",
                d->mma_type);
  if (d->out_features < 1 || d->out_features > (1 << 20))
    return fail(MOE_ERR_INVALID_ARG, "out_features %d outside [1, 2^20]", d->out_features);
  if (d->in_features < 32 || d->in_features % 32 || d->in_features > 65536)
    return fail(MOE_ERR_INVALID_ARG, "in_features %d must be a multiple of 32 in [32, 65536]",
                d->in_features);
  if (d->max_rows < 1 || d->max_rows > (1 << 20))
    return fail(MOE_ERR_INVALID_ARG, "max_rows %d outside [1, 2^20]", d->max_rows);
  return MOE_OK;
}

moe_status check_ws(const moe_linear_dims* d, const void* ws, size_t ws_bytes,
                    bool* give_up) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  const size_t need = ws_layout(*d).total;
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_linear.find(ws);
  if (it == g_linear.end())
    return fail(MOE_ERR_WORKSPACE_MISMATCH,
                "workspace %p was not initialised by moe_linear_workspace_init", ws);
  const moe_linear_dims& w = it->second.dims;
  if (w.out_features != d->out_features || w.in_features != d->in_features ||
      w.max_rows != d->max_rows || w.mma_type != d->mma_type)
    return fail(MOE_ERR_WORKSPACE_MISMATCH, "workspace %p was initialised for other dims", ws);
  *give_up = it->second.give_up;
  return MOE_OK;
}

moe_status check_call(const moe_linear_dims* d, const void* prepared, int64_t rows,
                      const void* out, int64_t ldo, int32_t out_type, const void* ws,
                      size_t ws_bytes, bool* give_up) {
  moe_status s = check_dims(d);
  if (s) return s;
  if ((s = check_ws(d, ws, ws_bytes, give_up))) return s;
  if (rows < 0 || rows > d->max_rows)
    return fail(MOE_ERR_INVALID_ARG, "rows %lld outside [0, max_rows=%d]", (long long)rows,
                d->max_rows);
  if (out_type != MOE_OUT_BF16 && out_type != MOE_OUT_F32)
    return fail(MOE_ERR_INVALID_ARG, "unknown out_type %d", out_type);
  if (rows == 0) return MOE_OK;
  if (!prepared || !aligned(prepared, 256))
    return fail(MOE_ERR_INVALID_ARG, "prepared weights NULL or not 256-byte aligned");
  if (!out || !aligned(out, out_type == MOE_OUT_F32 ? 4 : 2))
    return fail(MOE_ERR_INVALID_ARG, "out NULL or not aligned to its element");
  if (ldo < d->out_features)
    return fail(MOE_ERR_INVALID_ARG, "ldo %lld below out_features %d", (long long)ldo,
                d->out_features);
  return MOE_OK;
}

// The product of a pair (q, sf) or, q null, of a few bf16 rows x.
moe_status forward(const moe_linear_dims* d, const void* prepared, const void* q, const void* sf,
                   const void* x, int64_t ldx, int64_t rows, void* out, int64_t ldo,
                   int32_t out_type, void* ws, bool give_up, cudaStream_t st) {
  const LinWs L = ws_layout(*d);
  uint8_t* b = static_cast<uint8_t*>(ws);
  LinearLaunch g;
  g.shape = shape_of(*d);
  g.w_codes = static_cast<const uint8_t*>(prepared);
  g.q = static_cast<const uint8_t*>(q);
  g.sf = static_cast<const uint8_t*>(sf);
  g.x = x;
  g.ldx = ldx;
  g.rows = rows;
  g.out = out;
  g.ldo = ldo;
  g.out_f32 = out_type == MOE_OUT_F32;
  g.flags = reinterpret_cast<int32_t*>(b + L.flags);
  g.give_up = give_up;
  g.num_sms = moe_device_sm_count();
  if (g.num_sms <= 0 || cudaGetDevice(&g.device) != cudaSuccess) return fail(MOE_ERR_CUDA, "no CUDA device");
  const cudaError_t e = launch_linear(g, st);
  if (e != cudaSuccess) return cuda_fail(e, "linear kernel");
  return MOE_OK;
}

// A row stride: a multiple of 8 elements, at least K.
bool good_stride(int64_t ld, int64_t K) { return ld >= K && ld % 8 == 0; }

}  // namespace

extern "C" {

moe_status moe_rmsnorm_mxfp8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                             const void* gamma, float eps, int64_t rows, int64_t K,
                             void* residual_out, int64_t ldro, void* y, int64_t ldy, void* q,
                             void* sf, int32_t sf_layout, int64_t rows_cap, void* stream) {
  if (K < 128 || K % 128 || K > 65536)
    return fail(MOE_ERR_INVALID_ARG, "K = %lld: must be a multiple of 128 in [128, 65536]",
                (long long)K);
  if (!q && !sf) rows_cap = rows;
  if (rows < 0 || rows > rows_cap || rows_cap > ((int64_t)1 << 23))
    return fail(MOE_ERR_INVALID_ARG,
                "rows = %lld, rows_cap = %lld: need 0 <= rows <= rows_cap <= 2^23",
                (long long)rows, (long long)rows_cap);
  if (!(eps >= 0.f) || std::isinf(eps))
    return fail(MOE_ERR_INVALID_ARG, "eps must be a finite number of at least 0");
  if ((q == nullptr) != (sf == nullptr))
    return fail(MOE_ERR_INVALID_ARG, "q and sf are given together or not at all");
  if (!q && !y && !residual_out) return fail(MOE_ERR_INVALID_ARG, "no output is given");
  if (q && sf_layout != MOE_SF_PACKED && sf_layout != MOE_SF_128X4)
    return fail(MOE_ERR_INVALID_ARG, "unknown scale layout %d", sf_layout);
  if (q && (!aligned(q, 16) || !aligned(sf, 16)))
    return fail(MOE_ERR_INVALID_ARG, "q and sf must be 16-byte aligned");
  if (rows > 0) {
    if (!x || !gamma || !aligned(x, 16) || !aligned(gamma, 16) || !aligned(residual, 16) ||
        !aligned(residual_out, 16) || !aligned(y, 16))
      return fail(MOE_ERR_INVALID_ARG, "x and gamma must be given and every tensor 16-byte aligned");
    if (!good_stride(ldx, K) || (residual && !good_stride(ldr, K)) ||
        (residual_out && !good_stride(ldro, K)) || (y && !good_stride(ldy, K)))
      return fail(MOE_ERR_INVALID_ARG, "row strides must be multiples of 8 and at least K");
  }
  RmsnormArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.gamma = static_cast<const uint16_t*>(gamma);
  a.residual_out = static_cast<uint16_t*>(residual_out);
  a.y = static_cast<uint16_t*>(y);
  a.q = static_cast<uint8_t*>(q);
  a.sf = static_cast<uint8_t*>(sf);
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldro = ldro;
  a.ldy = ldy;
  a.rows = rows;
  a.K = (int)K;
  a.layout = sf_layout;
  a.eps = eps;
  const cudaError_t e = launch_rmsnorm_mxfp8(a, rows_cap, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rmsnorm kernel");
  return MOE_OK;
}

size_t moe_linear_weights_size(const moe_linear_dims* d) {
  if (check_dims(d) != MOE_OK) return 0;
  const LinearShape s = shape_of(*d);
  return (size_t)(linear_code_bytes(s) + linear_scale_bytes(s));
}

size_t moe_linear_workspace_size(const moe_linear_dims* d) {
  if (check_dims(d) != MOE_OK) return 0;
  return ws_layout(*d).total;
}

moe_status moe_linear_prepare(const moe_linear_dims* d, const uint8_t* codes,
                              const uint8_t* scales, void* prepared, size_t prepared_bytes,
                              void* stream) {
  moe_status s = check_dims(d);
  if (s) return s;
  if (!codes || !scales || !prepared) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(prepared, 256))
    return fail(MOE_ERR_INVALID_ARG, "codes and scales must be 16-byte, prepared 256-byte aligned");
  const size_t need = moe_linear_weights_size(d);
  if (prepared_bytes < need)
    return fail(MOE_ERR_INVALID_ARG, "prepared has %zu bytes, needs %zu", prepared_bytes, need);
  const cudaError_t e = launch_linear_prepare(shape_of(*d), codes, scales,
                                              static_cast<uint8_t*>(prepared),
                                              static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "linear prepare");
  return MOE_OK;
}

moe_status moe_linear_workspace_init(const moe_linear_dims* d, void* ws, size_t ws_bytes,
                                     void* stream) {
  moe_status s = check_dims(d);
  if (s) return s;
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  const LinWs L = ws_layout(*d);
  if (ws_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", ws_bytes,
                L.total);
  // only the flags need a defined start
  const cudaError_t e = cudaMemsetAsync(ws, 0, L.q, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "workspace clear");
  try {
    std::lock_guard<std::mutex> lk(g_mu);
    g_linear[ws] = LinState{*d, false};
  } catch (...) {
    return fail(MOE_ERR_CUDA, "out of host memory for the workspace registry");
  }
  return MOE_OK;
}

moe_status moe_linear_forward(const moe_linear_dims* d, const void* prepared, const void* x,
                              int64_t ldx, int64_t rows, void* out, int64_t ldo, int32_t out_type,
                              void* ws, size_t ws_bytes, void* stream) {
  bool give_up = false;
  moe_status s = check_call(d, prepared, rows, out, ldo, out_type, ws, ws_bytes, &give_up);
  if (s || rows == 0) return s;
  if (!x || !aligned(x, 16)) return fail(MOE_ERR_INVALID_ARG, "x NULL or not 16-byte aligned");
  if (!good_stride(ldx, d->in_features))
    return fail(MOE_ERR_INVALID_ARG, "ldx must be a multiple of 8 and at least in_features");
  const LinWs L = ws_layout(*d);
  uint8_t* b = static_cast<uint8_t*>(ws);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows <= kLinFusedRows)
    return forward(d, prepared, nullptr, nullptr, x, ldx, rows, out, ldo, out_type, ws, give_up,
                   st);
  const cudaError_t e =
      launch_linear_quantize(shape_of(*d), x, ldx, rows, b + L.q, b + L.sf, st);
  if (e != cudaSuccess) return cuda_fail(e, "linear quantise");
  return forward(d, prepared, b + L.q, b + L.sf, nullptr, 0, rows, out, ldo, out_type, ws,
                 give_up, st);
}

moe_status moe_linear_forward_pair(const moe_linear_dims* d, const void* prepared, const void* q,
                                   const void* sf, int64_t rows, void* out, int64_t ldo,
                                   int32_t out_type, void* ws, size_t ws_bytes, void* stream) {
  bool give_up = false;
  moe_status s = check_call(d, prepared, rows, out, ldo, out_type, ws, ws_bytes, &give_up);
  if (s) return s;
  if (d->mma_type != MOE_MMA_FP8xFP4 || d->in_features % 128)
    return fail(MOE_ERR_UNSUPPORTED,
                "a pair needs fp8xfp4 dims and in_features a multiple of 128");
  if (rows == 0) return MOE_OK;
  if (!q || !sf || !aligned(q, 16) || !aligned(sf, 16))
    return fail(MOE_ERR_INVALID_ARG, "q and sf must be 16-byte aligned pointers");
  return forward(d, prepared, q, sf, nullptr, 0, rows, out, ldo, out_type, ws, give_up,
                 static_cast<cudaStream_t>(stream));
}

moe_status moe_linear_check(void* ws, void* stream) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_linear.find(ws) == g_linear.end())
      return fail(MOE_ERR_WORKSPACE_MISMATCH, "workspace %p was not initialised", ws);
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t flag = 0;
  cudaError_t e = read_flags(&flag, ws, st);
  if (e != cudaSuccess) return cuda_fail(e, "flag read");
  if (flag && (e = clear_flags(ws, sizeof(flag), st))) return cuda_fail(e, "flag clear");
  if (flag & kErrTimeout) return fail(MOE_ERR_TIMEOUT, "a device wait ran past its limit");
  return MOE_OK;
}

moe_status moe_debug_linear_give_up(void* ws, int32_t on) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_linear.find(ws);
  if (it == g_linear.end())
    return fail(MOE_ERR_WORKSPACE_MISMATCH, "workspace %p was not initialised", ws);
  it->second.give_up = on != 0;
  return MOE_OK;
}

}  // extern "C"
