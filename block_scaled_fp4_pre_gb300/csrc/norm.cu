// Root-mean-square norm with the residual's addition and an MXFP8 output, for sm_103a.
//
//   r = x + residual                      (fp32; also stored as bf16)
//   y = r * gamma / sqrt(mean(r^2) + eps) (fp32; optionally stored as bf16)
//   q, sf = MXFP8 of y                    (E4M3, one UE8M0 scale per 32 elements)
//
// One pass: a row's values stay in registers between the sum of squares and the
// quantisation, so each input element is read once and each output written once.  y is
// quantised from its fp32 value, not from the bf16 one, so q carries one rounding.  The
// sum is fp32 in a fixed order (per thread, then a shuffle tree, then a tree over the
// warps) that depends on K and, above K = 1024, on whether the call has more rows than the
// device has SMs: the same call gives the same bits, whatever else runs.
//
// An element next to a rounding boundary of E4M3, or a group's largest next to a power of
// two's, flips with the last bits of y.  So the sums, the mean and the reciprocal root are
// pairs of floats, and where the nearest float of some y lies on a boundary (its last 19
// bits are 0, one float in 2^19) it is rounded to odd instead: a value that is not exactly a
// float gets the float next to it towards zero with its last bit set, which is on no
// boundary, and E4M3 of that is E4M3 of the unrounded value.  What is left are the sums' own
// roundings.  Codes a million that differ from those of 64 bits, on rows whose squares a few
// large channels dominate, here and in plain fp32: K = 768 0.08 and 1.2, 1152 0.18 and 0.87,
// 1408 0.12 and 0.70, 2048 0.16 and 0.60, 4096 0.15 and 0.64, for 4 us of 93 at 16384 x 4096.
// With the squares of each vector as a tree and pairs all through: 0.06, 0.10, 0.13 and 0.03
// from K = 1152 on, for another 1 us of 38 at 16384 x 1408 and 4 of 94 at 16384 x 4096.
//
// Layout: a thread holds V vectors of 8 consecutive elements (16 bytes of bf16), so four
// lanes hold a scale's 32 elements and reduce its amax with two shuffles, and sixteen
// lanes a whole scale word (four scales), which is stored as one 32-bit word in either
// layout.
//
// Bound by HBM at large row counts: 16384 x 4096 with residual and both outputs (606 MB)
// 93 us, 0.96 of the measured copy bandwidth; by launch and load latency at few: one row
// of 4096 2.2 us.
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mxmoe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarpRowThreads = 256;   // warp-per-row form: eight rows a block

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = lo_bf16(w.x); v[1] = hi_bf16(w.x);
  v[2] = lo_bf16(w.y); v[3] = hi_bf16(w.y);
  v[4] = lo_bf16(w.z); v[5] = hi_bf16(w.z);
  v[6] = lo_bf16(w.w); v[7] = hi_bf16(w.w);
}

// Two fp32 to packed bf16, round to nearest even, `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                    bf16x2(v[6], v[7]));
}

// Byte offset of the scale word (groups 4w..4w+3) of a row.
__device__ __forceinline__ size_t sf_word(int64_t row, int w, int words, int layout) {
  return layout == MOE_SF_128X4 ? sf_atom_offset((size_t)row, 4 * w, words)
                                : ((size_t)row * words + w) * 4;
}

// A value as the sum of two floats, |lo| at most half a unit of hi's last place.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
// Adds the pairs of the lanes that differ in `o`.
__device__ __forceinline__ Two lane_sum(Two a, int o) {
  const Two s = two_sum(a.hi, __shfl_xor_sync(kAll, a.hi, o));
  return {s.hi, s.lo + (a.lo + __shfl_xor_sync(kAll, a.lo, o))};
}
// r * g * inv, to nearest but for some 2^-24 of the cases next to a tie.
__device__ __forceinline__ float times(float r, float g, Two inv) {
  const float p = r * g, pl = fmaf(r, g, -p);
  return fmaf(p, inv.hi, fmaf(p, inv.lo, pl * inv.hi));
}
// The same rounded to odd.  hi is the product to nearest and lo what is left of it, to
// about 2^-45 of it: where lo is not 0 the value towards zero is hi, or one below where
// lo's sign differs.
__device__ __forceinline__ float times_to_odd(float r, float g, Two inv) {
  const float p = r * g, pl = fmaf(r, g, -p);
  const float t = p * inv.hi;
  const float tl = fmaf(p, inv.hi, -t) + fmaf(p, inv.lo, pl * inv.hi);
  const float hi = t + tl, lo = (t - hi) + tl;
  const uint32_t h = __float_as_uint(hi), l = __float_as_uint(lo);
  const uint32_t odd = (h - ((h ^ l) >> 31)) | 1u;
  // (NaN and infinities, whose lo is NaN, stay as they are)
  return fabsf(lo) > 0.f ? __uint_as_float(odd) : hi;
}
// 1 / sqrt(s / K + eps): the hardware's approximate root improved by one Newton step in
// two-float form (inv_k is 1 / K so).  Every thread of a row does this, so it has no
// division: with IEEE divisions and root here the large rows took 120 us instead of 96.
// Where the step is not a small correction (a sum of 0 with eps 0, one not finite) the
// approximate root stands.
__device__ __forceinline__ Two inverse_root(Two s, Two inv_k, float eps) {
  const float q = s.hi * inv_k.hi;
  const float ql = fmaf(s.hi, inv_k.hi, -q) + fmaf(s.hi, inv_k.lo, s.lo * inv_k.hi);
  Two m = two_sum(q, eps);
  m.lo += ql;
  const float r = rsqrtf(m.hi);
  const float t = r * r, tl = fmaf(r, r, -t);
  const float e = fmaf(-m.hi, t, 1.0f) - fmaf(m.hi, tl, m.lo * t);   // 1 - m r^2
  const float lo = 0.5f * r * e;
  return {r, fabsf(lo) < r ? lo : 0.0f};
}

// WARP_ROW: one warp a row (kWarpRowThreads / 32 rows a block); otherwise one block a row.
// V = 2 serves at most 512 threads; three such blocks an SM leave each thread 42 registers
// (without the bound: 50, and 104 us instead of 96 at 16384 x 4096).
template <int V, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowThreads : V == 2 ? 512 : 1024,
                                  WARP_ROW ? 5 : V == 2 ? 3 : 1)
    rmsnorm_mxfp8_kernel(const RmsnormArgs a) {
  __shared__ float2 part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nt = WARP_ROW ? 32 : (int)blockDim.x;       // threads of a row
  const int t = WARP_ROW ? lane : (int)threadIdx.x;
  const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * (kWarpRowThreads / 32) + warp
                               : (int64_t)blockIdx.x;
  const int vecs = a.K >> 3, words = a.K >> 7;
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  if (row >= a.rows) {
    // rows that pad the last 128-row scale block: zero scales
    if (row < a.sf_rows)
      for (int w = t; w < words; w += nt)
        *reinterpret_cast<uint32_t*>(a.sf + sf_word(row, w, words, a.layout)) = 0u;
    return;
  }
  uint4 xw[V], rw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * nt + t;
    xw[i] = rw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < vecs) {
      xw[i] = *reinterpret_cast<const uint4*>(a.x + row * a.ldx + c * 8);
      if (a.residual)
        rw[i] = *reinterpret_cast<const uint4*>(a.residual + row * a.ldr + c * 8);
    }
  }
  float r[V][8];
  Two sum = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * nt + t;
    unpack8(xw[i], r[i]);
    if (a.residual) {
      float b[8];
      unpack8(rw[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] += b[j];
    }
    if (a.residual_out && c < vecs)
      *reinterpret_cast<uint4*>(a.residual_out + row * a.ldro + c * 8) = pack8(r[i]);
    if (WARP_ROW) {   // eight squares as a tree, the vectors' sums as pairs
      float s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[j] = fmaf(r[i][2 * j], r[i][2 * j], r[i][2 * j + 1] * r[i][2 * j + 1]);
      const Two v = two_sum(sum.hi, (s[0] + s[1]) + (s[2] + s[3]));
      sum = {v.hi, sum.lo + v.lo};
    } else {          // one chain a thread: see the rates at the top of the file
#pragma unroll
      for (int j = 0; j < 8; ++j) sum.hi = fmaf(r[i][j], r[i][j], sum.hi);
    }
  }
  if (WARP_ROW || nt <= 128) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum = lane_sum(sum, o);
  } else {   // and so do the warps' trees'
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum.hi += __shfl_xor_sync(kAll, sum.hi, o);
  }
  if (!WARP_ROW) {
    if (lane == 0) part[warp] = make_float2(sum.hi, sum.lo);
    __syncthreads();
    // every warp adds the warps' sums, a lane each, as a tree of pairs
    const float2 mine = lane < (nt >> 5) ? part[lane] : make_float2(0.f, 0.f);
    sum = {mine.x, mine.y};
    const int top = 31 - __clz((nt >> 5) * 2 - 1);   // levels: 2^top lanes cover the warps
#pragma unroll 1
    for (int o = (1 << top) >> 1; o > 0; o >>= 1) sum = lane_sum(sum, o);
    sum.hi = __shfl_sync(kAll, sum.hi, 0);   // lanes past the 2^top hold other sums
    sum.lo = __shfl_sync(kAll, sum.lo, 0);
  }
  const Two inv = inverse_root(sum, Two{a.inv_k, a.inv_k_lo}, a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * nt + t;
    const bool live = c < vecs;
    float y[8], g[8];
    uint4 gw = make_uint4(0u, 0u, 0u, 0u);
    if (live) gw = *reinterpret_cast<const uint4*>(a.gamma + c * 8);
    unpack8(gw, g);
    float amax = 0.f;
    uint32_t tail = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = times(r[i][j], g[j], inv);
      tail = min(tail, __float_as_uint(y[j]) & 0x7FFFFu);
    }
    if (tail == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = times_to_odd(r[i][j], g[j], inv);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
    if (a.y && live) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c * 8) = pack8(y);
    if (a.q) {
      amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
      const int e = ptx::mxfp8_exponent(amax);
      const float m = ptx::pow2_neg(e);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= m;
      if (live) *reinterpret_cast<uint2*>(a.q + row * a.K + c * 8) = ptx::e4m3x8(y);
      uint32_t w = (uint32_t)(e + 127) << (((lane >> 2) & 3) * 8);
      w |= __shfl_xor_sync(kAll, w, 4);
      w |= __shfl_xor_sync(kAll, w, 8);
      if (live && (lane & 15) == 0)
        *reinterpret_cast<uint32_t*>(a.sf + sf_word(row, c >> 4, words, a.layout)) = w;
    }
  }
}

template <int V, bool WARP_ROW>
cudaError_t launch(const RmsnormArgs& a, int threads, cudaStream_t st) {
  const int64_t rows = a.sf_rows > a.rows ? a.sf_rows : a.rows;
  const int64_t per = WARP_ROW ? kWarpRowThreads / 32 : 1;
  return launch_pdl(rmsnorm_mxfp8_kernel<V, WARP_ROW>, dim3((unsigned)((rows + per - 1) / per)),
                    dim3(WARP_ROW ? kWarpRowThreads : threads), 0, st, a);
}

}  // namespace

cudaError_t launch_rmsnorm_mxfp8(const RmsnormArgs& args, int64_t rows_cap, cudaStream_t st) {
  RmsnormArgs a = args;
  a.sf_rows = 0;
  a.inv_k = (float)(1.0 / a.K);
  a.inv_k_lo = (float)(1.0 / a.K - (double)a.inv_k);
  if (a.q) {
    // Scales past the live rows' last block (4-D layout) or row (packed): one tail.
    const size_t live = mxfp8_scale_bytes(a.rows, a.K, a.layout);
    const size_t total = mxfp8_scale_bytes(rows_cap, a.K, a.layout);
    if (total > live) {
      cudaError_t e = cudaMemsetAsync(a.sf + live, 0, total - live, st);
      if (e != cudaSuccess) return e;
    }
    if (a.layout == MOE_SF_128X4) a.sf_rows = (a.rows + 127) / 128 * 128;
  }
  if (a.rows == 0) return cudaSuccess;
  const int vecs = a.K / 8;
  if (vecs <= 32) return launch<1, true>(a, 0, st);
  if (vecs <= 64) return launch<2, true>(a, 0, st);
  // (72 bytes a thread spilled under the bound of five blocks an SM: 16384 x 1024 in 28.8 us,
  // 0.78 of the measured copy bandwidth)
  if (vecs <= 128) return launch<4, true>(a, 0, st);
  auto threads = [&](int v) { return (vecs + v * 32 - 1) / (v * 32) * 32; };
  // With at most one block an SM the latency of a row counts: as many threads as the row
  // feeds.  With more, a row's fixed work (the sums' trees) is shared by more elements a
  // thread.  K = 4096, one vector a thread against two (before the care for ties): 1 row
  // 2.06 / 2.49 us, 16384 rows 104.3 / 89.3 us; K = 1408, 333 rows: 2.88 / 2.53 us.
  if (vecs <= 1024 && a.rows <= moe_device_sm_count()) return launch<1, false>(a, threads(1), st);
  if (vecs <= 1024) return launch<2, false>(a, threads(2), st);
  if (vecs <= 2048) return launch<4, false>(a, threads(4), st);
  // K above 16384: 64 values and as many words of loads in 64 registers; 360 bytes a thread are
  // spilled.  1024 x 32768 takes 79.6 us (its bytes at copy bandwidth 44.8), 1024 x 65536 166
  // (89.6).
  return launch<8, false>(a, threads(8), st);
}

}  // namespace mxmoe
