// Microscaled 4-bit linear product for sm_103a: out = Q(x) * W^T with MXFP4 weights.
//
//   out[m, n] = sum_k q(x)[m, k] * w[n, k]        (fp32 sums, one rounding to bf16)
//
// q(x) is MXFP4 (mxf4xmxf4) or MXFP8 (fp8xfp4), one UE8M0 scale per 32 elements of K,
// and the scales are applied by the block-scaled MMA, so nothing is dequantised.
//
// Kernels.  The weight slab (128 output features) is the MMA's M operand and up to TN
// activation rows are N, so one instruction serves one row as well as a prefill tile and
// both operands' scales are whole 128-row blocks.  Roles (192 threads, two blocks an SM):
// warp 0 TMA producer, warp 1 tensor memory and MMA issue, warps 2-5 epilogue.
//
// - linear_quantize_kernel writes the activation codes and their scale blocks, for more
//   than 32 bf16 rows.
// - linear_kernel: persistent, one block's epilogue overlapping the other's MMAs.
// - linear_pair_kernel: tiles of 256 features by 192 or 256 rows over SM pairs, for large products.
// - linear_split_kernel: where there are too few tiles for the SMs, a cluster of up to
//   eight blocks splits a tile's K.  The blocks exchange their sums through distributed
//   shared memory, each adding the parts of its share of the features in order: no
//   global scratch, no atomics, the same bits every time.  With at most 32 rows its
//   epilogue warps quantise bf16 rows into the operand stages themselves, so that the
//   call is one kernel.
//
// Every wait is bounded (kWaitLimitNs); a timeout sets the workspace's error flag, and a block
// leaves only when its copies and MMAs have ended.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "per_device.h"
#include "ptx.cuh"
#include "tmap.cuh"

namespace mxmoe {
namespace {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr int kLinThreads = 192;
constexpr int kLinBlocksPerSM = 2;
constexpr int kLinTmemCols = 256;
constexpr int kLinSfCol = 128;        // two buffers of scale registers after the accumulator
constexpr int kQuantThreads = 256;

// ---------------------------------------------------------------------------
// Weights: canonical MXFP4 [N, K/2], [N, K/32] into 128-row slabs of k-block tiles and
// 128x4 scale blocks.  Rows past N and elements past K are zero.

__global__ void linear_codes_kernel(const uint8_t* __restrict__ src, uint4* __restrict__ dst,
                                    int64_t chunks, int N, int K, int num_kb, int kb_bytes) {
  const int per_row = kb_bytes / 16;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < chunks;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int c = (int)(i % per_row);
    const int64_t tr = i / per_row;                 // row of a tile
    const int r = (int)(tr & 127);
    const int64_t tile = tr >> 7;
    const int kb = (int)(tile % num_kb);
    const int64_t row = tile / num_kb * 128 + r;
    const int64_t at = (int64_t)kb * kb_bytes + c * 16;   // byte of the canonical row
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row < N && at < K / 2) v = *reinterpret_cast<const uint4*>(src + row * (K / 2) + at);
    dst[i] = v;
  }
}

__global__ void linear_scales_kernel(const uint8_t* __restrict__ src, uint32_t* __restrict__ dst,
                                     int64_t words, int N, int K, int kc4) {
  for (int64_t w = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; w < words;
       w += (int64_t)gridDim.x * blockDim.x) {
    const int q = (int)(w & 3), i = (int)((w >> 2) & 31);
    const int64_t blk = w >> 7;
    const int kc = (int)(blk % kc4);
    const int64_t row = blk / kc4 * 128 + q * 32 + i;
    uint32_t v = 0;
    if (row < N)
      for (int j = 0; j < 4; ++j)
        if (kc * 4 + j < K / 32) v |= (uint32_t)src[row * (K / 32) + kc * 4 + j] << (8 * j);
    dst[w] = v;
  }
}

// ---------------------------------------------------------------------------
// Activations: a thread takes 8 elements of a row at a time, four lanes a scale, sixteen a
// scale word.  Elements past K (to the next multiple of 128) are zero.  A block covers
// 2^span_log vectors of kQuantThreads >> span_log rows at a time and R times as many rows,
// all of a thread's loads before any arithmetic; rows and columns need no division.
// Bound by HBM: 16384 x 4096 in 33 us, 172 MB at 0.77 of the measured copy bandwidth.
template <bool F8, int R>
__global__ void __launch_bounds__(kQuantThreads)
    linear_quantize_kernel(const uint16_t* __restrict__ x, int64_t ldx, int64_t rows, int K,
                           int Kp, uint8_t* __restrict__ q, uint8_t* __restrict__ sf,
                           int span_log) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int words = Kp / 128;
  const int c = ((int)blockIdx.y << span_log) + (threadIdx.x & ((1 << span_log) - 1));
  const int rows_once = kQuantThreads >> span_log;
  const int64_t row0 = (int64_t)blockIdx.x * R * rows_once + (threadIdx.x >> span_log);
  const bool in_k = c * 8 < K, in_kp = c * 8 < Kp;
  uint4 w[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * rows_once;
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < rows && in_k) w[i] = __ldcs(reinterpret_cast<const uint4*>(x + row * ldx + c * 8));
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * rows_once;
    float v[8] = {__uint_as_float(w[i].x << 16), __uint_as_float(w[i].x & 0xFFFF0000u),
                  __uint_as_float(w[i].y << 16), __uint_as_float(w[i].y & 0xFFFF0000u),
                  __uint_as_float(w[i].z << 16), __uint_as_float(w[i].z & 0xFFFF0000u),
                  __uint_as_float(w[i].w << 16), __uint_as_float(w[i].w & 0xFFFF0000u)};
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
    amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
    const int e = F8 ? ptx::mxfp8_exponent(amax) : ptx::mx_scale_exponent(amax);
    const float m = ptx::pow2_neg(e);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= m;
    uint32_t s = (uint32_t)(e + 127) << (((threadIdx.x >> 2) & 3) * 8);
    s |= __shfl_xor_sync(kFullMask, s, 4);
    s |= __shfl_xor_sync(kFullMask, s, 8);
    if (row < rows && in_kp) {
      if (F8)
        *reinterpret_cast<uint2*>(q + row * Kp + c * 8) = ptx::e4m3x8(v);
      else
        *reinterpret_cast<uint32_t*>(q + row * (Kp / 2) + c * 4) = ptx::e2m1x8(v);
      if ((c & 15) == 0)
        *reinterpret_cast<uint32_t*>(sf + sf_atom_offset((size_t)row, c >> 2, words)) = s;
    }
  }
}

// ---------------------------------------------------------------------------
struct LinArgs {
  const uint8_t* w_sf;
  const uint8_t* t_sf;
  void* out;
  int64_t ldo;
  const uint16_t* x;     // bf16 rows and their stride (fused quantisation only)
  int64_t ldx;
  int32_t* flags;
  int M, N, K;           // K padded to a multiple of 128
  int k_live;            // K as given
  int slabs, tiles, num_kb, kc4;
  int out_f32;
  int pairs16;           // bf16 rows whose features can be stored two at a time
  int give_up;           // the MMA warps give up before their first wait (a test of that path)
};

__host__ __device__ constexpr int lin_stages(int tn) { return tn == 128 ? 3 : tn == 64 ? 4 : 5; }

struct __align__(16) LinTail {
  uint64_t full[5];
  uint64_t empty[5];
  uint64_t acc_full, acc_empty, mma_done;
  uint32_t tmem_base;
  int abort;
  int issued;   // k-blocks whose copies were issued (linear_split_kernel)
};

template <bool F8, int TN>
struct LinSmem {
  static constexpr int kSt = lin_stages(TN);
  static constexpr size_t kBSlot = (size_t)TN * kBKBytes;
  static constexpr size_t kSF = (size_t)(F8 ? 1 : 2) * kSFAtomBytes;
  static constexpr size_t kB = (size_t)kSt * kATileBytes;
  static constexpr size_t kSFA = kB + kSt * kBSlot;
  static constexpr size_t kSFB = kSFA + kSt * kSF;
  static constexpr size_t kTail = kSFB + kSt * kSF;
  static constexpr size_t kBytes = kTail + sizeof(LinTail) + 1024;
  static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two blocks per SM");
};

__device__ __forceinline__ void lin_store(const LinArgs& a, int m, int n, float v) {
  if (a.out_f32)
    static_cast<float*>(a.out)[(int64_t)m * a.ldo + n] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[(int64_t)m * a.ldo + n] = __float2bfloat16(v);
}

// Stores up to 16 rows' values of feature n (a warp's lanes hold 32 consecutive features).
// bf16 pairs where rows allow it: neighbouring lanes exchange, so that each stores two
// features of every other row, and a whole block of 16 x 32 goes through one pointer.
__device__ __forceinline__ void lin_store16(const LinArgs& a, int m, int rows, int n,
                                            const float (&v)[16]) {
  if (a.pairs16) {
    const int odd = threadIdx.x & 1;
    __nv_bfloat162 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float got = __shfl_xor_sync(kFullMask, odd ? v[2 * j] : v[2 * j + 1], 1);
      w[j] = odd ? __floats2bfloat162_rn(got, v[2 * j + 1]) : __floats2bfloat162_rn(v[2 * j], got);
    }
    __nv_bfloat162* p =
        static_cast<__nv_bfloat162*>(a.out) + (((int64_t)(m + odd) * a.ldo + (n & ~1)) >> 1);
    if (rows == 16 && (n | 31) < a.N) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j * a.ldo] = w[j];   // two rows further on each time
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (2 * j + odd < rows && n < a.N) p[j * a.ldo] = w[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < rows && n < a.N) lin_store(a, m + j, n, v[j]);
  }
}

// The MMAs of one k-block: four, 32 bytes (+2 in a descriptor) further along every row.
// `shift`: where the tile's rows start in their 128-row scale block, in columns of 32 rows
// (2 for the odd ones of 64-row tiles).
template <bool F8, int TN>
__device__ __forceinline__ void lin_mma(uint32_t d, uint64_t da, uint64_t db, uint64_t dsa,
                                        uint64_t dsb, uint32_t sfa, uint32_t shift, uint32_t acc,
                                        bool whole) {
  const uint32_t sfb0 = sfa + 8, sfb = sfb0 + shift;
  ptx::tc_cp_sf(sfa, dsa);
  ptx::tc_cp_sf(sfb0, dsb);
  if constexpr (F8) {
    ptx::tc_mma_f8f4(d, da, db, ptx::idesc_f8f4(TN, 0), sfa, sfb, acc);
    ptx::tc_mma_f8f4(d, da + 2, db + 2, ptx::idesc_f8f4(TN, 1), sfa, sfb, 1u);
    ptx::tc_mma_f8f4(d, da + 4, db + 4, ptx::idesc_f8f4(TN, 2), sfa, sfb, 1u);
    ptx::tc_mma_f8f4(d, da + 6, db + 6, ptx::idesc_f8f4(TN, 3), sfa, sfb, 1u);
  } else {
    const uint32_t id0 = ptx::idesc_mxf4(TN, 0), id2 = ptx::idesc_mxf4(TN, 2);
    if (whole) {   // a last k-block may be half wide
      ptx::tc_cp_sf(sfa + 4, dsa + 32);
      ptx::tc_cp_sf(sfb0 + 4, dsb + 32);
    }
    ptx::tc_mma_mxf4(d, da, db, id0, sfa, sfb, acc);
    ptx::tc_mma_mxf4(d, da + 2, db + 2, id2, sfa, sfb, 1u);
    if (whole) {
      ptx::tc_mma_mxf4(d, da + 4, db + 4, id0, sfa + 4, sfb + 4, 1u);
      ptx::tc_mma_mxf4(d, da + 6, db + 6, id2, sfa + 4, sfb + 4, 1u);
    }
  }
}

template <bool F8, int TN>
__global__ void __launch_bounds__(kLinThreads, kLinBlocksPerSM)
    linear_kernel(const __grid_constant__ CUtensorMap tmap_w,
                  const __grid_constant__ CUtensorMap tmap_x, const LinArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using SM = LinSmem<F8, TN>;
  constexpr int kSt = SM::kSt;
  constexpr int kKb = F8 ? 128 : kBK;
  LinTail* tail = reinterpret_cast<LinTail*>(smem + SM::kTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      ptx::mbar_init(&tail->full[s], 1);
      ptx::mbar_init(&tail->empty[s], 1);
    }
    ptx::mbar_init(&tail->acc_full, 1);
    ptx::mbar_init(&tail->acc_empty, 128);
    ptx::mbar_init(&tail->mma_done, 1);
    tail->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmap_w);
    ptx::prefetch_tmap(&tmap_x);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&tail->tmem_base, kLinTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;
  volatile int* abort_flag = &tail->abort;
  ptx::pdl_launch_dependents();
  const int total = a.slabs * a.tiles;   // the slabs of a row tile follow one another

  if (warp == 0) {
    // the whole warp runs the loop; one lane issues
    ptx::pdl_wait();
    const uint64_t pol_w = ptx::policy_evict_normal();
    const uint64_t pol_t = ptx::policy_evict_last();
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int g = blockIdx.x; g < total && ok; g += gridDim.x) {
      const int slab = g % a.slabs, tile = g / a.slabs;
      const uint8_t* wsf = a.w_sf + (size_t)slab * a.kc4 * kSFAtomBytes;
      const uint8_t* tsf = a.t_sf + (size_t)(tile * TN >> 7) * a.kc4 * kSFAtomBytes;
      for (int kb = 0; kb < a.num_kb; ++kb) {
        ok = __all_sync(kFullMask, ptx::mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag,
                                                  kWaitLimitNs));
        if (!ok) break;
        if (ptx::elect_one()) {
          const int atoms = min(kKb, a.K - kb * kKb) / 128;
          const size_t at = (size_t)kb * (kKb / 128) * kSFAtomBytes;
          uint64_t* bar = &tail->full[stage];
          // a widened E2M1 box (F8) counts its packed bytes only
          ptx::mbar_arrive_expect_tx(bar, (uint32_t)((F8 ? kATileBytes / 2 : kATileBytes) +
                                                     SM::kBSlot + 2 * atoms * kSFAtomBytes));
          ptx::tma_load_2d(smem + (size_t)stage * kATileBytes, &tmap_w, 0,
                           (slab * a.num_kb + kb) * kBM, bar, pol_w);
          ptx::bulk_load(smem + SM::kSFA + (size_t)stage * SM::kSF, wsf + at,
                         atoms * kSFAtomBytes, bar, pol_w);
          ptx::tma_load_2d(smem + SM::kB + (size_t)stage * SM::kBSlot, &tmap_x, kb * kBKBytes,
                           tile * TN, bar, pol_t);
          ptx::bulk_load(smem + SM::kSFB + (size_t)stage * SM::kSF, tsf + at,
                         atoms * kSFAtomBytes, bar, pol_t);
        }
        __syncwarp();
        ++issued;
        if (++stage == kSt) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&a.flags[0], kErrTimeout);
    // every copy issued here must have landed before the block exits
    const int64_t first = issued > kSt ? issued - kSt : 0;
    for (int64_t i = first; i < issued; ++i) {
      int never = 0;
      ptx::mbar_wait(&tail->full[i % kSt], (uint32_t)((i / kSt) & 1), &never, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // the whole warp runs the loop; one lane issues
    {
      const uint64_t da0 = ptx::desc_sw128(ptx::smem_addr(smem));
      const uint64_t db0 = ptx::desc_sw128(ptx::smem_addr(smem + SM::kB));
      const uint64_t dsa0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFA));
      const uint64_t dsb0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFB));
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0, sfbuf = 0;
      bool ok = !a.give_up;
      if (!ok) *abort_flag = 1;
      for (int g = blockIdx.x; g < total && ok; g += gridDim.x) {
        ok = __all_sync(kFullMask, ptx::mbar_wait(&tail->acc_empty, acc_phase ^ 1u, abort_flag,
                                                  kWaitLimitNs));
        if (!ok) break;
        ptx::tc_fence_after();
        for (int kb = 0; kb < a.num_kb; ++kb) {
          ok = __all_sync(kFullMask,
                          ptx::mbar_wait(&tail->full[stage], phase, abort_flag, kWaitLimitNs));
          if (!ok) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            lin_mma<F8, TN>(tmem_base, da0 + (uint64_t)(stage * (kATileBytes >> 4)),
                            db0 + (uint64_t)(stage * (int)(SM::kBSlot >> 4)),
                            dsa0 + (uint64_t)(stage * (int)(SM::kSF >> 4)),
                            dsb0 + (uint64_t)(stage * (int)(SM::kSF >> 4)),
                            tmem_base + (uint32_t)kLinSfCol + (sfbuf ? 16u : 0u),
                            TN == 64 ? (uint32_t)(g / a.slabs & 1) * 2u : 0u, kb ? 1u : 0u,
                            a.K - kb * kKb >= kKb);
            ptx::tc_commit(&tail->empty[stage]);
          }
          __syncwarp();
          sfbuf ^= 1u;
          if (++stage == kSt) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (ptx::elect_one()) ptx::tc_commit(&tail->acc_full);
        __syncwarp();
        acc_phase ^= 1u;
      }
      if (!ok && lane == 0) atomicOr(&a.flags[0], kErrTimeout);
      // every MMA issued here has finished before the block frees its tensor memory
      if (ptx::elect_one()) ptx::tc_commit(&tail->mma_done);
      __syncwarp();
      int never = 0;
      ptx::mbar_wait(&tail->mma_done, 0, &never, kWaitLimitNs);
    }
  } else {
    const int q = warp & 3;   // tensor-memory lane quarter of this warp
    const int row = q * 32 + lane, ep_tid = threadIdx.x - 64;
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t acc_phase = 0;
    for (int g = blockIdx.x; g < total; g += gridDim.x) {
      const int slab = g % a.slabs, tile = g / a.slabs;
      if (!ptx::mbar_wait(&tail->acc_full, acc_phase, abort_flag, kWaitLimitNs)) {
        if (ep_tid == 0) atomicOr(&a.flags[0], kErrTimeout);
        break;
      }
      acc_phase ^= 1u;
      ptx::tc_fence_after();
      const int m0 = tile * TN, cols = min(TN, a.M - m0);
      const int n = slab * 128 + row;
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        ptx::tmem_ld16(taddr + (uint32_t)c0, v);
        lin_store16(a, m0 + c0, min(16, cols - c0), n, v);
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&tail->acc_empty);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kLinTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Large products: a pair of SMs (a 2-CTA cluster) shares a tile of 256 features by up to
// ROWS (192 or 256) rows, each MMA spanning both (tcgen05 cta_group::2, M = 256): each SM
// stages its own 128-feature slab and half of the rows, so it writes and reads 60% (192)
// or half (256) of the shared-memory bytes a 128 x 128 tile takes per product.  Two
// accumulators: two of 256 rows and the scale registers are more than the 512 columns of
// tensor memory, so these share 48 columns, which the epilogue reads first.  Roles (576
// threads, one block an SM): warp 0 producer, warp 1 of the leader MMA issue, warps 2-17
// epilogue, four a lane quarter (two: 39.5 us against 34.2 at 16384 x 4096 x 512).
// MXFP4, 16384 x 4096 x 4096: 85 us behind the quantisation (6.4 PFLOP/s, 0.66 of what the MMA
// alone reaches).  No unit is saturated (8192 rows: tensor pipe 64% of the launch, L2 54%,
// DRAM 12%), and what was measured explains half of the rest: without stores 10% less, without
// loads 3 to 4%, without copies of scales about 1%, on zeros, which draw less power, 3%.
// MXFP8: 78% of the launch in the tensor pipe, and bound by power (8192 cubed 331 us, on zeros
// 253, 0.89 of what the MMA alone reaches).
constexpr int kPairEpiWarps = 16;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kPairTmemCols = 512;
constexpr uint32_t kPairSfCols = 24;                // a buffer of scale registers: 8 of the
constexpr uint32_t kPairSfCol = kPairTmemCols - 2 * kPairSfCols;   // slab's, 16 of the rows'
__host__ __device__ constexpr int lin_pair_stages(int rows) { return rows == 256 ? 6 : 7; }
// first column of the second accumulator
__host__ __device__ constexpr uint32_t lin_pair_acc(int rows) {
  return 2 * rows <= (int)kPairSfCol ? (uint32_t)rows : kPairSfCol - (uint32_t)rows;
}

struct __align__(16) LinPairTail {
  uint64_t full[7];               // leader: both CTAs' loads of a stage landed
  uint64_t empty[7];              // each CTA: the pair's MMAs are done with its stage
  uint64_t acc_full[2];           // each CTA: the accumulator is complete
  uint64_t acc_empty[2];          // leader: both CTAs' epilogue warps have read it, or what
                                  // the other accumulator shares with it
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

template <bool F8, int ROWS>
struct LinPairSmem {
  static constexpr int kSt = lin_pair_stages(ROWS);
  static constexpr size_t kSF = (size_t)(F8 ? 1 : 2) * kSFAtomBytes;   // one 128-row block
  static constexpr size_t kBSlot = (size_t)(ROWS / 2) * kBKBytes;
  static constexpr size_t kB = (size_t)kSt * kATileBytes;
  static constexpr size_t kSFA = kB + kSt * kBSlot;
  static constexpr size_t kSFB = kSFA + kSt * kSF;
  static constexpr size_t kTail = kSFB + kSt * 2 * kSF;
  static constexpr size_t kBytes = kTail + sizeof(LinPairTail) + 1024;
  static_assert(kBytes <= 227 * 1024, "one block per SM");
};

struct LinPairMaps {
  CUtensorMap w, x, wsf, tsf;
};

template <bool F8, int ROWS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinPairMaps maps, const LinArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using SM = LinPairSmem<F8, ROWS>;
  constexpr int kKb = F8 ? 128 : kBK;
  constexpr int kSt = SM::kSt;
  constexpr uint32_t kAcc2 = lin_pair_acc(ROWS);
  constexpr bool kShared = kAcc2 < ROWS;   // the accumulators share columns
  LinPairTail* tail = reinterpret_cast<LinPairTail*>(smem + SM::kTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int first = (int)blockIdx.x / 2, step = (int)gridDim.x / 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      ptx::mbar_init(&tail->full[s], 1);
      ptx::mbar_init(&tail->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&tail->acc_full[b], 1);
      ptx::mbar_init(&tail->acc_empty[b], 2 * kPairEpiWarps);
    }
    ptx::mbar_init(&tail->mma_done, 1);
    tail->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&maps.w);
    ptx::prefetch_tmap(&maps.x);
    ptx::prefetch_tmap(&maps.wsf);
    ptx::prefetch_tmap(&maps.tsf);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&tail->tmem_base, kPairTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // both CTAs' barriers exist before either signals the other's
  ptx::tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;
  volatile int* abort_flag = &tail->abort;
  ptx::pdl_launch_dependents();
  const int pairs = (a.slabs + 1) / 2, total = pairs * a.tiles;

  if (warp == 0) {
    // the whole warp runs the loop; one lane issues
    ptx::pdl_wait();
    const uint64_t pol = ptx::policy_evict_normal();
    const uint32_t full0 = ptx::mapa_shared(ptx::smem_addr(&tail->full[0]), 0);
    const uint32_t s_a = ptx::smem_addr(smem), s_b = ptx::smem_addr(smem + SM::kB);
    const uint32_t s_sfa = ptx::smem_addr(smem + SM::kSFA);
    const uint32_t s_sfb = ptx::smem_addr(smem + SM::kSFB);
    // Both CTAs' bytes of a stage, all counted on the leader's barrier (a widened E2M1
    // box counts its packed bytes only).
    constexpr uint32_t kStageBytes = 2u * (uint32_t)((F8 ? kATileBytes / 2 : kATileBytes) +
                                                     SM::kBSlot + 3 * SM::kSF);
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int g = first; g < total && ok; g += step) {
      // an odd last slab is multiplied twice, and stored once
      const int slab = min(g % pairs * 2 + (int)rank, a.slabs - 1), m0 = g / pairs * ROWS;
      int wy = slab * a.num_kb * kBM, say = slab * a.kc4 * 2, sby = 0;
      const int row = m0 + (int)rank * (ROWS / 2), blk = m0 >> 7;
      for (int kb = 0; kb < a.num_kb; ++kb) {
        ok = __all_sync(kFullMask, ptx::mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag,
                                                  kWaitLimitNs));
        if (!ok) break;
        if (ptx::elect_one()) {
          const uint32_t bar = full0 + (uint32_t)stage * 8u;
          if (rank == 0) ptx::mbar_arrive_expect_tx(&tail->full[stage], kStageBytes);
          ptx::tma_load_2d_pair(s_a + (uint32_t)stage * kATileBytes, &maps.w, 0, wy, bar, pol);
          ptx::tma_load_2d_pair(s_b + (uint32_t)(stage * SM::kBSlot), &maps.x, kb * kBKBytes, row,
                                bar, pol);
          ptx::tma_load_3d_pair(s_sfa + (uint32_t)(stage * SM::kSF), &maps.wsf, 0, say, 0, bar, pol);
          // every MMA reads all the rows' scales in both CTAs
          ptx::tma_load_3d_pair(s_sfb + (uint32_t)(stage * 2 * SM::kSF), &maps.tsf, 0, sby, blk, bar,
                                pol);
        }
        __syncwarp();
        wy += kBM;
        say += F8 ? 2 : 4;
        sby += F8 ? 2 : 4;
        ++issued;
        if (++stage == kSt) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&a.flags[0], kErrTimeout);
    // the pair's MMAs are done reading this CTA's last stages before the block leaves
    const int64_t from = issued > kSt ? issued - kSt : 0;
    for (int64_t i = from; i < issued; ++i) {
      int never = 0;
      ptx::mbar_wait(&tail->empty[i % kSt], (uint32_t)((i / kSt) & 1), &never, kWaitLimitNs);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // the whole warp runs the loop; one lane issues
      const uint64_t da0 = ptx::desc_sw128(ptx::smem_addr(smem));
      const uint64_t db0 = ptx::desc_sw128(ptx::smem_addr(smem + SM::kB));
      const uint64_t dsa0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFA));
      const uint64_t dsb0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFB));
      const uint32_t id0 = ptx::idesc_mxf4_m(2 * kBM, ROWS, 0);
      const uint32_t id2 = ptx::idesc_mxf4_m(2 * kBM, ROWS, 2);
      int stage = 0, ab = 0;
      uint32_t phase = 0, acc_phase = 0, sfbuf = 0;
      bool ok = true;
      for (int g = first; g < total && ok; g += step) {
        // tiles start at a 128-row scale block or in the middle of one
        const uint32_t shift = (uint32_t)((g / pairs * ROWS & 127) >> 5);
        // free: read by the epilogue in its last tile, or, with shared columns, what the
        // tile before has in them
        ok = __all_sync(kFullMask,
                        kShared ? ptx::mbar_wait(&tail->acc_empty[ab ^ 1],
                                                 ab ? acc_phase : acc_phase ^ 1u, abort_flag,
                                                 kWaitLimitNs)
                                : ptx::mbar_wait(&tail->acc_empty[ab], acc_phase ^ 1u, abort_flag,
                                                 kWaitLimitNs));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + (ab ? kAcc2 : 0u);
        for (int kb = 0; kb < a.num_kb; ++kb) {
          ok = __all_sync(kFullMask,
                          ptx::mbar_wait(&tail->full[stage], phase, abort_flag, kWaitLimitNs));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t da = da0 + (uint64_t)(stage * (kATileBytes >> 4));
          const uint64_t db = db0 + (uint64_t)(stage * (int)(SM::kBSlot >> 4));
          const uint64_t dsa = dsa0 + (uint64_t)(stage * (int)(SM::kSF >> 4));
          const uint64_t dsb = dsb0 + (uint64_t)(stage * (int)(2 * SM::kSF >> 4));
          const uint32_t fa = tmem_base + kPairSfCol + (sfbuf ? kPairSfCols : 0u);
          const uint32_t fb0 = fa + 8, fb = fb0 + shift;
          const uint32_t acc = kb ? 1u : 0u;
          const bool whole = a.K - kb * kKb >= kKb;   // a last k-block may be half wide
          if (ptx::elect_one()) {
            constexpr int kBlk = (int)(SM::kSF >> 4);
            ptx::tc_cp_sf_pair(fa, dsa);
            ptx::tc_cp_sf_pair(fb0, dsb);
            ptx::tc_cp_sf_pair(fb0 + 4, dsb + kBlk);
            if constexpr (F8) {
              ptx::tc_mma_f8f4_pair(d, da, db, ptx::idesc_f8f4_m(2 * kBM, ROWS, 0), fa, fb, acc);
              ptx::tc_mma_f8f4_pair(d, da + 2, db + 2, ptx::idesc_f8f4_m(2 * kBM, ROWS, 1), fa,
                                    fb, 1u);
              ptx::tc_mma_f8f4_pair(d, da + 4, db + 4, ptx::idesc_f8f4_m(2 * kBM, ROWS, 2), fa,
                                    fb, 1u);
              ptx::tc_mma_f8f4_pair(d, da + 6, db + 6, ptx::idesc_f8f4_m(2 * kBM, ROWS, 3), fa,
                                    fb, 1u);
            } else {
              if (whole) {
                ptx::tc_cp_sf_pair(fa + 4, dsa + 32);
                ptx::tc_cp_sf_pair(fb0 + 8, dsb + 32);
                ptx::tc_cp_sf_pair(fb0 + 12, dsb + kBlk + 32);
              }
              ptx::tc_mma_mxf4_pair(d, da, db, id0, fa, fb, acc);
              ptx::tc_mma_mxf4_pair(d, da + 2, db + 2, id2, fa, fb, 1u);
              if (whole) {
                ptx::tc_mma_mxf4_pair(d, da + 4, db + 4, id0, fa + 4, fb + 8, 1u);
                ptx::tc_mma_mxf4_pair(d, da + 6, db + 6, id2, fa + 4, fb + 8, 1u);
              }
            }
            ptx::tc_commit_pair_both(&tail->empty[stage]);
          }
          __syncwarp();
          sfbuf ^= 1u;
          if (++stage == kSt) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (ptx::elect_one()) ptx::tc_commit_pair_both(&tail->acc_full[ab]);
        __syncwarp();
        if (ab) acc_phase ^= 1u;
        ab ^= 1;
      }
      if (!ok && lane == 0) atomicOr(&a.flags[0], kErrTimeout);
      // every MMA issued here finishes before the pair's memory goes
      if (ptx::elect_one()) ptx::tc_commit_pair(ptx::mapa_shared(ptx::smem_addr(&tail->mma_done), 0));
      __syncwarp();
      int never = 0;
      ptx::mbar_wait(&tail->mma_done, 0, &never, kWaitLimitNs);
    }
  } else {
    constexpr int kShare = kPairEpiWarps / 4;        // warps a lane quarter
    const int q = warp & 3, hh = (warp - 2) >> 2;    // lane quarter; first chunk
    const uint32_t acc_empty_l = ptx::mapa_shared(ptx::smem_addr(&tail->acc_empty[0]), 0);
    int ab = 0;
    uint32_t acc_phase = 0;
    for (int g = first; g < total; g += step) {
      const int m0 = g / pairs * ROWS, cols = min(ROWS, a.M - m0);
      const int n0 = (g % pairs * 2 + (int)rank) * 128 + q * 32, n = n0 + lane;
      if (!ptx::mbar_wait(&tail->acc_full[ab], acc_phase, abort_flag, kWaitLimitNs)) {
        if (lane == 0) atomicOr(&a.flags[0], kErrTimeout);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (ab ? kAcc2 : 0u);
      // Two chunks of 16 rows a turn; shared columns first, and handed back once read (a
      // half's two of the three chunks at that end).
      bool held = true;
      auto hand_back = [&] {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(acc_empty_l + (uint32_t)ab * 8u);
        held = false;
      };
      if (n0 < a.N) {
        const bool down = kShared && ab == 0;
        constexpr int kTurns = (ROWS + 32 * kShare - 1) / (32 * kShare);
#pragma unroll 1
        for (int u = 0; u < kTurns; ++u) {
          const int c0 = (down ? kTurns - 1 - u : u) * 32 * kShare + hh * 16, c1 = c0 + 16 * kShare;
          if (c0 < cols) {
            uint32_t r0[16], r1[16];
            const bool two = c1 < cols;
            ptx::tmem_ld16_issue(taddr + (uint32_t)c0, r0);
            if (two) ptx::tmem_ld16_issue(taddr + (uint32_t)c1, r1);
            ptx::tmem_wait_ld(r0);
            if (two) ptx::tmem_wait_ld(r1);
            if (held && (kShared || u == kTurns - 1)) hand_back();
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r0[j]);
            lin_store16(a, m0 + c0, min(16, cols - c0), n, v);
            if (two) {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r1[j]);
              lin_store16(a, m0 + c1, min(16, cols - c1), n, v);
            }
          }
        }
      }
      if (held) hand_back();
      if (ab) acc_phase ^= 1u;
      ab ^= 1;
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  // neither CTA leaves, nor frees its tensor memory, while the pair may still use it
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, kPairTmemCols);
  }
}

// ---------------------------------------------------------------------------
// One tile a cluster; block p of the cluster's `parts` takes the k-blocks [p * num_kb /
// parts, (p + 1) * num_kb / parts).  QUANT: bf16 rows quantised by the epilogue warps into
// the stages (TN = 32).
template <bool F8, int TN, bool QUANT>
__global__ void __launch_bounds__(kLinThreads, kLinBlocksPerSM)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmap_w,
                        const __grid_constant__ CUtensorMap tmap_x, const LinArgs a, int parts) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using SM = LinSmem<F8, TN>;
  constexpr int kSt = SM::kSt;
  constexpr int kKb = F8 ? 128 : kBK;
  static_assert(!QUANT || TN == 32, "fused quantisation");
  static_assert((size_t)(TN + 4) * 128 * 4 <= SM::kSFA, "sums fit the operand stages");
  LinTail* tail = reinterpret_cast<LinTail*>(smem + SM::kTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % parts), item = (int)(blockIdx.x / parts);
  const int slab = item % a.slabs, tile = item / a.slabs;
  const int kb0 = part * a.num_kb / parts, kb1 = (part + 1) * a.num_kb / parts;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      ptx::mbar_init(&tail->full[s], QUANT ? 129 : 1);   // the producer and the quantisers
      ptx::mbar_init(&tail->empty[s], 1);
    }
    ptx::mbar_init(&tail->acc_full, 1);
    ptx::mbar_init(&tail->mma_done, 1);
    tail->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmap_w);
    if (!QUANT) ptx::prefetch_tmap(&tmap_x);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&tail->tmem_base, kLinTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;
  volatile int* abort_flag = &tail->abort;
  ptx::pdl_launch_dependents();
  const int m0 = tile * TN, cols = min(TN, a.M - m0);
  const int q = warp & 3, ep = (int)threadIdx.x - 64, row = q * 32 + lane;
  bool ok = true;
  int done = 0;   // k-blocks issued (warp 0) or quantised (warps 2-5)

  if (warp == 0) {
    // the whole warp runs the loop; one lane issues
    const uint64_t pol_w = ptx::policy_evict_normal();
    const uint64_t pol_t = ptx::policy_evict_last();
    const uint8_t* wsf = a.w_sf + (size_t)slab * a.kc4 * kSFAtomBytes;
    const uint8_t* tsf = a.t_sf + (size_t)(tile * TN >> 7) * a.kc4 * kSFAtomBytes;
    // The first stages' weights are asked into L2 while the kernel before this one ends.
    if (ptx::elect_one()) {
      const int first = min(kb1 - kb0, kSt);
      for (int j = 0; j < first; ++j)
        ptx::tma_prefetch_2d(&tmap_w, 0, (slab * a.num_kb + kb0 + j) * kBM);
      const int atom0 = kb0 * (kKb / 128);
      ptx::bulk_prefetch(wsf + (size_t)atom0 * kSFAtomBytes,
                         (uint32_t)(min(first * (kKb / 128), a.kc4 - atom0) * kSFAtomBytes));
    }
    __syncwarp();
    ptx::pdl_wait();
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++done) {
      ok = __all_sync(kFullMask, ptx::mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag,
                                                kWaitLimitNs));
      if (!ok) break;
      if (ptx::elect_one()) {
        const int atoms = min(kKb, a.K - kb * kKb) / 128;
        uint64_t* bar = &tail->full[stage];
        // a widened E2M1 box (F8) counts its packed bytes only
        ptx::mbar_arrive_expect_tx(
            bar, (uint32_t)((F8 ? kATileBytes / 2 : kATileBytes) + atoms * kSFAtomBytes +
                            (QUANT ? 0 : SM::kBSlot + atoms * kSFAtomBytes)));
        ptx::tma_load_2d(smem + (size_t)stage * kATileBytes, &tmap_w, 0,
                         (slab * a.num_kb + kb) * kBM, bar, pol_w);
        ptx::bulk_load(smem + SM::kSFA + (size_t)stage * SM::kSF,
                       wsf + (size_t)kb * (kKb / 128) * kSFAtomBytes, atoms * kSFAtomBytes, bar,
                       pol_w);
        if (!QUANT) {
          ptx::tma_load_2d(smem + SM::kB + (size_t)stage * SM::kBSlot, &tmap_x, kb * kBKBytes, m0,
                           bar, pol_t);
          ptx::bulk_load(smem + SM::kSFB + (size_t)stage * SM::kSF,
                         tsf + (size_t)kb * (kKb / 128) * kSFAtomBytes, atoms * kSFAtomBytes, bar,
                         pol_t);
        }
      }
      __syncwarp();
      if (++stage == kSt) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (lane == 0) tail->issued = done;
  } else if (warp == 1) {
    {
      const uint64_t da0 = ptx::desc_sw128(ptx::smem_addr(smem));
      const uint64_t db0 = ptx::desc_sw128(ptx::smem_addr(smem + SM::kB));
      const uint64_t dsa0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFA));
      const uint64_t dsb0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFB));
      int stage = 0;
      uint32_t phase = 0, sfbuf = 0;
      ok = !a.give_up;
      if (!ok) *abort_flag = 1;
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = __all_sync(kFullMask,
                        ptx::mbar_wait(&tail->full[stage], phase, abort_flag, kWaitLimitNs));
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          lin_mma<F8, TN>(tmem_base, da0 + (uint64_t)(stage * (kATileBytes >> 4)),
                          db0 + (uint64_t)(stage * (int)(SM::kBSlot >> 4)),
                          dsa0 + (uint64_t)(stage * (int)(SM::kSF >> 4)),
                          dsb0 + (uint64_t)(stage * (int)(SM::kSF >> 4)),
                          tmem_base + (uint32_t)kLinSfCol + (sfbuf ? 16u : 0u),
                          TN == 64 ? (uint32_t)(tile & 1) * 2u : 0u, kb != kb0 ? 1u : 0u, a.K - kb * kKb >= kKb);
          ptx::tc_commit(&tail->empty[stage]);
        }
        __syncwarp();
        sfbuf ^= 1u;
        if (++stage == kSt) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ptx::elect_one()) ptx::tc_commit(&tail->acc_full);
      __syncwarp();
    }
  } else {
    if constexpr (QUANT) {
      ptx::pdl_wait();
      constexpr int kVecs = kKb / 8;              // 8-element vectors a row and k-block
      constexpr int kMost = TN * kVecs / 128;     // of a thread
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++done) {
        uint4 w[kMost];
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          const int at = ep + i * 128, r = at / kVecs, c = kb * kVecs + at % kVecs;
          w[i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < cols && c * 8 < a.k_live)
            w[i] = *reinterpret_cast<const uint4*>(a.x + (m0 + r) * a.ldx + c * 8);
        }
        ok = __all_sync(kFullMask, ptx::mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag,
                                                  kWaitLimitNs));
        if (!ok) break;
        uint8_t* b = smem + SM::kB + (size_t)stage * SM::kBSlot;
        uint8_t* sf = smem + SM::kSFB + (size_t)stage * SM::kSF;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          if (i * 128 >= cols * kVecs) break;     // rows past the live ones hold anything
          const int at = ep + i * 128, r = at / kVecs, v = at % kVecs;
          float f[8] = {__uint_as_float(w[i].x << 16), __uint_as_float(w[i].x & 0xFFFF0000u),
                        __uint_as_float(w[i].y << 16), __uint_as_float(w[i].y & 0xFFFF0000u),
                        __uint_as_float(w[i].z << 16), __uint_as_float(w[i].z & 0xFFFF0000u),
                        __uint_as_float(w[i].w << 16), __uint_as_float(w[i].w & 0xFFFF0000u)};
          float amax = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
          amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
          const int e = F8 ? ptx::mxfp8_exponent(amax) : ptx::mx_scale_exponent(amax);
          const float m = ptx::pow2_neg(e);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= m;
          uint32_t s = (uint32_t)(e + 127) << ((v >> 2 & 3) * 8);
          s |= __shfl_xor_sync(kFullMask, s, 4);
          s |= __shfl_xor_sync(kFullMask, s, 8);
          // 128-byte swizzle: 16-byte chunk c of row r at chunk c ^ (r % 8)
          if constexpr (F8)
            *reinterpret_cast<uint2*>(b + r * 128 + (((v >> 1) ^ (r & 7)) << 4) + (v & 1) * 8) =
                ptx::e4m3x8(f);
          else
            *reinterpret_cast<uint32_t*>(b + r * 128 + (((v >> 2) ^ (r & 7)) << 4) +
                                         (v & 3) * 4) = ptx::e2m1x8(f);
          if ((v & 15) == 0)
            *reinterpret_cast<uint32_t*>(sf + (v >> 4) * kSFAtomBytes + r * 16) = s;
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&tail->full[stage]);
        if (++stage == kSt) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    ok = ptx::mbar_wait(&tail->acc_full, 0, abort_flag, kWaitLimitNs) && ok;
    ptx::tc_fence_after();
  }
  __syncwarp();
  // The accumulator is complete, so every copy has landed and every MMA has read its
  // operands: the stages are free for the other blocks' sums.  (After a timeout the sums
  // are worthless and the flag says so; all barriers are still met, and copies and MMAs in
  // flight touch this block's memory only, which it keeps until they have ended.)
  if (!ok) atomicOr(&a.flags[0], kErrTimeout);
  const int n = slab * 128 + row;
  if (parts == 1) {
    if (warp >= 2) {
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        ptx::tmem_ld16(taddr + (uint32_t)c0, v);
        lin_store16(a, m0 + c0, min(16, cols - c0), n, v);
      }
    }
  } else {
    // Block p adds the features [p * share, ...): its buffer is [part][feature][column],
    // rows padded by 16 bytes so that 16-byte accesses of consecutive features spread over
    // the banks.
    constexpr int kRow = TN + 4;
    ptx::cluster_sync();
    const int share = 128 / parts;
    float* sums = reinterpret_cast<float*>(smem);
    if (warp >= 2) {
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
      const uint32_t to = ptx::mapa_shared(
          ptx::smem_addr(sums + (part * share + row % share) * kRow), (uint32_t)(row / share));
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        ptx::tmem_ld16(taddr + (uint32_t)c0, v);
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          if (c0 + j < cols)
            ptx::st_cluster_f32x4(to + (uint32_t)(c0 + j) * 4, v[j], v[j + 1], v[j + 2], v[j + 3]);
      }
    }
    ptx::cluster_sync();
    const int quads = (cols + 3) / 4;
    for (int i = threadIdx.x; i < quads * share; i += kLinThreads) {
      const int f = i % share, c = i / share * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int p = 0; p < parts; ++p) {
        const float4 s =
            *reinterpret_cast<const float4*>(sums + (p * share + f) * kRow + c);
        v.x += s.x; v.y += s.y; v.z += s.z; v.w += s.w;
      }
      const int nn = slab * 128 + part * share + f;
      if (nn < a.N) {
        lin_store(a, m0 + c, nn, v.x);
        if (c + 1 < cols) lin_store(a, m0 + c + 1, nn, v.y);
        if (c + 2 < cols) lin_store(a, m0 + c + 2, nn, v.z);
        if (c + 3 < cols) lin_store(a, m0 + c + 3, nn, v.w);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (*abort_flag) {   // the same in every thread: all waits that set it lie before the barrier
    int never = 0;
    // A stage's phase ends with its bytes and, with QUANT, every quantiser's arrival: those
    // that gave up arrive for what was issued, at most kSt k-blocks, a stage each.
    if (QUANT && warp >= 2)
      for (int i = done; i < tail->issued; ++i) ptx::mbar_arrive(&tail->full[i % kSt]);
    if (warp == 0)
      for (int i = max(done - kSt, 0); i < done; ++i)
        ptx::mbar_wait(&tail->full[i % kSt], (uint32_t)((i / kSt) & 1), &never, kWaitLimitNs);
    if (warp == 1) {
      if (ptx::elect_one()) ptx::tc_commit(&tail->mma_done);
      __syncwarp();
      ptx::mbar_wait(&tail->mma_done, 0, &never, kWaitLimitNs);
    }
    __syncthreads();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kLinTmemCols);
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int grid, int cluster, size_t smem,
                           cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Raises a kernel's shared-memory limit on the current device, `dev`, once; a failure is tried
// again.
template <typename K>
cudaError_t allow_smem(K* kernel, size_t bytes, PerDevice<bool>& done, int dev) {
  return once_a_device(done, dev, [&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  });
}

template <bool F8, int TN, bool QUANT>
cudaError_t launch_split(const CUtensorMap& tw, const CUtensorMap& tx, const LinArgs& a, int parts,
                         int dev, cudaStream_t st) {
  constexpr size_t kBytes = LinSmem<F8, TN>::kBytes;
  static PerDevice<bool> set;
  const cudaError_t e = allow_smem(linear_split_kernel<F8, TN, QUANT>, kBytes, set, dev);
  if (e != cudaSuccess) return e;
  return launch_cluster(linear_split_kernel<F8, TN, QUANT>, a.tiles * a.slabs * parts, parts,
                        kBytes, st, tw, tx, a, parts);
}

template <bool F8, int TN>
cudaError_t launch_tile(const LinearLaunch& g, LinArgs a, cudaStream_t st) {
  constexpr size_t kBytes = LinSmem<F8, TN>::kBytes;
  CUtensorMap tw, tx = {};
  const uint64_t w_rows = (uint64_t)a.slabs * a.num_kb * kBM;
  if (w_rows > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  cudaError_t e = F8 ? make_tmap_e2m1_wide(&tw, g.w_codes, 128, w_rows)
                     : make_tmap(&tw, g.w_codes, kBKBytes, w_rows, kBM);
  if (e != cudaSuccess) return e;
  const bool quant = g.q == nullptr;
  if (!quant) {
    e = make_tmap(&tx, g.q, F8 ? (uint64_t)a.K : (uint64_t)a.K / 2, (uint64_t)a.M, TN);
    if (e != cudaSuccess) return e;
  }
  a.tiles = (a.M + TN - 1) / TN;
  const int blocks = kLinBlocksPerSM * g.num_sms;
  const int64_t items = (int64_t)a.tiles * a.slabs;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // Splitting a tile's K in two saves half its k-blocks' time and costs an exchange of
  // about 2 us; it also spreads the weights' reads over more SMs.  Measured (us, parts 1 /
  // 2 / 4 / 8): 1 x 4096 x 4096 10.4 / 7.2 / 5.6 / 5.3, 40 x 1024 x 4096 11.4 / 9.9 / 7.9 /
  // 6.5, both with 2 k-blocks left a part; 100 x 4096 x 4096 on MXFP8 pairs 15.3 / 11.9 /
  // 9.5 (8 left); but 317 x 1001 x 1056 8.3 / 9.0 / 9.5 (40 tiles, 5 k-blocks).
  int parts = 1;
  while (parts < 8 && 2 * parts <= a.num_kb) {
    const int64_t after = 2 * parts * items;
    const int kb = a.num_kb / (2 * parts);      // k-blocks left a part
    const bool pays = TN == 32                  ? after <= blocks && kb >= 2
                      : after <= 64             ? kb >= 2
                      : after <= g.num_sms      ? kb >= 5
                                                : after <= blocks && kb >= 8;
    if (!pays) break;
    parts *= 2;
  }
  if constexpr (TN == 32) {
    return quant ? launch_split<F8, TN, true>(tw, tx, a, parts, g.device, st)
                 : launch_split<F8, TN, false>(tw, tx, a, parts, g.device, st);
  } else {
    if (parts > 1) return launch_split<F8, TN, false>(tw, tx, a, parts, g.device, st);
    static PerDevice<bool> set;
    if ((e = allow_smem(linear_kernel<F8, TN>, kBytes, set, g.device)) != cudaSuccess) return e;
    const int grid = (int)(items < blocks ? items : blocks);
    return launch_pdl(linear_kernel<F8, TN>, dim3(grid), dim3(kLinThreads), kBytes, st, tw, tx,
                      a);
  }
}

template <bool F8, int ROWS>
cudaError_t launch_pair(const LinearLaunch& g, LinArgs a, cudaStream_t st) {
  constexpr size_t kBytes = LinPairSmem<F8, ROWS>::kBytes;
  LinPairMaps m;
  const uint64_t w_rows = (uint64_t)a.slabs * a.num_kb * kBM;
  if (w_rows > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  cudaError_t e = F8 ? make_tmap_e2m1_wide(&m.w, g.w_codes, 128, w_rows)
                     : make_tmap(&m.w, g.w_codes, kBKBytes, w_rows, kBM);
  const uint64_t row_blocks = (uint64_t)(a.M + 127) / 128;
  if (e != cudaSuccess ||
      (e = make_tmap(&m.x, g.q, F8 ? (uint64_t)a.K : (uint64_t)a.K / 2, (uint64_t)a.M,
                     ROWS / 2)) ||
      (e = make_tmap_scales(&m.wsf, a.w_sf, (uint64_t)a.slabs * a.kc4, 1, F8 ? 1 : 2, 1)) ||
      (e = make_tmap_scales(&m.tsf, a.t_sf, (uint64_t)a.kc4, row_blocks, F8 ? 1 : 2, 2)))
    return e;
  a.tiles = (a.M + ROWS - 1) / ROWS;
  const int64_t items = (int64_t)a.tiles * ((a.slabs + 1) / 2);
  if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // clusters that fit at once (a GPC may have an odd number of SMs)
  static PerDevice<int> fit;
  int clusters = fit.get(g.device);
  if (clusters == 0) {
    if ((e = cudaFuncSetAttribute(linear_pair_kernel<F8, ROWS>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes)) !=
        cudaSuccess)
      return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(g.num_sms);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kBytes;
    int c = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&c, linear_pair_kernel<F8, ROWS>, &cfg)) != cudaSuccess)
      return e;
    if (c < 1) return cudaErrorInvalidConfiguration;
    clusters = c < g.num_sms / 2 ? c : g.num_sms / 2;
    fit.set(g.device, clusters);
  }
  const int grid = 2 * (int)(items < clusters ? items : clusters);
  return launch_pdl(linear_pair_kernel<F8, ROWS>, dim3(grid), dim3(kPairThreads), kBytes, st, m, a);
}

int grid_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (int)(b < 1 ? 1 : b > 16384 ? 16384 : b);
}

}  // namespace

cudaError_t launch_linear_prepare(const LinearShape& s, const uint8_t* codes,
                                  const uint8_t* scales, uint8_t* prep, cudaStream_t st) {
  const int64_t code_bytes = linear_code_bytes(s);
  linear_codes_kernel<<<grid_for(code_bytes / 16), 256, 0, st>>>(
      codes, reinterpret_cast<uint4*>(prep), code_bytes / 16, s.N, s.K, linear_num_kb(s),
      s.f8 ? 64 : 128);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t words = linear_scale_bytes(s) / 4;
  linear_scales_kernel<<<grid_for(words), 256, 0, st>>>(
      scales, reinterpret_cast<uint32_t*>(prep + code_bytes), words, s.N, s.K,
      linear_padded_k(s) / 128);
  return cudaGetLastError();
}

cudaError_t launch_linear_quantize(const LinearShape& s, const void* x, int64_t ldx, int64_t rows,
                                   uint8_t* q, uint8_t* sf, cudaStream_t st) {
  const int Kp = linear_padded_k(s);
  auto* xp = static_cast<const uint16_t*>(x);
  int span_log = 4;   // columns of a block: a power of two, at least a scale word
  while (span_log < 8 && (8 << span_log) < Kp) ++span_log;
  const unsigned spans = (unsigned)((Kp / 8 + (1 << span_log) - 1) >> span_log);
  auto go = [&](auto kernel, int r) {
    const int64_t per = (int64_t)r * (kQuantThreads >> span_log);
    return launch_pdl(kernel, dim3((unsigned)((rows + per - 1) / per), spans), dim3(kQuantThreads),
                      0, st, xp, ldx, rows, s.K, Kp, q, sf, span_log);
  };
  // four rows a thread once that leaves blocks enough for every SM
  if (rows * (Kp / 8) >= (int64_t)1 << 20)
    return s.f8 ? go(linear_quantize_kernel<true, 4>, 4) : go(linear_quantize_kernel<false, 4>, 4);
  return s.f8 ? go(linear_quantize_kernel<true, 1>, 1) : go(linear_quantize_kernel<false, 1>, 1);
}

cudaError_t launch_linear(const LinearLaunch& g, cudaStream_t st) {
  const LinearShape& s = g.shape;
  LinArgs a = {};
  a.w_sf = g.w_codes + linear_code_bytes(s);
  a.t_sf = g.sf;
  a.out = g.out;
  a.ldo = g.ldo;
  a.out_f32 = g.out_f32;
  a.pairs16 = !g.out_f32 && s.N % 2 == 0 && g.ldo % 2 == 0 &&
              reinterpret_cast<uintptr_t>(g.out) % 4 == 0;
  a.x = static_cast<const uint16_t*>(g.x);
  a.ldx = g.ldx;
  a.flags = g.flags;
  a.give_up = g.give_up;
  a.M = (int)g.rows;
  a.N = s.N;
  a.K = linear_padded_k(s);
  a.k_live = s.K;
  a.slabs = (s.N + 127) / 128;
  a.num_kb = linear_num_kb(s);
  a.kc4 = a.K / 128;
  if (a.M <= 32) return s.f8 ? launch_tile<true, 32>(g, a, st) : launch_tile<false, 32>(g, a, st);
  // Tiles: 64 rows while 128-row tiles would not give every SM one, else 128, or SM pairs'
  // 256 features by 192 or 256 rows, by an estimate in cycles: rounds of tiles times
  // (k-blocks times a tile's cycles a k-block, plus a tile's fixed part), fitted to timings of
  // pairs with eight epilogue warps.  Measured with the present sixteen (us, 256 / 192 / 128 / 64
  // rows; MXFP4 from bf16 rows, then MXFP8 pairs in):
  //   1024 x 4096 x 4096   12.7 / 16.2 / 13.3 / 17.9    14.1 / 18.8 / 14.8 / 24.7
  //   1536 x 4096 x 4096   19.7 / 18.2 / 20.8 / 25.5    23.7 / 19.7 / 26.9 / 35.7
  //   4096 x 4096 x 512    12.7 / 12.8 / 14.3 / 16.9    11.8 / 11.8 / 14.4 / 19.2
  //   4096 x 4096 x 2048   23.3 / 23.8 / 27.2 / 34.7    25.8 / 25.0 / 31.0 / 45.2
  //   4096 x 4096 x 4096   36.7 / 37.6 / 42.9 / 56.4    43.5 / 42.7 / 55.3 / 79.8
  //   16384 x 4096 x 512   34.1 / 35.6 / 42.3 / 55.7    32.2 / 32.9 / 44.1 / 66.4
  //   16384 x 4096 x 4096   118 / 127 / 145 / 203        154 / 160 / 188 / 299
  //   16384 x 512 x 1024   22.9 / 24.0 / 23.3 / 23.2    14.1 / 15.1 / 16.1 / 18.6
  //   8192 x 8192 x 8192    198 / 209 / 250 / 336        321 / 321 / 378 / 562
  //   700 x 2048 x 512      7.9 / 6.5 / 5.9 / 5.1        6.3 / 4.9 / 5.4 / 4.4
  //   1300 x 2200 x 256     7.4 / 6.8 / 6.3 / 5.7        6.0 / 5.3 / 5.3 / 5.4
  // The estimate takes the fastest but at 4096 cubed (192 rows, 2% slower in MXFP4) and in small
  // products, where it takes pairs that are 1 to 1.4 us behind 64-row tiles.  Fewer than 24
  // pairs leave most of the weights' reads to too few SMs (317 x 1001 x 1056: 12.9 / 8.8).
  const bool narrow = (int64_t)((a.M + 127) / 128) * a.slabs <= g.num_sms;
  const int64_t tiles =
      (int64_t)(narrow ? (a.M + 63) / 64 : (a.M + 127) / 128) * a.slabs;
  auto rounds = [](int64_t n, int64_t at_once) { return (n + at_once - 1) / at_once; };
  const int64_t kb_tile = narrow ? (s.f8 ? 750 : 600) : (s.f8 ? 850 : 1100);
  const int64_t t_tile = rounds(tiles, 2 * g.num_sms) * (a.num_kb * kb_tile + (narrow ? 1200 : 1500));
  auto pair_tiles = [&](int rows) {
    return (int64_t)((a.M + rows - 1) / rows) * ((a.slabs + 1) / 2);
  };
  auto t_pair = [&](int rows, int64_t kb) {
    return rounds(pair_tiles(rows), g.num_sms / 2) * (a.num_kb * kb + 1500);
  };
  const int64_t t192 = t_pair(192, s.f8 ? 560 : 590), t256 = t_pair(256, s.f8 ? 745 : 762);
  if (pair_tiles(256) >= 24 && t256 < t_tile && t256 < t192)
    return s.f8 ? launch_pair<true, 256>(g, a, st) : launch_pair<false, 256>(g, a, st);
  if (pair_tiles(192) >= 24 && t192 < t_tile)
    return s.f8 ? launch_pair<true, 192>(g, a, st) : launch_pair<false, 192>(g, a, st);
  if (narrow) return s.f8 ? launch_tile<true, 64>(g, a, st) : launch_tile<false, 64>(g, a, st);
  return s.f8 ? launch_tile<true, 128>(g, a, st) : launch_tile<false, 128>(g, a, st);
}

}  // namespace mxmoe
