// Microscaled 4-bit linear product for sm_103a: out = Q(x) * W^T with MXFP4 weights.
//
//   out[m, n] = sum_k q(x)[m, k] * w[n, k]        (fp32 sums, one rounding to bf16)
//
// q(x) is MXFP4 (mxf4xmxf4) or MXFP8 (fp8xfp4), one UE8M0 scale per 32 elements of K,
// and the scales are applied by the block-scaled MMA, so nothing is dequantised.
//
// Two kernels a call: linear_quantize_kernel writes the activation codes and their
// 128x4 scale blocks, linear_kernel multiplies.  A pair that is quantised already (the
// norm's output) takes the second kernel only.
//
// linear_kernel: the weight slab (128 output features) is the MMA's M operand and up to
// TN activation rows are N, so one instruction serves one row as well as a prefill tile
// and both operands' scales are whole 128-row blocks.  Roles (192 threads, two blocks an
// SM, so that one block's epilogue overlaps the other's MMAs): warp 0 TMA producer,
// warp 1 tensor memory and MMA issue, warps 2-5 epilogue.  When there are fewer tiles
// than blocks, K is split: each part leaves its fp32 sums in the workspace and the last
// part to finish adds them in the order of the parts, so results do not depend on timing.
// Every wait is bounded (kWaitLimitNs); a timeout sets the workspace's error flag.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
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
// Activations: a thread takes 8 elements of a row, four lanes a scale, sixteen a scale
// word.  Elements past K (to the next multiple of 128) are zero.
template <bool F8>
__global__ void __launch_bounds__(kQuantThreads)
    linear_quantize_kernel(const uint16_t* __restrict__ x, int64_t ldx, int64_t rows, int K,
                           int Kp, uint8_t* __restrict__ q, uint8_t* __restrict__ sf) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();   // after the wait: see linear_kernel's weight loads
  const int vecs = Kp / 8, words = Kp / 128;
  const int64_t total = rows * vecs;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  // whole warps stay in the loop: the shuffles below need every lane
  for (int64_t i = first; i - (threadIdx.x & 31) < total; i += step) {
    const bool live = i < total;
    const int64_t row = live ? i / vecs : 0;
    const int c = live ? (int)(i - row * vecs) : 0;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (live && c * 8 < K) w = *reinterpret_cast<const uint4*>(x + row * ldx + c * 8);
    float v[8] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                  __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u),
                  __uint_as_float(w.z << 16), __uint_as_float(w.z & 0xFFFF0000u),
                  __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xFFFF0000u)};
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
    if (live) {
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
  float* partial;        // [slab * split + part][TN][128] (split > 1, one row tile)
  int32_t* counters;     // [slab], zero between calls
  int32_t* flags;
  int M, N, K;           // K padded to a multiple of 128
  int slabs, tiles, split, num_kb, kc4;
  int out_f32;
};

__host__ __device__ constexpr int lin_stages(int tn) { return tn == 128 ? 3 : tn == 64 ? 4 : 5; }

struct __align__(16) LinTail {
  uint64_t full[5];
  uint64_t empty[5];
  uint64_t acc_full, acc_empty, mma_done;
  uint32_t tmem_base;
  int abort;
  int last;
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

struct LinItem {
  int slab, tile, part, kb0, kb1;
};
__device__ __forceinline__ LinItem lin_item(const LinArgs& a, int g) {
  LinItem it;
  it.part = g % a.split;
  const int r = g / a.split;
  it.slab = r % a.slabs;
  it.tile = r / a.slabs;
  it.kb0 = (int)((int64_t)it.part * a.num_kb / a.split);
  it.kb1 = (int)((int64_t)(it.part + 1) * a.num_kb / a.split);
  return it;
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
  const int total = a.slabs * a.tiles * a.split;

  if (warp == 0) {
    if (lane == 0) {
      ptx::pdl_wait();
      const uint64_t pol_w = ptx::policy_evict_normal();
      const uint64_t pol_t = ptx::policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int g = blockIdx.x; g < total && ok; g += gridDim.x) {
        const LinItem it = lin_item(a, g);
        const uint8_t* wsf = a.w_sf + (size_t)it.slab * a.kc4 * kSFAtomBytes;
        const uint8_t* tsf = a.t_sf + (size_t)(it.tile * TN >> 7) * a.kc4 * kSFAtomBytes;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          ok = ptx::mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs);
          if (!ok) break;
          const int atoms = min(kKb, a.K - kb * kKb) / 128;
          uint64_t* bar = &tail->full[stage];
          // a widened E2M1 box (F8) counts its packed bytes only
          ptx::mbar_arrive_expect_tx(bar, (uint32_t)((F8 ? kATileBytes / 2 : kATileBytes) +
                                                     SM::kBSlot + 2 * atoms * kSFAtomBytes));
          ptx::tma_load_2d(smem + (size_t)stage * kATileBytes, &tmap_w, 0,
                           (it.slab * a.num_kb + kb) * kBM, bar, pol_w);
          ptx::bulk_load(smem + SM::kSFA + (size_t)stage * SM::kSF,
                         wsf + (size_t)kb * (kKb / 128) * kSFAtomBytes, atoms * kSFAtomBytes, bar,
                         pol_w);
          ptx::tma_load_2d(smem + SM::kB + (size_t)stage * SM::kBSlot, &tmap_x, kb * kBKBytes,
                           it.tile * TN, bar, pol_t);
          ptx::bulk_load(smem + SM::kSFB + (size_t)stage * SM::kSF,
                         tsf + (size_t)kb * (kKb / 128) * kSFAtomBytes, atoms * kSFAtomBytes, bar,
                         pol_t);
          ++issued;
          if (++stage == kSt) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) atomicOr(&a.flags[0], kErrTimeout);
      // every copy issued here must have landed before the block exits
      const int64_t first = issued > kSt ? issued - kSt : 0;
      for (int64_t i = first; i < issued; ++i) {
        int never = 0;
        ptx::mbar_wait(&tail->full[i % kSt], (uint32_t)((i / kSt) & 1), &never, kWaitLimitNs);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint64_t da0 = ptx::desc_sw128(ptx::smem_addr(smem));
      const uint64_t db0 = ptx::desc_sw128(ptx::smem_addr(smem + SM::kB));
      const uint64_t dsa0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFA));
      const uint64_t dsb0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFB));
      const uint32_t id0 = ptx::idesc_mxf4(TN, 0), id2 = ptx::idesc_mxf4(TN, 2);
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0, sfbuf = 0;
      bool ok = true;
      for (int g = blockIdx.x; g < total && ok; g += gridDim.x) {
        const LinItem it = lin_item(a, g);
        ok = ptx::mbar_wait(&tail->acc_empty, acc_phase ^ 1u, abort_flag, kWaitLimitNs);
        if (!ok) break;
        ptx::tc_fence_after();
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          ok = ptx::mbar_wait(&tail->full[stage], phase, abort_flag, kWaitLimitNs);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t sfa = tmem_base + (uint32_t)kLinSfCol + (sfbuf ? 16u : 0u);
          const uint32_t sfb = sfa + 8;
          const uint64_t dsa = dsa0 + (uint64_t)(stage * (int)(SM::kSF >> 4));
          const uint64_t dsb = dsb0 + (uint64_t)(stage * (int)(SM::kSF >> 4));
          const uint64_t da = da0 + (uint64_t)(stage * (kATileBytes >> 4));
          const uint64_t db = db0 + (uint64_t)(stage * (int)(SM::kBSlot >> 4));
          const uint32_t acc = kb != it.kb0 ? 1u : 0u;
          // four MMAs a k-block, 32 bytes (+2 in a descriptor) further along every row
          ptx::tc_cp_sf(sfa, dsa);
          ptx::tc_cp_sf(sfb, dsb);
          if constexpr (F8) {
            ptx::tc_mma_f8f4(tmem_base, da, db, ptx::idesc_f8f4(TN, 0), sfa, sfb, acc);
            ptx::tc_mma_f8f4(tmem_base, da + 2, db + 2, ptx::idesc_f8f4(TN, 1), sfa, sfb, 1u);
            ptx::tc_mma_f8f4(tmem_base, da + 4, db + 4, ptx::idesc_f8f4(TN, 2), sfa, sfb, 1u);
            ptx::tc_mma_f8f4(tmem_base, da + 6, db + 6, ptx::idesc_f8f4(TN, 3), sfa, sfb, 1u);
          } else {
            const bool whole = a.K - kb * kKb >= kKb;   // a last k-block may be half wide
            if (whole) {
              ptx::tc_cp_sf(sfa + 4, dsa + 32);
              ptx::tc_cp_sf(sfb + 4, dsb + 32);
            }
            ptx::tc_mma_mxf4(tmem_base, da, db, id0, sfa, sfb, acc);
            ptx::tc_mma_mxf4(tmem_base, da + 2, db + 2, id2, sfa, sfb, 1u);
            if (whole) {
              ptx::tc_mma_mxf4(tmem_base, da + 4, db + 4, id0, sfa + 4, sfb + 4, 1u);
              ptx::tc_mma_mxf4(tmem_base, da + 6, db + 6, id2, sfa + 4, sfb + 4, 1u);
            }
          }
          ptx::tc_commit(&tail->empty[stage]);
          sfbuf ^= 1u;
          if (++stage == kSt) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::tc_commit(&tail->acc_full);
        acc_phase ^= 1u;
      }
      if (!ok) atomicOr(&a.flags[0], kErrTimeout);
      // every MMA issued here has finished before the block frees its tensor memory
      ptx::tc_commit(&tail->mma_done);
      int never = 0;
      ptx::mbar_wait(&tail->mma_done, 0, &never, kWaitLimitNs);
    }
  } else {
    const int q = warp & 3;   // tensor-memory lane quarter of this warp
    const int row = q * 32 + lane, ep_tid = threadIdx.x - 64;
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t acc_phase = 0;
    for (int g = blockIdx.x; g < total; g += gridDim.x) {
      const LinItem it = lin_item(a, g);
      bool ok = ptx::mbar_wait(&tail->acc_full, acc_phase, abort_flag, kWaitLimitNs);
      // the warps of a split item meet at named barriers further on: all stop or none
      if (a.split > 1) ok = ptx::named_bar_and(2, 128, ok);
      if (!ok) {
        if (ep_tid == 0) atomicOr(&a.flags[0], kErrTimeout);
        break;
      }
      acc_phase ^= 1u;
      ptx::tc_fence_after();
      const int m0 = it.tile * TN, cols = min(TN, a.M - m0);
      const int n = it.slab * 128 + row;
      auto store = [&](int c, float v) {
        if (n >= a.N) return;
        const int64_t at = (int64_t)(m0 + c) * a.ldo + n;
        if (a.out_f32)
          static_cast<float*>(a.out)[at] = v;
        else
          static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16(v);
      };
      float* mine = a.partial + (size_t)(it.slab * a.split + it.part) * TN * 128 + row;
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        ptx::tmem_ld16(taddr + (uint32_t)c0, v);
        const int nc = min(16, cols - c0);
        if (a.split == 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < nc) store(c0 + j, v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < nc) mine[(c0 + j) * 128] = v[j];
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&tail->acc_empty);
      if (a.split > 1) {
        // the last part of this slab to get here adds all of them
        ptx::named_bar_sync(1, 128);
        if (ep_tid == 0) {
          __threadfence();
          tail->last = atomicAdd(&a.counters[it.slab], 1) == a.split - 1;
          if (tail->last) a.counters[it.slab] = 0;
          __threadfence();
        }
        ptx::named_bar_sync(1, 128);
        if (tail->last) {
          const float* p0 = a.partial + (size_t)it.slab * a.split * TN * 128 + row;
          for (int c = 0; c < cols; ++c) {
            float v = 0.f;
            for (int p = 0; p < a.split; ++p) v += __ldcg(p0 + ((size_t)p * TN + c) * 128);
            store(c, v);
          }
        }
        ptx::named_bar_sync(1, 128);   // tail->last is read before the next item sets it
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kLinTmemCols);
  }
}

template <bool F8, int TN>
cudaError_t launch_tile(const LinearLaunch& g, LinArgs a, cudaStream_t st) {
  constexpr size_t kBytes = LinSmem<F8, TN>::kBytes;
  static bool set = false;
  if (!set) {
    cudaError_t e = cudaFuncSetAttribute(linear_kernel<F8, TN>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes);
    if (e != cudaSuccess) return e;
    set = true;
  }
  CUtensorMap tw, tx;
  const uint64_t w_rows = (uint64_t)a.slabs * a.num_kb * kBM;
  if (w_rows > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  cudaError_t e = F8 ? make_tmap_e2m1_wide(&tw, g.w_codes, 128, w_rows)
                     : make_tmap(&tw, g.w_codes, kBKBytes, w_rows, kBM);
  if (e != cudaSuccess) return e;
  e = make_tmap(&tx, g.q, F8 ? (uint64_t)a.K : (uint64_t)a.K / 2, (uint64_t)a.M, TN);
  if (e != cudaSuccess) return e;
  a.tiles = (a.M + TN - 1) / TN;
  const int blocks = kLinBlocksPerSM * g.num_sms;
  a.split = 1;
  if (a.tiles == 1 && 2 * a.slabs <= blocks) {
    a.split = blocks / a.slabs;
    if (a.split > a.num_kb) a.split = a.num_kb;
    if (a.split * a.slabs > kLinMaxParts) a.split = kLinMaxParts / a.slabs;
    if (a.split < 1) a.split = 1;
  }
  const int64_t items = (int64_t)a.tiles * a.slabs * a.split;
  const int grid = (int)(items < blocks ? items : blocks);
  return launch_pdl(linear_kernel<F8, TN>, dim3(grid), dim3(kLinThreads), kBytes, st, tw, tx, a);
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
  const int64_t vecs = rows * (Kp / 8);
  const dim3 grid((unsigned)grid_for(vecs));
  auto* xp = static_cast<const uint16_t*>(x);
  return s.f8 ? launch_pdl(linear_quantize_kernel<true>, grid, dim3(kQuantThreads), 0, st, xp, ldx,
                           rows, s.K, Kp, q, sf)
              : launch_pdl(linear_quantize_kernel<false>, grid, dim3(kQuantThreads), 0, st, xp,
                           ldx, rows, s.K, Kp, q, sf);
}

cudaError_t launch_linear(const LinearLaunch& g, cudaStream_t st) {
  const LinearShape& s = g.shape;
  LinArgs a = {};
  a.w_sf = g.w_codes + linear_code_bytes(s);
  a.t_sf = g.sf;
  a.out = g.out;
  a.ldo = g.ldo;
  a.out_f32 = g.out_f32;
  a.partial = g.partial;
  a.counters = g.counters;
  a.flags = g.flags;
  a.M = (int)g.rows;
  a.N = s.N;
  a.K = linear_padded_k(s);
  a.slabs = (s.N + 127) / 128;
  a.num_kb = linear_num_kb(s);
  a.kc4 = a.K / 128;
  if (s.f8)
    return a.M <= 32 ? launch_tile<true, 32>(g, a, st)
           : a.M <= 64 ? launch_tile<true, 64>(g, a, st) : launch_tile<true, 128>(g, a, st);
  return a.M <= 32 ? launch_tile<false, 32>(g, a, st)
         : a.M <= 64 ? launch_tile<false, 64>(g, a, st) : launch_tile<false, 128>(g, a, st);
}

}  // namespace mxmoe
