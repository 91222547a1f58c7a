// The whole expert layer for a few tokens (up to kFewTokens), router included, in two
// kernels for sm_103a:
//
//   few_logits_kernel   logits = x Wr^T (fp32); x quantised
//   few_expert_kernel   top-k (ties to the lowest expert) and softmax over the chosen k;
//                       gate/up products, SwiGLU, requantisation; down products; the
//                       weighted sum over the experts; bf16
//
// The same arithmetic and rounding points as the layer kernel (gemm.cu), on the same
// prepared weights; SwiGLU too is the layer's, exp and division in the hardware's
// approximate forms (some units of fp32's last place, before 4 or 8 bits).  With few tokens an expert has one or two of them, so the time is the
// touched experts' weight bytes, and what has to be right is that every SM streams the
// same number of them without a pause:
//
// - Every token is a column of every MMA (N = 16): no bucketing, no gather; an expert's
//   columns of tokens that did not choose it are not used.  The tensor core takes the
//   same time for 16 columns as for one.
// - Every block works the routing out for itself, from the logits: some hundred loads and a
//   few warp reductions, against an elected block's ticket, its list in global memory and
//   a second read of it (5 us less at one token).
// - Work is cut into ranges of k-block tiles (one 16 KiB weight box each): whole weight
//   slabs where that spreads well, else equal ranges that start and end inside a slab (see
//   Plan).  A slab that spans ranges leaves fp32 sums of each part in the workspace, and
//   the part that finishes last adds them in the order of the ranges, so the result does
//   not depend on timing.
// - Blocks claim ranges from a counter, all of phase 0 before any of phase 1, so the wait
//   for the intermediate rows ends however many blocks are resident.  The first stages of
//   a phase 1 range hold its weights before that wait.
// - Phase 1 (down) runs slab by slab over the experts, so a block adds the experts'
//   weighted products in registers and leaves one sum per slab.  A cluster of eight blocks
//   takes a slab and adds its eight sums in shared memory (joins through global memory at
//   the end took 3 us of 29 at one token, 10 of 175 at sixteen); where there are more slabs
//   than clusters fit (H above 4480), phase 1 is cut into ranges as phase 0 is.
//
// Roles (192 threads, two blocks an SM): warp 0 claims and issues the TMA copies, warp 1
// issues the MMAs, warps 2-5 read the accumulators (four of 16 columns each in flight).
//
// Measured (4096 x 2048, 256 experts, top-6): 16 tokens 170 us, 0.94 of the measured copy
// bandwidth on the touched experts' weights; 5 tokens with MXFP8 activations 75 us, 0.76; 1
// token 22.6 us, 0.54: 9 of them stream weights, the rest is the chain logits (2.4), routing
// (1.7), first copy (2.3), SwiGLU and the step to phase 1 (2), its five tiles (2), the
// cluster's sum and the launch (3).  A small layer (12 experts of 640 x 384) takes 12.7 us,
// all of it that chain.  In NVFP4, with four stages and twice the scales, 26.6 us at 1 token
// and 170 at 16, where the same tokens take 23.1 and 162 in MXFP4 (26.1 and 177 with MXFP8
// activations).
// Every wait is bounded (kWaitLimitNs); a timeout sets the workspace's error flag.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <stddef.h>

#include <type_traits>

#include "common.cuh"
#include "per_device.h"
#include "ptx.cuh"
#include "tmap.cuh"

namespace mxmoe {
namespace {

constexpr unsigned kFullW = 0xFFFFFFFFu;
constexpr int kLogitExperts = 2;          // experts a block
constexpr int kLogitSplit = 4;            // warps that share a row of Wr
constexpr int kFewThreads = 192;
constexpr int kFewBlocksPerSM = 2;
constexpr int kFewN = kFewTokens;         // MMA columns
constexpr int kFewAccs = 4;
constexpr int kFewLeast = 5;         // least tiles of a range (a whole line where that is less)
constexpr int kFewLong = 20;         // tiles of a line from which cutting it pays (see Plan)
constexpr int kFewTmemCols = 256;
constexpr int kFewSfCol = kFewAccs * kFewN;   // two buffers of scale registers
constexpr int kFewRing = 4;
constexpr int kFewCluster = 8;
constexpr int kTailTokens = 8;   // tokens whose cluster sums fit the block's tail
constexpr int kFewMaxSlots = kFewTokens * 32;

// ws.ctrl words, cleared by the logits kernel
constexpr int kCtlClaim = 0;     // next range
constexpr int kCtlDone = 32;     // intermediate slabs written (a cache line of its own)

enum Fmt { kMx4 = 0, kMx8 = 1, kNv4 = 2 };

// ---------------------------------------------------------------------------
// Routing

__device__ __forceinline__ void bf16x8(const uint4& w, float (&v)[8]) {
  v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xFFFF0000u);
  v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  v[4] = __uint_as_float(w.z << 16); v[5] = __uint_as_float(w.z & 0xFFFF0000u);
  v[6] = __uint_as_float(w.w << 16); v[7] = __uint_as_float(w.w & 0xFFFF0000u);
}

// fp32 as an unsigned key of the same order, at least 1 (0 marks a taken value); -0 as +0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return k == 0 ? 1u : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// One token's top-k by one warp: lane j ends with the j-th expert and its weight.
// R: logits a lane holds (lane l: experts l, l + 32, ...).
template <int R>
__device__ __forceinline__ void load_keys(const float* logits, int E, int lane,
                                          uint32_t (&key)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < E ? order_key(__ldcg(logits + e)) : 0u;
  }
}
template <int R>
__device__ __forceinline__ void top_k(uint32_t (&key)[R], int k, int lane, int& id,
                                      float& weight) {
  uint32_t my_key = 0;
  id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kFullW, best);
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = R - 1; i >= 0; --i)
      if (key[i] == top) at = i * 32 + lane;
    const uint32_t win = __reduce_min_sync(kFullW, at);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i * 32 + lane == (int)win) key[i] = 0u;
    if (lane == j) {
      id = (int)win;
      my_key = top;
    }
  }
  const float top = key_value(__shfl_sync(kFullW, my_key, 0));
  float w = lane < k ? expf(key_value(my_key) - top) : 0.f;
  float sum = w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullW, sum, o);
  weight = w / sum;
}

// LIGHT: at most two tokens, in blocks small enough (64 registers, 256 threads) to sit
// beside the expert kernel's two: in a decode loop the next call's blocks then wait on the
// SMs when an expert kernel ends, instead of being launched (1 token 23.5 -> 22.6 us).
// Otherwise 512 threads, the second half of the warps for tokens 8 to 15.
template <int FMT, bool LIGHT>
__global__ void __launch_bounds__(LIGHT ? 256 : 512, LIGHT ? 4 : 1)
    few_logits_kernel(const FewArgs a) {
  constexpr int kThreads = LIGHT ? 256 : 512, kHalves = LIGHT ? 1 : 2;
  constexpr int kTok = LIGHT ? 2 : kFewTokens / 2;   // tokens a warp takes
  __shared__ float part[kThreads / 32][kTok];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.T, H = a.H, E = a.E;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (blockIdx.x == 0 && tid == 0) {   // the expert kernel's counters, for this call
    a.ctrl[kCtlClaim] = 0;
    a.ctrl[kCtlDone] = 0;
  }
  // x quantised: a thread takes 8 elements, four lanes a scale (two for NVFP4)
  {
    const int vecs = H / 8, total = T * vecs;
    for (int i = (int)(blockIdx.x * kThreads) + tid; i - lane < total;
         i += (int)gridDim.x * kThreads) {
      const bool live = i < total;
      const int t = live ? i / vecs : 0, c = live ? i - t * vecs : 0;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (live) w = *reinterpret_cast<const uint4*>(a.x + (size_t)t * H + c * 8);
      float v[8];
      bf16x8(w, v);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
      amax = fmaxf(amax, __shfl_xor_sync(kFullW, amax, 1));
      if (FMT != kNv4) amax = fmaxf(amax, __shfl_xor_sync(kFullW, amax, 2));
      uint32_t sb;
      if (FMT == kNv4) {
        sb = ptx::nvfp4_scale_byte(amax);
        const float s = ptx::ue4m3_value(sb);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = s > 0.f ? __fdiv_rn(v[j], s) : copysignf(0.f, v[j]);
      } else {
        const int e = FMT == kMx8 ? ptx::mxfp8_exponent(amax) : ptx::mx_scale_exponent(amax);
        sb = (uint32_t)(e + 127);
        const float m = ptx::pow2_neg(e);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= m;
      }
      if (live) {
        if (FMT == kMx8)
          *reinterpret_cast<uint2*>(a.xq + (size_t)t * H + c * 8) = ptx::e4m3x8(v);
        else
          *reinterpret_cast<uint32_t*>(a.xq + (size_t)t * (H / 2) + c * 4) = ptx::e2m1x8(v);
        // token t is row t of its scale blocks
        const int s = FMT == kNv4 ? c >> 1 : c >> 2;
        if ((c & (FMT == kNv4 ? 1 : 3)) == 0)
          a.xsf[((size_t)(s >> 2) << 9) + t * 16 + (s & 3)] = (uint8_t)sb;
      }
    }
  }
  if (!a.router) return;
  // Warp (g, s, p): expert g of the block, half s of the tokens, part p of the row.  Loads
  // come in batches of four 16-byte vectors of the row and of B tokens, before any
  // arithmetic.
  const int g = warp / (kLogitSplit * kHalves), half = (warp >> 2) & (kHalves - 1), p = warp & 3;
  const int e = (int)blockIdx.x * kLogitExperts + g;
  const int tok0 = half * kTok;
  float acc[kTok];
#pragma unroll
  for (int t = 0; t < kTok; ++t) acc[t] = 0.f;
  auto dots = [&](auto batch) {
    constexpr int B = decltype(batch)::value;
    const uint16_t* wr = a.router + (size_t)e * H;
    const int vecs = H / 8;
    for (int c0 = p * 32 + lane; c0 < vecs; c0 += 4 * kLogitSplit * 32) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i * kLogitSplit * 32;
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c < vecs) w[i] = *reinterpret_cast<const uint4*>(wr + c * 8);
      }
#pragma unroll
      for (int t0 = 0; t0 < kTok; t0 += B) {
        if (tok0 + t0 >= T) break;
        uint4 xv[B][4];
#pragma unroll
        for (int t = 0; t < B; ++t) {
          const int tok = min(tok0 + t0 + t, T - 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + i * kLogitSplit * 32;
            xv[t][i] = make_uint4(0u, 0u, 0u, 0u);
            if (c < vecs) xv[t][i] = *reinterpret_cast<const uint4*>(a.x + (size_t)tok * H + c * 8);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float wf[8];
          bf16x8(w[i], wf);
#pragma unroll
          for (int t = 0; t < B; ++t) {
            float v[8];
            bf16x8(xv[t][i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[t0 + t] = fmaf(wf[j], v[j], acc[t0 + t]);
          }
        }
      }
    }
  };
  if (e < E && tok0 < T) {
    dots(std::integral_constant<int, LIGHT ? 1 : 4>());
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    if (tok0 + t < T) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(kFullW, acc[t], o);
      if (lane == 0) part[warp][t] = acc[t];
    }
  }
  __syncthreads();
  if (tid < kLogitExperts * kHalves * kTok) {
    const int gg = tid / (kHalves * kTok), t = tid % (kHalves * kTok);
    const int ee = (int)blockIdx.x * kLogitExperts + gg;
    const int w0 = (gg * kHalves + t / kTok) * kLogitSplit, tt = t % kTok;
    if (t < T && ee < E)
      a.logits[(size_t)t * E + ee] =
          (part[w0][tt] + part[w0 + 1][tt]) + (part[w0 + 2][tt] + part[w0 + 3][tt]);
  }
}

// ---------------------------------------------------------------------------
// Experts

template <int FMT>
struct FewSmem {
  static constexpr int kSt = FMT == kNv4 ? 4 : 5;
  static constexpr size_t kBSlot = (size_t)kFewN * kBKBytes;
  static constexpr size_t kSF = (size_t)(FMT == kNv4 ? 4 : FMT == kMx8 ? 1 : 2) * kSFAtomBytes;
  static constexpr size_t kB = (size_t)kSt * kATileBytes;
  static constexpr size_t kSFA = kB + kSt * kBSlot;
  static constexpr size_t kSFB = kSFA + kSt * kSF;
  static constexpr size_t kTail = kSFB + kSt * kSF;
};

struct __align__(16) FewTail {
  uint64_t full[5], empty[5];
  uint64_t acc_full[kFewAccs], acc_empty[kFewAccs];
  uint64_t ring_full[kFewRing], ring_empty[kFewRing];
  uint64_t mma_done;
  int ring[kFewRing];
  uint32_t tmem_base;
  int abort;
  int last;
  int slots, weights_used;
  // One slab's SwiGLU outputs (64 features, padded rows); at the end of a clustered call the
  // cluster's sums, stored 16 bytes at a time.
  alignas(16) float h[kFewN][68];
  // Touched experts: (expert | first weight << 16, tokens as bits), and their tokens'
  // routing weights.
  int2 list[kFewMaxSlots];
  float weight[kFewMaxSlots];
};

static_assert(offsetof(FewTail, h) % 16 == 0 && FewSmem<kMx4>::kTail % 16 == 0 &&
                  FewSmem<kMx8>::kTail % 16 == 0 && FewSmem<kNv4>::kTail % 16 == 0,
              "the cluster's sums are stored 16 bytes at a time");

// Scratch of the routing, in the operand stages before any copy into them.
struct RouteScratch {
  uint32_t mask[1024];       // tokens of each expert
  int16_t slot_of[1024];
  int16_t id[kFewTokens][32];
  float w[kFewTokens][32];
};

template <int FMT>
constexpr size_t few_smem_bytes() {
  return FewSmem<FMT>::kTail + sizeof(FewTail) + 1024;
}
static_assert(2 * (few_smem_bytes<kMx4>() + 1024) <= 228 * 1024, "two blocks per SM");
static_assert(2 * (few_smem_bytes<kMx8>() + 1024) <= 228 * 1024, "two blocks per SM");
static_assert(2 * (few_smem_bytes<kNv4>() + 1024) <= 228 * 1024, "two blocks per SM");

// Tiles of a phase: `kb` of them a line (an expert's weight slab), cut into ranges.  Phase 0
// lines are slot * m0 + slab, phase 1 lines slab * slots + slot.
//
// A cut line costs a join of about 3.5 us, the time of a dozen tiles of one block.  So
// phase 0 takes whole lines where every block gets one or none, cut into `per` equal parts
// where lines are long and leave blocks idle, and where blocks take many (they claim as
// they finish, so a faster SM takes more).  In between, equal ranges that start and end
// anywhere.  1 token of the full-size layer (192 lines): 25.4 us with equal ranges, 22.6
// with whole lines; 3 tokens of 2176 x 256, MXFP8: 18.1 and 16.1.  Ranges smaller than a
// block's share measured slower: 1 token 46 us against 33, 16 tokens 213 to 225 against 205
// (before the changes since).
struct Plan {
  int n, kb, ranges, q, rem;
  int span = 0, per = 0;   // per > 0: each `span` tiles are `per` ranges
  // Equal ranges of at least kFewLeast tiles (or a line).
  __device__ __forceinline__ Plan(int tiles, int kb_line, int blocks) : n(tiles), kb(kb_line) {
    ranges = max(1, min(blocks, tiles / min(kb_line, kFewLeast)));
    q = n / ranges;
    rem = n - q * ranges;
  }
  // `spans` times `tiles` tiles of `parts` ranges each.
  __device__ __forceinline__ Plan(int spans, int tiles, int kb_line, int parts)
      : n(spans * tiles), kb(kb_line), ranges(spans * parts), q(0), rem(0), span(tiles),
        per(parts) {}
  static __device__ __forceinline__ Plan phase0(int lines, int kb_line, int blocks) {
    if (lines > blocks && lines < 4 * blocks) return Plan(lines * kb_line, kb_line, blocks);
    const int parts = lines > blocks || kb_line < kFewLong ? 1 : min(blocks / max(lines, 1), kb_line / 6);
    return Plan(lines, kb_line, kb_line, max(parts, 1));
  }
  __device__ __forceinline__ int start(int r) const {
    if (per == 1) return r * span;
    if (per) return r / per * span + r % per * span / per;
    return r * q + min(r, rem);
  }
  // the range that holds tile t
  __device__ __forceinline__ int range_of(int t) const {
    if (per == 1) return t / span;
    if (per) {
      const int s = t / span;
      return s * per + ((t - s * span + 1) * per - 1) / span;
    }
    const int big = rem * (q + 1);
    return t < big ? t / (q + 1) : rem + (t - big) / q;
  }
};

// Every block: each token's top-k (or the given ids), the list of touched experts.
// All threads; ends with a block barrier.  `scratch.mask` is zero at the start.
__device__ __forceinline__ void route(const FewArgs& a, RouteScratch& sc, FewTail* tail) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k;
  auto note = [&](int t, int id, float w) {   // lane j < k: assignment (t, j)
    if (lane < k) {
      sc.id[t][lane] = (int16_t)id;
      sc.w[t][lane] = w;
      if (id >= 0) atomicOr(&sc.mask[id], 1u << t);
      if (a.router && blockIdx.x == 0) {
        a.ids[t * k + lane] = id;
        a.weights[t * k + lane] = w;
      }
    }
  };
  if (a.router && a.T == 1 && E <= 256) {
    // One token: its j-th expert is slot j, straight from the warp that chose it (1.7 us of
    // routing against 2.4 with the steps below).
    if (warp == 0) {
      uint32_t key[8];
      int id;
      float w;
      load_keys<8>(a.logits, E, lane, key);
      top_k<8>(key, k, lane, id, w);
      if (lane < k) {
        tail->list[lane] = make_int2(id | lane << 16, 1);
        tail->weight[lane] = w;
        if (blockIdx.x == 0) {
          a.ids[lane] = id;
          a.weights[lane] = w;
        }
      }
      if (lane == 0) tail->slots = k;
    }
    ptx::fence_proxy_async_smem();   // the cleared scratch is written by TMA copies next
    __syncthreads();
    return;
  }
  constexpr int kWarps = kFewThreads / 32, kRounds = (kFewTokens + kWarps - 1) / kWarps;
  if (!a.router) {
    for (int t = warp; t < a.T; t += kWarps) {
      int id = lane < k ? a.ids[t * k + lane] : 0;
      const float w = lane < k ? a.weights[t * k + lane] : 0.f;
      if (id < 0 || id >= E) {
        if (blockIdx.x == 0) atomicOr(&a.flags[0], kErrRouting);
        id = -1;
      }
      note(t, id, w);
    }
  } else if (E <= 256) {
    uint32_t key[kRounds][8];   // every token's loads before any selection
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (warp + r * kWarps < a.T)
        load_keys<8>(a.logits + (size_t)(warp + r * kWarps) * E, E, lane, key[r]);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int t = warp + r * kWarps;
      if (t < a.T) {
        int id;
        float w;
        top_k<8>(key[r], k, lane, id, w);
        note(t, id, w);
      }
    }
  } else {
    for (int t = warp; t < a.T; t += kWarps) {
      uint32_t key[32];
      int id;
      float w;
      load_keys<32>(a.logits + (size_t)t * E, E, lane, key);
      top_k<32>(key, k, lane, id, w);
      note(t, id, w);
    }
  }
  __syncthreads();
  // Slots in the order in which the assignments first name an expert.
  const int n = a.T * k;
  if (warp == 0) {
    int at = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane, t = i / k, j = i - t * k;
      const int id = i < n ? sc.id[t][j] : -1;
      uint32_t m = 0;
      if (id >= 0) {
        m = sc.mask[id];
        if (m & ((1u << t) - 1u)) m = 0;
        if (!a.router)
          for (int o = 0; o < j; ++o)
            if (sc.id[t][o] == id) m = 0;
      }
      const uint32_t firsts = __ballot_sync(kFullW, m != 0);
      if (m) {
        const int s = at + __popc(firsts & ((1u << lane) - 1u));
        // which stretch of the weights a slot gets does not matter
        const int w0 = atomicAdd(&tail->weights_used, __popc(m));
        tail->list[s] = make_int2(id | w0 << 16, (int)m);
        sc.slot_of[id] = (int16_t)s;
      }
      at += __popc(firsts);
    }
    if (lane == 0) tail->slots = at;
  }
  __syncthreads();
  // A token that names an expert twice gets the sum of the weights, in their order.
  for (int i = threadIdx.x; i < n; i += kFewThreads) {
    const int t = i / k, j = i - t * k, id = sc.id[t][j];
    bool first = id >= 0;
    float w = sc.w[t][j];
    if (!a.router) {
      for (int o = 0; o < j; ++o) first = first && sc.id[t][o] != id;
      for (int o = j + 1; o < k; ++o)
        if (sc.id[t][o] == id) w += sc.w[t][o];
    }
    if (first) {
      const int2 l = tail->list[sc.slot_of[id]];
      tail->weight[(l.x >> 16) + __popc((uint32_t)l.y & ((1u << t) - 1u))] = w;
    }
  }
  ptx::fence_proxy_async_smem();   // the scratch is written by TMA copies next
  __syncthreads();
}

// CLUSTER: launched in clusters of kFewCluster; phase 1 slab c is cluster c's.
// 128 registers at most (the bound for two blocks of 256 threads), so that the next call's
// light logits blocks find room beside two of these.
template <int FMT, bool CLUSTER>
__global__ void __launch_bounds__(256, kFewBlocksPerSM)
    few_expert_kernel(const __grid_constant__ CUtensorMap tmap_w1,
                      const __grid_constant__ CUtensorMap tmap_x,
                      const __grid_constant__ CUtensorMap tmap_w2,
                      const __grid_constant__ CUtensorMap tmap_h, const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using SM = FewSmem<FMT>;
  constexpr int kSt = SM::kSt;
  constexpr int kKb = FMT == kMx8 ? 128 : kBK;      // elements a k-block
  constexpr int kAtomK = FMT == kNv4 ? 64 : 128;    // elements a scale block
  FewTail* tail = reinterpret_cast<FewTail*>(smem + SM::kTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = a.T;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      ptx::mbar_init(&tail->full[s], 1);
      ptx::mbar_init(&tail->empty[s], 1);
    }
    for (int s = 0; s < kFewAccs; ++s) {
      ptx::mbar_init(&tail->acc_full[s], 1);
      ptx::mbar_init(&tail->acc_empty[s], 128);
    }
    for (int s = 0; s < kFewRing; ++s) {
      ptx::mbar_init(&tail->ring_full[s], 1);
      ptx::mbar_init(&tail->ring_empty[s], 5);   // the MMA thread + 4 epilogue warps
    }
    ptx::mbar_init(&tail->mma_done, 1);
    tail->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmap_w1);
    ptx::prefetch_tmap(&tmap_x);
    ptx::prefetch_tmap(&tmap_w2);
    ptx::prefetch_tmap(&tmap_h);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&tail->tmem_base, kFewTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // Met before the cluster's sums are exchanged: every block has started by then.
  if (CLUSTER) ptx::cluster_arrive_relaxed();
  const uint32_t tmem_base = tail->tmem_base;
  volatile int* abort_flag = &tail->abort;
  RouteScratch& scratch = *reinterpret_cast<RouteScratch*>(smem);
  for (int e = threadIdx.x; e < a.E; e += kFewThreads) scratch.mask[e] = 0u;
  if (threadIdx.x == 0) tail->weights_used = 0;
  __syncthreads();
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  int claim = 0;
  if (threadIdx.x == 0) claim = atomicAdd(&a.ctrl[kCtlClaim], 1);   // answered during route()
  route(a, scratch, tail);

  const int slots = tail->slots;
  const int m0 = 2 * a.I / kBM, m1 = a.H / kBM;
  const int kb0 = (a.H + kKb - 1) / kKb, kb1 = (a.I + kKb - 1) / kKb;
  const int blocks = (int)gridDim.x;
  const Plan P0 = Plan::phase0(slots * m0, kb0, blocks);
  const Plan P1 =
      CLUSTER ? Plan(m1, slots * kb1, kb1, kFewCluster) : Plan(slots * m1 * kb1, kb1, blocks);
  const int R0 = P0.ranges, R = R0 + P1.ranges;
  float sum[kFewN];   // phase 1: weighted sums of this thread's output feature
#pragma unroll
  for (int c = 0; c < kFewN; ++c) sum[c] = 0.f;

  if (slots == 0) {
    // no valid assignment: zeros
    for (int64_t i = (int64_t)blockIdx.x * kFewThreads + threadIdx.x; i < (int64_t)T * a.H;
         i += (int64_t)gridDim.x * kFewThreads)
      a.out[i] = 0;
  } else if (warp == 0) {
    // the whole warp runs the loop; one lane issues
    {
      claim = __shfl_sync(kFullW, claim, 0);
      const uint64_t pol_w = ptx::policy_evict_first();
      const uint64_t pol_t = ptx::policy_evict_last();
      // Where a range stands: its next tile.
      struct Cursor {
        int idx, t, t1, kb, slot, slab, wslab;
        bool down;
      };
      auto weight_slab = [&](Cursor& c) {
        c.wslab = (tail->list[c.slot].x & 0xFFFF) * (c.down ? m1 : m0) + c.slab;
      };
      auto open = [&](int idx) {
        Cursor c = {};
        c.idx = idx < R ? idx : -1;
        c.down = idx >= R0;
        if (c.idx < 0) return c;
        const Plan& P = c.down ? P1 : P0;
        const int rg = c.down ? idx - R0 : idx;
        c.t = P.start(rg);
        c.t1 = P.start(rg + 1);
        const int line = c.t / P.kb, per = c.down ? slots : m0;
        c.kb = c.t - line * P.kb;
        (c.down ? c.slab : c.slot) = line / per;
        (c.down ? c.slot : c.slab) = line % per;
        weight_slab(c);
        return c;
      };
      auto step = [&](Cursor& c) {
        ++c.t;
        if (++c.kb < (c.down ? kb1 : kb0)) return;
        c.kb = 0;
        if (c.down) {
          if (++c.slot == slots) {
            c.slot = 0;
            ++c.slab;
          }
        } else if (++c.slab == m0) {
          c.slab = 0;
          ++c.slot;
        }
        if (c.t < c.t1) weight_slab(c);
      };
      int stage = 0, r = 0;
      uint32_t phase = 0, rph = 0;
      int64_t issued = 0;
      bool ok = true, waited = false, own_left = true;
      // The range of a claim; past phase 0, with clusters, the block's own, once.
      auto take_claim = [&]() {
        if (CLUSTER && claim >= R0) {
          const int own = own_left && (int)blockIdx.x < P1.ranges ? R0 + (int)blockIdx.x : R;
          own_left = false;
          return open(own);
        }
        return open(claim);
      };
      Cursor next = take_claim();
      while (true) {
        Cursor c = next;
        ok = __all_sync(kFullW, ptx::mbar_wait(&tail->ring_empty[r], rph ^ 1u, abort_flag,
                                               kWaitLimitNs));
        if (!ok) break;
        if (lane == 0) {
          tail->ring[r] = c.idx;
          ptx::mbar_arrive(&tail->ring_full[r]);
        }
        __syncwarp();
        if (++r == kFewRing) {
          r = 0;
          rph ^= 1u;
        }
        if (c.idx < 0) break;
        const bool down = c.down;
        const int kb_line = down ? kb1 : kb0;
        const CUtensorMap* tw = down ? &tmap_w2 : &tmap_w1;
        const CUtensorMap* tt = down ? &tmap_h : &tmap_x;
        const uint8_t* wsf0 = down ? a.w2_sf : a.w1_sf;
        const uint8_t* tsf0 = down ? a.hsf : a.xsf;
        const int K = down ? a.I : a.H, kc = K / kAtomK;
        // The token side of a tile, into stage s: x's rows, or the expert's rows of h.
        auto tokens = [&](int slot, int kb, int s) {
          const int atoms = min(kKb, K - kb * kKb) / kAtomK;
          ptx::tma_load_2d(smem + SM::kB + (size_t)s * SM::kBSlot, tt, kb * kBKBytes,
                           slot * kFewN, &tail->full[s], pol_t);
          ptx::bulk_load(smem + SM::kSFB + (size_t)s * SM::kSF,
                         tsf0 + ((size_t)slot * kc + (size_t)kb * (kKb / kAtomK)) * kSFAtomBytes,
                         atoms * kSFAtomBytes, &tail->full[s], pol_t);
        };
        // tiles [held, c.t) of a phase 1 range have their weights only, in stages from
        // held_stage on
        const int t0 = c.t;
        int held = t0, held_stage = stage;
        auto release = [&](int upto) {
          ok = __all_sync(kFullW, ptx::wait_counter(&a.ctrl[kCtlDone], slots * m0, abort_flag,
                                                    kWaitLimitNs));
          if (!ok) return;
          ptx::fence_proxy_async_global();
          waited = true;
          for (; held < upto; ++held) {
            const int line = held / kb_line;
            if (ptx::elect_one()) tokens(line % slots, held - line * kb_line, held_stage);
            __syncwarp();
            if (++held_stage == kSt) held_stage = 0;
          }
        };
        for (; c.t < c.t1; step(c)) {
          if (down && !waited && c.t - t0 == kSt) {
            release(c.t);   // every stage holds weights of this range
            if (!ok) break;
          }
          ok = __all_sync(kFullW, ptx::mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag,
                                                 kWaitLimitNs));
          if (!ok) break;
          if (ptx::elect_one()) {
            const int atoms = min(kKb, K - c.kb * kKb) / kAtomK;
            uint64_t* bar = &tail->full[stage];
            // a widened E2M1 box counts its packed bytes only
            ptx::mbar_arrive_expect_tx(
                bar, (uint32_t)((FMT == kMx8 ? kATileBytes / 2 : kATileBytes) +
                                a.t_rows * kBKBytes + 2 * atoms * kSFAtomBytes));
            ptx::tma_load_2d(smem + (size_t)stage * kATileBytes, tw, 0,
                             (c.wslab * kb_line + c.kb) * kBM, bar, pol_w);
            ptx::bulk_load(
                smem + SM::kSFA + (size_t)stage * SM::kSF,
                wsf0 + ((size_t)c.wslab * kc + (size_t)c.kb * (kKb / kAtomK)) * kSFAtomBytes,
                atoms * kSFAtomBytes, bar, pol_w);
            if (!down || waited) tokens(down ? c.slot : 0, c.kb, stage);
          }
          __syncwarp();
          // The next range, claimed late: a block that runs behind should not hold one.
          // (In phase 1 after the last tile, so that no block takes two ranges while it
          // waits for the intermediate rows.)
          if (!down && c.t == max(t0, c.t1 - 2) && lane == 0)
            claim = atomicAdd(&a.ctrl[kCtlClaim], 1);
          ++issued;
          if (++stage == kSt) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok && down && !waited) release(c.t1);   // a range shorter than the stages
        if (!ok) break;
        if (!CLUSTER && down && lane == 0) claim = atomicAdd(&a.ctrl[kCtlClaim], 1);
        claim = __shfl_sync(kFullW, claim, 0);
        next = take_claim();
      }
      if (!ok && lane == 0) atomicOr(&a.flags[0], kErrTimeout);
      // Every copy issued here must have landed before the block exits.  (After a timeout
      // some stages may lack their token side: their waits run out.)
      const int64_t first = issued > kSt ? issued - kSt : 0;
      for (int64_t i = first; i < issued; ++i) {
        int never = 0;
        ptx::mbar_wait(&tail->full[i % kSt], (uint32_t)((i / kSt) & 1), &never,
                       ok ? kWaitLimitNs : kWaitLimitNs / 16);
      }
    }
  } else if (warp == 1) {
    // the whole warp runs the loop; one lane issues
    {
      const uint64_t da0 = ptx::desc_sw128(ptx::smem_addr(smem));
      const uint64_t db0 = ptx::desc_sw128(ptx::smem_addr(smem + SM::kB));
      const uint64_t dsa0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFA));
      const uint64_t dsb0 = ptx::desc_sf(ptx::smem_addr(smem + SM::kSFB));
      const uint32_t id0 = ptx::idesc_mxf4(kFewN, 0), id2 = ptx::idesc_mxf4(kFewN, 2);
      const uint32_t idn = ptx::idesc_nvf4(kFewN);
      constexpr uint32_t kSfCols = FMT == kNv4 ? 16 : 8;
      int stage = 0, r = 0, acc = 0;
      uint32_t phase = 0, rph = 0, acc_phase = 0, sfbuf = 0;
      bool ok = true;
      while (ok) {
        ok = __all_sync(kFullW, ptx::mbar_wait(&tail->ring_full[r], rph, abort_flag, kWaitLimitNs));
        if (!ok) break;
        const int idx = __shfl_sync(kFullW, tail->ring[r], 0);
        if (ptx::elect_one()) ptx::mbar_arrive(&tail->ring_empty[r]);
        if (++r == kFewRing) {
          r = 0;
          rph ^= 1u;
        }
        if (idx < 0) break;
        const bool down = idx >= R0;
        const Plan& P = down ? P1 : P0;
        const int rg = down ? idx - R0 : idx;
        const int t1 = P.start(rg + 1);
        const int K = down ? a.I : a.H;
        for (int t = P.start(rg), kbs = t % P.kb; t < t1 && ok; kbs = 0) {
          const int kbe = min(P.kb, kbs + t1 - t);
          t += kbe - kbs;
          ok = __all_sync(kFullW, ptx::mbar_wait(&tail->acc_empty[acc], acc_phase ^ 1u, abort_flag,
                                                 kWaitLimitNs));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * kFewN);
          for (int kb = kbs; kb < kbe; ++kb) {
            ok = __all_sync(kFullW, ptx::mbar_wait(&tail->full[stage], phase, abort_flag,
                                                   kWaitLimitNs));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t sfa = tmem_base + (uint32_t)kFewSfCol + (sfbuf ? 2 * kSfCols : 0u);
            const uint32_t sfb = sfa + kSfCols;
            const uint64_t dsa = dsa0 + (uint64_t)(stage * (int)(SM::kSF >> 4));
            const uint64_t dsb = dsb0 + (uint64_t)(stage * (int)(SM::kSF >> 4));
            const uint64_t da = da0 + (uint64_t)(stage * (kATileBytes >> 4));
            const uint64_t db = db0 + (uint64_t)(stage * (int)(SM::kBSlot >> 4));
            const uint32_t on = kb != kbs ? 1u : 0u;
            const bool whole = K - kb * kKb >= kKb;   // a last k-block may be half wide
            if (ptx::elect_one()) {
              if constexpr (FMT == kMx8) {
                ptx::tc_cp_sf(sfa, dsa);
                ptx::tc_cp_sf(sfb, dsb);
                ptx::tc_mma_f8f4(d, da, db, ptx::idesc_f8f4(kFewN, 0), sfa, sfb, on);
                ptx::tc_mma_f8f4(d, da + 2, db + 2, ptx::idesc_f8f4(kFewN, 1), sfa, sfb, 1u);
                ptx::tc_mma_f8f4(d, da + 4, db + 4, ptx::idesc_f8f4(kFewN, 2), sfa, sfb, 1u);
                ptx::tc_mma_f8f4(d, da + 6, db + 6, ptx::idesc_f8f4(kFewN, 3), sfa, sfb, 1u);
              } else if constexpr (FMT == kNv4) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                  if (s < 2 || whole) {
                    ptx::tc_cp_sf(sfa + s * 4, dsa + 32 * s);
                    ptx::tc_cp_sf(sfb + s * 4, dsb + 32 * s);
                  }
                }
#pragma unroll
                for (int s = 0; s < 4; ++s)
                  if (s < 2 || whole)
                    ptx::tc_mma_nvf4(d, da + 2 * s, db + 2 * s, idn, sfa + s * 4, sfb + s * 4,
                                     s == 0 ? on : 1u);
              } else {
                ptx::tc_cp_sf(sfa, dsa);
                ptx::tc_cp_sf(sfb, dsb);
                if (whole) {
                  ptx::tc_cp_sf(sfa + 4, dsa + 32);
                  ptx::tc_cp_sf(sfb + 4, dsb + 32);
                }
                ptx::tc_mma_mxf4(d, da, db, id0, sfa, sfb, on);
                ptx::tc_mma_mxf4(d, da + 2, db + 2, id2, sfa, sfb, 1u);
                if (whole) {
                  ptx::tc_mma_mxf4(d, da + 4, db + 4, id0, sfa + 4, sfb + 4, 1u);
                  ptx::tc_mma_mxf4(d, da + 6, db + 6, id2, sfa + 4, sfb + 4, 1u);
                }
              }
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
          if (ptx::elect_one()) ptx::tc_commit(&tail->acc_full[acc]);
          __syncwarp();
          if (++acc == kFewAccs) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (!ok && lane == 0) atomicOr(&a.flags[0], kErrTimeout);
      // every MMA issued here has finished before the block frees its tensor memory
      if (ptx::elect_one()) ptx::tc_commit(&tail->mma_done);
      __syncwarp();
      int never = 0;
      ptx::mbar_wait(&tail->mma_done, 0, &never, kWaitLimitNs);
    }
  } else {
    const int q = warp & 3, ep = (int)threadIdx.x - 64, row = q * 32 + lane;
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    int r = 0, acc = 0;
    uint32_t rph = 0, acc_phase = 0;
    bool ok = true;
    // Waits for the next accumulator and reads it.  Should the wait run out, all four
    // warps agree on it: they meet at named barriers further on.
    auto take = [&](float (&v)[kFewN]) {
      const bool got =
          ptx::mbar_wait(&tail->acc_full[acc], acc_phase, abort_flag, kWaitLimitNs);
      if (!ptx::named_bar_and(2, 128, got)) return false;
      ptx::tc_fence_after();
      ptx::tmem_ld16(taddr + (uint32_t)(acc * kFewN), v);
      ptx::tc_fence_before();
      ptx::mbar_arrive(&tail->acc_empty[acc]);
      if (++acc == kFewAccs) {
        acc = 0;
        acc_phase ^= 1u;
      }
      return true;
    };
    // Adds the parts of tiles [lo, hi), which span ranges first..last, of which this block
    // has range rg's in v.  Returns false in every part but the last one to finish.
    auto join = [&](float (&v)[kFewN], const Plan& P, float* parts, int32_t* counter, int rg,
                    int lo, int hi) {
      const int first = P.range_of(lo), last = P.range_of(hi - 1);
      if (first == last) return true;
      // A range's first line is its piece 0, a later one (its last) piece 1; a piece is
      // [128 features][16 columns].
      auto piece = [&](int rr) {
        return reinterpret_cast<float4*>(
            parts + ((size_t)rr * 2 + (P.start(rr) >= lo ? 0 : 1)) * (kFewN * kBM) + row * kFewN);
      };
      float4* mine = piece(rg);
#pragma unroll
      for (int c = 0; c < kFewN; c += 4)
        if (c < T) __stcg(mine + c / 4, make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]));
      ptx::named_bar_sync(1, 128);
      if (ep == 0) {
        tail->last = ptx::atomic_add_acq_rel(counter, 1) == last - first;
        if (tail->last) *counter = 0;
      }
      ptx::named_bar_sync(1, 128);
      if (tail->last == 0) return false;
      // eight parts' loads in flight, added in the order of the ranges
#pragma unroll
      for (int c = 0; c < kFewN; c += 4) {
        if (c >= T) break;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r0 = first; r0 <= last; r0 += 8) {
          float4 p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r0 + i <= last) p[i] = __ldcg(piece(r0 + i) + c / 4);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s.x += p[i].x;
            s.y += p[i].y;
            s.z += p[i].z;
            s.w += p[i].w;
          }
        }
        v[c] = s.x;
        v[c + 1] = s.y;
        v[c + 2] = s.z;
        v[c + 3] = s.w;
      }
      return true;
    };
    while (ok) {
      ok = ptx::named_bar_and(
          2, 128, ptx::mbar_wait(&tail->ring_full[r], rph, abort_flag, kWaitLimitNs));
      if (!ok) break;
      const int idx = tail->ring[r];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&tail->ring_empty[r]);
      if (++r == kFewRing) {
        r = 0;
        rph ^= 1u;
      }
      if (idx < 0) break;
      float v[kFewN];
      if (idx < R0) {
        // ---- gate/up: sums, SwiGLU, requantisation
        const int rg = idx, t1 = P0.start(rg + 1);
        int line = P0.start(rg) / kb0, slot = line / m0, slab = line - slot * m0;
        for (int t = P0.start(rg); t < t1; ++line, ++slab) {
          const int lo = line * kb0, hi = lo + kb0;
          t = min(hi, t1);
          if (slab == m0) {
            slab = 0;
            ++slot;
          }
          const uint32_t chosen = (uint32_t)tail->list[slot].y;
          if (!(ok = take(v))) break;
          if (!join(v, P0, a.parts0, a.counters + line, rg, lo, hi)) continue;
          // Rows of this warp: [gate 8 | up 8 | gate 8 | up 8], so lane l and l ^ 8 hold
          // one feature's gate and up: gate lanes take the even columns, up lanes the odd.
          const bool up = (lane & 8) != 0;
          const int f = q * 16 + (FMT == kMx8 ? (lane & 7) + ((lane >> 4) << 3)
                                              : (lane & 7) * 2 + (lane >> 4));
#pragma unroll
          for (int p = 0; p < kFewN / 2; ++p) {
            if (2 * p < T) {
              const float x = __shfl_xor_sync(kFullW, up ? v[2 * p] : v[2 * p + 1], 8);
              const float g = up ? x : v[2 * p], u = up ? v[2 * p + 1] : x;
              tail->h[2 * p + (up ? 1 : 0)][f] = __fdividef(g, 1.0f + __expf(-g)) * u;
            }
          }
          ptx::named_bar_sync(1, 128);
          // 16 columns x 64 features: eight threads a column, eight features each
          const int c = ep >> 3, piece = ep & 7;
          float hv[8], amax = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            hv[j] = tail->h[c][piece * 8 + j];
            amax = fmaxf(amax, fabsf(hv[j]));
          }
          amax = fmaxf(amax, __shfl_xor_sync(kFullW, amax, 1));
          if (FMT != kNv4) amax = fmaxf(amax, __shfl_xor_sync(kFullW, amax, 2));
          uint32_t sb;
          if (FMT == kNv4) {
            sb = ptx::nvfp4_scale_byte(amax);
            const float s = ptx::ue4m3_value(sb);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              hv[j] = s > 0.f ? __fdiv_rn(hv[j], s) : copysignf(0.f, hv[j]);
          } else {
            const int e = FMT == kMx8 ? ptx::mxfp8_exponent(amax) : ptx::mx_scale_exponent(amax);
            sb = (uint32_t)(e + 127);
            const float m = ptx::pow2_neg(e);
#pragma unroll
            for (int j = 0; j < 8; ++j) hv[j] *= m;
          }
          if ((chosen >> c) & 1u) {
            const size_t hrow = (size_t)slot * kFewN + c;
            if (FMT == kMx8)
              *reinterpret_cast<uint2*>(a.hq + hrow * a.I + (size_t)slab * 64 + piece * 8) =
                  ptx::e4m3x8(hv);
            else
              *reinterpret_cast<uint32_t*>(a.hq + hrow * (a.I / 2) + (size_t)slab * 32 +
                                           piece * 4) = ptx::e2m1x8(hv);
            const int s = FMT == kNv4 ? slab * 4 + (piece >> 1) : slab * 2 + (piece >> 2);
            if ((piece & (FMT == kNv4 ? 1 : 3)) == 0)
              a.hsf[(((size_t)slot * (a.I / kAtomK) + (s >> 2)) << 9) + c * 16 + (s & 3)] =
                  (uint8_t)sb;
          }
          ptx::named_bar_sync(1, 128);   // all stored; the buffer is free again
          if (ep == 0) {
            ptx::fence_proxy_async_global();
            ptx::red_add_release(&a.ctrl[kCtlDone], 1);
          }
        }
      } else {
        // ---- down: the experts' products, weighted, summed slab by slab
        const int rg = idx - R0, t1 = P1.start(rg + 1);
        const int span = slots * kb1;   // tiles of one output slab
        int line = P1.start(rg) / kb1, slab = line / slots, slot = line - slab * slots;
        for (int t = P1.start(rg); t < t1; ++line, ++slot) {
          t = min((line + 1) * kb1, t1);
          if (slot == slots) {
            slot = 0;
            ++slab;
          }
          const int2 l = tail->list[slot];
          const uint32_t chosen = (uint32_t)l.y;
          const float* w = tail->weight + (l.x >> 16);
          if (!(ok = take(v))) break;
          // columns of other tokens hold anything, NaN too: skipped, not multiplied by 0
#pragma unroll
          for (int c = 0; c < kFewN; ++c)
            if ((chosen >> c) & 1u) sum[c] = fmaf(*w++, v[c], sum[c]);
          if (!CLUSTER && (t == t1 || t == (slab + 1) * span)) {
            if (join(sum, P1, a.parts1, a.counters1 + slab, rg, slab * span, (slab + 1) * span)) {
              const int n = slab * kBM + row;
#pragma unroll
              for (int c = 0; c < kFewN; ++c)
                if (c < T)
                  a.out[(size_t)c * a.H + n] = __bfloat16_as_ushort(__float2bfloat16(sum[c]));
            }
#pragma unroll
            for (int c = 0; c < kFewN; ++c) sum[c] = 0.f;
          }
        }
      }
    }
    if (!ok && ep == 0) atomicOr(&a.flags[0], kErrTimeout);
  }

  __syncwarp();
  if (CLUSTER) ptx::cluster_wait();
  if (CLUSTER && slots > 0 && (int)blockIdx.x < P1.ranges) {
    // The cluster's sums of its slab: block p adds features [16 p, 16 p + 16), in the order
    // of the blocks; the buffer is [part][feature][token].  Few tokens fit the room of phase
    // 0's h, which every block has left (their sums rest on all of it); more take the
    // operand stages, free once every block has read its accumulators.
    constexpr int kShare = kBM / kFewCluster;
    const int cols = T <= 4 ? 4 : T <= kTailTokens ? kTailTokens : kFewN;
    static_assert(kFewCluster * kShare * kTailTokens * 4 <= sizeof(tail->h), "room of h");
    float* const sums = T <= kTailTokens ? &tail->h[0][0] : reinterpret_cast<float*>(smem);
    const int part = (int)blockIdx.x % kFewCluster, slab = (int)blockIdx.x / kFewCluster;
    if (T > kTailTokens) ptx::cluster_sync();
    if (warp >= 2) {
      const int row = (warp & 3) * 32 + lane;
      const uint32_t to =
          ptx::mapa_shared(ptx::smem_addr(sums + (part * kShare + row % kShare) * cols),
                           (uint32_t)(row / kShare));
#pragma unroll
      for (int c = 0; c < kFewN; c += 4)
        if (c < T)
          ptx::st_cluster_f32x4(to + (uint32_t)c * 4, sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
    }
    ptx::cluster_sync();
    for (int i = threadIdx.x; i < kShare * T; i += kFewThreads) {
      const int f = i % kShare, c = i / kShare;
      float v = 0.f;
#pragma unroll
      for (int p = 0; p < kFewCluster; ++p) v += sums[(p * kShare + f) * cols + c];
      a.out[(size_t)c * a.H + slab * kBM + part * kShare + f] =
          __bfloat16_as_ushort(__float2bfloat16(v));
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kFewTmemCols);
  }
}

// Launch attributes of the expert kernel in clusters: the cluster, then programmatic
// stream serialisation.
struct ClusterConfig {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  ClusterConfig(int blocks, size_t smem, cudaStream_t st) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kFewCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

// Stands for the expert kernel's threads and shared memory when asking how many clusters fit:
// for kernels that allocate tensor memory the runtime answers as if one block filled an SM
// (15 clusters instead of 36).  Never launched.
__global__ void __launch_bounds__(kFewThreads, kFewBlocksPerSM) few_shape_kernel(int* p) {
  extern __shared__ int shape_smem[];
  if (p) *p = shape_smem[0];
}

// Blocks of the expert kernel that run at once on the current device, `dev` (found once; a
// failure is tried again), at most `most`.
template <int FMT, bool CLUSTER>
cudaError_t resident_blocks(int dev, int most, int& blocks) {
  static PerDevice<int> fit;
  constexpr size_t kBytes = few_smem_bytes<FMT>();
  blocks = fit.get(dev);
  if (blocks == 0) {
    cudaError_t e = cudaFuncSetAttribute(few_expert_kernel<FMT, CLUSTER>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes);
    if (e != cudaSuccess) return e;
    blocks = most;
    if (CLUSTER) {
      int n = 0;
      ClusterConfig c(most / kFewCluster * kFewCluster, kBytes, nullptr);
      if ((e = cudaFuncSetAttribute(few_shape_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kBytes)) != cudaSuccess ||
          (e = cudaOccupancyMaxActiveClusters(&n, few_shape_kernel, &c.cfg)) != cudaSuccess)
        return e;
      blocks = n < 1 ? -1 : n * kFewCluster;
      if (blocks > most) blocks = most / kFewCluster * kFewCluster;
    }
    fit.set(dev, blocks);
  }
  return cudaSuccess;
}

template <int FMT>
cudaError_t launch_fmt(const FewLaunch& g, cudaStream_t st) {
  FewArgs a = g.args;
  const Shape& s = g.shape;
  constexpr bool f8 = FMT == kMx8;
  const uint64_t w1_rows = (uint64_t)s.E * 2 * s.I * weight_num_kb(s, s.H);
  const uint64_t w2_rows = (uint64_t)s.E * s.H * weight_num_kb(s, s.I);
  if (w1_rows > 0x7FFFFFFFull || w2_rows > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  a.t_rows = a.T <= 8 ? 8 : kFewN;
  CUtensorMap m1, mx, m2, mh;
  cudaError_t e;
  if (f8) {
    if ((e = make_tmap_e2m1_wide(&m1, g.w1_codes, 128, w1_rows)) ||
        (e = make_tmap_e2m1_wide(&m2, g.w2_codes, 128, w2_rows)))
      return e;
  } else if ((e = make_tmap(&m1, g.w1_codes, kBKBytes, w1_rows, kBM)) ||
             (e = make_tmap(&m2, g.w2_codes, kBKBytes, w2_rows, kBM))) {
    return e;
  }
  if ((e = make_tmap(&mx, a.xq, f8 ? s.H : s.H / 2, kFewN, a.t_rows)) ||
      (e = make_tmap(&mh, a.hq, f8 ? s.I : s.I / 2, (uint64_t)g.slots_cap * kFewN, a.t_rows)))
    return e;
  const bool light = a.T <= 2;
  const int threads = light ? 256 : 512;
  // enough blocks for the experts' logits and for a vector of x a thread
  int blocks = (a.T * (s.H / 8) + threads - 1) / threads;
  if (a.router && blocks < (s.E + kLogitExperts - 1) / kLogitExperts)
    blocks = (s.E + kLogitExperts - 1) / kLogitExperts;
  e = light ? launch_pdl(few_logits_kernel<FMT, true>, dim3(blocks), dim3(threads), 0, st, a)
            : launch_pdl(few_logits_kernel<FMT, false>, dim3(blocks), dim3(threads), 0, st, a);
  if (e != cudaSuccess) return e;
  constexpr size_t kBytes = few_smem_bytes<FMT>();
  int most = kFewBlocksPerSM * g.num_sms, grid = 0;
  if (most > kFewBlocks) most = kFewBlocks;
  // A slab a cluster: as many clusters as slabs, at least 32 (phase 0 wants the blocks), and
  // fewer than fit an empty GPU, where the last one started late (1 token: 25.2 us with 32
  // clusters, 25.5 with 35, 27.8 with all 36).
  if ((e = resident_blocks<FMT, true>(g.device, most, grid)) != cudaSuccess) return e;
  // Small layers launch no more than phase 0 has ranges for.
  const int slabs = s.H / kBM, fit = grid / kFewCluster - 1;
  if (slabs <= fit) {
    const int64_t touched = (int64_t)a.T * s.k < s.E ? (int64_t)a.T * s.k : s.E;
    const int64_t kb0 = weight_num_kb(s, s.H);
    const int64_t ranges0 = touched * (2 * s.I / kBM) * (kb0 < kFewLong ? 1 : kb0 / 6);
    const int64_t want = (ranges0 + kFewCluster - 1) / kFewCluster;
    int clusters = want < 32 ? (int)want : 32;
    if (clusters > fit) clusters = fit;
    if (clusters < slabs) clusters = slabs;
    ClusterConfig c(clusters * kFewCluster, kBytes, st);
    c.cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&c.cfg, few_expert_kernel<FMT, true>, m1, mx, m2, mh, a);
  }
  if ((e = resident_blocks<FMT, false>(g.device, most, grid)) != cudaSuccess) return e;
  return launch_pdl(few_expert_kernel<FMT, false>, dim3(grid), dim3(kFewThreads), kBytes, st, m1,
                    mx, m2, mh, a);
}

}  // namespace

cudaError_t launch_few(const FewLaunch& g, cudaStream_t st) {
  if (g.shape.f8) return launch_fmt<kMx8>(g, st);
  if (g.shape.nv) return launch_fmt<kNv4>(g, st);
  return launch_fmt<kMx4>(g, st);
}

}  // namespace mxmoe
