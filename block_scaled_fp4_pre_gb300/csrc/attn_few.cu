// Attention with at most 16 query rows an item (a sequence's new tokens times the heads that
// share a kv head): decode steps and short drafts, for sm_103a.
//
//   S = scale q K^T, p = exp2(S - m), O = sum p V, l = sum p over an item's keys in one pass
//
// Bound by the cache's bytes: 16 rows use each loaded key and value 16 times, far below what
// the tensor cores take, so tiles arrive by TMA into a ring as deep as shared memory holds
// (six of 32 KiB at D = 128) and eight warps go through each tile together, 16 keys a warp,
// with mma.sync on registers: M = 16 is the rows there are, where a tcgen05 tile would carry 112
// rows of padding through tensor memory.  Each warp keeps its own running maximum, sum and
// output; they meet in shared memory at the end of an item.  The maximum is raised, and the output
// scaled, only where a logit passes it by 2^8: the sums have room for that in fp32, and so has a
// probability in bf16, whose rounding is relative.
//
// One token on 131 k keys, 32 heads of 128 on 8: 84.9 us (537 MB, 0.95 of the measured copy
// bandwidth).  48 ragged sequences of up to 6000 keys, 64 elements a head, pages of 16: 17 to 20
// us for 66 MB: an item's lookups and end are as long as three of its tiles.
//
// Work is cut as attn.cuh says; a cut item's parts are joined by the block that comes last.
#include "attn.cuh"
#include "per_device.h"
#include "tmap.cuh"

namespace mxmoe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kRows = 16;
constexpr int kWarps = 8;                       // of consumers
constexpr int kLoaders = 2;                     // warps that load keys, and values
constexpr int kThreads = 32 * (kWarps + 2 * kLoaders);
constexpr int kGroup = 8;                       // rows that the warps add up at a time

template <int D>
struct Ring {
  static constexpr int kBytes = kAttnTile * D * 2;
  static constexpr int kStages = 196608 / kBytes;   // keys and values in turn
  static_assert(kStages % 2 == 0, "keys keep to the even stages");
};

template <int D>
struct Smem {
  uint8_t ring[Ring<D>::kStages][Ring<D>::kBytes];
  float sums[kWarps][kGroup][D];
  float2 stats[kWarps][kRows];
  int64_t scan[kThreads / 32];
  uint64_t full[Ring<D>::kStages], empty[Ring<D>::kStages];
  int start_left, start_seq, start_head, start_tile;
  int issued[2][kLoaders];                      // tiles of keys, and of values, by each loader
  int abort, joins;
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What an item costs beside its tiles (its queries, its end), in tiles: positions of the line
// before its first.  us with 1, 2, 3, 4: 48 ragged sequences of 64 elements a head 19.1, 17.4,
// 17.1, 17.3; 64 sequences behind common tokens, with the prefix's part, 93.7, 86.2, 85.0, 84.6; 7
// drafts of 4 over 9 k tokens 16.4, 15.8, 15.4, 15.8.
constexpr int kItemCost = 3;

// Items of up to this many tiles are not cut: a block takes all of one whose first tile is in its
// range.  us with 0, 2, 4, 8: 112 sequences of 265 tokens 31.9, 31.9, 29.1, 29.4; 128 of 182 22.4,
// 21.5, 20.5, 20.5; one of 1000 8.0, 8.1, 8.1, 11.8.
constexpr int kShortItem = 4;

// Length on the line of a sequence's items: their tiles, one, of no keys, where the tokens see
// none from kstart on.
__device__ __forceinline__ int length_of(const AttnArgs& a, const Sequence& s) {
  if (s.taken == 0) return 0;
  return kItemCost + max(1, (s.kend - a.kstart + kAttnTile - 1) / kAttnTile);
}

// Walks the items of a block's range.
struct Walk {
  int64_t at;         // position of the current item's first tile on the line
  int left;           // positions of the range not yet given out
  int seq, head, tile;
  Sequence s;
  int tiles, first, last;   // the current item's tiles, and those of them in the range
  __device__ __forceinline__ bool next(const AttnArgs& a, bool begin) {
    for (;; begin = false) {
      if (left <= 0) return false;
      if (begin) {
        s = sequence(a, seq);
        tiles = length_of(a, s) - kItemCost;
      } else {
        at += tiles + kItemCost;
        tile = -kItemCost;
        if (++head == a.kv_heads) {
          head = 0;
          do {
            s = sequence(a, ++seq);
            tiles = length_of(a, s) - kItemCost;
          } while (tiles < 0);
        }
      }
      if (tile < 0) {                        // the positions before its first tile
        left += tile;
        if (left <= 0) return false;
        tile = 0;
      }
      first = tile;
      last = min(tiles, tile + left);
      left -= last - first;
      if (tiles > kShortItem) return true;
      last = tiles;                          // whole, the block's that its first tile is in
      if (first == 0) return true;
    }
  }
};

// Four elements of a row of an item.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs& a, const Sequence& s, int kv_head, int r,
                                          int quad, float4 acc, float sum, float top) {
  const int i = token_of(a, r), head = kv_head * a.group + r - i * a.group;
  const int64_t t = s.first + i;
  const Finish f = finish_begin<D, false>(a, kv_head, (int64_t)s.first * a.group + r, top, sum);
  finish_quad<D, false>(a, f, t, head, quad, acc);
  if (a.lse && quad == 0) a.lse[t * a.q_heads + head] = f.lse;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attention_few_kernel(const __grid_constant__ AttnArgs a,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  constexpr int STAGES = Ring<D>::kStages;
  extern __shared__ uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(
      raw + ((1024 - (ptx::smem_addr(raw) & 1023)) & 1023));
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      ptx::mbar_init(&sm.full[i], kLoaders);
      ptx::mbar_init(&sm.empty[i], kWarps);
    }
    ptx::fence_mbar_init();
    sm.abort = 0;
    ptx::prefetch_tmap(&kmap);
    ptx::prefetch_tmap(&vmap);
  }
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();

  // The block's range of the line.
  const int per = (a.batch.batch + kThreads - 1) / kThreads;
  const int b0 = min((int)threadIdx.x * per, a.batch.batch), b1 = min(b0 + per, a.batch.batch);
  int64_t mine = 0, line = 0;
  for (int b = b0; b < b1; ++b) mine += length_of(a, sequence(a, b));
  int64_t at = block_exclusive_sum(mine, sm.scan, &line) * a.kv_heads;
  line *= a.kv_heads;
  const int N = (int)min((int64_t)gridDim.x, line);
  if (line == 0 || (int)blockIdx.x >= N) return;
  const int64_t begin = range_start(line, N, blockIdx.x);
  const int64_t end = range_start(line, N, blockIdx.x + 1);
  if (begin >= at && begin < at + mine * a.kv_heads) {
    int b = b0, t = (int)mine;
    for (; per > 1; ++b) {
      t = length_of(a, sequence(a, b));
      if (begin < at + (int64_t)t * a.kv_heads) break;
      at += (int64_t)t * a.kv_heads;
    }
    sm.start_seq = b;
    sm.start_head = (int)((begin - at) / t);
    sm.start_tile = (int)((begin - at) % t) - kItemCost;
    sm.start_left = (int)(end - begin);
  }
  __syncthreads();
  Walk w;
  w.left = sm.start_left;
  w.seq = sm.start_seq;
  w.head = sm.start_head;
  w.tile = sm.start_tile;
  w.at = begin - w.tile;
  // A warp whose wait has run out, or that finds that another's has, loads, reads and releases
  // nothing more.
  volatile int* abort = &sm.abort;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(kAll, ptx::mbar_wait(bar, parity, abort, kAttnWaitNs));
  };
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&] {
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
  };

  if (warp >= kWarps) {
    // ---- loads: keys into the even stages, values into the odd ----
    const int v = (warp - kWarps) & 1, part = (warp - kWarps) >> 1;
    stage = v;
    auto advance2 = [&] {
      if ((stage += 2) >= STAGES) {
        stage -= STAGES;
        phase ^= 1;
      }
    };
    Pages pages;
    int seq = -1, issued = 0;
    for (bool first = true; ok && __any_sync(kAll, w.next(a, first)); first = false) {
      if (__any_sync(kAll, w.seq != seq)) pages.start(a, seq = w.seq);
      const int head = __shfl_sync(kAll, w.head, 0), kend = __shfl_sync(kAll, w.s.kend, 0);
      int k0 = __shfl_sync(kAll, a.kstart + w.first * kAttnTile, 0);
      const int n = __shfl_sync(kAll, w.last - w.first, 0);
      for (int i = 0; i < n && k0 < kend; ++i, k0 += kAttnTile) {
        ok = wait(&sm.empty[stage], phase ^ 1);
        if (!ok) break;
        load_tile<D, kAttnTile, kLoaders>(a, v ? &vmap : &kmap, pages, head, k0,
                                          min(kAttnTile, kend - k0), part, sm.ring[stage],
                                          &sm.full[stage]);
        advance2();
        ++issued;
      }
    }
    if (!ok && lane == 0) atomicOr(a.flags, kErrTimeout);
    // Every copy issued here must have landed before the block exits.  A stage's phase takes an
    // arrival of each loader: after a wait that ran out, the one that stopped first makes up for
    // the tiles that the other has gone on with (at most a ring's, as no stage is released
    // before all have arrived for it).
    static_assert(kLoaders == 2, "a loader and the other");
    constexpr int kMine = STAGES / 2;
    if (lane == 0) sm.issued[v][part] = issued;
    ptx::named_bar_sync(2 + v, 32 * kLoaders);
    const int other = sm.issued[v][part ^ 1], all = max(issued, other);
    if (lane == 0)
      for (int i = issued; i < other; ++i) ptx::mbar_arrive(&sm.full[2 * (i % kMine) + v]);
    int never = 0;
    for (int i = max(all - kMine, 0); i < all; ++i)
      ptx::mbar_wait(&sm.full[2 * (i % kMine) + v], (i / kMine) & 1, &never, kAttnWaitNs);
    return;
  }

  // ---- rows against tiles: 16 keys of a tile a warp ----
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = ptx::smem_addr(sm.ring);
  const int k_row = (lane >> 4) * 8 + (lane & 7), k_chunk = (lane >> 3) & 1;
  const int v_row = ((lane >> 3) & 1) * 8 + (lane & 7), v_chunk = lane >> 4;
  const uint32_t k_base = (warp * 16 + k_row) * 128, v_base = (warp * 16 + v_row) * 128;
  const int swizzle = lane & 7;
  for (bool first = true; ok && w.next(a, first); first = false) {
    const Sequence& s = w.s;
    const int rows = s.taken * a.group;
    uint32_t q[D / 16][4];
    int limit[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      const bool live = r < rows;
      const int token = token_of(a, r), head = w.head * a.group + r - token * a.group;
      const uint16_t* src = a.q + (int64_t)(s.first + token) * a.ldq + head * D + 2 * c;
      limit[i] = live ? limit_of(s, token) : 0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][i] = live ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
        q[k][i + 2] = live ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
      }
    }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][j] = 0.f;

    for (int t = w.first; t < w.last; ++t) {
      if (a.kstart + t * kAttnTile >= s.kend) continue;
      const int tok = a.kstart + t * kAttnTile + warp * 16;      // the warp's first key
      const bool some = tok < s.kend;
      float x[2][4] = {};
      ok = wait(&sm.full[stage], phase);
      if (!ok) break;
      if (some) {
        float y[2][4] = {};                            // two chains a key group
        const uint32_t base = ring + stage * Ring<D>::kBytes + k_base;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t f[4];
          const int chunk = 2 * k + k_chunk;
          ldmatrix4(base + (chunk >> 3) * (kAttnTile * 128) + (((chunk & 7) ^ swizzle) << 4), f);
          if (k & 1) {
            mma(y[0], q[k], f[0], f[1]);
            mma(y[1], q[k], f[2], f[3]);
          } else {
            mma(x[0], q[k], f[0], f[1]);
            mma(x[1], q[k], f[2], f[3]);
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[n][j] += y[n][j];
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.empty[stage]);
      advance();
      uint32_t p[4] = {};
      if (some) {
        const int key = tok + 2 * c;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[n][j] = key + n * 8 + (j & 1) < limit[j >> 1] ? x[n][j] * a.scale_log2 : -INFINITY;
        float top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
        }
        if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float up = fmaxf(m[i], top[i]);
            const float f = up == m[i] ? 1.f : exp2_approx(m[i] - up);
            m[i] = up;
            l[i] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * i] *= f;
              o[n][2 * i + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float from = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float u = exp2_approx(x[n][2 * i] - from);
            const float v = exp2_approx(x[n][2 * i + 1] - from);
            l[i] += u + v;
            p[2 * n + i] = pack_bf16(u, v);
          }
        }
      }
      ok = wait(&sm.full[stage], phase);
      if (!ok) break;
      if (some) {
        const uint32_t base = ring + stage * Ring<D>::kBytes + v_base;
        // values behind the last key may be anything: 0 times them must be 0
        uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        const bool tail = tok + 16 > s.kend;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = tok + i * 8 + 2 * c;
          keep[i] = (key < s.kend ? 0xFFFFu : 0u) | (key + 1 < s.kend ? 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t f[4];
          const int chunk = 2 * n + v_chunk;
          ldmatrix4_t(base + (chunk >> 3) * (kAttnTile * 128) + (((chunk & 7) ^ swizzle) << 4), f);
          if (tail) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] &= keep[j & 1];
          }
          mma(o[2 * n], p, f[0], f[1]);
          mma(o[2 * n + 1], p, f[2], f[3]);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.empty[stage]);
      advance();
    }

    // ---- the warps' sums to one, eight rows at a time ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      if (c == 0) sm.stats[warp][g + 8 * i] = make_float2(m[i], l[i]);
    }
    ok = ptx::named_bar_and(1, 32 * kWarps, ok);
    if (!ok) break;
    const bool whole = w.first == 0 && w.last == w.tiles;
    // parts: a block's second is one that begins an item, its first one that does not
    const int slot = 2 * blockIdx.x + (w.first == 0);
    constexpr int kQuads = D / 4;
    const int quad = threadIdx.x % kQuads, row8 = threadIdx.x / kQuads;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kGroup) {
      const int i = r0 / kGroup;
      float top = -INFINITY;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) top = fmaxf(top, sm.stats[v][r0 + g].x);
      const float f = top == -INFINITY ? 0.f : exp2_approx((i ? m[1] : m[0]) - top);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        const int pair = (n * 4 + c) ^ ((g & 3) * 4);     // spreads the rows over the banks
        *reinterpret_cast<float2*>(&sm.sums[warp][g][2 * pair]) =
            make_float2((i ? o[n][2] : o[n][0]) * f, (i ? o[n][3] : o[n][1]) * f);
      }
      ptx::named_bar_sync(1, 32 * kWarps);
      for (int rr = row8; rr < kGroup; rr += 32 * kWarps / kQuads) {
        const int r = r0 + rr;
        if (r >= rows) continue;
        float rowtop = -INFINITY, sum = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) rowtop = fmaxf(rowtop, sm.stats[v][r].x);
        const float from = rowtop == -INFINITY ? 0.f : rowtop;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          const float2 st = sm.stats[v][r];
          sum += st.y * exp2_approx(st.x - from);
          const float4 y = *reinterpret_cast<const float4*>(
              &sm.sums[v][rr][4 * (quad ^ ((rr & 3) * 2))]);
          acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
        }
        if (whole) {
          store_row<D>(a, s, w.head, r, quad, acc, sum, rowtop);
        } else {
          *reinterpret_cast<float4*>(a.parts + ((int64_t)slot * kRows + r) * D + quad * 4) = acc;
          if (quad == 0) a.part_stats[slot * kRows + r] = make_float2(rowtop, sum);
        }
      }
      ptx::named_bar_sync(1, 32 * kWarps);
    }
    if (whole) continue;

    // ---- a cut item: the block that comes last joins its parts ----
    const int from = block_of(line, N, w.at), to = block_of(line, N, w.at + w.tiles - 1);
    ptx::named_bar_sync(1, 32 * kWarps);
    if (threadIdx.x == 0) {
      const bool last = ptx::atomic_add_acq_rel(a.counters + from, 1) == to - from;
      if (last) a.counters[from] = 0;
      sm.joins = last;
    }
    ptx::named_bar_sync(1, 32 * kWarps);
    if (!sm.joins) continue;
    for (int r = row8; r < rows; r += 32 * kWarps / kQuads) {
      const Joined j = join_parts<D>(a, from, to, kRows, r, quad);
      store_row<D>(a, s, w.head, r, quad, j.acc, j.sum, j.top);
    }
  }
  if (!ok && lane == 0) atomicOr(a.flags, kErrTimeout);
}

template <int D>
cudaError_t launch(const AttnLaunch& g, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t st) {
  static PerDevice<bool> raised;
  constexpr size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(smem <= 232448, "a block's shared memory");
  const cudaError_t e = once_a_device(raised, g.device, [] {
    return cudaFuncSetAttribute(attention_few_kernel<D>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  const int blocks = g.num_sms < kAttnBlocks ? g.num_sms : kAttnBlocks;
  return launch_pdl(attention_few_kernel<D>, dim3(blocks), dim3(kThreads), smem, st, g.args, k, v);
}

}  // namespace

cudaError_t launch_attention_few(const AttnLaunch& g, const CUtensorMap& k, const CUtensorMap& v,
                                 cudaStream_t st) {
  return g.head_dim == 64 ? launch<64>(g, k, v, st) : launch<128>(g, k, v, st);
}

}  // namespace mxmoe
