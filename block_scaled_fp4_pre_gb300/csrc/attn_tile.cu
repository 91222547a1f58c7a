// Attention with many query rows an item, on tensor memory, for sm_103a: prompts, drafts, and
// the prefix that a batch shares.
//
// A row is a new token and one of the heads that share a kv head; an item is up to 256 rows of
// one kv head, in two tiles of 128, against the keys that the last of them sees:
//   main     rows of one sequence, keys from `kstart` on
//   SHARED   rows of all sequences, the common prefix's keys [0, kstart): one pass over the
//            prefix serves the whole batch; its unfinished sums go to the workspace, where
//            the main part's rows pick them up
// A tile of keys (128) goes through S = Q K^T (both operands in shared memory, 128 x 128 fp32 in
// tensor memory), a thread a row for the softmax, and O += P V with P as bf16 in tensor memory,
// in the columns of S that it came from, and V as the transposed operand.
//
// The tensor cores alternate between the two row tiles: while one tile's scores are in the hands
// of its warpgroup, the other's products run.  The loader keeps a ring of key and value tiles
// full.  The running maximum is raised only where a logit passes it by 2^8 (the sums and the
// rounding of P allow it), so the output in tensor memory is rarely scaled; its warpgroup does that
// before it hands over the next P, when no product on it is in flight.
//
// Bound by the tensor cores: 4 x 128 x 128 x D operations a tile pair at the dense bf16 rate.
#include "attn.cuh"
#include "per_device.h"
#include "tmap.cuh"

namespace mxmoe {
namespace {

constexpr int kTileRows = 128;
constexpr int kLoader = 8, kIssuer = 9;         // warps; eight before them hold a row a thread
constexpr int kThreads = 384;                   // whole warpgroups, as register shares go by
// 384 threads start with 168 registers: the softmax's two warpgroups take 208, the third 88
// (2 x 208 + 88 = 3 x 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "the launch's registers");

template <int D>
struct Sizes {
  static constexpr int kTileBytes = kTileRows * D * 2;      // of queries, keys or values
  static constexpr int kStages = (229376 - 2 * kTileBytes) / kTileBytes;
  static constexpr int kHalf = kTileRows * 128;             // 64 columns of a tile
};

template <int D>
struct Smem {
  uint8_t q[2][Sizes<D>::kTileBytes];
  uint8_t ring[Sizes<D>::kStages][Sizes<D>::kTileBytes];
  int64_t scan[kThreads / 32];
  uint64_t full[Sizes<D>::kStages], empty[Sizes<D>::kStages];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], done;
  int64_t start_left, start_at;
  int start_seq, start_head, start_rt, start_tile;
  int kend;                                     // SHARED: keys that some row sees
  uint32_t tmem;
  int abort;
};

// tensor memory: scores (and P) of both tiles, then the outputs
constexpr uint32_t kColS = 0, kColO = 256;

// D[tmem] (+)= A[smem] B[smem]^T and A[tmem] B[smem], bf16.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor: fp32 sums of bf16 products, M = 128; bit 16: B with N contiguous.
__device__ __forceinline__ uint32_t idesc_bf16(int N, bool b_transposed) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_transposed ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTileRows >> 4) << 24);
}
// Operand with N contiguous, 128-byte swizzle: atoms of 64 columns x 8 rows of K, 1024 bytes
// from 8 rows to the next, `atom` bytes from 64 columns to the next.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t atom) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(atom >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for this thread's loads; r is tied to the wait so that no use of it moves above.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// ---- the line ----

// Row tiles (of 256 rows) of a sequence, and the keys that row tile rt's last row sees.
__device__ __forceinline__ int row_tiles(const AttnArgs& a, const Sequence& s) {
  return (int)(((int64_t)s.t.taken * a.group + kAttnRows - 1) / kAttnRows);
}
__device__ __forceinline__ int kend_of(const AttnArgs& a, const Sequence& s, int rt) {
  const int64_t rows = min((int64_t)(rt + 1) * kAttnRows, (int64_t)s.t.taken * a.group);
  return limit_of(s, (int)((rows - 1) / a.group));
}
__device__ __forceinline__ int key_tiles(int kstart, int kend) {
  return max(1, (kend - kstart + kAttnTile - 1) / kAttnTile);
}
// Tiles of a sequence's items of one head.
__device__ __forceinline__ int64_t tiles_of(const AttnArgs& a, const Sequence& s) {
  int64_t n = 0;
  const int rts = row_tiles(a, s);
  for (int rt = 0; rt < rts; ++rt) n += key_tiles(a.kstart, kend_of(a, s, rt));
  return n;
}

// An item: rows [row0, row0 + rows) of a kv head, counted from token `token0`'s first, and the
// keys [k0, kend) of tiles [first, last) out of `tiles`, at position `at` of the line.
template <bool SHARED>
struct Walk {
  int64_t left, at;
  int seq, head, rt, tile;
  Sequence s;
  int rts, kend, tiles, first, last, rows;
  __device__ __forceinline__ void measure(const AttnArgs& a) {
    const int64_t all = SHARED ? (int64_t)a.batch.tokens * a.group : (int64_t)s.t.taken * a.group;
    rows = (int)min((int64_t)kAttnRows, all - (int64_t)rt * kAttnRows);
    if (!SHARED) {
      kend = kend_of(a, s, rt);
      tiles = key_tiles(a.kstart, kend);
    }
  }
  __device__ __forceinline__ bool next(const AttnArgs& a, bool begin) {
    if (left <= 0) return false;
    if (begin) {
      if (!SHARED) {
        s = sequence(a, seq);
        rts = row_tiles(a, s);
      }
    } else {
      at += tiles;
      tile = 0;
      if (++rt == rts) {
        rt = 0;
        if (++head == a.kv_heads && !SHARED) {
          head = 0;
          do {
            s = sequence(a, ++seq);
            rts = row_tiles(a, s);
          } while (rts == 0);
        }
      }
    }
    measure(a);
    first = tile;
    last = (int)min((int64_t)tiles, tile + left);
    left -= last - first;
    return true;
  }
  // Tiles of [first, last) that hold a key; the others are behind the last one.
  __device__ __forceinline__ int busy(int kstart) const {
    const int from = SHARED ? 0 : kstart;
    const int n = kend > from ? (kend - from + kAttnTile - 1) / kAttnTile : 0;
    return max(0, min(last, n) - first);
  }
};

// Where the row r of an item lies: its token (-1: none) and head, and the keys it sees.
struct Row {
  int token, head, limit;
  int64_t index;      // among the kv head's rows of all tokens
};
template <bool SHARED>
__device__ __forceinline__ Row row_of(const AttnArgs& a, const Walk<SHARED>& w, int r) {
  Row x = {-1, 0, w.kend, 0};
  if (r >= w.rows) return x;
  const int R = w.rt * kAttnRows + r;                 // (tokens * heads: below 2^30)
  const int i = R / a.group;
  x.head = w.head * a.group + R % a.group;
  if (SHARED) {
    const int b = sequence_of(a.batch, i);
    if (b < 0) return x;
    const Sequence s = sequence(a, b);
    const int at = i - s.t.first;
    if (at < 0 || at >= s.t.taken) return x;
    x.token = i;
    x.limit = min(limit_of(s, at), w.kend);
    x.index = R;
  } else {
    x.token = w.s.t.first + i;
    x.limit = limit_of(w.s, i);
    x.index = (int64_t)w.s.t.first * a.group + R;
  }
  return x;
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tile_kernel(const __grid_constant__ AttnArgs a,
                          const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap) {
  constexpr int STAGES = Sizes<D>::kStages;
  extern __shared__ uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(
      raw + ((1024 - (ptx::smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      ptx::mbar_init(&sm.full[i], 1);
      ptx::mbar_init(&sm.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&sm.q_full[t], 4);
      ptx::mbar_init(&sm.s_full[t], 1);
      ptx::mbar_init(&sm.p_full[t], 4);
      ptx::mbar_init(&sm.o_full[t], 1);
    }
    ptx::mbar_init(&sm.done, 1);
    ptx::fence_mbar_init();
    sm.abort = 0;
    sm.kend = 0;
    ptx::prefetch_tmap(&kmap);
    ptx::prefetch_tmap(&vmap);
  }
  // Tensor memory after the wait and before the next kernel may start: no block holds all of
  // it while one that it waits for has yet to ask.
  ptx::pdl_wait();
  if (warp == kIssuer) {
    ptx::tmem_alloc(&sm.tmem, 512);
    ptx::tmem_relinquish();
  }
  __syncthreads();
  ptx::pdl_launch_dependents();

  // The block's range of the line.
  int64_t line = 0;
  int N;
  if (SHARED) {
    const int rts = (int)(((int64_t)a.batch.tokens * a.group + kAttnRows - 1) / kAttnRows);
    const int tiles = (a.kstart + kAttnTile - 1) / kAttnTile;
    line = (int64_t)a.kv_heads * rts * tiles;
    N = (int)min((int64_t)gridDim.x, line);
    int most = 0;
    for (int b = threadIdx.x; b < a.batch.batch; b += kThreads)
      most = max(most, sequence(a, b).kend);
    atomicMax(&sm.kend, min(most, a.kstart));
    if (threadIdx.x == 0 && (int)blockIdx.x < N) {
      const int64_t begin = range_start(line, N, blockIdx.x);
      const int64_t item = begin / tiles;
      sm.start_tile = (int)(begin % tiles);
      sm.start_rt = (int)(item % rts);
      sm.start_head = (int)(item / rts);
      sm.start_at = item * tiles;
      sm.start_seq = 0;
      sm.start_left = range_start(line, N, blockIdx.x + 1) - begin;
    }
  } else {
    const int per = (a.batch.batch + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.batch.batch), b1 = min(b0 + per, a.batch.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += tiles_of(a, sequence(a, b));
    int64_t at = block_exclusive_sum(mine, sm.scan, &line) * a.kv_heads;
    line *= a.kv_heads;
    N = (int)min((int64_t)gridDim.x, line);
    if ((int)blockIdx.x < N) {
      const int64_t begin = range_start(line, N, blockIdx.x);
      if (begin >= at && begin < at + mine * a.kv_heads) {
        int b = b0;
        int64_t n;
        for (;; ++b) {
          n = tiles_of(a, sequence(a, b));
          if (begin < at + n * a.kv_heads) break;
          at += n * a.kv_heads;
        }
        const Sequence s = sequence(a, b);
        int head = (int)((begin - at) / n), rt = 0;
        at += head * n;
        for (;; ++rt) {
          const int t = key_tiles(a.kstart, kend_of(a, s, rt));
          if (begin < at + t) break;
          at += t;
        }
        sm.start_seq = b;
        sm.start_head = head;
        sm.start_rt = rt;
        sm.start_tile = (int)(begin - at);
        sm.start_at = at;
        sm.start_left = range_start(line, N, blockIdx.x + 1) - begin;
      }
    }
  }
  if (threadIdx.x == 0) a.cuts[blockIdx.x].to = -1;      // no item begins here and goes on
  __syncthreads();
  const bool working = (int)blockIdx.x < N;
  Walk<SHARED> w = {};
  w.left = working ? sm.start_left : 0;
  w.at = sm.start_at;
  w.seq = sm.start_seq;
  w.head = sm.start_head;
  w.rt = sm.start_rt;
  w.tile = sm.start_tile;
  if (SHARED) {
    w.rts = (int)(((int64_t)a.batch.tokens * a.group + kAttnRows - 1) / kAttnRows);
    w.tiles = (a.kstart + kAttnTile - 1) / kAttnTile;
    w.kend = sm.kend;
  }
  const int key0 = SHARED ? 0 : a.kstart;
  const uint32_t tmem = sm.tmem;
  volatile int* abort = &sm.abort;

  if (warp >= kLoader) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoader) {
      // ---- loads: keys and values of a tile, one stage each ----
      int stage = 0;
      uint32_t phase = 0;
      auto advance = [&] {
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      };
      Pages pages;
      int seq = -1;
      for (bool first = true; w.next(a, first); first = false) {
        if (w.seq != seq) pages.start(a, seq = w.seq);
        const int n = w.busy(a.kstart);
        for (int t = w.first; t < w.first + n; ++t) {
          const int k0 = key0 + t * kAttnTile;
          const int keys = min(kAttnTile, w.kend - k0);
          for (int v = 0; v < 2; ++v) {
            ptx::mbar_wait(&sm.empty[stage], phase ^ 1, abort, kAttnWaitNs);
            load_tile<D>(a, v ? &vmap : &kmap, pages, w.head, k0, keys, sm.ring[stage],
                         &sm.full[stage]);
            advance();
          }
        }
      }
      // After a wait that ran out, copies may still be in flight: the block stays for them.
      if (*abort) {
        int never = 0;
        for (int i = 0; i < STAGES; ++i) {
          ptx::mbar_wait(&sm.full[stage], phase ^ 1, &never, kAttnWaitNs);
          advance();
        }
      }
    } else if (warp == kIssuer) {
      // ---- products ----
      int stage = 0;
      uint32_t phase = 0, q_phase = 0, q1_phase = 0, p_phase[2] = {0, 0};
      auto advance = [&] {
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      };
      const uint32_t q_addr = ptx::smem_addr(sm.q), ring = ptx::smem_addr(sm.ring);
      const uint32_t id_s = idesc_bf16(kAttnTile, false), id_o = idesc_bf16(D, true);
      auto scores = [&](int t, uint32_t k_addr) {
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * Sizes<D>::kHalf + (k & 3) * 32;
            mma_ss(tmem + kColS + t * 128, ptx::desc_sw128(q_addr + t * Sizes<D>::kTileBytes + off),
                   ptx::desc_sw128(k_addr + off), id_s, k > 0);
          }
          ptx::tc_commit(&sm.s_full[t]);
        }
        __syncwarp();
      };
      for (bool first = true; w.next(a, first); first = false) {
        const int n = w.busy(a.kstart);
        if (n == 0) continue;
        const int active = w.rows > kTileRows ? 2 : 1;
        ptx::mbar_wait(&sm.q_full[0], q_phase, abort, kAttnWaitNs);
        q_phase ^= 1;
        if (active == 2) {
          ptx::mbar_wait(&sm.q_full[1], q1_phase, abort, kAttnWaitNs);
          q1_phase ^= 1;
        }
        ptx::mbar_wait(&sm.full[stage], phase, abort, kAttnWaitNs);
        ptx::tc_fence_after();
        for (int t = 0; t < active; ++t) scores(t, ring + stage * Sizes<D>::kTileBytes);
        if (ptx::elect_one()) ptx::tc_commit(&sm.empty[stage]);
        __syncwarp();
        advance();
        for (int i = 0; i < n; ++i) {
          const int v_stage = stage;
          ptx::mbar_wait(&sm.full[v_stage], phase, abort, kAttnWaitNs);
          advance();
          const int keys = min(kAttnTile, w.kend - (key0 + (w.first + i) * kAttnTile));
          const int steps = (keys + 15) / 16;
          const uint32_t v_addr = ring + v_stage * Sizes<D>::kTileBytes;
          for (int t = 0; t < active; ++t) {
            ptx::mbar_wait(&sm.p_full[t], p_phase[t], abort, kAttnWaitNs);
            p_phase[t] ^= 1;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              for (int k = 0; k < steps; ++k)
                mma_ts(tmem + kColO + t * 128, tmem + kColS + t * 128 + k * 8,
                       desc_rows(v_addr + k * 2048, Sizes<D>::kHalf), id_o, i > 0 || k > 0);
              if (i + 1 == n) ptx::tc_commit(&sm.o_full[t]);
            }
            __syncwarp();
            if (i + 1 < n) {
              if (t == 0) {
                ptx::mbar_wait(&sm.full[stage], phase, abort, kAttnWaitNs);
                ptx::tc_fence_after();
              }
              scores(t, ring + stage * Sizes<D>::kTileBytes);
            }
          }
          if (ptx::elect_one()) {
            ptx::tc_commit(&sm.empty[v_stage]);
            if (i + 1 < n) ptx::tc_commit(&sm.empty[stage]);
          }
          __syncwarp();
          if (i + 1 < n) advance();
        }
      }
      // no product may be in flight when tensor memory is given back
      if (ptx::elect_one()) ptx::tc_commit(&sm.done);
      __syncwarp();
      int never = 0;
      ptx::mbar_wait(&sm.done, 0, &never, kAttnWaitNs);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax: a thread a row ----
    const int t = warp >> 2, r = threadIdx.x;             // row of the item
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);   // 32 lanes a warp
    const uint32_t s_col = lanes + kColS + t * 128, o_col = lanes + kColO + t * 128;
    uint32_t s_phase = 0, o_phase = 0;
    int loads = 0;                                         // stages that earlier items took
    for (bool first = true; w.next(a, first); first = false) {
      const int n = w.busy(a.kstart);
      const int v0 = loads;
      loads += 2 * n;
      if (t == 1 && w.rows <= kTileRows) continue;
      const Row row = row_of<SHARED>(a, w, r);
      if (n > 0) {
        // queries: 16-byte pieces, neighbouring lanes neighbouring pieces of a row
        constexpr int PIECES = D / 8;
        const int in = threadIdx.x & 127;
#pragma unroll 4
        for (int i = in; i < kTileRows * PIECES; i += 128) {
          const int qr = i / PIECES, piece = i % PIECES;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          const int rr = t * kTileRows + qr;
          if (rr < w.rows) {
            const int R = w.rt * kAttnRows + rr;
            const int64_t token = R / a.group + (SHARED ? 0 : w.s.t.first);
            const int head = w.head * a.group + R % a.group;
            v = *reinterpret_cast<const uint4*>(a.q + token * a.ldq + head * D + piece * 8);
          }
          *reinterpret_cast<uint4*>(sm.q[t] + (piece >> 3) * Sizes<D>::kHalf + qr * 128 +
                                    (((piece & 7) ^ (qr & 7)) << 4)) = v;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.q_full[t]);
      }
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i) {
        const int k0 = key0 + (w.first + i) * kAttnTile;
        ptx::mbar_wait(&sm.s_full[t], s_phase, abort, kAttnWaitNs);
        s_phase ^= 1;
        ptx::tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld32_issue(s_col + j * 32, x + j * 32);
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_wait_ld32(x + j * 32);
        if (__any_sync(0xFFFFFFFFu, k0 + kAttnTile > row.limit)) {
          const int seen = row.limit - k0;
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= seen) x[j] = 0xFF800000u;
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 128; ++j) top[j & 3] = fmaxf(top[j & 3], __uint_as_float(x[j]));
        const float up = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
        if (__any_sync(0xFFFFFFFFu, up > m + 8.f)) {
          const float to = fmaxf(m, up);
          const float f = to == m ? 1.f : exp2_approx(m - to);
          m = to;
          l *= f;
          if (i > 0) {
#pragma unroll 1
            for (int j = 0; j < D; j += 32) {
              uint32_t o[32];
              tmem_ld32_issue(o_col + j, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              ptx::tmem_st16(o_col + j, *reinterpret_cast<uint32_t(*)[16]>(o));
              ptx::tmem_st16(o_col + j + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
            }
          }
        }
        const float from = m == -INFINITY ? 0.f : m;
        const uint64_t scale2 = pair(a.scale_log2, a.scale_log2), from2 = pair(-from, -from);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t z =
                fma2(pair(__uint_as_float(x[32 * j + 2 * e]),
                          __uint_as_float(x[32 * j + 2 * e + 1])),
                     scale2, from2);
            const float u = exp2_approx(lo_of(z)), v = exp2_approx(hi_of(z));
            sum[e & 1] = add2(sum[e & 1], pair(u, v));
            p[e] = pack_bf16(u, v);
          }
          ptx::tmem_st16(s_col + j * 16, p);
        }
        sum[0] = add2(sum[0], sum[1]);
        l += lo_of(sum[0]) + hi_of(sum[0]);
        if (t == 0 && (w.kend - k0) % 16 != 0 && w.kend - k0 < kAttnTile) {
          // values behind the last key may be anything, and 0 times them must be 0: the rows
          // that share the last key's sixteen are cleared
          const int at = v0 + 2 * i + 1, stage = at % STAGES;
          ptx::mbar_wait(&sm.full[stage], (at / STAGES) & 1, abort, kAttnWaitNs);
          const int from_row = w.kend - k0, to_row = (from_row + 15) / 16 * 16;
          for (int e = threadIdx.x; e < (to_row - from_row) * (D / 8); e += 128) {
            const int vr = from_row + e / (D / 8), piece = e % (D / 8);
            *reinterpret_cast<uint4*>(sm.ring[stage] + (piece >> 3) * Sizes<D>::kHalf + vr * 128 +
                                      ((piece & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.p_full[t]);
      }

      // ---- the item's end ----
      if (n > 0) {
        ptx::mbar_wait(&sm.o_full[t], o_phase, abort, kAttnWaitNs);
        o_phase ^= 1;
        ptx::tc_fence_after();
      }
      const bool whole = w.first == 0 && w.last == w.tiles;
      const int slot = 2 * blockIdx.x + (w.first == 0);
      if (w.first == 0 && !whole && r == 0) {
        AttnCut cut;
        cut.first = SHARED ? 0 : w.s.t.first;
        cut.rt = w.rt;
        cut.rows = w.rows;
        cut.head = w.head;
        cut.from = blockIdx.x;
        cut.to = block_of(line, N, w.at + w.tiles - 1);
        a.cuts[blockIdx.x] = cut;
      }
      Finish fin;
      if (whole && row.token >= 0) fin = finish_begin<D, SHARED>(a, w.head, row.index, m, l);
#pragma unroll 1
      for (int j = 0; j < D; j += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32_issue(o_col + j, o);
          tmem_wait_ld32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (r < w.rows && !whole) {
          float4* dst =
              reinterpret_cast<float4*>(a.parts + ((int64_t)slot * kAttnRows + r) * D + j);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                 __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        } else if (whole && row.token >= 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            finish_quad<D, SHARED>(a, fin, row.token, row.head, j / 4 + e,
                                   make_float4(__uint_as_float(o[4 * e]),
                                               __uint_as_float(o[4 * e + 1]),
                                               __uint_as_float(o[4 * e + 2]),
                                               __uint_as_float(o[4 * e + 3])));
        }
      }
      if (r < w.rows && !whole) a.part_stats[slot * kAttnRows + r] = make_float2(m, l);
      if (whole && row.token >= 0 && !SHARED && a.lse)
        a.lse[(int64_t)row.token * a.q_heads + row.head] = fin.lse;
      ptx::tc_fence_before();
    }
  }
  __syncthreads();
  if (*abort && threadIdx.x == 0) atomicOr(a.flags, kErrTimeout);
  if (warp == kIssuer) ptx::tmem_dealloc(tmem, 512);
}

// Joins the parts of the items that the blocks of a tile kernel cut: block (c, y) the rows
// [y kJoinRows, ..) of the item that begins in block c's range and goes on behind it.
constexpr int kJoinRows = 8;
template <int D, bool SHARED>
__global__ void __launch_bounds__(kJoinRows * D / 4)
    attention_join_kernel(const __grid_constant__ AttnArgs a) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const AttnCut cut = a.cuts[blockIdx.x];
  const int quad = threadIdx.x % (D / 4);
  const int r = blockIdx.y * kJoinRows + threadIdx.x / (D / 4);
  if (cut.to < 0 || r >= cut.rows) return;
  const int64_t R = (int64_t)cut.rt * kAttnRows + r;
  const int token = cut.first + (int)(R / a.group);
  auto part = [&](int b) { return (int64_t)(2 * b + (b == cut.from)) * kAttnRows + r; };
  float top = -INFINITY, sum = 0.f;
#pragma unroll 8
  for (int b = cut.from; b <= cut.to; ++b) top = fmaxf(top, a.part_stats[part(b)].x);
  const float base = top == -INFINITY ? 0.f : top;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int b = cut.from; b <= cut.to; ++b) {
    const float2 st = a.part_stats[part(b)];
    const float4 y = *(reinterpret_cast<const float4*>(a.parts + part(b) * D) + quad);
    const float f = exp2_approx(st.x - base);
    sum += st.y * f;
    acc.x += y.x * f; acc.y += y.y * f; acc.z += y.z * f; acc.w += y.w * f;
  }
  const int head = cut.head * a.group + (int)(R % a.group);
  const Finish fin =
      finish_begin<D, SHARED>(a, cut.head, (int64_t)cut.first * a.group + R, top, sum);
  finish_quad<D, SHARED>(a, fin, token, head, quad, acc);
  if (!SHARED && a.lse && quad == 0) a.lse[(int64_t)token * a.q_heads + head] = fin.lse;
}

template <int D, bool SHARED>
cudaError_t launch(const AttnLaunch& g, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t st) {
  static PerDevice<bool> raised;
  constexpr size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(smem <= 232448, "a block's shared memory");
  cudaError_t e = once_a_device(raised, g.device, [] {
    return cudaFuncSetAttribute(attention_tile_kernel<D, SHARED>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (e != cudaSuccess) return e;
  const int blocks = g.num_sms < kAttnBlocks ? g.num_sms : kAttnBlocks;
  e = launch_pdl(attention_tile_kernel<D, SHARED>, dim3(blocks), dim3(kThreads), smem, st, g.args,
                 k, v);
  if (e != cudaSuccess) return e;
  const int64_t rows =
      (int64_t)(SHARED ? g.args.batch.tokens : g.args.batch.max_new) * g.args.group;
  const int most = (int)(rows < kAttnRows ? rows : kAttnRows);
  return launch_pdl(attention_join_kernel<D, SHARED>,
                    dim3(blocks, (most + kJoinRows - 1) / kJoinRows), dim3(kJoinRows * D / 4), 0,
                    st, g.args);
}

}  // namespace

cudaError_t launch_attention_tile(const AttnLaunch& g, const CUtensorMap& k, const CUtensorMap& v,
                                  bool shared, cudaStream_t st) {
  if (g.head_dim == 64)
    return shared ? launch<64, true>(g, k, v, st) : launch<64, false>(g, k, v, st);
  return shared ? launch<128, true>(g, k, v, st) : launch<128, false>(g, k, v, st);
}

}  // namespace mxmoe
