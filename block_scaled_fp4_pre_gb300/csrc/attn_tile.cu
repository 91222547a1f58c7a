// Attention with many query rows an item, on tensor memory, for sm_103a: prompts, drafts, and
// the prefix that a batch shares.
//
// A row is a new token and one of the heads that share a kv head; an item is up to 256 rows of
// one kv head, in two tiles of 128, against the keys that the last of them sees:
//   main     rows of one sequence, keys from `kstart` on
//   SHARED   rows of all sequences, the common prefix's keys [0, kstart): one pass over the
//            prefix serves the whole batch; its unfinished sums go to the workspace, where
//            the main part's rows pick them up
// A tile of 64 keys goes through S = Q K^T (both operands in shared memory, 128 x 64 fp32 in
// tensor memory), a thread a row for the softmax, and O += P V with P as bf16 in tensor memory,
// in the columns of S that it came from, and V as the transposed operand.
//
// A row tile has a warp that issues its products, a warpgroup for its softmax and two buffers of
// scores: the next tile's scores are made during this one's softmax, and the tensor cores alternate
// between the row tiles.  Where an item's rows fill one row tile at most, the two take every other
// tile of its keys instead and add up at its end.  The loaders keep a ring of key and value
// tiles full.  The running maximum is raised only where a logit passes it by 2^8 (the sums
// and the rounding of P allow it), so the output in tensor memory is rarely scaled; its warpgroup
// does that before it hands over the next P, when no product on it is in flight.
//
// Bound by the tensor cores: 4 x 128 x 64 x D operations a row tile and tile of keys at the dense
// bf16 rate.  1424 us for a prompt of 16384 tokens, 32 heads of 128 on 8 (1544 TFLOP/s, 0.82 of the
// measured rate of a library's product; 1532 us once the board's power limit sets in); the scores'
// products, 64 columns wide, read more of shared memory than they compute, and tiles of 128 columns
// would leave no room for two buffers a row tile beside the outputs.  At 64 elements a head the
// softmax's instructions take longer than the products: 4 prompts of 2048 105 us.  With one row
// tile an item it is bound by HBM: 19 drafts of 8 tokens over 8192 keys 103 us (0.92 of the
// measured copy bandwidth).
#include <algorithm>

#include "attn.cuh"
#include "per_device.h"
#include "tmap.cuh"

namespace mxmoe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kTileRows = 128;
// Warps: eight with a row a thread, one that loads keys and one for values and queries, one a row
// tile that issues its products.
constexpr int kLoader = 8, kIssuer = 10;
constexpr int kThreads = 384;                   // whole warpgroups, as register shares go by
// 384 threads start with 168 registers: the softmax's two warpgroups take 208, the third 88
// (2 x 208 + 88 = 3 x 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "the launch's registers");

constexpr int kTile = 64;                       // keys of a tile

template <int D>
struct Sizes {
  static constexpr int kBytes = kTile * D * 2;              // a tile of keys or values
  static constexpr int kHalf = kTile * 128;                 // 64 columns of it
  static constexpr int kQueries = kAttnRows * D * 2;
  static constexpr int kQueryHalf = kAttnRows * 128;
  static constexpr int kStage = 8 * 4096;                   // 32 rows of 128 bytes a warp
  static constexpr int kStages = (229376 - kStage - kQueries) / kBytes;
  static_assert(kStages % 2 == 0, "keys keep to the even stages");
};

template <int D>
struct Smem {
  uint8_t q[Sizes<D>::kQueries];                // [D / 64][256 rows][128 bytes]
  uint8_t ring[Sizes<D>::kStages][Sizes<D>::kBytes];
  uint8_t stage[8][4096];
  float2 split[kTileRows];                      // a split item's second share: maximum, sum
  int64_t scan[kThreads / 32];
  uint64_t full[Sizes<D>::kStages], empty[Sizes<D>::kStages];
  uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], o_prev[2], o_full[2], done;
  int64_t start_at;
  int start_left, start_seq, start_head, start_rt, start_tile;
  int kend;                                     // SHARED: keys that some row sees
  uint32_t tmem;
  int abort, joins[2];
};

// Tensor memory: scores of both row tiles (each of two tiles of keys, and, in their place, P),
// then the outputs.
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
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

// 64 scores to terms exp2(x scale - from), packed, and their sums.
__device__ __forceinline__ void terms(uint32_t (&p)[32], const uint32_t* x, uint64_t scale2,
                                      float from, uint64_t (&sum)[2]) {
  const uint64_t from2 = pair(-from, -from);
  sum[0] = sum[1] = 0;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const uint64_t z =
        fma2(pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, from2);
    const float u = exp2_approx(lo_of(z)), v = exp2_approx(hi_of(z));
    sum[e & 1] = add2(sum[e & 1], pair(u, v));
    p[e] = pack_bf16(u, v);
  }
}

// ---- the line ----

// sum over i in [0, n) of floor((a i + b) / m), by Euclid's steps on (m, a).
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += (int64_t)n * (n - 1) / 2 * (a / m) + (int64_t)n * (b / m);
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    n = top / m;
    b = top % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// What an item costs beside its tiles (its queries, its end), in tiles: positions of the line
// before its first.  us with 2, 3, 4, 5, 6: a prompt of 16384 tokens 1462, 1428, 1415, 1416, 1422;
// of 4096 129, 120, 116, 117, 118; 4 of 2048 at 64 elements a head 108, 104, 103, 105, 106.
constexpr int kItemCost = 4;

// Items of up to this many tiles are not cut: a block takes all of one whose first tile is in its
// range.  us with 0, 3, 6, 12, 32 heads of 128 on 8: 54 prompts of 110 tokens 44.8, 43.0, 43.0,
// 43.0; 106 of 12 tokens 32.7, 31.3, 31.3, 31.3; 117 drafts of 8 over 300 tokens 57.0, 57.4, 51.8,
// 51.6; 8 drafts of 5 behind 16384 common tokens 58.7, 59.0, 59.1, 64.4.
constexpr int kShortItem = 6;

// An item has whole tokens, `step` of them (256 / group) but for a sequence's last.
__device__ __forceinline__ int key_tiles(int keys) {
  return max(1, (keys + kTile - 1) / kTile);
}
// Keys from kstart on that row tile rt's last row sees (below 1: none).
__device__ __forceinline__ int keys_of(const AttnArgs& a, const Sequence& s, int rt, int step) {
  return s.base - a.kstart + min((rt + 1) * step, s.taken);
}
// Length on the line of a sequence's first k row tiles of one head.
__device__ __forceinline__ int64_t line_before(const AttnArgs& a, const Sequence& s, int k,
                                                int step) {
  const int rts = (s.taken + step - 1) / step;
  int64_t n = (int64_t)k * kItemCost;
  if (k == rts && k > 0) {                  // the last has its own number of tokens
    --k;
    n += key_tiles(keys_of(a, s, k, step));
  }
  const int unseen = a.kstart - s.base;     // new tokens that see no key from kstart on
  const int none = min(k, max(0, unseen / step));
  n += none;
  if (k > none)
    n += floor_sum(k - none, kTile, step,
                   (uint32_t)((none + 1) * step - unseen + kTile - 1));
  return n;
}

// An item: `rows` rows, of the tokens from `token` on, and of the keys [key0, kend) in `tiles`
// tiles those of tiles [first, last); its first tile is at position `at` of the line.
template <bool SHARED>
struct Walk {
  int64_t at;
  int left, seq, head, rt, tile;             // tile < 0: -tile positions before the first
  int step, rts;
  Sequence s;
  int token, rows, kend, tiles, first, last;
  __device__ __forceinline__ void enter(const AttnArgs& a) {     // a sequence
    if (!SHARED) {
      s = sequence(a, seq);
      rts = (s.taken + step - 1) / step;
    }
  }
  __device__ __forceinline__ bool next(const AttnArgs& a, bool begin) {
    for (;; begin = false) {
      if (left <= 0) return false;
      if (begin) {
        enter(a);
      } else {
        at += tiles + kItemCost;
        tile = -kItemCost;
        if (++rt == rts) {
          rt = 0;
          if (++head == a.kv_heads && !SHARED) {
            head = 0;
            do {
              ++seq;
              enter(a);
            } while (rts == 0);
          }
        }
      }
      if (tile < 0) {                        // the positions before its first tile
        left += tile;
        if (left <= 0) return false;
        tile = 0;
      }
      const int tokens = min(step, (SHARED ? a.batch.tokens : s.taken) - rt * step);
      token = rt * step + (SHARED ? 0 : s.first);
      rows = tokens * a.group;
      if (!SHARED) {
        const int keys = keys_of(a, s, rt, step);
        kend = a.kstart + keys;
        tiles = key_tiles(keys);
      }
      first = tile;
      last = min(tiles, tile + left);
      left -= last - first;
      if (SHARED || tiles > kShortItem) return true;
      last = tiles;                          // whole, the block's that its first tile is in
      if (first == 0) return true;
    }
  }
  // Tiles of [first, last) that hold a key; the others are behind the last one.
  __device__ __forceinline__ int busy(int key0) const {
    const int n = kend > key0 ? (kend - key0 + kTile - 1) / kTile : 0;
    return max(0, min(last, n) - first);
  }
};

// What row tile t does of an item: with rows for both, all of its `n` tiles of keys; where the
// rows fill one at most, every other tile (t 0 the first), the sums joined at the end.
struct Share {
  bool split;
  int tiles, base, t;
  // The share's tile j among the item's, counted from the block's first, and its first key.
  __device__ __forceinline__ int tile(int j) const { return split ? 2 * j + t : j; }
  __device__ __forceinline__ int key_of(int j) const { return base + tile(j) * kTile; }
};
template <bool SHARED>
__device__ __forceinline__ Share share_of(const Walk<SHARED>& w, int key0, int n, int t) {
  Share s;
  s.split = w.rows <= kTileRows;
  s.t = t;
  s.base = key0 + w.first * kTile;
  s.tiles = s.split ? (n + 1 - t) >> 1 : n;
  return s;
}

// Keys that row r of an item sees; all of its keys where the row is none.
template <bool SHARED>
__device__ __forceinline__ int row_limit(const AttnArgs& a, const Walk<SHARED>& w, int r) {
  if (r >= w.rows) return w.kend;
  const int i = token_of(a, r);
  if (!SHARED) return limit_of(w.s, w.rt * w.step + i);
  const int b = sequence_of(a.batch, w.token + i);
  if (b < 0) return w.kend;
  const Sequence s = sequence(a, b);
  const int at = w.token + i - s.first;
  return at < 0 || at >= s.taken ? w.kend : min(limit_of(s, at), w.kend);
}

// A warp's 32 rows of 128 bytes (8 pieces) go through its part of shared memory, so that global
// memory sees whole rows: a lane's own row on one side, neighbouring lanes neighbouring pieces of
// a row on the other.
__device__ __forceinline__ uint4* staged(uint8_t* stage, int row, int piece) {
  return reinterpret_cast<uint4*>(stage + row * 128 + ((piece ^ (row & 7)) << 4));
}
__device__ __forceinline__ void write_row(uint8_t* stage, int row, const uint32_t* v) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *staged(stage, row, e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
  __syncwarp();
}
template <typename F>
__device__ __forceinline__ void each_piece(int rows, F f) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int row = 4 * k + (lane >> 3);
    if (row < rows) f(row, lane & 7);
  }
}
// 32 columns of a row's output; zeros where nothing was computed.
__device__ __forceinline__ void load_output(uint32_t (&o)[32], uint32_t col, bool any) {
  if (any) {
    tmem_ld32_issue(col, o);
    tmem_wait_ld32(o);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0u;
  }
}
__device__ __forceinline__ uint32_t add_bits(uint32_t x, float f, uint32_t y, float g) {
  return __float_as_uint(add_scaled(__uint_as_float(x), f, __uint_as_float(y), g));
}

// A warp joins the parts of its rows [row0, row0 + rows) of an item, in the order of the line.
// Seldom needed, and short: code that runs once a block is read from L2 as it goes (unrolled for
// eight rows at a time this took 33 thousand cycles).
template <int D>
__device__ __noinline__ void join_rows(const AttnArgs& a, int kv_head, int token, int from, int to,
                                       int row0, int rows) {
  constexpr int QUADS = D / 4, PASS = 32 / QUADS;
  const int lane = threadIdx.x & 31, quad = lane % QUADS;
#pragma unroll 1
  for (int r = row0 + lane / QUADS; r < row0 + rows; r += PASS) {
    const Joined j = join_parts<D>(a, from, to, kAttnRows, r, quad);
    const int i = token_of(a, r), head = kv_head * a.group + r - i * a.group;
    const Finish fin =
        finish_begin<D, false>(a, kv_head, (int64_t)token * a.group + r, j.top, j.sum);
    finish_quad<D, false>(a, fin, token + i, head, quad, j.acc);
    if (a.lse && quad == 0) a.lse[(int64_t)(token + i) * a.q_heads + head] = fin.lse;
  }
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tile_kernel(const __grid_constant__ AttnArgs a,
                          const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap) {
  constexpr int STAGES = Sizes<D>::kStages;
  extern __shared__ uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(
      raw + ((1024 - (ptx::smem_addr(raw) & 1023)) & 1023));
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      ptx::mbar_init(&sm.full[i], 1);
      ptx::mbar_init(&sm.empty[i], 2);
    }
    ptx::mbar_init(&sm.q_full, 1);
    ptx::mbar_init(&sm.q_empty, 2);
    for (int t = 0; t < 2; ++t) {
      for (int u = 0; u < 2; ++u) {
        ptx::mbar_init(&sm.s_full[t][u], 1);
        ptx::mbar_init(&sm.p_full[t][u], 4);
      }
      ptx::mbar_init(&sm.o_prev[t], 1);
      ptx::mbar_init(&sm.o_full[t], 1);
    }
    ptx::mbar_init(&sm.done, 2);
    ptx::fence_mbar_init();
    sm.abort = 0;
    sm.kend = 0;
    sm.start_left = 0;
    ptx::prefetch_tmap(&qmap);
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
  const int step = kAttnRows / a.group;
  const int shared_rts = (a.batch.tokens + step - 1) / step;
  const int shared_tiles = (a.kstart + kTile - 1) / kTile;
  int64_t line = 0;
  int N;
  if (SHARED) {
    const int length = shared_tiles + kItemCost;
    line = (int64_t)a.kv_heads * shared_rts * length;
    N = (int)min((int64_t)gridDim.x, line);
    int most = 0;
    for (int b = threadIdx.x; b < a.batch.batch; b += kThreads)
      most = max(most, sequence(a, b).kend);
    atomicMax(&sm.kend, min(most, a.kstart));
    if (threadIdx.x == 0 && (int)blockIdx.x < N) {
      const int64_t begin = range_start(line, N, blockIdx.x);
      const int item = (int)(begin / length);
      sm.start_at = (int64_t)item * length + kItemCost;
      sm.start_tile = (int)(begin - sm.start_at);
      sm.start_rt = item % shared_rts;
      sm.start_head = item / shared_rts;
      sm.start_seq = 0;
      sm.start_left = (int)(range_start(line, N, blockIdx.x + 1) - begin);
    }
  } else {
    const int per = (a.batch.batch + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.batch.batch), b1 = min(b0 + per, a.batch.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Sequence s = sequence(a, b);
      mine += line_before(a, s, (s.taken + step - 1) / step, step);
    }
    const int64_t before = block_exclusive_sum(mine, sm.scan, &line) * a.kv_heads;
    line *= a.kv_heads;
    N = (int)min((int64_t)gridDim.x, line);
    if ((int)blockIdx.x < N) {
      const int64_t begin = range_start(line, N, blockIdx.x);
      if (begin >= before && begin < before + mine * a.kv_heads) {
        int64_t at = before, n;
        int b = b0;
        for (;; ++b) {
          const Sequence s = sequence(a, b);
          n = line_before(a, s, (s.taken + step - 1) / step, step);
          if (begin < at + n * a.kv_heads) break;
          at += n * a.kv_heads;
        }
        sm.start_head = (int)((begin - at) / n);
        sm.start_at = at + sm.start_head * n;
        sm.start_seq = b;
        sm.start_left = (int)(range_start(line, N, blockIdx.x + 1) - begin);
      }
      __syncthreads();
      if (warp == 0) {                                     // the row tile that holds begin
        const Sequence s = sequence(a, sm.start_seq);
        const int64_t rest = begin - sm.start_at;
        int lo = 0, hi = (s.taken + step - 1) / step;
        while (hi - lo > 1) {
          const int every = (hi - lo + 31) / 32;
          const int mine = lo + lane * every;
          const bool before = mine < hi && line_before(a, s, mine, step) <= rest;
          lo += (__popc(__ballot_sync(0xFFFFFFFFu, before)) - 1) * every;
          hi = min(hi, lo + every);
        }
        if (lane == 0) {
          const int64_t n = line_before(a, s, lo, step);
          sm.start_rt = lo;
          sm.start_tile = (int)(rest - n) - kItemCost;
          sm.start_at += n + kItemCost;
        }
      }
    }
  }
  // Entries of the cuts: an item's where the prefix's are fewer than the blocks, else the
  // block's that the item begins in.
  const bool by_item = SHARED && a.kv_heads * shared_rts <= (int)gridDim.x;
  if (threadIdx.x == 0 && !by_item && !a.join_here) a.cuts[blockIdx.x].to = -1;
  __syncthreads();
  Walk<SHARED> w = {};
  w.left = sm.start_left;
  w.at = sm.start_at;
  w.seq = sm.start_seq;
  w.head = sm.start_head;
  w.rt = sm.start_rt;
  w.tile = sm.start_tile;
  w.step = step;
  if (SHARED) {
    w.rts = shared_rts;
    w.tiles = shared_tiles;
    w.kend = sm.kend;
  }
  const int key0 = SHARED ? 0 : a.kstart;
  const uint32_t tmem = sm.tmem;
  // Once a wait has run out every other one gives up too.  The loaders stop there, and the issuers
  // issue and release nothing more, so that no load meets a copy in flight.  The softmax's warps
  // hand over no more terms and go through their items: those that meet at barriers have the same
  // ones.  What they read and store then is undefined, within the call's tensors.
  volatile int* abort = &sm.abort;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(kAll, ptx::mbar_wait(bar, parity, abort, kAttnWaitNs));
  };

  if (warp >= kLoader) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    uint32_t q_phase = 0;
    auto advance2 = [](int& stage, uint32_t& phase) {     // keys and values have every other stage
      if ((stage += 2) >= STAGES) {
        stage -= STAGES;
        phase ^= 1;
      }
    };
    if (warp < kIssuer) {
      // ---- loads: keys into the even stages; values into the odd, and an item's queries, which
      // wait for the last item's scores: the next keys do not wait with them ----
      const int v = warp - kLoader;
      int stage = v;
      uint32_t phase = 0;
      Pages pages;
      int seq = -1;
      for (bool first = true; ok && __any_sync(kAll, w.next(a, first)); first = false) {
        const int n = __shfl_sync(kAll, w.busy(key0), 0);
        if (n == 0) continue;
        if (__any_sync(kAll, w.seq != seq)) pages.start(a, seq = w.seq);
        const int head = __shfl_sync(kAll, w.head, 0);
        int k0 = __shfl_sync(kAll, key0 + w.first * kTile, 0);
        const int kend = __shfl_sync(kAll, w.kend, 0);
        if (v == 1) {
          const int token = __shfl_sync(kAll, w.token, 0);
          ok = wait(&sm.q_empty, q_phase ^ 1);
          if (!ok) break;
          q_phase ^= 1;
          if (ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(&sm.q_full, step * a.group * 2 * D);
            for (int h = 0; h < D / 64; ++h)
              ptx::tma_load_3d(sm.q + h * Sizes<D>::kQueryHalf, &qmap, h * 64, head * a.group,
                               token, &sm.q_full, ptx::policy_evict_first());
          }
          __syncwarp();
        }
        for (int i = 0; i < n; ++i, k0 += kTile) {
          ok = wait(&sm.empty[stage], phase ^ 1);
          if (!ok) break;
          load_tile<D, kTile, 1>(a, v ? &vmap : &kmap, pages, head, k0, min(kTile, kend - k0), 0,
                                 sm.ring[stage], &sm.full[stage]);
          advance2(stage, phase);
        }
      }
      // Every copy issued here must have landed before the block exits.
      int never = 0;
      if (v == 1) ptx::mbar_wait(&sm.q_full, q_phase ^ 1, &never, kAttnWaitNs);
#pragma unroll 1
      for (int i = 0; i < STAGES; i += 2) {
        ptx::mbar_wait(&sm.full[stage], phase ^ 1, &never, kAttnWaitNs);
        advance2(stage, phase);
      }
    } else {
      // ---- products: a warp a row tile, so that neither waits for the other's softmax ----
      // What steers the loops comes from votes and shuffles, and descriptors grow by sums, so
      // that the compiler keeps them in uniform registers: each of a product's operands would
      // be moved there first otherwise (100 cycles a product, where the tensor cores take 32
      // to 64).  For the same reason a wait that gave up leaves no loop before its item's end (a
      // prompt of 16384 tokens 1421 us, with a way out behind each wait 1450).
      const int t = warp - kIssuer;
      int k_stage = 0, v_stage = 1;
      uint32_t k_phase = 0, v_phase = 0, p_phase = 0;
      const uint32_t s_col = tmem + kColS + t * 128, o_col = tmem + kColO + t * 128;
      const uint32_t id_s = idesc_bf16(kTile, false), id_o = idesc_bf16(D, true);
      const uint64_t q_desc = ptx::desc_sw128(ptx::smem_addr(sm.q));
      const uint64_t k_desc = ptx::desc_sw128(ptx::smem_addr(sm.ring));
      const uint64_t v_desc = desc_rows(ptx::smem_addr(sm.ring), Sizes<D>::kHalf);
      auto pass = [&](int& stage, uint32_t& phase) {       // a tile of the other row tile's share
        ok &= wait(&sm.full[stage], phase);
        if (ptx::elect_one() && ok) ptx::mbar_arrive(&sm.empty[stage]);
        __syncwarp();
        advance2(stage, phase);
      };
      for (bool first = true; ok && __any_sync(kAll, w.next(a, first)); first = false) {
        const int n = __shfl_sync(kAll, w.busy(key0), 0);
        if (n == 0) continue;
        const bool split = __any_sync(kAll, w.rows <= kTileRows);
        const int tiles = split ? (n + 1 - t) >> 1 : n;
        // keys from the block's first tile on
        const int keys = __shfl_sync(kAll, w.kend - key0 - w.first * kTile, 0);
        const uint64_t q_tile = q_desc + (split ? 0 : t * ((kTileRows * 128) >> 4));
        ok &= wait(&sm.q_full, q_phase);
        q_phase ^= 1;
        auto scores = [&](int j) {                         // into their half of the columns
          if (split && j + t > 0) pass(k_stage, k_phase);
          ok &= wait(&sm.full[k_stage], k_phase);
          ptx::tc_fence_after();
          const uint64_t kd = k_desc + (uint64_t)(k_stage * (Sizes<D>::kBytes >> 4));
          const uint32_t col = s_col + (j & 1) * kTile;
          if (ptx::elect_one() && ok) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(col, q_tile + (k >> 2) * (Sizes<D>::kQueryHalf >> 4) + (k & 3) * 2,
                     kd + (k >> 2) * (Sizes<D>::kHalf >> 4) + (k & 3) * 2, id_s, k > 0);
            ptx::tc_commit(&sm.s_full[t][j & 1]);
            ptx::tc_commit(&sm.empty[k_stage]);
            if (j + 1 == tiles) ptx::tc_commit(&sm.q_empty);
          }
          __syncwarp();
          advance2(k_stage, k_phase);
        };
        if (tiles > 0) scores(0);
        if (tiles > 1) scores(1);
        for (int j = 0; j < tiles; ++j) {
          if (split && j + t > 0) pass(v_stage, v_phase);
          ok &= wait(&sm.full[v_stage], v_phase);
          ok &= wait(&sm.p_full[t][j & 1], (p_phase >> (j & 1)) & 1);
          p_phase ^= 1u << (j & 1);
          ptx::tc_fence_after();
          const uint64_t vd = v_desc + (uint64_t)(v_stage * (Sizes<D>::kBytes >> 4));
          const uint32_t col = s_col + (j & 1) * kTile;
          const int left = keys - (split ? 2 * j + t : j) * kTile;
          const uint32_t more = j > 0;
          if (ptx::elect_one() && ok) {
            mma_ts(o_col, col, vd, id_o, more);
#pragma unroll
            for (int k = 1; k < kTile / 16; ++k)
              if (k * 16 < left) mma_ts(o_col, col + k * 8, vd + k * (2048 >> 4), id_o, 1u);
            if (j + 2 == tiles) ptx::tc_commit(&sm.o_prev[t]);
            if (j + 1 == tiles) ptx::tc_commit(&sm.o_full[t]);
            ptx::tc_commit(&sm.empty[v_stage]);
          }
          __syncwarp();
          advance2(v_stage, v_phase);
          if (j + 2 < tiles) scores(j + 2);
        }
        if (tiles == 0 && ptx::elect_one() && ok) ptx::mbar_arrive(&sm.q_empty);
        __syncwarp();
        if (split && n > 2 * tiles - 1 + t) {              // one behind the share's last
          pass(k_stage, k_phase);
          pass(v_stage, v_phase);
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
    const int t = warp >> 2, peers = 1 + (warp & 3);      // barrier of the two warps of 32 rows
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);   // 32 lanes a warp
    const uint32_t s_col = lanes + kColS + t * 128, o_col = lanes + kColO + t * 128;
    const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
    uint32_t s_phase = 0, prev_phase = 0, o_phase = 0;
    int loads = 0;                                        // tiles of values that earlier items took
    for (bool first = true; w.next(a, first); first = false) {
      const int n = w.busy(key0);
      const int v0 = loads;
      loads += n;
      const Share share = share_of(w, key0, n, t);
      const int tiles = share.tiles;
      if (share.split && t == 1 && tiles == 0) continue;
      const int r = share.split ? threadIdx.x & 127 : threadIdx.x;     // row of the item
      const int limit = row_limit(a, w, r);
      const int all_see = __reduce_min_sync(kAll, limit);    // keys that every row of the warp sees
      float m = -INFINITY, l = 0.f;
      int k0 = share.key_of(0);
      for (int j = 0; j < tiles; ++j, k0 += share.split ? 2 * kTile : kTile) {
        const uint32_t x_col = s_col + (j & 1) * kTile;
        ptx::mbar_wait(&sm.s_full[t][j & 1], (s_phase >> (j & 1)) & 1, abort, kAttnWaitNs);
        bool gave_up = *abort;            // (what the wait returns costs 1% more)
        s_phase ^= 1u << (j & 1);
        ptx::tc_fence_after();
        uint32_t x[kTile];
        tmem_ld32_issue(x_col, x);
        tmem_ld32_issue(x_col + 32, x + 32);
        tmem_wait_ld32(x);
        tmem_wait_ld32(x + 32);
        if (all_see - k0 < kTile) {
          const int seen = limit - k0;
#pragma unroll
          for (int e = 0; e < kTile; ++e)
            if (e >= seen) x[e] = 0xFF800000u;
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kTile; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(x[e]));
        const float up = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
        if (__any_sync(0xFFFFFFFFu, up > m + 8.f)) {
          const float to = fmaxf(m, up);
          const float f = to == m ? 1.f : exp2_approx(m - to);
          m = to;
          l *= f;
          if (j > 0) {
            // No product may be in flight on the output: tile j - 1's end comes before the scores
            // of tile j + 1, or has a barrier of its own before the item's last.
            if (j + 1 < tiles)
              gave_up |= !wait(&sm.s_full[t][(j + 1) & 1], (s_phase >> ((j + 1) & 1)) & 1);
            else
              gave_up |= !wait(&sm.o_prev[t], prev_phase);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int e0 = 0; e0 < D; e0 += 32) {
              uint32_t o[32];
              tmem_ld32_issue(o_col + e0, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_col + e0, o);
            }
          }
        }
        if (j + 1 == tiles && w.kend - k0 < kTile && (w.kend - k0) % 16 != 0) {
          // values behind the last key may be anything, and 0 times them must be 0: the rows
          // that share the last key's sixteen are cleared, by each row tile before its own
          // products (the second to come writes zeros over zeros)
          const int at = v0 + share.tile(j), v = 2 * (at % (STAGES / 2)) + 1;
          if (!wait(&sm.full[v], (at / (STAGES / 2)) & 1)) break;
          const int from_row = w.kend - k0, to_row = (from_row + 15) / 16 * 16;
          for (int e = threadIdx.x & 127; e < (to_row - from_row) * (D / 8); e += 128) {
            const int vr = from_row + e / (D / 8), piece = e % (D / 8);
            *reinterpret_cast<uint4*>(sm.ring[v] + (piece >> 3) * Sizes<D>::kHalf + vr * 128 +
                                      ((piece & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
        }
        const float from = m == -INFINITY ? 0.f : m;
        uint64_t sum[2] = {0, 0};
        uint32_t p[32];
        terms(p, x, scale2, from, sum);
        tmem_st32(x_col, p);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0 && !gave_up) ptx::mbar_arrive(&sm.p_full[t][j & 1]);
        l += lo_of(sum[0]) + hi_of(sum[0]) + (lo_of(sum[1]) + hi_of(sum[1]));
      }

      // ---- the item's end ----
      float f0 = 1.f, f1 = 0.f;
      const bool joined = share.split && n > 1;              // a second share
      if (joined) {
        if (t == 1) sm.split[r] = make_float2(m, l);
        ptx::named_bar_sync(peers, 64);
        if (t == 0) {
          const float2 other = sm.split[r];
          const float up = fmaxf(m, other.x), base = up == -INFINITY ? 0.f : up;
          f0 = exp2_approx(m - base);
          f1 = exp2_approx(other.x - base);
          m = up;
          l = l * f0 + other.y * f1;
        }
      }
      const bool keeper = !share.split || t == 0;            // has the rows' end
      bool whole = w.first == 0 && w.last == w.tiles;
      const int slot = 2 * blockIdx.x + (w.first == 0);
      int from = 0, to = 0;                                  // blocks of a cut item
      if (!whole) {
        from = w.first == 0 ? blockIdx.x : block_of(line, N, w.at);
        to = block_of(line, N, w.at + w.tiles - 1);
      }
      if (w.first == 0 && (by_item || (!whole && !a.join_here)) && threadIdx.x == 0) {
        AttnCut cut;
        cut.first = w.token;
        cut.rows = w.rows;
        cut.head = w.head;
        cut.from = blockIdx.x;
        cut.to = whole ? -1 : to;
        a.cuts[by_item ? w.head * shared_rts + w.rt : blockIdx.x] = cut;
      }
      const int row0 = r - lane, live = w.rows - row0;      // the warp's rows of the item
      const int64_t index = (int64_t)w.token * a.group + r;
      const float* other = a.shared_parts + ((int64_t)w.head * a.batch.tokens * a.group +
                                             (int64_t)w.token * a.group + row0) * D;
      bool merge = a.kstart > 0;                             // with what `other` points to
      Finish fin = {};
      if (!SHARED && !whole && a.join_here && keeper && to == from + 1 && !merge) {
        // An item of two parts whose other one is there: joined on the way out.
        if ((threadIdx.x & 127) == 0) {
          int32_t* counter = a.counters + 2 * from + t;
          sm.joins[t] = ptx::ld_acquire(counter) == 1;
          if (sm.joins[t]) *counter = 0;
        }
        ptx::named_bar_sync(5 + t, 128);
        if (sm.joins[t]) {
          const int64_t at = (int64_t)(w.first == 0 ? 2 * to : 2 * from + 1) * kAttnRows;
          if (r < w.rows) finish_sums(fin, m, l, __ldcg(&a.part_stats[at + r]));
          other = a.parts + (at + row0) * D;
          whole = merge = true;
        }
        ptx::named_bar_sync(5 + t, 128);
      } else if (whole && r < w.rows && keeper) {
        fin = finish_begin<D, SHARED>(a, w.head, index, m, l);
      }
      float* keep = SHARED && whole
                        ? a.shared_parts + ((int64_t)w.head * a.batch.tokens * a.group +
                                            (int64_t)w.token * a.group + row0) * D
                        : a.parts + ((int64_t)slot * kAttnRows + row0) * D;
      // this lane's eighth of every fourth row of the output
      uint16_t* dst[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = row0 + 4 * k + (lane >> 3), i = token_of(a, at);
        dst[k] = a.out + (int64_t)(w.token + i) * a.ldo +
                 (w.head * a.group + at - i * a.group) * D + (lane & 7) * 8;
      }
      uint8_t* stage = sm.stage[warp];
      if (n > 0) {
        if (tiles > 1) {
          ptx::mbar_wait(&sm.o_prev[t], prev_phase, abort, kAttnWaitNs);
          prev_phase ^= 1;
        }
        ptx::mbar_wait(&sm.o_full[t], o_phase, abort, kAttnWaitNs);
        o_phase ^= 1;
        ptx::tc_fence_after();
      }
      // 32 columns of the row's output, of both shares
      auto output = [&](uint32_t (&o)[32], int j) {
        load_output(o, o_col + j, n > 0);
        if (joined) {
          ptx::named_bar_sync(peers, 64);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 y = *staged(sm.stage[warp + 4], lane, e);
            o[4 * e] = add_bits(o[4 * e], f0, y.x, f1);
            o[4 * e + 1] = add_bits(o[4 * e + 1], f0, y.y, f1);
            o[4 * e + 2] = add_bits(o[4 * e + 2], f0, y.z, f1);
            o[4 * e + 3] = add_bits(o[4 * e + 3], f0, y.w, f1);
          }
          ptx::named_bar_sync(peers, 64);
        }
      };
      if (share.split && t == 1) {               // to the other warpgroup
#pragma unroll 1
        for (int j = 0; j < D; j += 32) {
          uint32_t o[32];
          load_output(o, o_col + j, true);
          write_row(stage, lane, o);
          ptx::named_bar_sync(peers, 64);
          ptx::named_bar_sync(peers, 64);
        }
      } else if (SHARED || !whole) {
#pragma unroll 1
        for (int j = 0; j < D; j += 32) {
          uint32_t o[32];
          output(o, j);
          write_row(stage, lane, o);
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = *staged(stage, 4 * k + (lane >> 3), lane & 7);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = 4 * k + (lane >> 3);
            if (row < live) *reinterpret_cast<uint4*>(keep + row * D + j + (lane & 7) * 4) = v[k];
          }
          __syncwarp();
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < D; j += 64) {
          uint32_t z[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t o[32];
            output(o, j + 32 * half);
            if (merge) {
              each_piece(live, [&](int row, int piece) {
                *staged(stage, row, piece) = __ldcg(reinterpret_cast<const uint4*>(
                    other + row * D + j + 32 * half + piece * 4));
              });
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint4 y = *staged(stage, lane, e);
                o[4 * e] = add_bits(o[4 * e], fin.mine, y.x, fin.theirs);
                o[4 * e + 1] = add_bits(o[4 * e + 1], fin.mine, y.y, fin.theirs);
                o[4 * e + 2] = add_bits(o[4 * e + 2], fin.mine, y.z, fin.theirs);
                o[4 * e + 3] = add_bits(o[4 * e + 3], fin.mine, y.w, fin.theirs);
              }
              __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              z[16 * half + e] = pack_bf16(__uint_as_float(o[2 * e]) * fin.inv,
                                           __uint_as_float(o[2 * e + 1]) * fin.inv);
          }
          write_row(stage, lane, z);
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = *staged(stage, 4 * k + (lane >> 3), lane & 7);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (4 * k + (lane >> 3) < live) *reinterpret_cast<uint4*>(dst[k] + j) = v[k];
          __syncwarp();
        }
      }
      if (keeper && r < w.rows && !whole) a.part_stats[slot * kAttnRows + r] = make_float2(m, l);
      if (keeper && r < w.rows && whole && !SHARED && a.lse) {
        const int i = token_of(a, r);
        a.lse[(int64_t)(w.token + i) * a.q_heads + w.head * a.group + r - i * a.group] = fin.lse;
      }
      ptx::tc_fence_before();
      if (!SHARED && !whole && a.join_here && keeper) {
        // Else the rows' parts are joined by the block that comes last.
        ptx::named_bar_sync(5 + t, 128);
        if ((threadIdx.x & 127) == 0) {
          int32_t* counter = a.counters + 2 * from + t;
          const bool last = ptx::atomic_add_acq_rel(counter, 1) == to - from;
          if (last) *counter = 0;
          sm.joins[t] = last;
        }
        ptx::named_bar_sync(5 + t, 128);
        if (sm.joins[t])
          join_rows<D>(a, w.head, w.token, from, to, row0, min(live, 32));
      }
    }
  }
  __syncthreads();
  if (*abort && threadIdx.x == 0) atomicOr(a.flags, kErrTimeout);
  if (warp == kIssuer) ptx::tmem_dealloc(tmem, 512);
}

// Joins the parts of the items that the blocks of a tile kernel cut: block (c, y) the rows
// [y rows_a_block, ..) of entry c of the cuts.
template <int D, bool SHARED>
__global__ void __launch_bounds__(256)
    attention_join_kernel(const __grid_constant__ AttnArgs a, int rows_a_block) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const AttnCut cut = a.cuts[blockIdx.x];
  if (cut.to < 0) return;
  constexpr int kQuads = D / 4;
  const int quad = threadIdx.x % kQuads;
  const int end = min(cut.rows, ((int)blockIdx.y + 1) * rows_a_block);
  for (int r = blockIdx.y * rows_a_block + threadIdx.x / kQuads; r < end; r += 256 / kQuads) {
    const int i = token_of(a, r), head = cut.head * a.group + r - i * a.group;
    const int64_t token = cut.first + i;
    const Joined j = join_parts<D>(a, cut.from, cut.to, kAttnRows, r, quad);
    const Finish fin =
        finish_begin<D, SHARED>(a, cut.head, (int64_t)cut.first * a.group + r, j.top, j.sum);
    finish_quad<D, SHARED>(a, fin, token, head, quad, j.acc);
    if (!SHARED && a.lse && quad == 0) a.lse[token * a.q_heads + head] = fin.lse;
  }
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
  AttnArgs a = g.args;
  const int step = kAttnRows / a.group;
  // An item's parts are joined within the kernel where they are few: with twice as many items as
  // SMs a block's range is longer than most.  Elsewhere (a launch more, 4 to 10 us) many
  // blocks join an item's many parts together.  A short row of the page table leaves no item
  // that is cut.
  a.join_here = !SHARED && ((int64_t)a.kv_heads * (a.batch.tokens / step) >= 2 * g.num_sms ||
                            ((int64_t)a.batch.pages_ld << a.page_shift) <= kShortItem * kTile);
  CUtensorMap q;
  e = make_tmap_heads(&q, a.q, D, a.q_heads, a.batch.tokens, a.ldq, a.group, kAttnRows / a.group);
  if (e != cudaSuccess) return e;
  const int blocks = g.num_sms < kAttnBlocks ? g.num_sms : kAttnBlocks;
  e = launch_pdl(attention_tile_kernel<D, SHARED>, dim3(blocks), dim3(kThreads), smem, st, a, q,
                 k, v);
  if (e != cudaSuccess || a.join_here) return e;
  const int64_t rows = (int64_t)(SHARED ? a.batch.tokens : a.batch.max_new) * a.group;
  const int most = (int)(rows < kAttnRows ? rows : kAttnRows);
  // 8 rows a block, or more where that would be more blocks than are resident together
  const int eights = (most + 7) / 8;
  const int64_t items = (int64_t)a.kv_heads * ((a.batch.tokens + step - 1) / step);
  const int cuts = SHARED && items <= blocks ? (int)items : blocks;
  const int y = std::min(eights, std::max(1, 8 * g.num_sms / cuts));
  return launch_pdl(attention_join_kernel<D, SHARED>, dim3(cuts, y), dim3(256), 0, st, a,
                    (eights + y - 1) / y * 8);
}

}  // namespace

cudaError_t launch_attention_tile(const AttnLaunch& g, const CUtensorMap& k, const CUtensorMap& v,
                                  bool shared, cudaStream_t st) {
  if (g.head_dim == 64)
    return shared ? launch<64, true>(g, k, v, st) : launch<64, false>(g, k, v, st);
  return shared ? launch<128, true>(g, k, v, st) : launch<128, false>(g, k, v, st);
}

}  // namespace mxmoe
