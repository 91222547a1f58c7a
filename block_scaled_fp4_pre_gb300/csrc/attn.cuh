// What the attention kernels share: the line of work that they cut into equal ranges, and the
// loads of keys and values by page.
//
// The work of a call is a line of tiles (128 or 64 keys of one item), item after item; block c of N
// takes the tiles [c W / N, (c + 1) W / N).  So every block streams the same number of keys,
// whatever the sequences' lengths, and an item is cut only where a block's range ends: a block
// has at most two parts of items, its first and its last.  Parts go to the workspace, and the
// block that finishes an item's last part joins them, in the order of the line.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mxmoe {

constexpr int kAttnTile = 128;            // keys of a tile of the few-row kernel
constexpr int kAttnBox = 64;              // most keys of a box that is loaded
constexpr int kAttnMostKeys = 1 << 30;    // of a sequence
constexpr unsigned long long kAttnWaitNs = 2000000000ull;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A sequence in a call: its first new token, how many are computed, the position of the first,
// and the keys [0, kend) that the last of them sees.
struct Sequence {
  int first, taken, base, kend;
};
__device__ __forceinline__ Sequence sequence(const AttnArgs& a, int b) {
  const NewTokens t = new_tokens(a.batch, b);
  Sequence s = {t.first, t.taken, max(a.batch.seq_lens[b], 0) - t.n, 0};
  const int64_t cap = min((int64_t)a.batch.pages_ld << a.page_shift, (int64_t)kAttnMostKeys);
  if ((int64_t)s.base + s.taken > cap) {      // behind the end of its row of the page table
    atomicOr(a.flags, kErrPage);
    s.base = (int)cap - s.taken;
  }
  s.kend = s.taken > 0 ? max(s.base + s.taken, 0) : 0;
  return s;
}
// Keys that new token i sees.
__device__ __forceinline__ int limit_of(const Sequence& s, int i) {
  return max(s.base + i + 1, 0);
}
// r / group for a row of an item.
__device__ __forceinline__ int token_of(const AttnArgs& a, int r) {
  return (int)(((uint32_t)r * (uint32_t)a.group_inv) >> 16);
}

// Position of a block's range on a line of W tiles, and the block that has position p.
__device__ __forceinline__ int64_t range_start(int64_t W, int N, int c) { return c * W / N; }
__device__ __forceinline__ int block_of(int64_t W, int N, int64_t p) {
  return (int)(((p + 1) * N - 1) / W);
}

// Sums of each thread's value over the threads before it; total in *total.  All threads of
// the block (a whole number of warps, at most 32).
__device__ __forceinline__ int64_t block_exclusive_sum(int64_t v, int64_t* warp_sums,
                                                       int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  *total = all;
  return before + s - v;
}

// A sequence's row of the page table, 32 entries at a time in the lanes of a warp.
struct Pages {
  const int32_t* row;
  const int32_t* shared;    // the first sequence's, for entries below shared_pages
  int shared_pages, base, mine;
  __device__ __forceinline__ void start(const AttnArgs& a, int b) {
    row = a.batch.pages + (int64_t)b * a.batch.pages_ld;
    shared = a.batch.pages;
    shared_pages = a.batch.shared_len >> a.page_shift;
    base = -64;
  }
  // Makes the entries [first, first + n), n at most 32, ready for at (converged warp).
  __device__ __forceinline__ void fetch(const AttnArgs& a, int first, int n) {
    if (first < base || first + n > base + 32) {
      base = first;
      const int at = first + (int)(threadIdx.x & 31);
      mine = -1;
      if (at < a.batch.pages_ld) mine = at < shared_pages ? shared[at] : row[at];
    }
  }
  __device__ __forceinline__ int at(int i) const {
    return __shfl_sync(0xFFFFFFFFu, mine, i - base);
  }
};

// Row of the cache's arrays, as the tensor map counts them, of row r of a page and head; the
// row behind the last, which loads read as zeros, for a page outside the cache.
__device__ __forceinline__ int cache_row(const AttnArgs& a, int page, int head, int r) {
  if (page < 0 || page >= a.num_pages) {
    atomicOr(a.flags, kErrPage);
    return (a.num_pages * a.kv_heads) << a.page_shift;
  }
  return ((page * a.kv_heads + head) << a.page_shift) + r;
}

// Loads one tile of keys (or values) from key k0 of a sequence, `keys` of them (1 .. TILE), into
// dst: [D / 64][TILE rows][128 bytes], swizzled; what no box covers keeps its old contents.
// PARTS converged warps share the boxes, each its own with an arrival of its own on bar.  The
// boxes' places come from shuffles and the loop's bounds from values that the caller made uniform,
// so that a copy's operands stay in uniform registers (see attn_tile.cu).
template <int D, int TILE, int PARTS>
__device__ __forceinline__ void load_tile(const AttnArgs& a, const CUtensorMap* map, Pages& pages,
                                          int head, int k0, int keys, int part, uint8_t* dst,
                                          uint64_t* bar) {
  constexpr int HALVES = D / 64;
  constexpr int MOST = TILE / 16 * HALVES / PARTS;        // boxes of a part, pages of 16 keys
  const int box = min(1 << a.page_shift, kAttnBox);
  const int boxes = (keys + box - 1) / box, mine = (boxes * HALVES - part + PARTS - 1) / PARTS;
  const int first = k0 >> a.page_shift, r = k0 & ((1 << a.page_shift) - 1);
  pages.fetch(a, first, ((r + (boxes - 1) * box) >> a.page_shift) + 1);
  // each lane the row of one box
  const int lane = threadIdx.x & 31;
  const int which = max(min(lane, mine - 1) * PARTS + part, 0), i = which / HALVES;
  const int at = r + i * box;                             // (a page may hold several boxes)
  const int page = pages.at(first + (at >> a.page_shift));
  const int y = cache_row(a, page, head, at & ((1 << a.page_shift) - 1));
  __syncwarp();
  if (ptx::elect_one()) ptx::mbar_arrive_expect_tx(bar, mine * box * 128);
  __syncwarp();
  const uint64_t policy = ptx::policy_evict_normal();
#pragma unroll
  for (int e = 0; e < MOST; ++e) {
    const int row = __shfl_sync(0xFFFFFFFFu, y, e);
    if (e < mine) {
      const int w = e * PARTS + part, h = w % HALVES;
      if (ptx::elect_one())
        ptx::tma_load_2d(dst + (h * TILE + w / HALVES * box) * 128, map, h * 64, row, bar, policy);
    }
  }
  __syncwarp();
}

// x f + y g, each product rounded: the same from either side, so that an item of two parts has the
// same bits whichever of its blocks joins them, and by whichever way.
__device__ __forceinline__ float add_scaled(float x, float f, float y, float g) {
  return __fadd_rn(__fmul_rn(x, f), __fmul_rn(y, g));
}

// What ends a row: its sums, with m the log2 of the term they are relative to, join the shared
// prefix's (main part) and become the output, or are kept (SHARED).  `index` is the row among
// its kv head's rows of all tokens.
struct Finish {
  float4* keep;
  const float4* other;
  float mine, theirs, inv, lse;
};
// The row's factors where its sums are joined with another part's (maximum, sum).
__device__ __forceinline__ void finish_sums(Finish& f, float m, float l, float2 part) {
  const float top = fmaxf(m, part.x), base = top == -INFINITY ? 0.f : top;
  f.mine = exp2_approx(m - base);
  f.theirs = exp2_approx(part.x - base);
  l = add_scaled(l, f.mine, part.y, f.theirs);
  // 0: no key; NaN where a key's logit is, for both outputs
  f.inv = l == 0.f ? 0.f : 1.f / l;
  f.lse = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
}
template <int D, bool SHARED>
__device__ __forceinline__ Finish finish_begin(const AttnArgs& a, int kv_head, int64_t index,
                                               float m, float l) {
  Finish f = {};
  const int64_t at = (int64_t)kv_head * a.batch.tokens * a.group + index;
  f.keep = reinterpret_cast<float4*>(a.shared_parts + at * D);
  f.other = nullptr;
  if (SHARED) {
    a.shared_stats[at] = make_float2(m, l);
    return f;
  }
  if (a.kstart > 0) {
    f.other = f.keep;
    finish_sums(f, m, l, a.shared_stats[at]);
  } else {
    finish_sums(f, m, l, make_float2(-INFINITY, 0.f));
  }
  return f;
}
// Four elements of the row.
template <int D, bool SHARED>
__device__ __forceinline__ void finish_quad(const AttnArgs& a, const Finish& f, int64_t token,
                                            int head, int quad, float4 v) {
  if (SHARED) {
    f.keep[quad] = v;
    return;
  }
  if (f.other) {
    const float4 y = f.other[quad];
    v.x = add_scaled(v.x, f.mine, y.x, f.theirs);
    v.y = add_scaled(v.y, f.mine, y.y, f.theirs);
    v.z = add_scaled(v.z, f.mine, y.z, f.theirs);
    v.w = add_scaled(v.w, f.mine, y.w, f.theirs);
  }
  *reinterpret_cast<uint2*>(a.out + token * a.ldo + head * D + quad * 4) = make_uint2(
      pack_bf16(v.x * f.inv, v.y * f.inv), pack_bf16(v.z * f.inv, v.w * f.inv));
}

// Row r's four elements `quad` of a cut item, over its parts of blocks [from, to] in their
// order: the sum of its terms, relative to 2^top, and of their products.  A block's parts lie at
// [2 block + whether the item begins there], `rows` rows each.  Eight parts' loads at a time.
struct Joined {
  float4 acc;
  float sum, top;
};
template <int D>
__device__ __forceinline__ Joined join_parts(const AttnArgs& a, int from, int to, int rows, int r,
                                             int quad) {
  constexpr int kAtOnce = 8;
  Joined j = {make_float4(0.f, 0.f, 0.f, 0.f), 0.f, -INFINITY};
  for (int b0 = from; b0 <= to; b0 += kAtOnce) {
    float2 st[kAtOnce];
    float4 y[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const int b = min(b0 + e, to);
      const int64_t at = (int64_t)(2 * b + (b == from)) * rows + r;
      st[e] = __ldcg(&a.part_stats[at]);
      y[e] = __ldcg(reinterpret_cast<const float4*>(a.parts + at * D) + quad);
    }
    float up = j.top;
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) up = fmaxf(up, st[e].x);
    const float base = up == -INFINITY ? 0.f : up, f = exp2_approx(j.top - base);
    j.top = up;
    j.sum = __fmul_rn(j.sum, f);
    j.acc.x = __fmul_rn(j.acc.x, f); j.acc.y = __fmul_rn(j.acc.y, f);
    j.acc.z = __fmul_rn(j.acc.z, f); j.acc.w = __fmul_rn(j.acc.w, f);
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const float g = b0 + e <= to ? exp2_approx(st[e].x - base) : 0.f;
      j.sum = add_scaled(j.sum, 1.f, st[e].y, g);
      j.acc.x = add_scaled(j.acc.x, 1.f, y[e].x, g);
      j.acc.y = add_scaled(j.acc.y, 1.f, y[e].y, g);
      j.acc.z = add_scaled(j.acc.z, 1.f, y[e].z, g);
      j.acc.w = add_scaled(j.acc.w, 1.f, y[e].w, g);
    }
  }
  return j;
}

// Items of at most 16 rows (attn_few.cu).
constexpr int kAttnFewRows = 16;
cudaError_t launch_attention_few(const AttnLaunch& g, const CUtensorMap& k, const CUtensorMap& v,
                                 cudaStream_t st);
// Items of any number of rows (attn_tile.cu); shared: the prefix's part for all rows.
cudaError_t launch_attention_tile(const AttnLaunch& g, const CUtensorMap& k, const CUtensorMap& v,
                                  bool shared, cudaStream_t st);

}  // namespace mxmoe
