// Internal definitions shared by the CUDA translation units of libmxmoe.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "mxmoe.h"

namespace mxmoe {

// ---------------------------------------------------------------------------
// Tile geometry of the grouped GEMMs (weights on the MMA M side, tokens on N).
constexpr int kBM = 128;            // weight rows per tile (MMA M)
constexpr int kBN = 128;            // token rows per tile (max MMA N); expert segments are
                                    // padded to multiples of kBN rows
constexpr int kBK = 256;            // FP4 elements per k-block = one 128-byte swizzle row
constexpr int kBKBytes = kBK / 2;   // 128
constexpr int kATileBytes = kBM * kBKBytes;   // 16 KiB
constexpr int kBTileBytes = kBN * kBKBytes;   // 16 KiB
constexpr int kBBoxRows = 32;                 // token rows per TMA box
constexpr int kSFAtomBytes = 512;             // 128 rows x 4 scale bytes
constexpr int kSFStageBytes = 2 * kSFAtomBytes;  // 8 scale columns per k-block
// Narrower token tiles for lighter loads: 32 (decode-sized) or 64 token rows a tile,
// expert segments padded to that many rows, each tile's token scales in 128x4 blocks
// of its own (its rows in the first quarter or half of each block).
constexpr int kBNNarrow = 32;
constexpr int kBNMedium = 64;
// Token tiles of the pair kernel (two SMs share each item, tcgen05 cta_group::2): up
// to kBNPair rows, each starting at a whole 128-row scale block, so a tile spans
// kPairStride workspace rows of which it uses kBNPair.
constexpr int kBNPair = 192;
constexpr int kPairStride = 256;

// Workspace row, from its expert's segment start, of the expert's r-th assignment
// under a dispatch with token tiles of tile_rows rows.
__host__ __device__ __forceinline__ int tile_row_of_rank(int r, int tile_rows) {
  return tile_rows == kBNPair ? (r / kBNPair) * kPairStride + r % kBNPair : r;
}

// Workspace rows of an expert segment holding n assignments: whole tiles (tiles of up
// to 128 rows), or whole kPairStride spans and a last partial tile padded to 128 rows.
__host__ __device__ __forceinline__ int segment_rows(int n, int tile_rows) {
  if (tile_rows == kBNPair) {
    const int rem = n % kBNPair;
    return n / kBNPair * kPairStride + (rem + kBN - 1) / kBN * kBN;
  }
  return (n + tile_rows - 1) / tile_rows * tile_rows;
}

// Device error bits in ws.flags[0].
constexpr int kErrRouting = 1;
constexpr int kErrTimeout = 2;
constexpr int kErrPage = 4;

// A check's read of the error bits and its clear of them.  Both on its own stream and done when
// they return: a clear on the default stream could still run, or fall between two kernels, when
// the next call's kernels set the bits again on a stream that does not wait for that one.
inline cudaError_t read_flags(int32_t* flag, const void* dev, cudaStream_t st) {
  const cudaError_t e = cudaMemcpyAsync(flag, dev, sizeof(*flag), cudaMemcpyDeviceToHost, st);
  const cudaError_t waited = cudaStreamSynchronize(st);
  return e != cudaSuccess ? e : waited;
}
inline cudaError_t clear_flags(void* dev, size_t bytes, cudaStream_t st) {
  const cudaError_t e = cudaMemsetAsync(dev, 0, bytes, st);
  return e != cudaSuccess ? e : cudaStreamSynchronize(st);
}

// Other words of ws.flags: [1] number of token tiles, [2] valid assignments,
// [3] next work item of the layer kernel, [4] blocks of the layer kernel done.
constexpr int kFlagTiles = 1;
constexpr int kFlagValid = 2;
constexpr int kFlagSched = 3;
constexpr int kFlagExit = 4;
constexpr int kFlagBucketTicket = 5;   // blocks of the bucketing kernel done
constexpr int kFlagBucketBad = 6;      // ids outside [0, E) seen by the bucketing kernel

constexpr int kFlagProbe = 8;          // a counter nothing increments (wait probe)

// Assignments (t*k + j) ranked by one block of the bucketing kernel.
constexpr int kBucketChunk = 8192;

// Bounded waits give up after this many nanoseconds of %globaltimer.
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

// Byte offset of scale column s of row `row` in the 128x4 block layout
// (int32 view [rows/128][Kc/4][32][4]); kc4 = Kc / 4.
__host__ __device__ __forceinline__ size_t sf_atom_offset(size_t row, int s, int kc4) {
  return (((row >> 7) * (size_t)kc4 + (size_t)(s >> 2)) << 9) + ((row & 31) << 4) +
         (((row >> 5) & 3) << 2) + (size_t)(s & 3);
}

// Canonical row (gate 0..I-1, up I..2I-1) of the first weight stored at prepared
// row r under the gran=16 even/odd interleave.
__host__ __device__ __forceinline__ int gate_up_source_row(int r, int I) {
  const int chunk = r >> 5, within = r & 31;
  const int odd = within >> 4;
  const int is_up = (within >> 3) & 1;
  return is_up * I + chunk * 16 + (within & 7) * 2 + odd;
}

// The same under the gran=8 contiguous interleave of FP8 activations: prepared rows
// [gate 0..7, up 0..7, gate 8..15, up 8..15, ...].
__host__ __device__ __forceinline__ int gate_up_source_row8(int r, int I) {
  const int chunk = r >> 4, within = r & 15;
  return (within >> 3) * I + chunk * 8 + (within & 7);
}

// Interleave by activation format: gran=8 when f8, else gran=16.
__host__ __device__ __forceinline__ int gate_up_source_row_for(int r, int I, int f8) {
  return f8 ? gate_up_source_row8(r, I) : gate_up_source_row(r, I);
}

// Byte of token-side scale (row, scale column s) in a workspace of tiles of tile_rows
// rows (32, 64 or 128): the tile of rows tile_rows*t.. owns its scale blocks, with its
// row r in line r % 32, 4-byte word r / 32.  For 128-row tiles this is sf_atom_offset.
__host__ __device__ __forceinline__ size_t sf_tile_offset(size_t row, int s, int kc4,
                                                          int tile_rows) {
  const size_t tile = row / (size_t)tile_rows, r = row % (size_t)tile_rows;
  return ((tile * (size_t)kc4 + (size_t)(s >> 2)) << 9) + ((r & 31) << 4) + ((r >> 5) << 2) +
         (size_t)(s & 3);
}

// ---------------------------------------------------------------------------
// Workspace layout (computed on the host from the dims, passed to kernels).
struct WsLayout {
  int64_t T_cap, A_cap, R_cap, tiles_cap;
  size_t off_header, off_flags, off_counts, off_seg, off_tiles, off_tile_done, off_assign,
      off_local_rank, off_blk_base, off_tile_start,
      off_slot_token, off_slot_assign, off_slot_weight, off_xb, off_xsf, off_xq, off_xs, off_hb,
      off_hsf, off_acc, off_stage_x, off_stage_ids, off_stage_w, off_stage_out, off_few_ctrl,
      off_few_counters, off_few_logits, off_few_xq, off_few_xsf,
      off_few_hq, off_few_hsf, off_few_parts, total;
  int64_t few_slots;      // experts the few-token form can touch
};

struct WsPtrs {
  int32_t* flags;        // error bits and counters, see kFlag*
  int32_t* counts;       // [E]
  int32_t* seg;          // [E+1] first workspace row of each expert (multiples of kBN)
  int4* tiles;           // [tiles_cap] (expert, first row, rows, 0), experts in order
  int32_t* tile_start;   // [E+1] first tile of each expert (exclusive prefix of tiles)
  int32_t* tile_done;    // [tiles_cap] gate/up items finished per token tile
  int32_t* assign_slot;  // [A_cap] workspace row of assignment t*k+j, -1 if skipped
  int32_t* local_rank;   // [A_cap] rank of an assignment among its expert's, in its chunk
  int32_t* blk_base;     // [A_cap/kBucketChunk + 1][E] rows of an expert in earlier chunks
  int32_t* slot_token;   // [R_cap]
  int32_t* slot_assign;  // [R_cap]
  float* slot_weight;    // [R_cap]
  uint8_t* xb;           // [R_cap, H/2] (FP4) or [R_cap, H] (FP8) quantised token rows
  uint8_t* xsf;          // 128x4 blocks of [R_cap, H/32] (H/16 for NVFP4)
  uint8_t* xq;           // [T_cap, H/2] quantised token rows, one per token (pull dispatch)
  uint8_t* xs;           // [T_cap, H/32] their scales, row-major (pull dispatch)
  uint8_t* hb;           // [R_cap, I/2] (FP4) or [R_cap, I] (FP8) requantised intermediate rows
  uint8_t* hsf;          // 128x4 blocks of [R_cap, I/32] (I/16 for NVFP4)
  float* acc;            // [T_cap, H] fp32 combine accumulator, cleared by pre_dispatch
};

struct PrepLayout {
  size_t off_w1c, off_w1s, off_w2c, off_w2s, total;
};

struct Shape {
  int H, I, E, k;
  int f8;   // 1: fp8xfp4 (E4M3 activations, gran=8 interleave)
  int nv;   // 1: nvf4xnvf4 (E4M3 scale per 16 elements); both 0: mxf4xmxf4
};

// Elements per scale of the format: 16 (NVFP4) or 32 (MXFP4, MXFP8).
__host__ __device__ __forceinline__ int sf_group(const Shape& s) { return s.nv ? 16 : 32; }

// Prepared weight codes are stored in k-block tiles: the 128 rows of one weight slab
// over one k-block are contiguous, row after row, so each TMA box of the layer
// kernel reads one contiguous 16 KiB (8 KiB for fp8xfp4) run of memory.  A tile row
// holds one k-block's packed E2M1 bytes: 128 (256 elements) or, for fp8xfp4, whose
// k-blocks are 128 elements, 64.  Byte j of weight row R of a matrix with K elements
// a row sits at ((R / 128 * num_kb + j / kb_bytes) * 128 + R % 128) * kb_bytes +
// j % kb_bytes; a last k-block shorter than the others is zero-padded to full width.
__host__ __device__ __forceinline__ int weight_kb_bytes(const Shape& s) { return s.f8 ? 64 : 128; }
__host__ __device__ __forceinline__ int64_t weight_num_kb(const Shape& s, int64_t K) {
  const int64_t elems = 2 * (int64_t)weight_kb_bytes(s);
  return (K + elems - 1) / elems;
}
// Bytes of the tiled codes of `rows` weight rows (a multiple of 128) of K elements.
__host__ __device__ __forceinline__ int64_t weight_code_bytes(const Shape& s, int64_t rows,
                                                              int64_t K) {
  return rows * weight_num_kb(s, K) * weight_kb_bytes(s);
}

// Launch with programmatic stream serialisation: the kernel may start before the
// previous kernel in the stream finishes and must call ptx::pdl_wait() before it
// touches that kernel's output.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------------------
// Launchers implemented in dispatch.cu / gemm.cu.  Each returns the cudaError_t
// of its launch.
// Bucketing: per-expert counts and segment starts, the tile list, and each
// assignment's rank; the quantiser (or launch_assign_slots) turns ranks into rows.
// tile_rows: kBN (wide tiles), kBNMedium, kBNNarrow or kBNPair.
cudaError_t launch_bucket(const Shape& s, const int32_t* ids, int T, const WsPtrs& ws,
                          int tile_rows, cudaStream_t st);
// Quantise the tokens, give every assignment its row and copy the token there.
// pull: write each token's row once (xq/xs) instead of copying it to its k rows; the
// layer kernel then gathers token rows itself.
// tile_rows: the dispatch's token tiles (rows from tile_row_of_rank; token scales in the
// layout of tiles of min(tile_rows, 128) rows, sf_tile_offset).
cudaError_t launch_quantize_scatter(const Shape& s, const void* x, const int32_t* ids,
                                    const float* tw, int T, const WsPtrs& ws, bool pull,
                                    int tile_rows, cudaStream_t st);
// Rows of all assignments (128-row tiles) and the per-row tables, without quantising
// anything.
cudaError_t launch_assign_slots(const Shape& s, const int32_t* ids, const float* tw, int T,
                                const WsPtrs& ws, cudaStream_t st);
// acc [n] fp32 -> out [n] bf16 (round to nearest even).
cudaError_t launch_convert_out(const float* acc, void* out, int64_t n, cudaStream_t st);
cudaError_t launch_quantize_rows(const float* src, int64_t rows, int K, uint8_t* codes,
                                 uint8_t* sf, cudaStream_t st);
// fp32 rows -> NVFP4 codes and E4M3 scales (one per 16 elements).
cudaError_t launch_quantize_rows_nv(const float* src, int64_t rows, int K, uint8_t* codes,
                                 uint8_t* sf, cudaStream_t st);
cudaError_t launch_prepare(const Shape& s, const uint8_t* w1c, const uint8_t* w1s,
                           const uint8_t* w2c, const uint8_t* w2s, uint8_t* prep,
                           const PrepLayout& pl, cudaStream_t st);

// One block waiting, with the given limit, on an mbarrier no one arrives at and on a
// counter no one increments, through the same bounded waits as the layer kernel.
cudaError_t launch_wait_probe(int32_t* flags, unsigned long long limit_ns, cudaStream_t st);
size_t mxfp8_scale_bytes(int64_t rows_cap, int64_t K, int layout);
cudaError_t launch_mxfp8_quantize(const void* x, int64_t rows, int64_t K, void* q, void* sf,
                                  int layout, int64_t rows_cap, cudaStream_t st);
cudaError_t launch_fp4_mma_probe(int n, int blocks_per_sm, int blocks, long long mma_count,
                                 int32_t* flags, cudaStream_t st);
// M=256 across SM pairs (2-CTA clusters, tcgen05 cta_group::2), `pairs` clusters.
cudaError_t launch_fp4_mma_probe_pair(int n, int pairs, long long mma_count, int32_t* flags,
                                      cudaStream_t st);

// Records the message moe_last_error() returns on this thread.
void set_last_error(const char* msg);

// The layer kernel: gate/up GEMM + SwiGLU + requantisation, then down GEMM +
// weighted combine into the fp32 accumulator, in one persistent launch.  With num_phases == 1
// and gate_up_debug set it runs only the gate/up GEMM and writes raw accumulators.
struct LayerLaunch {
  const uint8_t* w1_codes;   // prepared gate/up codes [E*2I, H/2]
  const uint8_t* w1_sf;      // their scale blocks
  const uint8_t* w2_codes;   // prepared down codes [E*H, I/2]
  const uint8_t* w2_sf;
  int64_t R_cap;
  Shape shape;
  int T;
  int num_phases;
  WsPtrs ws;
  float* gate_up_debug;      // [T*k, 2I] (num_phases == 1)
  int num_sms;
  bool pull;                 // gate/up token rows gathered from ws.xq/xs (pull dispatch)
  int tile_rows;             // token rows a tile: 32, 64, 128 or kBNPair (the dispatch's choice)
};
cudaError_t launch_layer(const LayerLaunch& g, cudaStream_t st);
// The layer on SM pairs (pair.cu): kBNPair-row token tiles, mxf4xmxf4 only, bucketed
// dispatch; pair_shape_ok says whether the shape allows it (H and 2I multiples of 256).
bool pair_shape_ok(const Shape& s);
cudaError_t launch_layer_pair(const LayerLaunch& g, cudaStream_t st);

// ---------------------------------------------------------------------------
// RMSNorm with the residual's addition and an MXFP8 output (norm.cu).  Strides in
// elements.  residual, residual_out and y may be null; so may q and sf, together.
struct RmsnormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* gamma;
  uint16_t* residual_out;
  uint16_t* y;
  uint8_t* q;
  uint8_t* sf;
  int64_t ldx, ldr, ldro, ldy;
  int64_t rows, sf_rows;     // sf_rows: rows whose scales the kernel writes (zero past rows)
  int K, layout;
  float eps;
  float inv_k, inv_k_lo;     // 1 / K as two floats (set at the launch)
};
cudaError_t launch_rmsnorm_mxfp8(const RmsnormArgs& a, int64_t rows_cap, cudaStream_t st);

// ---------------------------------------------------------------------------
// The MXFP4 linear product (linear.cu).
struct LinearShape {
  int N, K;   // output and input features
  int f8;     // 1: fp8xfp4 (E4M3 activations); 0: mxf4xmxf4
};
// K and N as the weights are stored: whole scale blocks, whole 128-row slabs.
__host__ __device__ __forceinline__ int linear_padded_k(const LinearShape& s) {
  return (s.K + 127) / 128 * 128;
}
__host__ __device__ __forceinline__ int linear_slabs(const LinearShape& s) {
  return (s.N + 127) / 128;
}
__host__ __device__ __forceinline__ int linear_num_kb(const LinearShape& s) {
  const int kb = s.f8 ? 128 : kBK;
  return (linear_padded_k(s) + kb - 1) / kb;
}
inline int64_t linear_code_bytes(const LinearShape& s) {
  return (int64_t)linear_slabs(s) * linear_num_kb(s) * kBM * (s.f8 ? 64 : 128);
}
inline int64_t linear_scale_bytes(const LinearShape& s) {
  return (int64_t)linear_slabs(s) * (linear_padded_k(s) / 128) * kSFAtomBytes;
}
constexpr int kLinFusedRows = 32;   // bf16 rows up to which the product quantises itself
struct LinearLaunch {
  LinearShape shape;
  const uint8_t* w_codes;    // prepared: codes, then scale blocks
  const uint8_t* q;          // activation codes [rows, K bytes or K/2], or null: from x
  const uint8_t* sf;         // their 128x4 scale blocks
  const void* x;             // bf16 rows, at most kLinFusedRows (q null)
  int64_t ldx;
  int64_t rows;
  void* out;
  int64_t ldo;
  int out_f32;
  int32_t* flags;
  int give_up;               // as LinArgs
  int device, num_sms;       // the current device
};
cudaError_t launch_linear_prepare(const LinearShape& s, const uint8_t* codes,
                                  const uint8_t* scales, uint8_t* prep, cudaStream_t st);
cudaError_t launch_linear_quantize(const LinearShape& s, const void* x, int64_t ldx, int64_t rows,
                                   uint8_t* q, uint8_t* sf, cudaStream_t st);
cudaError_t launch_linear(const LinearLaunch& g, cudaStream_t st);

// ---------------------------------------------------------------------------
// The whole layer for a few tokens (few.cu).
constexpr int kFewTokens = 16;     // tokens a call takes: the columns of one MMA
constexpr int kFewBlocks = 304;    // most blocks of the expert kernel
struct FewArgs {
  const uint16_t* x;         // bf16 [T, H]
  const uint16_t* router;    // bf16 [E, H], or null: ids and weights are given
  int32_t* ids;              // [T, k]
  float* weights;            // [T, k]
  uint16_t* out;             // bf16 [T, H]
  const uint8_t* w1_sf;
  const uint8_t* w2_sf;
  float* logits;             // [T, E]
  uint8_t* xq;               // [kFewTokens, H or H/2] and its scale blocks
  uint8_t* xsf;
  uint8_t* hq;               // [slots * kFewTokens, I or I/2] and, a slot, its scale blocks
  uint8_t* hsf;
  float* parts0;             // [ranges][2][128][kFewTokens] fp32 sums of cut lines
  float* parts1;
  int32_t* counters;         // [slots * 2I/128], zero between calls
  int32_t* counters1;        // [H/128], zero between calls
  int32_t* ctrl;
  int32_t* flags;
  int T, H, I, E, k;
  int t_rows;                // token rows a TMA box holds: 8 or kFewTokens
};
struct FewLaunch {
  FewArgs args;
  Shape shape;
  const uint8_t* w1_codes;
  const uint8_t* w2_codes;
  int64_t slots_cap;
  int device, num_sms;       // the current device
};
cudaError_t launch_few(const FewLaunch& g, cudaStream_t st);

// ---------------------------------------------------------------------------
// Rotary positions and the append to a paged cache (rope.cu).
constexpr int kMostSequences = 4096;
constexpr int kMostPairs = 256;    // rotated pairs of a head of at most 512 elements
struct RopeTable {
  uint64_t turn[kMostPairs];       // 2^64 w / (2 pi): the angle of one position
};
// The step's batch on the device; pages through row 0 below shared_len.
struct KvBatch {
  const int32_t* seq_lens;
  const int32_t* cu_new;           // or null: n_each tokens a sequence
  const int32_t* pages;
  int batch, tokens, max_new, n_each, pages_ld, shared_len;
};
struct RopeSection {               // heads of one tensor
  const uint16_t* src;
  uint16_t* dst;                   // null in the cache's sections
  int64_t lds, ldd;
  int heads;
};
struct RopeArgs {
  const uint64_t* turn;            // table, or null: nothing is rotated
  const int32_t* positions;        // or null: the place in the sequence
  RopeSection q, k, v;             // moe_rope: q alone
  uint16_t* k_cache;               // [num_pages, k.heads, page_size, head_dim]
  uint16_t* v_cache;
  KvBatch batch;                   // append only
  int32_t* flags;
  int64_t tokens;
  float magnitude;
  int head_dim, rotary_dim, layout;
  int num_pages, page_shift;
};
cudaError_t launch_rope_prepare(const RopeTable& t, int pairs, void* table, cudaStream_t st);
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st);
cudaError_t launch_kv_append(const RopeArgs& a, cudaStream_t st);

// ---------------------------------------------------------------------------
// Attention over a paged cache (attention.cu).
constexpr int kAttnBlocks = 160;   // most blocks of a kernel
constexpr int kAttnRows = 256;     // most rows of an item
// The item of a tile kernel that begins in a block's range and goes on behind it: rows of the
// tokens from `first` on, in the parts of blocks [from, to]; to < 0: none.
struct AttnCut {
  int first, rows, head, from, to;
};
struct AttnArgs {
  const uint16_t* q;               // [tokens, q_heads, head_dim], stride ldq
  const uint16_t* k_cache;         // [num_pages, kv_heads, page_size, head_dim]
  const uint16_t* v_cache;
  uint16_t* out;
  float* lse;                      // [tokens, q_heads], or null
  int64_t ldq, ldo;
  float scale_log2;                // scale * log2(e)
  KvBatch batch;
  int q_heads, kv_heads, group, num_pages, page_shift;
  int group_inv;                   // ceil(2^16 / group)
  int32_t* flags;
  int kstart;                      // keys below it are the shared prefix's, computed apart
  int join_here;                   // tile kernel: the last block joins an item's parts
  // workspace: parts of cut items, two a block, and two counters a block (zero between calls)
  float* parts;                    // [blocks][2][rows][head_dim]
  float2* part_stats;              // [blocks][2][rows]: log2 of the largest term, sum
  int32_t* counters;
  AttnCut* cuts;                   // [blocks]
  // the prefix's sums of every row: [kv_heads][tokens * group], as parts
  float* shared_parts;
  float2* shared_stats;
};
struct AttnLaunch {
  AttnArgs args;
  int head_dim;
  int shared;                      // MOE_SHARED_*
  int device, num_sms;             // the current device
};
cudaError_t launch_attention(const AttnLaunch& g, cudaStream_t st);

// A sequence's new tokens in a call: the first, how many, and how many of them are computed.
struct NewTokens {
  int first, n, taken;
};
__device__ __forceinline__ NewTokens new_tokens(const KvBatch& b, int seq) {
  if (!b.cu_new) return {seq * b.n_each, b.n_each, b.n_each};
  const int first = min(max(b.cu_new[seq], 0), b.tokens);
  const int n = min(max(b.cu_new[seq + 1], first), b.tokens) - first;
  return {first, n, min(n, b.max_new)};
}

// The sequence that new token t belongs to: the last with first token at most t that is not
// empty there.  -1 behind the last one's tokens.
__device__ __forceinline__ int sequence_of(const KvBatch& b, int t) {
  if (!b.cu_new) return t / b.n_each;
  int lo = 0, hi = b.batch;            // cu[lo] <= t < cu[hi] where the entries are in order
  if (t >= b.cu_new[hi] || t < b.cu_new[0]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.cu_new[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace mxmoe
