// Rotary positions, and the append of keys and values to a paged cache with the keys (and
// queries) rotated on the way, for sm_103a.
//
//   pair i of a head, (a, b):  (a, b) -> m (a cos t - b sin t, b cos t + a sin t),  t = p w_i
//
// The angle: the table holds w_i as a fraction of a turn in 64-bit fixed point, so p times it
// modulo 2^64 is the angle modulo one turn with no rounding, whatever the position (fp32
// angles are off by 0.03 rad at p = 10^6).  Its cosine and sine are fp32, and so is the
// rotation; one rounding to bf16.
//
// Layout: a thread holds 16 bytes of a head (and, in the half layout, the 16 bytes that they
// pair with) and goes through up to HP heads of one token with the same cosines and sines,
// four heads' loads in flight at a time.  Sharing them pays where the call is bound by HBM;
// with few tokens latency counts, and a thread takes one head.  Queries, keys and values of an
// append are one launch: thread groups of the three tensors side by side.
//
// Bound by HBM at large token counts: 8191 tokens of 40 heads of 128, half of them rotated, 27.7
// us (168 MB, 0.91 of the measured copy bandwidth); an append of 15.3 k tokens of 32 query and
// 8 + 8 key and value heads 61.5 us (382 MB, 0.93).  By latency at few: one token 2.6 us, its
// append with queries 3.2 us (its page is looked up in three dependent loads).  Halves that are not
// whole 16-byte pieces are bound by their 2-byte loads and stores: 8191 tokens of 32 heads of 80
// with 20 rotated 34.9 us (84 MB, 0.36), adjacent pairs of the same 15.4.
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mxmoe {
namespace {

constexpr int kThreads = 256;

__global__ void rope_prepare_kernel(const __grid_constant__ RopeTable t, int pairs,
                                    uint64_t* out) {
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) out[i] = t.turn[i];
}

template <int VEC>
struct Piece;
template <>
struct Piece<8> {
  typedef uint4 T;
};
template <>
struct Piece<1> {
  typedef uint16_t T;
};

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Pairs (a, b) of the same places of two pieces.
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float (&c)[8],
                                       const float (&s)[8]) {
  uint32_t* x = &a.x;
  uint32_t* y = &b.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = lo_bf16(x[i]), a1 = hi_bf16(x[i]), b0 = lo_bf16(y[i]), b1 = hi_bf16(y[i]);
    x[i] = bf16x2(fmaf(a0, c[2 * i], -b0 * s[2 * i]), fmaf(a1, c[2 * i + 1], -b1 * s[2 * i + 1]));
    y[i] = bf16x2(fmaf(b0, c[2 * i], a0 * s[2 * i]), fmaf(b1, c[2 * i + 1], a1 * s[2 * i + 1]));
  }
}
__device__ __forceinline__ void rotate(uint16_t& a, uint16_t& b, const float (&c)[1],
                                       const float (&s)[1]) {
  const float x = lo_bf16(a), y = lo_bf16(b);
  const uint32_t r = bf16x2(fmaf(x, c[0], -y * s[0]), fmaf(y, c[0], x * s[0]));
  a = (uint16_t)r;
  b = (uint16_t)(r >> 16);
}
// The first `pairs` of the four adjacent pairs of a piece.
__device__ __forceinline__ void rotate_adjacent(uint4& a, const float (&c)[8],
                                                const float (&s)[8], int pairs) {
  uint32_t* x = &a.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p = lo_bf16(x[i]), q = hi_bf16(x[i]);
    const uint32_t r = bf16x2(fmaf(p, c[i], -q * s[i]), fmaf(q, c[i], p * s[i]));
    if (i < pairs) x[i] = r;
  }
}

struct Threads {
  int chunks;          // pieces (or pairs of pieces) of a head that threads hold
  int per_token;       // threads of a token
  int groups_q, groups_k;
  int64_t threads;     // of all tokens
};

// VEC elements a piece: 8, or 1 in a half layout whose halves are not whole 16-byte pieces.
template <int VEC, bool HALF, bool APPEND, int HP>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a,
                                                        const __grid_constant__ Threads g) {
  typedef typename Piece<VEC>::T T;
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int D = a.head_dim, half = a.rotary_dim >> 1;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= g.threads) return;
  const int64_t t = g.threads >> 32 ? id / g.per_token
                                    : (int64_t)((uint32_t)id / (uint32_t)g.per_token);
  const int u = (int)(id - t * g.per_token), c = u % g.chunks;
  int group = u / g.chunks;
  const bool is_q = group < g.groups_q;
  if (!is_q) group -= g.groups_q;
  const bool is_v = APPEND && !is_q && group >= g.groups_k;
  if (is_v) group -= g.groups_k;
  const RopeSection& sec = is_q ? a.q : is_v ? a.v : a.k;

  // where the token goes
  int pos = 0;
  int64_t row = 0;           // of the cache, in rows of head_dim
  if (APPEND) {
    const int seq = sequence_of(a.batch, (int)t);
    if (seq < 0) return;
    const NewTokens nt = new_tokens(a.batch, seq);
    const int at = (int)t - nt.first;
    pos = max(a.batch.seq_lens[seq], 0) - nt.n + at;
    if (at < 0 || at >= nt.taken || pos < 0) return;
    if (!is_q) {
      const int slot = pos >> a.page_shift;
      int page = -1;
      if (slot < a.batch.pages_ld)
        page = a.batch.pages[(pos < a.batch.shared_len ? 0 : (int64_t)seq * a.batch.pages_ld) +
                             slot];
      if (page < 0 || page >= a.num_pages) {
        if (c == 0 && group == 0) atomicOr(a.flags, kErrPage);
        return;
      }
      row = (((int64_t)page * sec.heads) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    }
    if (a.positions) pos = a.positions[t];
  } else {
    pos = a.positions[t];
  }

  // which elements, and their rotation
  int ea, eb = -1, pairs = 0;
  if (is_v) {
    ea = c * VEC;
    eb = D / 2 + ea;
    if (ea >= D / 2) return;
  } else if (HALF) {
    ea = c * VEC;
    if (ea < half) {
      eb = half + ea;
      pairs = a.turn ? VEC : 0;
    } else {
      ea += half;
    }
  } else {
    ea = c * 8;
    pairs = a.turn ? min(4, half - c * 4) : 0;
  }
  float cs[VEC], sn[VEC];
  if (pairs > 0) {
#pragma unroll
    for (int j = 0; j < (HALF ? VEC : 4); ++j) {
      const int p = (HALF ? ea : c * 4) + j;
      const uint64_t turns = p < half ? (uint64_t)(int64_t)pos * a.turn[p] : 0;
      sincospif((float)(int64_t)turns * 0x1p-63f, &sn[j], &cs[j]);
      sn[j] *= a.magnitude;
      cs[j] *= a.magnitude;
    }
  }

  const bool cache = APPEND && !is_q;
  const uint16_t* src = sec.src + t * sec.lds;
  uint16_t* dst = !cache ? sec.dst + t * sec.ldd : (is_v ? a.v_cache : a.k_cache) + row * D;
  const int64_t head_step = cache ? (int64_t)D << a.page_shift : D;
  constexpr int U = HP < 4 ? HP : 4;
#pragma unroll 1
  for (int h0 = group * HP; h0 < min((group + 1) * HP, sec.heads); h0 += U) {
    T x[U], y[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (h0 + j < sec.heads) {
        x[j] = *reinterpret_cast<const T*>(src + (int64_t)(h0 + j) * D + ea);
        if (eb >= 0) y[j] = *reinterpret_cast<const T*>(src + (int64_t)(h0 + j) * D + eb);
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (h0 + j < sec.heads) {
        if (pairs > 0) {
          if constexpr (HALF) rotate(x[j], y[j], cs, sn);
          else rotate_adjacent(x[j], cs, sn, pairs);
        }
        uint16_t* d = dst + (h0 + j) * head_step;
        *reinterpret_cast<T*>(d + ea) = x[j];
        if (eb >= 0) *reinterpret_cast<T*>(d + eb) = y[j];
      }
    }
  }
}

template <int VEC, bool HALF, bool APPEND, int HP>
cudaError_t launch(const RopeArgs& a, cudaStream_t st) {
  auto groups = [](int heads) { return (heads + HP - 1) / HP; };
  Threads g;
  const int half = a.rotary_dim / 2;
  g.chunks = HALF ? half / VEC + (a.head_dim - a.rotary_dim) / VEC : a.head_dim / 8;
  g.groups_q = groups(a.q.heads);
  g.groups_k = groups(a.k.heads);
  g.per_token = (g.groups_q + g.groups_k + groups(a.v.heads)) * g.chunks;
  g.threads = a.tokens * g.per_token;
  const int64_t blocks = (g.threads + kThreads - 1) / kThreads;
  if (blocks >= (int64_t)1 << 31) return cudaErrorInvalidConfiguration;
  return launch_pdl(rope_kernel<VEC, HALF, APPEND, HP>, dim3((unsigned)blocks), dim3(kThreads), 0,
                    st, a, g);
}

template <int VEC, bool HALF, bool APPEND>
cudaError_t choose(const RopeArgs& a, cudaStream_t st) {
  // Threads of one head each.  us with 1, 4 and 8 heads a thread, 128 elements a head: 16 tokens
  // of 40 heads 2.5, 2.9, 3.9; 256 tokens 5.2, 3.6, 4.1; 2048 tokens 13.0, 7.6, 7.6; 8191
  // tokens 45.9, 29.8, 28.5; an append of 15.3 k tokens of 32 + 16 heads 116, 65, 61.
  const int64_t pieces = a.tokens * (a.q.heads + a.k.heads + a.v.heads) * (a.head_dim / 16);
  if (pieces < (int64_t)1 << 15) return launch<VEC, HALF, APPEND, 1>(a, st);
  if (pieces < (int64_t)1 << 20) return launch<VEC, HALF, APPEND, 4>(a, st);
  return launch<VEC, HALF, APPEND, 8>(a, st);
}

template <bool APPEND>
cudaError_t by_layout(const RopeArgs& a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  if (a.layout == MOE_ROPE_INTERLEAVED) return choose<8, false, APPEND>(a, st);
  if (a.rotary_dim % 16 == 0) return choose<8, true, APPEND>(a, st);
  return choose<1, true, APPEND>(a, st);
}

}  // namespace

cudaError_t launch_rope_prepare(const RopeTable& t, int pairs, void* table, cudaStream_t st) {
  rope_prepare_kernel<<<1, 256, 0, st>>>(t, pairs, static_cast<uint64_t*>(table));
  return cudaGetLastError();
}
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) { return by_layout<false>(a, st); }
cudaError_t launch_kv_append(const RopeArgs& a, cudaStream_t st) { return by_layout<true>(a, st); }

}  // namespace mxmoe
