// Attention of a batch's new tokens over a paged cache of keys and values, for sm_103a.
//
//   out[t, h] = sum_j p_j v[j] / sum_j p_j,  p_j = exp(scale q . k[j]),  j <= position of t
//
// One warp a query head of a token: a pass over its keys with the running maximum and sum.
#include <cuda_runtime.h>

#include "attn.cuh"
#include "tmap.cuh"

namespace mxmoe {
namespace {

template <int D>
__global__ void __launch_bounds__(256) attention_row_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int t = (int)(row / a.q_heads), h = (int)(row % a.q_heads);
  if (t >= a.batch.tokens) return;
  int seq = -1;
  NewTokens nt = {};
  for (int b = 0; b < a.batch.batch; ++b) {
    const NewTokens x = new_tokens(a.batch, b);
    if (t >= x.first && t < x.first + x.taken) { seq = b; nt = x; }
  }
  if (seq < 0) return;
  const int limit = a.batch.seq_lens[seq] - nt.n + (t - nt.first) + 1;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e)
    q[e] = __uint_as_float((uint32_t)a.q[t * a.ldq + h * D + lane * E + e] << 16) * a.scale_log2;
  const int kvh = h / a.group;
  for (int j = 0; j < limit; ++j) {
    const int slot = j >> a.page_shift;
    int page = -1;
    if (slot < a.batch.pages_ld)
      page = a.batch.pages[(j < a.batch.shared_len ? 0 : (int64_t)seq * a.batch.pages_ld) + slot];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(a.flags, kErrPage);
      break;
    }
    const int64_t at = ((((int64_t)page * a.kv_heads + kvh) << a.page_shift) +
                        (j & ((1 << a.page_shift) - 1))) * D + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * __uint_as_float((uint32_t)a.k_cache[at + e] << 16);
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, w);
    const float top = fmaxf(m, s), f = exp2f(m - top), p = exp2f(s - top);
    m = top;
    l = l * f + p;
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * f + p * __uint_as_float((uint32_t)a.v_cache[at + e] << 16);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int e = 0; e < E; ++e) {
    const float v = o[e] * inv;
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(v));
    a.out[t * a.ldo + h * D + lane * E + e] = (uint16_t)r;
  }
  if (a.lse && lane == 0)
    a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_attention(const AttnLaunch& g, cudaStream_t st) {
  const AttnArgs& a = g.args;
  const uint64_t rows = ((uint64_t)a.num_pages * a.kv_heads) << a.page_shift;
  const uint32_t box = a.page_shift < 7 ? 1u << a.page_shift : kAttnTile;
  CUtensorMap k, v;
  cudaError_t e = make_tmap_bf16(&k, a.k_cache, g.head_dim, rows, box);
  if (e == cudaSuccess) e = make_tmap_bf16(&v, a.v_cache, g.head_dim, rows, box);
  if (e != cudaSuccess) return e;
  if ((int64_t)a.batch.max_new * a.group <= kAttnFewRows)
    return launch_attention_few(g, k, v, st);
  const int64_t warps = (int64_t)g.args.batch.tokens * g.args.q_heads;
  const dim3 grid((unsigned)((warps + 7) / 8));
  if (g.head_dim == 64) return launch_pdl(attention_row_kernel<64>, grid, dim3(256), 0, st, g.args);
  return launch_pdl(attention_row_kernel<128>, grid, dim3(256), 0, st, g.args);
}

}  // namespace mxmoe
