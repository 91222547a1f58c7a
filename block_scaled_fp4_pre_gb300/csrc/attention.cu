// Which kernels a call of attention takes (attn_few.cu, attn_tile.cu).
#include "attn.cuh"
#include "tmap.cuh"

namespace mxmoe {
namespace {

// Whether the shared prefix is worth a pass of its own (attn_tile.cu, SHARED), from estimates of
// what it takes and what it saves, in us.
//
// Apart, each sequence streams the prefix: in the few-row kernel at 11 TB/s, mostly from L2; in
// the tile kernel as tiles of its own items, 1.55 us for 128 keys and 256 rows on an SM (1.1 at 64
// elements a head), the last item of a sequence as long as a whole one.  Together it is the tiles
// of the whole batch's rows, two launches, and the hand-over of each row's sums.  Measured, apart /
// shared, 32 heads of 128 on 8 kv heads: 32 sequences of one token behind 1024 common ones 29.7 /
// 33.4 us, behind 4096 63.8 / 37.4; 4 behind 16384 33.4 / 31.6, 8 56.8 / 34.2; 16 of 5 tokens
// behind 1024 26.3 / 35.0, behind 4096 46.3 / 42.0; 32 of 30 tokens behind 4096 81.0 / 97.2, behind
// 16384 252 / 223; 8 of 400 tokens behind 16384 625 / 679; 4 of 130 155 / 138, where the estimate
// takes the slower way, as with 16 of 5 at 64 elements a head on 2 kv heads (35.5 / 32.1).
bool worth_sharing(const AttnLaunch& g, bool few) {
  const AttnArgs& a = g.args;
  const double batch = a.batch.batch, prefix = a.batch.shared_len, D = g.head_dim;
  const int step = kAttnRows / a.group;
  const double tile_us = (g.head_dim == 64 ? 1.1 : 1.55) * a.kv_heads * (prefix / kAttnTile) /
                         g.num_sms;
  const double together = tile_us * ((a.batch.tokens + step - 1) / step);
  if (few)
    return 12.0 + 0.008 * batch * a.kv_heads + together <
           (batch - 1) * prefix * a.kv_heads * D * 4 / 11e6;
  const double tokens = a.batch.tokens / batch;
  const double items = a.batch.cu_new ? tokens / step + 0.5 : (a.batch.n_each + step - 1) / step;
  return 25.0 + a.batch.tokens * (double)a.q_heads * D * 8 * 0.65e-6 + together <
         tile_us * batch * items;
}

}  // namespace

cudaError_t launch_attention(const AttnLaunch& call, cudaStream_t st) {
  AttnLaunch g = call;
  AttnArgs& a = g.args;
  const uint64_t rows = ((uint64_t)a.num_pages * a.kv_heads) << a.page_shift;
  const uint32_t box = 1u << a.page_shift < kAttnBox ? 1u << a.page_shift : kAttnBox;
  CUtensorMap k, v;
  cudaError_t e = make_tmap_bf16(&k, a.k_cache, g.head_dim, rows, box);
  if (e == cudaSuccess) e = make_tmap_bf16(&v, a.v_cache, g.head_dim, rows, box);
  if (e != cudaSuccess) return e;
  const bool few = (int64_t)a.batch.max_new * a.group <= kAttnFewRows;
  a.kstart = 0;
  if (g.shared == MOE_SHARED_ALWAYS || (g.shared == MOE_SHARED_AUTO && worth_sharing(g, few))) {
    a.kstart = a.batch.shared_len;
    if ((e = launch_attention_tile(g, k, v, true, st)) != cudaSuccess) return e;
  }
  return few ? launch_attention_few(g, k, v, st) : launch_attention_tile(g, k, v, false, st);
}

}  // namespace mxmoe
