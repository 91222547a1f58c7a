// Which kernels a call of attention takes (attn_few.cu, attn_tile.cu).
#include "attn.cuh"
#include "tmap.cuh"

namespace mxmoe {

cudaError_t launch_attention(const AttnLaunch& call, cudaStream_t st) {
  AttnLaunch g = call;
  AttnArgs& a = g.args;
  const uint64_t rows = ((uint64_t)a.num_pages * a.kv_heads) << a.page_shift;
  const uint32_t box = a.page_shift < 7 ? 1u << a.page_shift : kAttnTile;
  CUtensorMap k, v;
  cudaError_t e = make_tmap_bf16(&k, a.k_cache, g.head_dim, rows, box);
  if (e == cudaSuccess) e = make_tmap_bf16(&v, a.v_cache, g.head_dim, rows, box);
  if (e != cudaSuccess) return e;
  const int64_t item_rows = (int64_t)a.batch.max_new * a.group;
  // A prefix is worth a pass of its own where a sequence's rows do not fill an item.
  a.kstart = 0;
  if (g.shared && a.batch.batch > 1 && item_rows < kAttnRows) {
    a.kstart = a.batch.shared_len;
    if ((e = launch_attention_tile(g, k, v, true, st)) != cudaSuccess) return e;
  }
  if (item_rows <= kAttnFewRows) return launch_attention_few(g, k, v, st);
  return launch_attention_tile(g, k, v, false, st);
}

}  // namespace mxmoe
