// C ABI of the attention half of a decoder block (declared in include/mxmoe.h): rotary
// positions, the append to a paged cache, and attention over it.  Argument checks, layouts and
// the registry of workspaces; nothing here allocates device memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>

#include "common.cuh"
#include "mxmoe.h"

using namespace mxmoe;

namespace {

moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

moe_status cuda_fail(cudaError_t e, const char* what) {
  return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool given(const void* p) { return p && aligned(p, 16); }
// A token stride: a multiple of 8 elements, at least a row.
bool good_stride(int64_t ld, int64_t row) { return ld >= row && ld % 8 == 0; }

// ---- rotary positions ----

moe_status check_rope(const moe_rope_dims* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARG, "rope dims is NULL");
  if (d->head_dim < 8 || d->head_dim % 8 || d->head_dim > 2 * kMostPairs)
    return fail(MOE_ERR_INVALID_ARG, "head_dim %d must be a multiple of 8 in [8, %d]", d->head_dim,
                2 * kMostPairs);
  if (d->rotary_dim < 2 || d->rotary_dim % 2 || d->rotary_dim > d->head_dim)
    return fail(MOE_ERR_INVALID_ARG, "rotary_dim %d must be even in [2, head_dim=%d]",
                d->rotary_dim, d->head_dim);
  if (d->layout != MOE_ROPE_HALF && d->layout != MOE_ROPE_INTERLEAVED)
    return fail(MOE_ERR_INVALID_ARG, "unknown rotary layout %d", d->layout);
  if (d->scaling < MOE_ROPE_UNSCALED || d->scaling > MOE_ROPE_YARN)
    return fail(MOE_ERR_INVALID_ARG, "unknown rotary scaling %d", d->scaling);
  if (!(d->base > 1.0) || std::isinf(d->base))
    return fail(MOE_ERR_INVALID_ARG, "base must be finite and above 1");
  if (!(d->magnitude >= 0.0) || std::isinf((float)d->magnitude))
    return fail(MOE_ERR_INVALID_ARG, "magnitude must be finite and at least 0");
  if (d->scaling != MOE_ROPE_UNSCALED && (!(d->factor >= 1.0) || std::isinf(d->factor)))
    return fail(MOE_ERR_INVALID_ARG, "factor must be finite and at least 1");
  if (d->scaling == MOE_ROPE_NTK && d->rotary_dim == 2)
    return fail(MOE_ERR_INVALID_ARG, "MOE_ROPE_NTK needs a rotary_dim above 2");
  if (d->scaling == MOE_ROPE_YARN) {
    if (!(d->original_length > 0.0) || std::isinf(d->original_length))
      return fail(MOE_ERR_INVALID_ARG, "original_length must be finite and above 0");
    if (!(d->beta_slow >= 0.0) || !(d->beta_fast > d->beta_slow) || std::isinf(d->beta_fast))
      return fail(MOE_ERR_INVALID_ARG, "need beta_fast > beta_slow >= 0, finite");
  }
  return MOE_OK;
}

float magnitude_of(const moe_rope_dims& d) {
  if (d.magnitude > 0.0) return (float)d.magnitude;
  return d.scaling == MOE_ROPE_YARN ? (float)(0.1 * std::log(d.factor) + 1.0) : 1.f;
}

constexpr double kTurn = 6.283185307179586476925;

// Radians that pair i rotates by from one position to the next.
double frequency_of(const moe_rope_dims& d, int i) {
  const double n = d.rotary_dim;
  double base = d.base;
  if (d.scaling == MOE_ROPE_NTK) base *= std::pow(d.factor, n / (n - 2.0));
  double w = std::pow(base, -2.0 * i / n);
  if (d.scaling == MOE_ROPE_LINEAR) w /= d.factor;
  if (d.scaling == MOE_ROPE_YARN) {
    const double turns = d.original_length * w / kTurn;
    const double g =
        std::fmin(1.0, std::fmax(0.0, (turns - d.beta_slow) / (d.beta_fast - d.beta_slow)));
    w = w * g + w / d.factor * (1.0 - g);
  }
  return w;   // at most 1
}

void set_rope(RopeArgs& a, const moe_rope_dims& d, const void* table) {
  a.turn = static_cast<const uint64_t*>(table);
  a.magnitude = magnitude_of(d);
  a.head_dim = d.head_dim;
  a.rotary_dim = d.rotary_dim;
  a.layout = d.layout;
}

// The table, of w (radians a position) or, where that is null, of the dims' frequencies.
moe_status prepare_rope(const moe_rope_dims* d, const double* w, void* table, size_t table_bytes,
                        void* stream) {
  const moe_status s = check_rope(d);
  if (s) return s;
  if (!given(table)) return fail(MOE_ERR_INVALID_ARG, "table NULL or not 16-byte aligned");
  const int pairs = d->rotary_dim / 2;
  if (table_bytes < pairs * sizeof(uint64_t))
    return fail(MOE_ERR_INVALID_ARG, "table has %zu bytes, needs %zu", table_bytes,
                pairs * sizeof(uint64_t));
  RopeTable t = {};   // parts of a turn, times 2^64
  for (int i = 0; i < pairs; ++i) {
    const double part = (w ? w[i] : frequency_of(*d, i)) / kTurn;
    if (!(part >= 0.0 && part < 1.0))
      return fail(MOE_ERR_INVALID_ARG, "frequency %d must be in [0, 2 pi)", i);
    t.turn[i] = (uint64_t)std::ldexp(part, 64);
  }
  const cudaError_t e = launch_rope_prepare(t, pairs, table, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope prepare");
  return MOE_OK;
}

// ---- workspaces ----

struct AttnWs {
  size_t flags, counters, cuts, stats, parts, shared_stats, shared_parts, total;
};

AttnWs ws_layout(const moe_attention_dims& d) {
  AttnWs L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 1023) / 1024 * 1024;
    return at;
  };
  L.flags = take(4);
  L.counters = take(2 * kAttnBlocks * sizeof(int32_t));
  L.cuts = take(kAttnBlocks * sizeof(AttnCut));
  L.stats = take((size_t)kAttnBlocks * 2 * kAttnRows * sizeof(float2));
  L.parts = take((size_t)kAttnBlocks * 2 * kAttnRows * d.head_dim * sizeof(float));
  const size_t rows = (size_t)d.max_shared_tokens * d.q_heads;
  L.shared_stats = take(rows * sizeof(float2));
  L.shared_parts = take(rows * d.head_dim * sizeof(float));
  L.total = o;
  return L;
}

std::mutex g_mu;
struct AttnState {
  moe_attention_dims dims;
  int32_t shared;   // moe_attention_set_shared
};
std::map<const void*, AttnState> g_attention;

bool power_of_two(int v) { return v > 0 && (v & (v - 1)) == 0; }
int shift_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

moe_status check_dims(const moe_attention_dims* d) {
  if (!d) return fail(MOE_ERR_INVALID_ARG, "dims is NULL");
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(MOE_ERR_UNSUPPORTED, "head_dim %d: attention is built for 64 and 128",
                d->head_dim);
  if (d->kv_heads < 1 || d->q_heads < d->kv_heads || d->q_heads > 1024 ||
      d->q_heads % d->kv_heads)
    return fail(MOE_ERR_INVALID_ARG, "q_heads %d must be a multiple of kv_heads %d, at most 1024",
                d->q_heads, d->kv_heads);
  if (d->q_heads / d->kv_heads > kAttnRows)
    return fail(MOE_ERR_INVALID_ARG, "q_heads %d: more than %d for each of kv_heads %d",
                d->q_heads, kAttnRows, d->kv_heads);
  if (!power_of_two(d->page_size) || d->page_size < 16 || d->page_size > 256)
    return fail(MOE_ERR_INVALID_ARG, "page_size %d must be a power of two in [16, 256]",
                d->page_size);
  if (d->num_pages < 1 ||
      (int64_t)d->num_pages * d->kv_heads * d->page_size >= ((int64_t)1 << 31))
    return fail(MOE_ERR_INVALID_ARG, "num_pages %d: need 1 <= num_pages * kv_heads * page_size < 2^31",
                d->num_pages);
  if (d->max_tokens < 1 || d->max_tokens > (1 << 20))
    return fail(MOE_ERR_INVALID_ARG, "max_tokens %d outside [1, 2^20]", d->max_tokens);
  if (d->max_shared_tokens < 0 || d->max_shared_tokens > d->max_tokens)
    return fail(MOE_ERR_INVALID_ARG, "max_shared_tokens %d outside [0, max_tokens=%d]",
                d->max_shared_tokens, d->max_tokens);
  return MOE_OK;
}

bool same(const moe_attention_dims& a, const moe_attention_dims& b) {
  return a.q_heads == b.q_heads && a.kv_heads == b.kv_heads && a.head_dim == b.head_dim &&
         a.num_pages == b.num_pages && a.page_size == b.page_size &&
         a.max_tokens == b.max_tokens && a.max_shared_tokens == b.max_shared_tokens;
}

moe_status check_ws(const moe_attention_dims* d, const void* ws, size_t ws_bytes,
                    int32_t* shared) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  const size_t need = ws_layout(*d).total;
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_attention.find(ws);
  if (it == g_attention.end())
    return fail(MOE_ERR_WORKSPACE_MISMATCH,
                "workspace %p was not initialised by moe_attention_workspace_init", ws);
  if (!same(it->second.dims, *d))
    return fail(MOE_ERR_WORKSPACE_MISMATCH, "workspace %p was initialised for other dims", ws);
  *shared = it->second.shared;
  return MOE_OK;
}

// Checks a call's batch and fills in the kernels' view of it.
moe_status check_batch(const moe_attention_dims* d, const moe_kv_batch* b, KvBatch* out) {
  if (!b) return fail(MOE_ERR_INVALID_ARG, "batch is NULL");
  if (b->batch < 1 || b->batch > kMostSequences)
    return fail(MOE_ERR_INVALID_ARG, "batch %d outside [1, %d]", b->batch, kMostSequences);
  if (b->tokens < 0 || b->tokens > d->max_tokens)
    return fail(MOE_ERR_INVALID_ARG, "tokens %d outside [0, max_tokens=%d]", b->tokens,
                d->max_tokens);
  if (!b->seq_lens_dev || !b->pages_dev || !aligned(b->seq_lens_dev, 4) ||
      !aligned(b->pages_dev, 4) || !aligned(b->cu_new_dev, 4))
    return fail(MOE_ERR_INVALID_ARG,
                "seq_lens_dev and pages_dev must be given, and arrays aligned to their element");
  if (b->pages_ld < 1) return fail(MOE_ERR_INVALID_ARG, "pages_ld %d below 1", b->pages_ld);
  if (b->cu_new_dev && (b->max_new < 1 || b->max_new > d->max_tokens))
    return fail(MOE_ERR_INVALID_ARG, "max_new %d outside [1, max_tokens=%d]", b->max_new,
                d->max_tokens);
  if (!b->cu_new_dev && b->tokens % b->batch)
    return fail(MOE_ERR_INVALID_ARG, "tokens %d is not a multiple of batch %d and cu_new is NULL",
                b->tokens, b->batch);
  if (b->shared_len < 0 || b->shared_len % d->page_size ||
      b->shared_len / d->page_size > b->pages_ld)
    return fail(MOE_ERR_INVALID_ARG,
                "shared_len %d must be a multiple of page_size %d within a row of the page table",
                b->shared_len, d->page_size);
  out->seq_lens = b->seq_lens_dev;
  out->cu_new = b->cu_new_dev;
  out->pages = b->pages_dev;
  out->batch = b->batch;
  out->tokens = b->tokens;
  out->n_each = b->tokens / b->batch;
  out->max_new = b->cu_new_dev ? b->max_new : out->n_each;
  out->pages_ld = b->pages_ld;
  out->shared_len = b->shared_len;
  return MOE_OK;
}

int32_t* flags_of(const moe_attention_dims& d, void* ws) {
  return reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + ws_layout(d).flags);
}

}  // namespace

extern "C" {

size_t moe_rope_table_size(const moe_rope_dims* d) {
  if (check_rope(d) != MOE_OK) return 0;
  return (size_t)(d->rotary_dim / 2) * sizeof(uint64_t);
}

moe_status moe_rope_prepare(const moe_rope_dims* d, void* table, size_t table_bytes,
                            void* stream) {
  return prepare_rope(d, nullptr, table, table_bytes, stream);
}

moe_status moe_rope_prepare_frequencies(const moe_rope_dims* d, const double* w, void* table,
                                        size_t table_bytes, void* stream) {
  if (!w) return fail(MOE_ERR_INVALID_ARG, "w is NULL");
  return prepare_rope(d, w, table, table_bytes, stream);
}

moe_status moe_rope(const moe_rope_dims* d, const void* table, const void* x, int64_t ldx,
                    const int32_t* positions, int64_t tokens, int32_t heads, void* out,
                    int64_t ldo, void* stream) {
  const moe_status s = check_rope(d);
  if (s) return s;
  if (tokens < 0 || tokens >= ((int64_t)1 << 31))
    return fail(MOE_ERR_INVALID_ARG, "tokens %lld outside [0, 2^31)", (long long)tokens);
  if (heads < 1 || heads > 65536)
    return fail(MOE_ERR_INVALID_ARG, "heads %d outside [1, 65536]", heads);
  if (tokens == 0) return MOE_OK;
  if (!given(table) || !given(x) || !given(out) || !positions || !aligned(positions, 4))
    return fail(MOE_ERR_INVALID_ARG,
                "table, x, out and positions must be given, 16-byte aligned (positions 4)");
  const int64_t row = (int64_t)heads * d->head_dim;
  if (!good_stride(ldx, row) || !good_stride(ldo, row))
    return fail(MOE_ERR_INVALID_ARG, "strides must be multiples of 8 and at least heads * head_dim");
  if (x == out && ldx != ldo)
    return fail(MOE_ERR_INVALID_ARG, "in place, both strides must be the same");
  RopeArgs a = {};
  set_rope(a, *d, table);
  a.positions = positions;
  a.q = {static_cast<const uint16_t*>(x), static_cast<uint16_t*>(out), ldx, ldo, heads};
  a.tokens = tokens;
  const cudaError_t e = launch_rope(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope kernel");
  return MOE_OK;
}

size_t moe_attention_workspace_size(const moe_attention_dims* d) {
  if (check_dims(d) != MOE_OK) return 0;
  return ws_layout(*d).total;
}

moe_status moe_attention_workspace_init(const moe_attention_dims* d, void* ws, size_t ws_bytes,
                                        void* stream) {
  const moe_status s = check_dims(d);
  if (s) return s;
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  const AttnWs L = ws_layout(*d);
  if (ws_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, needs %zu", ws_bytes,
                L.total);
  // only the flags and counters need a defined start
  const cudaError_t e = cudaMemsetAsync(ws, 0, L.stats, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "workspace clear");
  try {
    std::lock_guard<std::mutex> lk(g_mu);
    g_attention[ws] = AttnState{*d, MOE_SHARED_AUTO};
  } catch (...) {
    return fail(MOE_ERR_CUDA, "out of host memory for the workspace registry");
  }
  return MOE_OK;
}

moe_status moe_attention_set_shared(void* ws, int32_t mode) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (mode < MOE_SHARED_AUTO || mode > MOE_SHARED_NEVER)
    return fail(MOE_ERR_INVALID_ARG, "unknown mode %d", mode);
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_attention.find(ws);
  if (it == g_attention.end())
    return fail(MOE_ERR_WORKSPACE_MISMATCH, "workspace %p was not initialised", ws);
  it->second.shared = mode;
  return MOE_OK;
}

moe_status moe_kv_append(const moe_attention_dims* d, const moe_kv_batch* batch,
                         const moe_rope_dims* rope, const void* table, const int32_t* positions,
                         const void* q, int64_t ldq, void* q_out, int64_t ldqo, const void* k,
                         int64_t ldk, const void* v, int64_t ldv, void* k_cache, void* v_cache,
                         void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_dims(d);
  if (s) return s;
  int32_t shared;
  if ((s = check_ws(d, ws, ws_bytes, &shared))) return s;
  RopeArgs a = {};
  if ((s = check_batch(d, batch, &a.batch))) return s;
  if ((rope == nullptr) != (table == nullptr))
    return fail(MOE_ERR_INVALID_ARG, "rope and its table are given together or not at all");
  if ((q == nullptr) != (q_out == nullptr))
    return fail(MOE_ERR_INVALID_ARG, "q and q_out are given together or not at all");
  if (q && !rope) return fail(MOE_ERR_INVALID_ARG, "q is given without a rotation");
  if (rope) {
    if ((s = check_rope(rope))) return s;
    if (rope->head_dim != d->head_dim)
      return fail(MOE_ERR_INVALID_ARG, "the rotation's head_dim %d is not the cache's %d",
                  rope->head_dim, d->head_dim);
  }
  if (batch->tokens == 0) return MOE_OK;
  if (!given(k) || !given(v) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(table, 16) ||
      !aligned(positions, 4))
    return fail(MOE_ERR_INVALID_ARG, "k and v must be given and every tensor 16-byte aligned");
  if (!k_cache || !v_cache || !aligned(k_cache, 128) || !aligned(v_cache, 128))
    return fail(MOE_ERR_INVALID_ARG, "caches NULL or not 128-byte aligned");
  const int64_t kv_row = (int64_t)d->kv_heads * d->head_dim;
  const int64_t q_row = (int64_t)d->q_heads * d->head_dim;
  if (!good_stride(ldk, kv_row) || !good_stride(ldv, kv_row) ||
      (q && (!good_stride(ldq, q_row) || !good_stride(ldqo, q_row))))
    return fail(MOE_ERR_INVALID_ARG, "strides must be multiples of 8 and at least a row");
  if (q && q == q_out && ldq != ldqo)
    return fail(MOE_ERR_INVALID_ARG, "in place, both strides must be the same");
  if (rope) {
    set_rope(a, *rope, table);
  } else {   // whole pieces, none rotated
    a.head_dim = a.rotary_dim = d->head_dim;
    a.layout = MOE_ROPE_HALF;
  }
  a.positions = rope ? positions : nullptr;
  if (q)
    a.q = {static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), ldq, ldqo, d->q_heads};
  a.k = {static_cast<const uint16_t*>(k), nullptr, ldk, 0, d->kv_heads};
  a.v = {static_cast<const uint16_t*>(v), nullptr, ldv, 0, d->kv_heads};
  a.k_cache = static_cast<uint16_t*>(k_cache);
  a.v_cache = static_cast<uint16_t*>(v_cache);
  a.flags = flags_of(*d, ws);
  a.tokens = batch->tokens;
  a.num_pages = d->num_pages;
  a.page_shift = shift_of(d->page_size);
  const cudaError_t e = launch_kv_append(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "append kernel");
  return MOE_OK;
}

moe_status moe_attention(const moe_attention_dims* d, const moe_kv_batch* batch, const void* q,
                         int64_t ldq, const void* k_cache, const void* v_cache, float scale,
                         void* out, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                         void* stream) {
  moe_status s = check_dims(d);
  if (s) return s;
  int32_t shared = 0;
  if ((s = check_ws(d, ws, ws_bytes, &shared))) return s;
  AttnLaunch g = {};
  if ((s = check_batch(d, batch, &g.args.batch))) return s;
  const float scale_log2 = (float)(scale * 1.4426950408889634);
  if (!(scale > 0.f) || std::isinf(scale_log2))    // (a logit of 0 would become NaN)
    return fail(MOE_ERR_INVALID_ARG, "scale and scale * log2(e) must be finite and above 0");
  if (batch->tokens == 0) return MOE_OK;
  if (!given(q) || !given(out) || !aligned(lse, 4))
    return fail(MOE_ERR_INVALID_ARG, "q and out must be given and every tensor 16-byte aligned");
  if (!k_cache || !v_cache || !aligned(k_cache, 128) || !aligned(v_cache, 128))
    return fail(MOE_ERR_INVALID_ARG, "caches NULL or not 128-byte aligned");
  const int64_t row = (int64_t)d->q_heads * d->head_dim;
  if (!good_stride(ldq, row) || !good_stride(ldo, row))
    return fail(MOE_ERR_INVALID_ARG, "strides must be multiples of 8 and at least a row");
  AttnArgs& a = g.args;
  a.q = static_cast<const uint16_t*>(q);
  a.k_cache = static_cast<const uint16_t*>(k_cache);
  a.v_cache = static_cast<const uint16_t*>(v_cache);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.ldq = ldq;
  a.ldo = ldo;
  a.scale_log2 = scale_log2;
  a.q_heads = d->q_heads;
  a.kv_heads = d->kv_heads;
  a.group = d->q_heads / d->kv_heads;
  a.group_inv = (65536 + a.group - 1) / a.group;
  a.num_pages = d->num_pages;
  a.page_shift = shift_of(d->page_size);
  const AttnWs L = ws_layout(*d);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.flags = reinterpret_cast<int32_t*>(w + L.flags);
  a.counters = reinterpret_cast<int32_t*>(w + L.counters);
  a.cuts = reinterpret_cast<AttnCut*>(w + L.cuts);
  a.part_stats = reinterpret_cast<float2*>(w + L.stats);
  a.shared_stats = reinterpret_cast<float2*>(w + L.shared_stats);
  a.shared_parts = reinterpret_cast<float*>(w + L.shared_parts);
  a.parts = reinterpret_cast<float*>(w + L.parts);
  g.head_dim = d->head_dim;
  g.shared = batch->shared_len > 0 && batch->tokens <= d->max_shared_tokens ? shared
                                                                            : MOE_SHARED_NEVER;
  g.num_sms = moe_device_sm_count();
  if (g.num_sms <= 0 || cudaGetDevice(&g.device) != cudaSuccess)
    return fail(MOE_ERR_CUDA, "no CUDA device");
  const cudaError_t e = launch_attention(g, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "attention kernel");
  return MOE_OK;
}

moe_status moe_attention_check(void* ws, void* stream) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  moe_attention_dims dims;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    const auto it = g_attention.find(ws);
    if (it == g_attention.end())
      return fail(MOE_ERR_WORKSPACE_MISMATCH, "workspace %p was not initialised", ws);
    dims = it->second.dims;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t flag = 0;
  cudaError_t e = read_flags(&flag, ws, st);
  if (e != cudaSuccess) return cuda_fail(e, "flag read");
  // a call that gave up may have left its counters of parts behind
  const size_t clear = flag & kErrTimeout ? ws_layout(dims).cuts : sizeof(flag);
  if (flag && (e = clear_flags(ws, clear, st))) return cuda_fail(e, "flag clear");
  if (flag & kErrTimeout) return fail(MOE_ERR_TIMEOUT, "a device wait ran past its limit");
  if (flag & kErrPage)
    return fail(MOE_ERR_PAGE, "a token's page is outside its table or the cache");
  return MOE_OK;
}

}  // extern "C"
