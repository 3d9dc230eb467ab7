// C ABI of the decoder-layer operators beside the linears (include/patch.h):
// argument checks and dispatch of rotary positions, the paged 8-bit cache,
// attention over it and 4-bit linears.
#include <cmath>

#include "decoder.cuh"
#include "host_checks.cuh"
#include "kernels.cuh"

using namespace patch;

namespace {

constexpr int64_t kMaxCount = int64_t(1) << 30;  // tokens, positions, sequences

int elem_size(int dtype) { return dtype == PATCH_DTYPE_FP32 ? 4 : 2; }
bool half_type(int dtype) { return dtype == PATCH_DTYPE_BF16 || dtype == PATCH_DTYPE_FP16; }

// Strides of an axis of one element do not matter and may be anything.
patch_status_t check_heads(const patch_heads* x, int64_t n_tokens, int dtype) {
  if (!x->data || x->heads < 1) return PATCH_ERR_INVALID_ARG;
  if (x->heads > 65535) return PATCH_ERR_SHAPE;
  const int64_t v = 16 / elem_size(dtype);
  if (!aligned16(x->data) || (n_tokens > 1 && x->token_stride % v) || (x->heads > 1 && x->head_stride % v))
    return PATCH_ERR_ALIGN;
  return PATCH_OK;
}

patch_status_t check_cache(const patch_kv8_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return PATCH_ERR_INVALID_ARG;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return PATCH_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return PATCH_ERR_SHAPE;
  if (c->n_pages < 1 || c->kv_heads < 1 || c->kv_heads > 65535 || c->n_pages >= (int64_t(1) << 31) / c->kv_heads)
    return PATCH_ERR_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale)) return PATCH_ERR_ALIGN;
  return PATCH_OK;
}

bool positive(double x) { return x > 0.0 && std::isfinite(x); }

}  // namespace

extern "C" {

patch_status_t patch_rope_table(int64_t n_pos, int64_t rot_dim, const patch_rope_config* c, float* table,
                                void* stream) {
  if (!c || !table) return PATCH_ERR_INVALID_ARG;
  if (!(c->base > 1.0) || !std::isfinite(c->base) || c->kind < PATCH_ROPE_PLAIN || c->kind > PATCH_ROPE_YARN ||
      !std::isfinite(c->amplitude))
    return PATCH_ERR_INVALID_ARG;
  if (c->kind != PATCH_ROPE_PLAIN && !positive(c->factor)) return PATCH_ERR_INVALID_ARG;
  if (c->kind >= PATCH_ROPE_BANDS && (!positive(c->original_positions) || !positive(c->low_freq) ||
                                      !positive(c->high_freq) || !(c->low_freq < c->high_freq)))
    return PATCH_ERR_INVALID_ARG;
  if (n_pos < 1 || n_pos > kMaxCount || rot_dim < 2 || rot_dim > 1024 || rot_dim % 2) return PATCH_ERR_SHAPE;
  if (!aligned16(table)) return PATCH_ERR_ALIGN;
  int sms = 0;
  const patch_status_t st = device_sms(&sms);
  if (st != PATCH_OK) return st;
  RopeTableParams P = {c->kind, std::log(c->base), c->factor, c->original_positions, c->low_freq, c->high_freq,
                       c->amplitude, 0.0, 1.0};
  if (c->kind == PATCH_ROPE_YARN) {
    // the (real-valued) pair index whose wavelength makes `turns` turns in original_positions
    auto pair_of = [&](double turns) {
      return double(rot_dim) * std::log(c->original_positions / (turns * 6.283185307179586)) / (2.0 * P.log_base);
    };
    P.ramp_lo = std::fmax(std::floor(pair_of(c->high_freq)), 0.0);
    P.ramp_hi = std::fmin(std::ceil(pair_of(c->low_freq)), double(rot_dim - 1));
    if (P.ramp_hi - P.ramp_lo < 0.001) P.ramp_hi = P.ramp_lo + 0.001;  // a step, not a division by zero
  }
  return launch_rope_table(n_pos, int(rot_dim / 2), P, table, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PATCH_OK
             : PATCH_ERR_CUDA;
}

patch_status_t patch_rope(const patch_heads* q, const patch_heads* k, const patch_heads* q_out,
                          const patch_heads* k_out, int64_t n_tokens, int64_t head_dim, int dtype,
                          const int32_t* positions, const float* table, int64_t n_pos, int64_t rot_dim, int layout,
                          int backward, int32_t* dev_status, void* stream) {
  if (!q || !q_out || (k != nullptr) != (k_out != nullptr) || n_tokens < 0) return PATCH_ERR_INVALID_ARG;
  if (dtype != PATCH_DTYPE_FP32 && !half_type(dtype)) return PATCH_ERR_INVALID_ARG;
  if (layout != PATCH_ROPE_HALF && layout != PATCH_ROPE_INTERLEAVED) return PATCH_ERR_INVALID_ARG;
  if (q->heads != q_out->heads || (k && k->heads != k_out->heads)) return PATCH_ERR_INVALID_ARG;
  if (q->heads > 65535 || (k && k->heads > 65535 - q->heads)) return PATCH_ERR_SHAPE;  // a launch's grid
  if (n_tokens > kMaxCount || n_pos < 1 || n_pos > kMaxCount || head_dim < 16 || head_dim > 1024 || head_dim % 8 ||
      rot_dim < 16 || rot_dim > head_dim || rot_dim % 16)
    return PATCH_ERR_SHAPE;
  if (n_tokens == 0) return PATCH_OK;
  if (!positions || !table) return PATCH_ERR_INVALID_ARG;
  if (!aligned16(table) || reinterpret_cast<uintptr_t>(positions) % 4) return PATCH_ERR_ALIGN;
  for (const patch_heads* x : {q, q_out, k, k_out}) {
    if (!x) continue;
    const patch_status_t st = check_heads(x, n_tokens, dtype);
    if (st != PATCH_OK) return st;
  }
  int sms = 0;
  const patch_status_t st = device_sms(&sms);
  if (st != PATCH_OK) return st;
  auto heads = [](const patch_heads* x, const patch_heads* y) {
    return RopeHeads{x->data, y->data, x->token_stride, x->head_stride, y->token_stride, y->head_stride, int(x->heads)};
  };
  RopeParams P = {};
  P.q = heads(q, q_out);
  if (k) P.k = heads(k, k_out);
  P.positions = positions;
  P.table = table;
  P.status = dev_status;
  P.n_pos = n_pos;
  const int v = 16 / elem_size(dtype);
  P.rot_units = int(rot_dim / (2 * v));
  P.units = P.rot_units + int((head_dim - rot_dim) / v);
  P.sign = backward ? -1.0f : 1.0f;
  return launch_rope(P, n_tokens, dtype, layout, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PATCH_OK
             : PATCH_ERR_CUDA;
}

patch_status_t patch_kv8_append(const patch_heads* k, const patch_heads* v, int64_t n_tokens, int dtype,
                                const patch_kv8_cache* cache, const int32_t* block_table, int64_t max_pages,
                                const int32_t* past_lens, const int32_t* cu_new, int64_t batch, const float* table,
                                int64_t n_pos, int64_t rot_dim, int layout, int32_t* dev_status, void* stream) {
  if (!k || !v || n_tokens < 0 || batch < 0 || !half_type(dtype)) return PATCH_ERR_INVALID_ARG;
  if (layout != PATCH_ROPE_HALF && layout != PATCH_ROPE_INTERLEAVED) return PATCH_ERR_INVALID_ARG;
  if (!cu_new && n_tokens != batch) return PATCH_ERR_INVALID_ARG;
  patch_status_t st = check_cache(cache);
  if (st != PATCH_OK) return st;
  if (k->heads != cache->kv_heads || v->heads != cache->kv_heads) return PATCH_ERR_INVALID_ARG;
  if (n_tokens > kMaxCount || batch > kMaxCount / 4 || max_pages < 0 || max_pages > kMaxCount) return PATCH_ERR_SHAPE;
  if (table ? (rot_dim < 16 || rot_dim > cache->head_dim || rot_dim % 16 || n_pos < 1 || n_pos > kMaxCount) : rot_dim != 0)
    return PATCH_ERR_SHAPE;
  if (n_tokens == 0 || batch == 0) return PATCH_OK;
  if (!block_table || !past_lens) return PATCH_ERR_INVALID_ARG;
  for (const patch_heads* x : {k, v}) {
    st = check_heads(x, n_tokens, dtype);
    if (st != PATCH_OK) return st;
  }
  if ((table && !aligned16(table)) || reinterpret_cast<uintptr_t>(block_table) % 4 ||
      reinterpret_cast<uintptr_t>(past_lens) % 4 || (cu_new && reinterpret_cast<uintptr_t>(cu_new) % 4))
    return PATCH_ERR_ALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != PATCH_OK) return st;
  AppendParams P = {};
  const patch_heads* x[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    P.x[i] = x[i]->data;
    P.ts[i] = x[i]->token_stride;
    P.hs[i] = x[i]->head_stride;
    P.cache[i] = static_cast<uint8_t*>(i ? cache->v : cache->k);
    P.scale[i] = i ? cache->v_scale : cache->k_scale;
  }
  P.block_table = block_table;
  P.past_lens = past_lens;
  P.cu_new = cu_new;
  P.table = table;
  P.status = dev_status;
  P.n_pages = cache->n_pages;
  P.max_pages = max_pages;
  P.n_pos = n_pos;
  P.n_tokens = int(n_tokens);
  P.batch = int(batch);
  P.kv_heads = int(cache->kv_heads);
  P.page = int(cache->page);
  P.rot_units = table ? int(rot_dim / 16) : 0;
  return launch_kv8_append(P, int(cache->head_dim), dtype, layout, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PATCH_OK
             : PATCH_ERR_CUDA;
}

static patch_status_t check_attn_sizes(int64_t n_tokens, int64_t batch, int64_t q_heads, const patch_kv8_cache* cache) {
  if (n_tokens < 0 || batch < 0 || q_heads < 1) return PATCH_ERR_INVALID_ARG;
  const patch_status_t st = check_cache(cache);
  if (st != PATCH_OK) return st;
  if (q_heads % cache->kv_heads || q_heads / cache->kv_heads > 16 || q_heads > 65535) return PATCH_ERR_SHAPE;
  if (n_tokens > kMaxCount / 16 || batch > kMaxCount / 4) return PATCH_ERR_SHAPE;
  return PATCH_OK;
}

patch_status_t patch_attn_kv8_workspace_size(int64_t n_tokens, int64_t batch, int64_t q_heads,
                                             const patch_kv8_cache* cache, size_t* bytes) {
  if (!bytes) return PATCH_ERR_INVALID_ARG;
  patch_status_t st = check_attn_sizes(n_tokens, batch, q_heads, cache);
  if (st != PATCH_OK) return st;
  *bytes = 0;
  if (n_tokens == 0 || batch == 0) return PATCH_OK;
  int sms = 0;
  st = device_sms(&sms);
  if (st != PATCH_OK) return st;
  *bytes = attn_kv8_workspace_bytes(n_tokens, batch, q_heads, cache->kv_heads, cache->head_dim, sms);
  return PATCH_OK;
}

patch_status_t patch_attn_kv8(const patch_heads* q, int64_t n_tokens, int dtype, const patch_kv8_cache* cache,
                              const int32_t* block_table, int64_t max_pages, const int32_t* kv_lens,
                              const int32_t* cu_q, int64_t batch, float scale, int causal, int64_t window,
                              const patch_heads* out, float* lse, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream, uint64_t wait_limit_us) {
  if (!q || !out || !half_type(dtype) || !std::isfinite(scale) || window < 0 || (window > 0 && !causal))
    return PATCH_ERR_INVALID_ARG;
  patch_status_t st = check_attn_sizes(n_tokens, batch, q->heads, cache);
  if (st != PATCH_OK) return st;
  if (out->heads != q->heads || (!cu_q && n_tokens != batch)) return PATCH_ERR_INVALID_ARG;
  if (max_pages < 0 || max_pages > kMaxCount / cache->page) return PATCH_ERR_SHAPE;
  if (n_tokens == 0 || batch == 0) return PATCH_OK;
  if (!kv_lens || (!block_table && max_pages > 0)) return PATCH_ERR_INVALID_ARG;
  for (const patch_heads* x : {q, out}) {
    st = check_heads(x, n_tokens, dtype);
    if (st != PATCH_OK) return st;
  }
  if (reinterpret_cast<uintptr_t>(block_table) % 4 || reinterpret_cast<uintptr_t>(kv_lens) % 4 ||
      reinterpret_cast<uintptr_t>(cu_q) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
    return PATCH_ERR_ALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != PATCH_OK) return st;
  const size_t need = attn_kv8_workspace_bytes(n_tokens, batch, q->heads, cache->kv_heads, cache->head_dim, sms);
  if (need && (!workspace || workspace_bytes < need || !aligned16(workspace))) return PATCH_ERR_WORKSPACE;
  AttnParams P = {};
  P.q = q->data;
  P.out = out->data;
  P.q_ts = q->token_stride;
  P.q_hs = q->head_stride;
  P.o_ts = out->token_stride;
  P.o_hs = out->head_stride;
  P.k = static_cast<const uint8_t*>(cache->k);
  P.v = static_cast<const uint8_t*>(cache->v);
  P.k_scale = cache->k_scale;
  P.v_scale = cache->v_scale;
  P.block_table = block_table;
  P.kv_lens = kv_lens;
  P.cu_q = cu_q;
  P.lse = lse;
  P.status = dev_status;
  P.n_pages = cache->n_pages;
  P.max_pages = max_pages;
  P.window = window;
  P.n_tokens = int(n_tokens);
  P.batch = int(batch);
  P.heads = int(q->heads);
  P.kv_heads = int(cache->kv_heads);
  P.page = int(cache->page);
  P.causal = causal ? 1 : 0;
  P.scale = scale;
  const uint64_t limit_ns = (wait_limit_us ? wait_limit_us : 2000000ull) * 1000ull;
  return launch_attn_kv8(P, int(cache->head_dim), dtype, workspace, sms, limit_ns,
                         static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PATCH_OK
             : PATCH_ERR_CUDA;
}

static patch_status_t check_weight4(const patch_weight4* W) {
  if (!W || !W->codes || !W->scales) return PATCH_ERR_INVALID_ARG;
  if (W->group != 32 && W->group != 64 && W->group != 128) return PATCH_ERR_INVALID_ARG;
  if (!half_type(W->scale_dtype)) return PATCH_ERR_INVALID_ARG;
  if (W->N < 1 || W->K < 1 || W->K % W->group || W->N > kMaxCount || W->K > kMaxCount)
    return PATCH_ERR_SHAPE;
  if (!aligned16(W->codes) || !aligned16(W->scales)) return PATCH_ERR_ALIGN;
  return PATCH_OK;
}

patch_status_t patch_quantize4(const void* W, int dtype, const patch_weight4* out, void* stream) {
  if (!W || (dtype != PATCH_DTYPE_FP32 && !half_type(dtype))) return PATCH_ERR_INVALID_ARG;
  patch_status_t st = check_weight4(out);
  if (st != PATCH_OK) return st;
  if (!aligned16(W)) return PATCH_ERR_ALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != PATCH_OK) return st;
  return launch_quantize4(W, dtype, *out, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PATCH_OK
                                                                                               : PATCH_ERR_CUDA;
}

patch_status_t patch_gemm4(const void* X, int64_t M, int dtype, const patch_weight4* W, void* Y,
                           int32_t* dev_status, void* stream) {
  if (M < 0 || M > PATCH_DECODE_MAX_M || !half_type(dtype)) return PATCH_ERR_INVALID_ARG;
  patch_status_t st = check_weight4(W);
  if (st != PATCH_OK) return st;
  if (M == 0) return PATCH_OK;
  if (!X || !Y) return PATCH_ERR_INVALID_ARG;
  if (!aligned16(X) || reinterpret_cast<uintptr_t>(Y) % 2) return PATCH_ERR_ALIGN;
  int sms = 0;
  st = device_sms(&sms);
  if (st != PATCH_OK) return st;
  return launch_gemm4(X, int(M), dtype, *W, Y, dev_status, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PATCH_OK
             : PATCH_ERR_CUDA;
}

}  // extern "C"
