// Shared by the decoder-layer kernels beside the linears: rotary positions,
// the paged 8-bit cache, attention over it, 4-bit linears.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace patch {

// ---- host-side parameters

struct RopeTableParams {
  int kind;
  double log_base, factor, original, low, high, amplitude, ramp_lo, ramp_hi;
};

struct RopeHeads {  // strides in elements
  const void* src;
  void* dst;
  int64_t src_ts, src_hs, dst_ts, dst_hs;
  int heads;
};

struct RopeParams {
  RopeHeads q, k;
  const int32_t* positions;
  const float* table;
  int32_t* status;
  int64_t n_pos;
  int rot_units, units;  // units of a head: rotated ones first
  int heads_per_pass;    // set by the launcher
  float sign;                            // of the sines
};

cudaError_t launch_rope_table(int64_t n_pos, int half, const RopeTableParams& P, float* table, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_rope(const RopeParams& P, int64_t n_tokens, int dtype, int layout, int num_sms, cudaStream_t stream);

struct AppendParams {
  const void* x[2];  // k, v
  int64_t ts[2], hs[2];
  uint8_t* cache[2];
  float* scale[2];
  const int32_t *block_table, *past_lens, *cu_new;
  const float* table;
  int32_t* status;
  int64_t n_pages, max_pages, n_pos;
  int n_tokens, batch, kv_heads, page, rot_units;
  int heads_per_cta;  // set by the launcher
};
cudaError_t launch_kv8_append(AppendParams P, int head_dim, int dtype, int layout, int num_sms, cudaStream_t stream);

struct AttnParams {
  const void* q;
  void* out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *kv_lens, *cu_q;
  float* lse;
  int32_t* status;
  int64_t n_pages, max_pages, window;  // window 0: none
  int n_tokens, batch, heads, kv_heads, page, causal;
  float scale;
};
size_t attn_kv8_workspace_bytes(int64_t n_tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                int num_sms);
cudaError_t launch_attn_kv8(const AttnParams& P, int head_dim, int dtype, void* workspace, int num_sms,
                            uint64_t limit_ns, cudaStream_t stream);
// the form for many query rows per sequence and head (launch_attn_kv8 chooses)
size_t attn_kv8_rows_workspace_bytes(int64_t head_dim, int num_sms);
cudaError_t launch_attn_kv8_rows(const AttnParams& P, int head_dim, int dtype, void* workspace,
                                 int num_sms, uint64_t limit_ns, cudaStream_t stream);

cudaError_t launch_quantize4(const void* W, int dtype, const patch_weight4& out, int num_sms, cudaStream_t stream);
cudaError_t launch_gemm4(const void* X, int M, int dtype, const patch_weight4& W, void* Y, int32_t* status,
                         int num_sms, cudaStream_t stream);

// ---- device helpers

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }

// 16 aligned bytes of T to fp32 and back
template <typename T>
__device__ __forceinline__ void load16(const T* p, float* x) {
  constexpr int V = 16 / sizeof(T);
  const uint4 raw = *reinterpret_cast<const uint4*>(p);
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = to_f32(e[i]);
}
template <typename T>
__device__ __forceinline__ void store16(T* p, const float* x) {
  constexpr int V = 16 / sizeof(T);
  uint4 raw;
  T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = from_f32<T>(x[i]);
  *reinterpret_cast<uint4*>(p) = raw;
}

// Turn a unit's V pairs by V (cos, sin) pairs.  Interleaved: pairs (x[2i],
// x[2i+1]); halves: (x[i], x[V+i]).  Products and sums are rounded one by one
// (no fused multiply-add), so that every operator that rotates gives the same
// bits as the formula in plain fp32.
template <int V, bool kInterleaved>
__device__ __forceinline__ void rotate_unit(float (&x)[2 * V], const float (&cs)[2 * V], float sign) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : V + i;
    const float a = x[ia], b = x[ib], c = cs[2 * i], s = sign * cs[2 * i + 1];
    x[ia] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    x[ib] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  }
}

// 2^e for e in -126 .. 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Last index b of a non-decreasing sequence f(0) <= ... <= f(n) with f(b) <= x
// (f(0) <= x), found by a whole warp 32 places at a time: two rounds of loads
// for a thousand sequences.
template <typename F>
__device__ __forceinline__ int warp_find(int n, int64_t x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // answer in lo .. hi
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, i <= hi && f(i) <= x);
    const int c = __popc(le);  // the first c probes hold (f does not decrease)
    lo += c * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

}  // namespace patch
