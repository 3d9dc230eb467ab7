// Attention of new tokens over the paged 8-bit cache (include/patch.h:
// patch_attn_kv8).
//
// One CTA per query token and head; each of its warps takes every fourth key,
// keeps a running maximum m, sum l and output o of the softmax,
//   m' = max(m, s), l' = l e^(m - m') + e^(s - m'), o' = o e^(m - m') + e^(s - m') v,
// and the warps' states are joined at the end.
#include "common.cuh"
#include "decoder.cuh"
#include "kernels.cuh"

namespace patch {

__device__ __forceinline__ float attn_e4m3(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(byte), __NV_E4M3);
  return __half2float(__half(h));
}

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_kv8_kernel(const __grid_constant__ AttnParams P) {
  constexpr int E = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b = t;
  int64_t first = t, m_new = 1;
  if (P.cu_q) {
    const int32_t* cu = P.cu_q;
    b = warp_find(P.batch, t, [&](int i) { return int64_t(cu[i]); });
    if (b >= P.batch) return;
    first = cu[b];
    m_new = cu[b + 1] - first;
  }
  int64_t len = P.kv_lens[b];
  if (len < 0 || len > P.max_pages * P.page) {
    if (threadIdx.x == 0) set_status(P.status, PATCH_DEV_BOUNDS);
    len = len < 0 ? 0 : P.max_pages * P.page;
  }
  const int64_t pos = len - m_new + (t - first);
  const int64_t hi = P.causal ? min(len, pos + 1) : len;
  const int64_t lo = P.window > 0 ? max(int64_t(0), pos - P.window + 1) : 0;
  const int hk = h / (P.heads / P.kv_heads);
  const T* q = static_cast<const T*>(P.q) + t * P.q_ts + h * P.q_hs;
  float qv[E], o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qv[i] = to_f32(q[lane * E + i]) * P.scale;
    o[i] = 0.0f;
  }
  float mx = -INFINITY, l = 0.0f;
  for (int64_t p = lo + warp; p < hi; p += 4) {
    const int64_t phys = P.block_table[b * P.max_pages + p / P.page];
    if (phys < 0 || phys >= P.n_pages) {
      if (lane == 0) set_status(P.status, PATCH_DEV_BOUNDS);
    }
    const bool ok = phys >= 0 && phys < P.n_pages;
    const int64_t blk = ok ? phys * P.kv_heads + hk : 0;
    const int64_t at = (blk * P.page + p % P.page) * D + lane * E;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += ok ? qv[i] * attn_e4m3(P.k[at + i]) : 0.0f;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (ok) s *= P.k_scale[blk];
    const float m2 = fmaxf(mx, s), a = expf(mx - m2), e = expf(s - m2);
    const float ev = ok ? e * P.v_scale[blk] : 0.0f;
    l = l * a + e;
    mx = m2;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * a + (ok ? ev * attn_e4m3(P.v[at + i]) : 0.0f);
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) {
    sm[warp] = mx;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[i];
  __syncthreads();
  if (warp) return;
  float M = -INFINITY, L = 0.0f;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w]);
  float f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = M == -INFINITY ? 0.0f : expf(sm[w] - M);
    L += sl[w] * f[w];
  }
  T* out = static_cast<T*>(P.out) + t * P.o_ts + h * P.o_hs;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float v = 0.0f;
    for (int w = 0; w < 4; ++w) v += so[w][lane * E + i] * f[w];
    out[lane * E + i] = from_f32<T>(M == -INFINITY ? 0.0f : v / L);
  }
  if (P.lse && lane == 0) P.lse[int64_t(t) * P.heads + h] = M == -INFINITY ? -INFINITY : M + logf(L);
}

size_t attn_kv8_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int) { return 0; }

cudaError_t launch_attn_kv8(const AttnParams& P, int head_dim, int dtype, void*, int, uint64_t, cudaStream_t stream) {
  const dim3 grid(unsigned(P.n_tokens), unsigned(P.heads));
  if (dtype == PATCH_DTYPE_BF16)
    return launch_pdl(head_dim == 128 ? attn_kv8_kernel<__nv_bfloat16, 128> : attn_kv8_kernel<__nv_bfloat16, 64>, grid,
                      dim3(128), 0, stream, P);
  return launch_pdl(head_dim == 128 ? attn_kv8_kernel<__half, 128> : attn_kv8_kernel<__half, 64>, grid, dim3(128), 0,
                    stream, P);
}

}  // namespace patch
