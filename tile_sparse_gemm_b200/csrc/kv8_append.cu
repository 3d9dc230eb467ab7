// New keys and values into the paged 8-bit cache, keys rotated on the way
// (include/patch.h: patch_kv8_append).
//
// One CTA per touched page, head and tensor (k or v): its new tokens stay in
// registers (fp32) between the pass that finds their largest magnitude and the
// one that rounds them, so each input is read once and each output written
// once.  The scale is a power of two: e4m3 keeps its relative precision under
// any scale, scaling is exact, and a page whose scale grows as tokens arrive is
// stored again without a second rounding.
#include "common.cuh"
#include "decoder.cuh"
#include "kernels.cuh"

namespace patch {

constexpr int kScaleExpMin = -100, kScaleExpMax = 119;

// The least e in kScaleExpMin .. kScaleExpMax with amax <= 448 * 2^e (448 =
// 1.75 * 2^8), from the bits of a finite amax >= 0.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int x = int(amax_bits >> 23) - 127;  // amax = m * 2^x, m in [1, 2); subnormals clamp below
  const int e = (amax_bits & 0x7FFFFFu) <= 0x600000u ? x - 8 : x - 7;
  return min(max(e, kScaleExpMin), kScaleExpMax);
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(byte), __NV_E4M3);
  return __half2float(__half(h));
}

// kUnits units of 16 elements per thread: a rotated unit is 8 pairs (two
// 8-element pieces), one behind the rotated part 16 elements in a row.
template <typename T, int D, bool kInterleaved, int kThreads, int kUnits>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const __grid_constant__ AppendParams P) {
  constexpr int kPerToken = D / 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Item -> (sequence, page of it).  Sequence b owns the items from
  // cu[b] / page + 2 b on: at least as many as the pages its tokens touch.
  const int64_t item = blockIdx.x;
  int b, j;
  int64_t row0, n;
  if (P.cu_new) {
    const int32_t* cu = P.cu_new;
    const int page = P.page;
    b = warp_find(P.batch, item, [&](int i) { return int64_t(cu[i]) / page + 2 * i; });
    if (b >= P.batch) return;
    row0 = cu[b];
    n = min(int64_t(cu[b + 1]), int64_t(P.n_tokens)) - row0;
    if (row0 < 0) return;
    j = int(item - (row0 / page + 2 * b));
  } else {
    b = int(item);
    j = 0;
    row0 = b;
    n = 1;
  }
  const int64_t past = P.past_lens[b];
  const int64_t page_no = past / P.page + j;
  const int64_t begin = max(past, page_no * P.page), end = min(past + n, (page_no + 1) * P.page);
  if (begin >= end) return;
  const int h = blockIdx.y, which = blockIdx.z;
  const int64_t phys = past >= 0 && page_no < P.max_pages ? P.block_table[b * P.max_pages + page_no] : -1;
  const bool turn = which == 0 && P.rot_units > 0;
  if (phys < 0 || phys >= P.n_pages || (turn && end > P.n_pos)) {
    if (threadIdx.x == 0) set_status(P.status, PATCH_DEV_BOUNDS);
    return;
  }
  const int off = int(begin - page_no * P.page), count = int(end - begin);
  const T* src = static_cast<const T*>(P.x[which]) + (row0 + begin - past) * P.ts[which] + h * P.hs[which];

  float x[kUnits][16];
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int idx = u * kThreads + threadIdx.x, tok = idx / kPerToken, unit = idx % kPerToken;
    if (tok >= count) continue;
    const T* row = src + tok * P.ts[which];
    const bool pair = turn && unit < P.rot_units;
    const int d0 = pair && !kInterleaved ? 8 * unit : 16 * unit;
    const int d1 = pair && !kInterleaved ? d0 + 8 * P.rot_units : d0 + 8;
    load16(row + d0, x[u]);
    load16(row + d1, x[u] + 8);
    if (pair) {
      float cs[16];
      const float4* tab =
          reinterpret_cast<const float4*>(P.table + (begin + tok) * (16 * P.rot_units) + 16 * unit);
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(cs + 4 * i) = __ldg(tab + i);
      rotate_unit<8, kInterleaved>(x[u], cs, 1.0f);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t m = __float_as_uint(x[u][i]) & 0x7FFFFFFFu;
      if (m < 0x7F800000u) amax = max(amax, m);  // infinities and NaN do not set the scale
    }
  }
  // largest magnitude over the CTA
  __shared__ uint32_t part[kThreads / 32];
  amax = __reduce_max_sync(0xFFFFFFFFu, amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) amax = max(amax, part[i]);
  float* scale_at = P.scale[which] + phys * P.kv_heads + h;
  float scale = pow2i(scale_exponent(amax));
  const float held = off > 0 ? *scale_at : 0.0f;
  scale = fmaxf(scale, held);
  const float inv = 1.0f / scale;  // exact: a power of two
  __syncthreads();                 // everyone has read the old scale
  if (threadIdx.x == 0) *scale_at = scale;

  uint8_t* dst = P.cache[which] + (phys * P.kv_heads + h) * (int64_t(P.page) * D);
  if (off > 0 && scale > held) {  // store the tokens the page holds again
    const float f = held * inv;
    for (int i = threadIdx.x; i < off * (D / 16); i += kThreads) {
      uint4 w = reinterpret_cast<uint4*>(dst)[i];
      uint32_t* e = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        e[q] = pack_e4m3x4(e4m3_to_f32(e[q] & 255) * f, e4m3_to_f32((e[q] >> 8) & 255) * f,
                           e4m3_to_f32((e[q] >> 16) & 255) * f, e4m3_to_f32(e[q] >> 24) * f);
      reinterpret_cast<uint4*>(dst)[i] = w;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int idx = u * kThreads + threadIdx.x, tok = idx / kPerToken, unit = idx % kPerToken;
    if (tok >= count) continue;
    const bool pair = turn && unit < P.rot_units;
    const int d0 = pair && !kInterleaved ? 8 * unit : 16 * unit;
    const int d1 = pair && !kInterleaved ? d0 + 8 * P.rot_units : d0 + 8;
    uint8_t* row = dst + (off + tok) * D;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack_e4m3x4(x[u][4 * i] * inv, x[u][4 * i + 1] * inv, x[u][4 * i + 2] * inv, x[u][4 * i + 3] * inv);
    *reinterpret_cast<uint2*>(row + d0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + d1) = make_uint2(w[2], w[3]);
  }
}

template <typename T, int D, bool kInterleaved>
static cudaError_t launch_append(const AppendParams& P, cudaStream_t stream) {
  const int64_t items = P.cu_new ? P.n_tokens / P.page + 2 * int64_t(P.batch) : P.batch;
  const dim3 grid(unsigned(items), unsigned(P.kv_heads), 2);
  const int units = P.page * (D / 16);  // of a full page: 64 ... 1024
  if (units <= 64) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 64, 1>, grid, dim3(64), 0, stream, P);
  if (units <= 128) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 128, 1>, grid, dim3(128), 0, stream, P);
  if (units <= 256) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 256, 1>, grid, dim3(256), 0, stream, P);
  if (units <= 512) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 256, 2>, grid, dim3(256), 0, stream, P);
  return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 256, 4>, grid, dim3(256), 0, stream, P);
}

cudaError_t launch_kv8_append(const AppendParams& P, int head_dim, int dtype, int layout, cudaStream_t stream) {
  const bool il = layout == PATCH_ROPE_INTERLEAVED && P.rot_units > 0;
  if (dtype == PATCH_DTYPE_BF16) {
    if (head_dim == 128)
      return il ? launch_append<__nv_bfloat16, 128, true>(P, stream) : launch_append<__nv_bfloat16, 128, false>(P, stream);
    return il ? launch_append<__nv_bfloat16, 64, true>(P, stream) : launch_append<__nv_bfloat16, 64, false>(P, stream);
  }
  if (head_dim == 128) return il ? launch_append<__half, 128, true>(P, stream) : launch_append<__half, 128, false>(P, stream);
  return il ? launch_append<__half, 64, true>(P, stream) : launch_append<__half, 64, false>(P, stream);
}

}  // namespace patch
