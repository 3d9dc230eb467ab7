// Linears with 4-bit weights and group scales (include/patch.h:
// patch_quantize4, patch_gemm4):  y[m][n] = sum_k x[m][k] (c[n][k] - 8) s[n][k / g].
#include "common.cuh"
#include "decoder.cuh"
#include "kernels.cuh"

namespace patch {

__device__ __forceinline__ float scale4_at(const void* scales, int dtype, int64_t i) {
  if (dtype == PATCH_DTYPE_BF16) return to_f32(static_cast<const __nv_bfloat16*>(scales)[i]);
  if (dtype == PATCH_DTYPE_FP16) return to_f32(static_cast<const __half*>(scales)[i]);
  return static_cast<const float*>(scales)[i];
}

// One thread per 8 weights (4 bytes of codes); the threads of a group (4, 8 or
// 16 neighbouring lanes) find its largest magnitude together.  Bandwidth-bound.
template <typename T>
__global__ void __launch_bounds__(256) quantize4_kernel(const T* __restrict__ W, int64_t n8, int lanes, int sdtype,
                                                        uint32_t* __restrict__ codes, void* __restrict__ scales) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t stride = int64_t(gridDim.x) * blockDim.x;
  // n8 is a multiple of `lanes`, so a group's lanes leave the loop together
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n8; i += stride) {
    float x[8];
    if constexpr (sizeof(T) == 2) {
      load16(W + 8 * i, x);
    } else {
      load16(W + 8 * i, x);
      load16(W + 8 * i + 4, x + 4);
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(x[j]);
      if (a < INFINITY) amax = fmaxf(amax, a);
    }
    const unsigned group = ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
    for (int d = lanes >> 1; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, d));
    const float s0 = __fdiv_rn(amax, 7.0f);
    const int64_t gi = i / lanes;
    const bool lead = (threadIdx.x & (lanes - 1)) == 0;
    float s = s0;
    if (sdtype == PATCH_DTYPE_BF16) {
      const __nv_bfloat16 r = __float2bfloat16_rn(s0);
      s = to_f32(r);
      if (lead) static_cast<__nv_bfloat16*>(scales)[gi] = r;
    } else if (sdtype == PATCH_DTYPE_FP16) {
      const __half r = __float2half_rn(s0);
      s = to_f32(r);
      if (lead) static_cast<__half*>(scales)[gi] = r;
    } else if (lead) {
      static_cast<float*>(scales)[gi] = s0;
    }
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = s > 0.0f ? __fdiv_rn(x[j], s) : 0.0f;
      const int c = q != q ? 0 : int(rintf(fminf(fmaxf(q, -8.0f), 7.0f)));
      w |= uint32_t(c + 8) << (4 * j);
    }
    codes[i] = w;
  }
}

cudaError_t launch_quantize4(const void* W, int dtype, const patch_weight4& out, int num_sms, cudaStream_t stream) {
  const int64_t n8 = out.N * out.K / 8;
  int64_t blocks = (n8 + 255) / 256;
  if (blocks > int64_t(num_sms) * 16) blocks = int64_t(num_sms) * 16;
  uint32_t* codes = static_cast<uint32_t*>(const_cast<void*>(out.codes));
  void* scales = const_cast<void*>(out.scales);
  const int lanes = out.group / 8;
  const dim3 grid{unsigned(blocks)};
  if (dtype == PATCH_DTYPE_BF16)
    return launch_pdl(quantize4_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream,
                      static_cast<const __nv_bfloat16*>(W), n8, lanes, int(out.scale_dtype), codes, scales);
  if (dtype == PATCH_DTYPE_FP16)
    return launch_pdl(quantize4_kernel<__half>, grid, dim3(256), 0, stream, static_cast<const __half*>(W), n8, lanes,
                      int(out.scale_dtype), codes, scales);
  return launch_pdl(quantize4_kernel<float>, grid, dim3(256), 0, stream, static_cast<const float*>(W), n8, lanes,
                    int(out.scale_dtype), codes, scales);
}

// One warp per output row, lanes along k (8 weights of 4 bytes each at a time).
template <typename T>
__global__ void __launch_bounds__(256) gemm4_kernel(const T* __restrict__ X, int M, patch_weight4 W,
                                                    T* __restrict__ Y) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t n = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (n >= W.N) return;
  float acc[16];
#pragma unroll
  for (int m = 0; m < 16; ++m) acc[m] = 0.0f;
  const uint32_t* row = static_cast<const uint32_t*>(W.codes) + n * (W.K / 8);
  for (int64_t i = lane; i < W.K / 8; i += 32) {
    const uint32_t c = row[i];
    const float s = scale4_at(W.scales, W.scale_dtype, n * (W.K / W.group) + 8 * i / W.group);
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = (float((c >> (4 * j)) & 15) - 8.0f) * s;
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      if (m < M) {
        float x[8];
        load16(X + m * W.K + 8 * i, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[m] = fmaf(w[j], x[j], acc[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 16; ++m) {
    if (m < M) {
      float v = acc[m];
#pragma unroll
      for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
      if (lane == 0) Y[m * W.N + n] = from_f32<T>(v);
    }
  }
}

cudaError_t launch_gemm4(const void* X, int M, int dtype, const patch_weight4& W, void* Y, int, cudaStream_t stream) {
  const dim3 grid(unsigned((W.N + 7) / 8));
  if (dtype == PATCH_DTYPE_BF16)
    return launch_pdl(gemm4_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, static_cast<const __nv_bfloat16*>(X), M,
                      W, static_cast<__nv_bfloat16*>(Y));
  return launch_pdl(gemm4_kernel<__half>, grid, dim3(256), 0, stream, static_cast<const __half*>(X), M, W,
                    static_cast<__half*>(Y));
}

}  // namespace patch
