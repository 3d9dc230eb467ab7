// Rotary positions: the table of angles and its application to query and key
// heads (include/patch.h: patch_rope_table, patch_rope).
//
// A pair (a, b) of a head turns by its position's angle t:
//   (a cos t - b sin t, b cos t + a sin t).
// The gradient is the transpose, the same with -sin t.
#include "common.cuh"
#include "decoder.cuh"
#include "kernels.cuh"

namespace patch {

// One thread per (position, pair).  Angles pass 1e5 radians at far positions,
// where fp32 has steps of 0.01: frequency, angle, sine and cosine are taken in
// 64 bits and rounded once.
__global__ void __launch_bounds__(256) rope_table_kernel(int64_t n, int half, RopeTableParams P,
                                                         float2* __restrict__ table) {
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t pos = i / half;
    const int j = int(i - pos * half);
    double w = exp(-P.log_base * (double(j) / half));
    if (P.kind == PATCH_ROPE_LINEAR) {
      w /= P.factor;
    } else if (P.kind == PATCH_ROPE_BANDS) {
      const double turns = P.original * w * 0.15915494309189535;  // c / wavelength; 1 / (2 pi)
      if (turns < P.low) {
        w /= P.factor;
      } else if (turns <= P.high) {
        const double s = (turns - P.low) / (P.high - P.low);
        w = (1.0 - s) * w / P.factor + s * w;
      }
    } else if (P.kind == PATCH_ROPE_YARN) {
      const double r = fmin(fmax((j - P.ramp_lo) / (P.ramp_hi - P.ramp_lo), 0.0), 1.0);
      w = w * (1.0 - r) + w / P.factor * r;
    }
    double s, c;
    sincos(double(pos) * w, &s, &c);
    table[i] = make_float2(float(c * P.amplitude), float(s * P.amplitude));
  }
}

cudaError_t launch_rope_table(int64_t n_pos, int half, const RopeTableParams& P, float* table, int num_sms,
                              cudaStream_t stream) {
  const int64_t n = n_pos * half;
  int64_t blocks = (n + 255) / 256;
  if (blocks > int64_t(num_sms) * 16) blocks = int64_t(num_sms) * 16;
  rope_table_kernel<<<unsigned(blocks), 256, 0, stream>>>(n, half, P, reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

// A unit is one thread's work on one head: V pairs (two 16-byte pieces, V = 8
// elements of 16 bits or 4 of 32 each) inside the rotated part, one 16-byte
// piece behind it.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeParams P) {
  constexpr int V = 16 / sizeof(T);
  const int64_t t = blockIdx.x;
  const int unit = threadIdx.x % P.units, sub = threadIdx.x / P.units;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // heads and positions come from earlier kernels
  const int32_t pos = P.positions[t];
  if (pos < 0 || pos >= P.n_pos) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && pos != -1) set_status(P.status, PATCH_DEV_BOUNDS);
    return;
  }
  const bool rotated = unit < P.rot_units;
  float cs[2 * V];
  if (rotated) {
    const float4* tab =
        reinterpret_cast<const float4*>(P.table + int64_t(pos) * (2 * V) * P.rot_units + unit * (2 * V));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) *reinterpret_cast<float4*>(cs + 4 * i) = __ldg(tab + i);
  }
  // element offsets of the unit's pieces
  const int d0 = !rotated ? 2 * V * P.rot_units + V * (unit - P.rot_units) : kInterleaved ? 2 * V * unit : V * unit;
  const int d1 = kInterleaved ? d0 + V : d0 + V * P.rot_units;
  for (int i = 0; i < P.heads_per_thread; ++i) {
    int h = (blockIdx.y * P.heads_per_thread + i) * P.heads_per_pass + sub;
    if (h >= P.q.heads + P.k.heads) break;
    const bool is_k = h >= P.q.heads;
    if (is_k) h -= P.q.heads;
    const T* src = static_cast<const T*>(is_k ? P.k.src : P.q.src) + t * (is_k ? P.k.src_ts : P.q.src_ts) +
                   h * (is_k ? P.k.src_hs : P.q.src_hs);
    T* dst = static_cast<T*>(is_k ? P.k.dst : P.q.dst) + t * (is_k ? P.k.dst_ts : P.q.dst_ts) +
             h * (is_k ? P.k.dst_hs : P.q.dst_hs);
    if (!rotated) {
      if (src != dst) *reinterpret_cast<uint4*>(dst + d0) = *reinterpret_cast<const uint4*>(src + d0);
      continue;
    }
    float x[2 * V];
    load16(src + d0, x);
    load16(src + d1, x + V);
    rotate_unit<V, kInterleaved>(x, cs, P.sign);
    store16(dst + d0, x);
    store16(dst + d1, x + V);
  }
}

cudaError_t launch_rope(RopeParams P, int64_t n_tokens, int dtype, int layout, int num_sms, cudaStream_t stream) {
  const int heads = P.q.heads + P.k.heads;
  P.heads_per_pass = P.units >= 128 ? 1 : 128 / P.units;
  if (P.heads_per_pass > heads) P.heads_per_pass = heads;
  const int passes = (heads + P.heads_per_pass - 1) / P.heads_per_pass;
  P.heads_per_thread = 1;
  const dim3 grid{unsigned(n_tokens), unsigned(passes)}, block{unsigned(P.heads_per_pass * P.units)};
  const bool il = layout == PATCH_ROPE_INTERLEAVED;
  if (dtype == PATCH_DTYPE_BF16)
    return launch_pdl(il ? rope_kernel<__nv_bfloat16, true> : rope_kernel<__nv_bfloat16, false>, grid, block, 0,
                      stream, P);
  if (dtype == PATCH_DTYPE_FP16)
    return launch_pdl(il ? rope_kernel<__half, true> : rope_kernel<__half, false>, grid, block, 0, stream, P);
  return launch_pdl(il ? rope_kernel<float, true> : rope_kernel<float, false>, grid, block, 0, stream, P);
}

}  // namespace patch
