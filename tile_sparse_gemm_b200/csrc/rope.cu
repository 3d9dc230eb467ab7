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

// Bandwidth-bound: each element is read and written once, but a token's row of
// the table (64 bytes per 32 bytes of a head) would pass through L1 again for
// every head.  A unit is one thread's work on one head: V pairs (two 16-byte
// pieces, V = 8 elements of 16 bits or 4 of 32 each) inside the rotated part, one
// 16-byte piece behind it.  A thread keeps its unit's V angles in registers and
// takes kHeads heads with them, their loads under way together.  8192 tokens of
// 32 + 32 heads of 128 in bf16, 268 MB: 45 us, 5.9 TB/s.
template <typename T, bool kInterleaved, int kHeads>
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
  // element offsets of the unit's pieces
  const int d0 = !rotated ? 2 * V * P.rot_units + V * (unit - P.rot_units) : kInterleaved ? 2 * V * unit : V * unit;
  const int d1 = kInterleaved ? d0 + V : d0 + V * P.rot_units;
  const T* src[kHeads];
  T* dst[kHeads];
  uint4 x0[kHeads], x1[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int head = (blockIdx.y * kHeads + i) * P.heads_per_pass + sub;
    src[i] = nullptr;
    if (head >= P.q.heads + P.k.heads) continue;
    const bool is_k = head >= P.q.heads;
    const RopeHeads& H = is_k ? P.k : P.q;
    const int h = is_k ? head - P.q.heads : head;
    src[i] = static_cast<const T*>(H.src) + t * H.src_ts + h * H.src_hs;
    dst[i] = static_cast<T*>(H.dst) + t * H.dst_ts + h * H.dst_hs;
    x0[i] = *reinterpret_cast<const uint4*>(src[i] + d0);
    if (rotated) x1[i] = *reinterpret_cast<const uint4*>(src[i] + d1);
  }
  float cs[2 * V];
  if (rotated) {
    const float4* tab =
        reinterpret_cast<const float4*>(P.table + int64_t(pos) * (2 * V) * P.rot_units + unit * (2 * V));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) *reinterpret_cast<float4*>(cs + 4 * i) = __ldg(tab + i);
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (!src[i]) continue;
    if (!rotated) {
      if (src[i] != dst[i]) *reinterpret_cast<uint4*>(dst[i] + d0) = x0[i];
      continue;
    }
    float x[2 * V];
    load16(reinterpret_cast<const T*>(&x0[i]), x);
    load16(reinterpret_cast<const T*>(&x1[i]), x + V);
    rotate_unit<V, kInterleaved>(x, cs, P.sign);
    store16(dst[i] + d0, x);
    store16(dst[i] + d1, x + V);
  }
}

template <typename T>
static cudaError_t launch_rope_type(RopeParams P, int64_t n_tokens, bool interleaved, int num_sms, cudaStream_t stream) {
  const int heads = P.q.heads + P.k.heads;
  P.heads_per_pass = P.units >= 128 ? 1 : 128 / P.units;
  if (P.heads_per_pass > heads) P.heads_per_pass = heads;
  const int passes = (heads + P.heads_per_pass - 1) / P.heads_per_pass;
  const dim3 block{unsigned(P.heads_per_pass * P.units)};
  // Four heads a thread where that still leaves more than a CTA per SM, else one (40 heads of 128: 16 tokens
  // 1.5 us with one, 1.8 with four; 128 tokens 1.8, 1.9; 256 tokens 2.4, 2.2; 2048 tokens 8.1, 6.7).
  if (passes > 1 && n_tokens * ((passes + 3) / 4) * 2 >= 3 * int64_t(num_sms)) {
    const dim3 grid{unsigned(n_tokens), unsigned((passes + 3) / 4)};
    return launch_pdl(interleaved ? rope_kernel<T, true, 4> : rope_kernel<T, false, 4>, grid, block, 0, stream, P);
  }
  const dim3 grid{unsigned(n_tokens), unsigned(passes)};
  return launch_pdl(interleaved ? rope_kernel<T, true, 1> : rope_kernel<T, false, 1>, grid, block, 0, stream, P);
}

cudaError_t launch_rope(const RopeParams& P, int64_t n_tokens, int dtype, int layout, int num_sms, cudaStream_t stream) {
  const bool il = layout == PATCH_ROPE_INTERLEAVED;
  if (dtype == PATCH_DTYPE_BF16) return launch_rope_type<__nv_bfloat16>(P, n_tokens, il, num_sms, stream);
  if (dtype == PATCH_DTYPE_FP16) return launch_rope_type<__half>(P, n_tokens, il, num_sms, stream);
  return launch_rope_type<float>(P, n_tokens, il, num_sms, stream);
}

}  // namespace patch
