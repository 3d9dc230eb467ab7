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

// ---- Y = X W^T for up to 16 tokens.
//
// Bound by the bytes of the codes: 6.5 TB/s are 13 codes a picosecond, about 90
// a nanosecond and SM, so what counts is instructions per code.  The codes
// become tensor-core operands (mma.sync m16n8k16, 16 rows of W by 8 tokens; W is
// the operand with 16 rows since 1 to 8 tokens would leave most of it empty)
// with 5 integer instructions for 8 codes: a code in the low bits of an fp16 is
// the subnormal c 2^-24 exactly (one AND for two codes), one 4 bits higher is
// c 2^-20, whose partner in X is stored divided by 16.  The offset 8 is taken
// off in the accumulator, which starts at -8 2^-24 sum x of its group.
//
// X is put in shared memory once per CTA as fp16 in operand order (per 8 k: the
// pairs (0,4) (1,5) (2,6) (3,7)), every 128 elements of a token divided by a
// power of two that brings their largest into [2^14, 2^15): bf16 and fp16 values
// down to 2^-28 of it stay exact, smaller ones are off by less than 2^-39 of it.
//
// A CTA takes 16 rows at a time, its 8 warps every eighth 128-element block of
// them (64 bytes of each row, 512 adjacent bytes per CTA), and their sums are
// added in shared memory in warp order (deterministic).  Groups of 32 and 64:
// a lane's 16 bytes are one group of 32, so the four lanes of a row exchange
// words (4 shuffles for 32 codes) until each holds a quarter of every group.
// K beyond what fits is taken in slices, with the sums kept in shared memory.
namespace g4 {

constexpr int kWarps = 8, kThreads = 256;
constexpr int kBatch = 4;           // blocks a warp has in flight
constexpr int kSliceBytes = 73728;  // of X and its sums: two CTAs per SM
constexpr int kAccBytes = 28672;    // of sums kept over slices

struct Params {
  const void *X, *codes, *scales;
  void* Y;
  int N, K, M, group_shift, scale_dtype;
  int blocks, slice_blocks, n_rb, rb_chunk;  // 128-element blocks of K and of a slice; row blocks, those of a CTA at a time
};

// Shared memory: X [M][slice_blocks * 16 + 4] units of 16 bytes, sums and scales per group and block, partial sums.
struct Layout {
  int x_row, neg_sum, x_scale, reduce, acc, bytes;
};
__host__ __device__ inline Layout layout(int M, int nt, int slice_blocks, int group_shift, int rb_chunk, bool slices) {
  Layout l;
  l.x_row = slice_blocks * 16 + 4;  // 64 bytes beyond a multiple of 128: 8 tokens' pieces lie in different banks
  l.neg_sum = M * l.x_row * 16;
  l.x_scale = l.neg_sum + (slice_blocks << (7 - group_shift)) * 8 * nt * 4;
  l.reduce = l.x_scale + slice_blocks * 8 * nt * 4;
  l.acc = l.reduce + 2 * kWarps * 128 * nt * 4;
  l.bytes = l.acc + (slices ? rb_chunk * 128 * nt * 4 : 0);
  return l;
}

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_sum(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return f.x + f.y;
}
// 4 x 4 words over the four lanes of a row: lane q's word j becomes lane j's word q
__device__ __forceinline__ void exchange(uint4& v, int q) {
  const bool hi = q & 2, odd = q & 1;
  uint32_t s0 = hi ? v.x : v.z, s1 = hi ? v.y : v.w;
  s0 = __shfl_xor_sync(0xFFFFFFFFu, s0, 2);
  s1 = __shfl_xor_sync(0xFFFFFFFFu, s1, 2);
  uint32_t a = hi ? s0 : v.x, b = hi ? s1 : v.y, c = hi ? v.z : s0, d = hi ? v.w : s1;
  uint32_t t0 = odd ? a : b, t1 = odd ? c : d;
  t0 = __shfl_xor_sync(0xFFFFFFFFu, t0, 1);
  t1 = __shfl_xor_sync(0xFFFFFFFFu, t1, 1);
  v.x = odd ? t0 : a;
  v.y = odd ? b : t0;
  v.z = odd ? t1 : c;
  v.w = odd ? d : t1;
}

// NT: 8-token tiles; kWide: groups of 128 (no exchange).
template <typename T, int NT, bool kWide>
__global__ void __launch_bounds__(kThreads, 2) gemm4_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, q = lane & 3;
  const bool slices = P.slice_blocks < P.blocks;
  const Layout L = layout(P.M, NT, P.slice_blocks, P.group_shift, P.rb_chunk, slices);
  uint4* xs = reinterpret_cast<uint4*>(smem);
  float* neg_sum = reinterpret_cast<float*>(smem + L.neg_sum);
  float* x_scale = reinterpret_cast<float*>(smem + L.x_scale);
  float* reduce = reinterpret_cast<float*>(smem + L.reduce);
  float* acc_kept = reinterpret_cast<float*>(smem + L.acc);
  const uint8_t* codes = static_cast<const uint8_t*>(P.codes);
  const int64_t row_bytes = P.K / 2, row_groups = P.K >> P.group_shift;
  // tokens beyond M read the last one's X (their columns are not stored)
  const uint4* x_lane[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) x_lane[t] = xs + min(8 * t + n, P.M - 1) * L.x_row + q;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  struct Batch {
    uint4 w[kBatch][2];
    float s[kBatch][2];
  };
  int parity = 0;
  for (int rb0 = blockIdx.x; rb0 < P.n_rb; rb0 += gridDim.x * P.rb_chunk) {
    for (int b0 = 0; b0 < P.blocks; b0 += P.slice_blocks) {
      const int nb = min(P.slice_blocks, P.blocks - b0);  // blocks of this slice
      // Rows 16 rb + n and + 8, blocks b0 + blk + 8 i: codes, and the scale of this lane's group times 2^12
      auto load = [&](Batch& B, int rb, int blk) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int k = (b0 + blk + kWarps * i) * 128 + 32 * q;
          const bool in = blk + kWarps * i < nb && k < P.K;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t row = min(16 * rb + n + 8 * h, P.N - 1);
            B.w[i][h] = make_uint4(0, 0, 0, 0);
            B.s[i][h] = 0.0f;
            if (in) {
              B.w[i][h] = ldg_stream(codes + row * row_bytes + (k >> 1));
              B.s[i][h] = scale4_at(P.scales, P.scale_dtype, row * row_groups + (k >> P.group_shift)) * 4096.0f;
            }
          }
        }
      };
      Batch cur, nxt;
      if (warp < nb) load(cur, rb0, warp);

      // ---- X of the slice: 16 threads per token and block
      __syncthreads();  // the last slice's is read
      for (int u = threadIdx.x; u < P.M * nb * 16; u += kThreads) {
        const int blk = (u >> 4) % nb, m = (u >> 4) / nb, p = u & 15;
        const int k = (b0 + blk) * 128 + 8 * p;
        float x[8];
        if (k < P.K) {
          load16(static_cast<const T*>(P.X) + int64_t(m) * P.K + k, x);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
        const unsigned half = 0xFFFFu << (threadIdx.x & 16);  // the block's 16 threads leave the loop together
#pragma unroll
        for (int d = 8; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, d));
        const int e = max(int(__float_as_uint(amax) >> 23) - 127, -113);
        const float f = e == 128 ? 1.0f : pow2i(14 - e);
        uint4 v;
        v.x = pack_f16(x[0] * f, x[4] * f);
        v.y = pack_f16(x[1] * f * 0.0625f, x[5] * f * 0.0625f);
        v.z = pack_f16(x[2] * f, x[6] * f);
        v.w = pack_f16(x[3] * f * 0.0625f, x[7] * f * 0.0625f);
        xs[m * L.x_row + 16 * blk + (kWide ? (p & 3) * 4 + (p >> 2) : p)] = v;
        float sum = f16_sum(v.x) + f16_sum(v.z) + 16.0f * (f16_sum(v.y) + f16_sum(v.w));
        const int lanes = 1 << (P.group_shift - 3);  // of a group
        for (int d = 1; d < lanes; d <<= 1) sum += __shfl_xor_sync(half, sum, d);
        if ((p & (lanes - 1)) == 0)
          neg_sum[(((blk * 128 + 8 * p) >> P.group_shift) * NT + (m >> 3)) * 8 + (m & 7)] = sum * (-8.0f / 16777216.0f);
        if (p == 0) x_scale[(blk * NT + (m >> 3)) * 8 + (m & 7)] = e == 128 ? 4096.0f : pow2i(e - 2);
      }
      __syncthreads();

      for (int i_rb = 0; i_rb < P.rb_chunk; ++i_rb) {
        const int rb = rb0 + i_rb * gridDim.x;
        if (rb >= P.n_rb) break;
        float y[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[t][i] = 0.0f;
        for (int blk = warp; blk < nb; blk += kWarps * kBatch) {
          // what comes next: this row block's next blocks, or the next row block's first
          const int nblk = blk + kWarps * kBatch;
          if (nblk < nb)
            load(nxt, rb, nblk);
          else if (i_rb + 1 < P.rb_chunk && rb + int(gridDim.x) < P.n_rb)
            load(nxt, rb + gridDim.x, warp);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int b = blk + kWarps * i;
            if (b >= nb) break;
            uint4 w0 = cur.w[i][0], w1 = cur.w[i][1];
            if (!kWide) {
              exchange(w0, q);
              exchange(w1, q);
            }
            const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
            float c[NT][4], sum[NT][4];
            const int per_group = 4 >> (7 - P.group_shift);  // words of a lane in a group
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // word j of both rows: 8 codes each, two k steps
              const uint32_t r0 = a0[j] >> 8, r1 = a1[j] >> 8;
              if (kWide ? j == 0 : (j & (per_group - 1)) == 0) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  const int g = ((b * 128 + 32 * j) >> P.group_shift) * NT + t;
                  const float2 s = *reinterpret_cast<const float2*>(neg_sum + g * 8 + 2 * q);
                  c[t][0] = c[t][2] = s.x;
                  c[t][1] = c[t][3] = s.y;
                }
              }
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint4 x = x_lane[t][16 * b + 4 * j];
                mma(c[t], a0[j] & 0x000F000Fu, a1[j] & 0x000F000Fu, a0[j] & 0x00F000F0u, a1[j] & 0x00F000F0u, x.x, x.y);
                mma(c[t], r0 & 0x000F000Fu, r1 & 0x000F000Fu, r0 & 0x00F000F0u, r1 & 0x00F000F0u, x.z, x.w);
              }
              if (kWide ? j == 3 : (j & (per_group - 1)) == per_group - 1) {
                // the group's scale is with the lane that loaded its first code
                const float s0 = kWide ? cur.s[i][0] : __shfl_sync(0xFFFFFFFFu, cur.s[i][0], (lane & ~3) | j);
                const float s1 = kWide ? cur.s[i][1] : __shfl_sync(0xFFFFFFFFu, cur.s[i][1], (lane & ~3) | j);
                const bool first = kWide || j == per_group - 1;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  sum[t][0] = first ? c[t][0] * s0 : fmaf(c[t][0], s0, sum[t][0]);
                  sum[t][1] = first ? c[t][1] * s0 : fmaf(c[t][1], s0, sum[t][1]);
                  sum[t][2] = first ? c[t][2] * s1 : fmaf(c[t][2], s1, sum[t][2]);
                  sum[t][3] = first ? c[t][3] * s1 : fmaf(c[t][3], s1, sum[t][3]);
                }
              }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float2 f = *reinterpret_cast<const float2*>(x_scale + (b * NT + t) * 8 + 2 * q);
              y[t][0] = fmaf(sum[t][0], f.x, y[t][0]);
              y[t][1] = fmaf(sum[t][1], f.y, y[t][1]);
              y[t][2] = fmaf(sum[t][2], f.x, y[t][2]);
              y[t][3] = fmaf(sum[t][3], f.y, y[t][3]);
            }
          }
          cur = nxt;
        }
        // ---- add the warps' sums: [warp][token][row], two buffers in turn
        float* buf = reduce + parity * kWarps * 128 * NT;
        parity ^= 1;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            buf[warp * 128 * NT + (8 * t + 2 * q + (i & 1)) * 16 + n + 8 * (i >> 1)] = y[t][i];
        __syncthreads();
        const int o = threadIdx.x;  // output: token o / 16, row o % 16
        if (o < 128 * NT && (o >> 4) < P.M) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += buf[w * 128 * NT + o];
          if (slices) {
            float* kept = acc_kept + i_rb * 128 * NT + o;
            if (b0 > 0) v += *kept;
            *kept = v;
          }
          const int row = 16 * rb + (o & 15);
          if (b0 + nb == P.blocks && row < P.N) static_cast<T*>(P.Y)[int64_t(o >> 4) * P.N + row] = from_f32<T>(v);
        }
      }
    }
  }
}

template <typename T, int NT>
static cudaError_t launch(Params P, int num_sms, cudaStream_t stream) {
  P.n_rb = (P.N + 15) / 16;
  P.blocks = (P.K + 127) / 128;
  const int grid = P.n_rb < 2 * num_sms ? P.n_rb : 2 * num_sms;
  const int per_cta = (P.n_rb + grid - 1) / grid;
  // a slice: whole rounds of the warps, as many as fit
  const Layout one = layout(P.M, NT, 8, P.group_shift, 0, false);
  const int round = one.reduce - P.M * 64;  // bytes of 8 blocks
  int rounds = (kSliceBytes - P.M * 64) / round;
  if (rounds * 8 >= P.blocks) {
    P.slice_blocks = P.blocks;
    P.rb_chunk = per_cta;
  } else {
    P.slice_blocks = rounds * 8;
    P.rb_chunk = kAccBytes / (128 * NT * 4);
    if (P.rb_chunk > per_cta) P.rb_chunk = per_cta;
  }
  const Layout L = layout(P.M, NT, P.slice_blocks, P.group_shift, P.rb_chunk, P.slice_blocks < P.blocks);
  auto kernel = P.group_shift == 7 ? gemm4_kernel<T, NT, true> : gemm4_kernel<T, NT, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L.bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(unsigned(grid)), dim3(kThreads), size_t(L.bytes), stream, P);
}

}  // namespace g4

cudaError_t launch_gemm4(const void* X, int M, int dtype, const patch_weight4& W, void* Y, int num_sms,
                         cudaStream_t stream) {
  g4::Params P = {};
  P.X = X;
  P.codes = W.codes;
  P.scales = W.scales;
  P.Y = Y;
  P.N = int(W.N);
  P.K = int(W.K);
  P.M = M;
  P.group_shift = W.group == 32 ? 5 : W.group == 64 ? 6 : 7;
  P.scale_dtype = W.scale_dtype;
  if (dtype == PATCH_DTYPE_BF16)
    return M <= 8 ? g4::launch<__nv_bfloat16, 1>(P, num_sms, stream) : g4::launch<__nv_bfloat16, 2>(P, num_sms, stream);
  return M <= 8 ? g4::launch<__half, 1>(P, num_sms, stream) : g4::launch<__half, 2>(P, num_sms, stream);
}

}  // namespace patch
