// Linears with 4-bit weights and group scales (include/patch.h:
// patch_quantize4, patch_gemm4):  y[m][n] = sum_k x[m][k] (c[n][k] - 8) s[n][k / g].
#include "common.cuh"
#include "decoder.cuh"
#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace patch {

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
// a nanosecond and SM, so what counts next is instructions per code.  The codes
// become tensor-core operands (mma.sync m16n8k16, 16 rows of W by 8 tokens; W is
// the operand with 16 rows since 1 to 8 tokens would leave most of it empty)
// with 5 integer instructions for 8 codes: a code in the low bits of an fp16 is
// the subnormal c 2^-24 exactly (one AND for two codes), one 4 bits higher is
// c 2^-20, whose partner in X is stored divided by 16.  The offset 8 is taken
// off in the accumulator, which starts at -8 2^-24 sum x of its group.
//
// X is put in shared memory as fp16 in operand order (per 8 k: the pairs (0,4)
// (1,5) (2,6) (3,7)), every 128 elements of a token divided by a power of two
// that brings their largest into [2^14, 2^15): bf16 and fp16 values down to 2^-28
// of it stay exact, smaller ones are off by less than 2^-39 of it.
//
// A CTA takes 16 rows at a time; its warps take the blocks of 256 k in turn, 128
// bytes of each row, fetched by TMA into a ring of the warp's own (no registers
// held while bytes are on their way), and their sums are added in shared memory
// in warp order (deterministic).  A lane reads 4 bytes at a time, so that the
// four lanes of a row hold a quarter each of every group of 32.  Up to 8 tokens:
// 8 warps, two CTAs per SM; up to 16: 16 warps, one CTA, whose X is twice as
// large.  K beyond what fits is taken in slices, the sums kept in shared memory.
namespace g4 {

constexpr int kBlockK = 256, kStageBytes = 16 * 128;

struct Params {
  CUtensorMap codes;
  const void *X, *scales;
  void* Y;
  int32_t* status;
  int N, K, M, scale_dtype;
  int blocks, slice_blocks, n_rb, rb_chunk;  // 256-k blocks of K and of a slice; row blocks, those of a CTA at a time
};

template <int NT>
struct Cfg {
  static constexpr int kWarps = NT == 1 ? 8 : 16, kThreads = 32 * kWarps, kCtas = NT == 1 ? 2 : 1;
  static constexpr int kStages = NT == 1 ? 3 : 2;
  static constexpr int kBuffers = NT == 1 ? 2 : 1;       // of the warps' sums
  static constexpr int kSum = 128 * NT;                  // outputs of a row block
  static constexpr int kXBytes = NT == 1 ? 40960 : 132096;
  static constexpr int kAccBytes = 7168;                 // of sums kept over slices
  static constexpr int kRing = kWarps * kStages * kStageBytes;
};

// Behind the ring: X [M][slice_blocks * 32 + 4] units of 16 bytes, sums per group, scales per 128 k, the warps' sums.
struct Layout {
  int x, x_row, neg_sum, x_scale, reduce, acc, bars, bytes;
};
template <int NT, int GS>
__host__ __device__ inline Layout layout(int M, int slice_blocks, int rb_chunk, bool slices) {
  using C = Cfg<NT>;
  Layout l;
  l.x = C::kRing;
  l.x_row = slice_blocks * 32 + 4;  // 64 bytes beyond a multiple of 128: 8 tokens' pieces lie in different banks
  l.neg_sum = l.x + M * l.x_row * 16;
  l.x_scale = l.neg_sum + slice_blocks * (kBlockK >> GS) * 8 * NT * 4;
  l.reduce = l.x_scale + slice_blocks * 2 * 8 * NT * 4;
  l.acc = l.reduce + C::kBuffers * C::kWarps * C::kSum * 4;
  l.bars = l.acc + (slices ? rb_chunk * C::kSum * 4 : 0);
  l.bytes = l.bars + C::kWarps * C::kStages * 8 + 16;
  return l;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
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

// NT: 8-token tiles; GS: log2 of the group.
template <typename T, int NT, int GS>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, Cfg<NT>::kCtas) gemm4_kernel(const __grid_constant__ Params P) {
  using C = Cfg<NT>;
  constexpr int kWarps = C::kWarps, kStages = C::kStages;
  constexpr int kGroups = kBlockK >> GS;              // of a block: 8, 4, 2
  constexpr int kHeld = kGroups > 4 ? kGroups / 4 : 1;  // scales of a row that a lane loads
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, q = lane & 3;
  const bool slices = P.slice_blocks < P.blocks;
  const Layout L = layout<NT, GS>(P.M, P.slice_blocks, P.rb_chunk, slices);
  uint4* xs = reinterpret_cast<uint4*>(smem + L.x);
  float* neg_sum = reinterpret_cast<float*>(smem + L.neg_sum);
  float* x_scale = reinterpret_cast<float*>(smem + L.x_scale);
  float* reduce = reinterpret_cast<float*>(smem + L.reduce);
  float* acc_kept = reinterpret_cast<float*>(smem + L.acc);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars) + warp * kStages;
  int* abort_flag = reinterpret_cast<int*>(smem + L.bars + kWarps * kStages * 8);
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(bars + s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.codes)) : "memory");
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // This CTA's row blocks are blockIdx.x + i gridDim.x, rb_chunk of them at a time; for
  // these, slice after slice, the warp's blocks are warp, warp + kWarps, ... of the slice.
  // The cursor of what is fetched next runs ahead through the same order.
  struct Place {
    int chunk0, b0, i, blk;  // first row block of the chunk, first block of the slice, row block of the chunk, block of the slice
  };
  auto nb_of = [&](int b0) { return min(P.slice_blocks, P.blocks - b0); };
  auto valid = [&](const Place& p) { return p.chunk0 < P.n_rb; };
  // the next place with a block for this warp, from one whose block may lie behind the slice's last
  auto settle = [&](Place& p) {
    while (valid(p) && p.blk >= nb_of(p.b0)) {
      p.blk = warp;
      if (++p.i >= P.rb_chunk || p.chunk0 + p.i * int(gridDim.x) >= P.n_rb) {
        p.i = 0;
        p.b0 += P.slice_blocks;
        if (p.b0 >= P.blocks) {
          p.b0 = 0;
          p.chunk0 += P.rb_chunk * gridDim.x;
        }
      }
    }
  };
  const uint32_t ring = tc::smem_u32(smem) + warp * kStages * kStageBytes;
  Place fet = {int(blockIdx.x), 0, 0, warp};
  settle(fet);
  int issued = 0, done = 0;
  auto fetch = [&]() {
    if (!valid(fet)) return;
    const int st = issued % kStages;
    if (lane == 0) {
      tc::mbar_expect_tx(bars + st, kStageBytes);
      tc::tma_load_2d(smem + warp * kStages * kStageBytes + st * kStageBytes, &P.codes, bars + st,
                      (fet.b0 + fet.blk) * 128, (fet.chunk0 + fet.i * int(gridDim.x)) * 16);
    }
    ++issued;
    fet.blk += kWarps;
    settle(fet);
  };
  for (int s = 0; s < kStages; ++s) fetch();

  const int row_groups = P.K >> GS;
  // scales as stored, of rows 16 rb + n and + 8, this lane's groups of a block
  auto load_scales = [&](uint32_t (&s)[2][kHeld], int rb, int block) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = int64_t(min(16 * rb + n + 8 * h, P.N - 1)) * row_groups;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int g = block * kGroups + 4 * i + (q & (kGroups - 1));
        s[h][i] = 0;
        if (g < row_groups)
          s[h][i] = P.scale_dtype == PATCH_DTYPE_FP32 ? static_cast<const uint32_t*>(P.scales)[at + g]
                                                      : static_cast<const uint16_t*>(P.scales)[at + g];
      }
    }
  };
  auto scale_of = [&](uint32_t raw) {  // times 2^12
    const float s = P.scale_dtype == PATCH_DTYPE_BF16   ? __uint_as_float(raw << 16)
                    : P.scale_dtype == PATCH_DTYPE_FP16 ? __half2float(__ushort_as_half(uint16_t(raw)))
                                                        : __uint_as_float(raw);
    return s * 4096.0f;
  };
  uint32_t x_lane[NT];  // tokens beyond M read the last one's X: their columns are not stored
#pragma unroll
  for (int t = 0; t < NT; ++t) x_lane[t] = tc::smem_u32(xs) + uint32_t(min(8 * t + n, P.M - 1) * L.x_row + q) * 16;
  // the lane's words: row n, chunk c of 16 bytes at c ^ n (128-byte swizzle); row n + 8 is 1024 bytes on
  const uint32_t word0 = ring + n * 128 + n * 16 + 4 * q;

  int parity = 0;
  for (int chunk0 = blockIdx.x; chunk0 < P.n_rb; chunk0 += gridDim.x * P.rb_chunk) {
    for (int b0 = 0; b0 < P.blocks; b0 += P.slice_blocks) {
      const int nb = nb_of(b0);
      // ---- X of the slice: 16 threads per token and 128 k
      if (slices || chunk0 == int(blockIdx.x)) {
        __syncthreads();  // the last slice's is read
        for (int u = threadIdx.x; u < P.M * nb * 32; u += C::kThreads) {
          const int half_blk = (u >> 4) % (2 * nb), m = (u >> 4) / (2 * nb), p = u & 15;
          const int k = b0 * kBlockK + half_blk * 128 + 8 * p;
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
          const unsigned half = 0xFFFFu << (threadIdx.x & 16);  // these 16 threads leave the loop together
#pragma unroll
          for (int d = 8; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, d));
          const int e = max(int(__float_as_uint(amax) >> 23) - 127, -113);
          const float f = e == 128 ? 1.0f : pow2i(14 - e);
          uint4 v;
          v.x = pack_f16(x[0] * f, x[4] * f);
          v.y = pack_f16(x[1] * f * 0.0625f, x[5] * f * 0.0625f);
          v.z = pack_f16(x[2] * f, x[6] * f);
          v.w = pack_f16(x[3] * f * 0.0625f, x[7] * f * 0.0625f);
          xs[m * L.x_row + 16 * half_blk + p] = v;
          float sum = f16_sum(v.x) + f16_sum(v.z) + 16.0f * (f16_sum(v.y) + f16_sum(v.w));
          constexpr int kLanes = 1 << (GS - 3);  // of a group
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(half, sum, d);
          if ((p & (kLanes - 1)) == 0)
            neg_sum[((half_blk * 128 + 8 * p) >> GS) * 8 * NT + m] = sum * (-8.0f / 16777216.0f);
          if (p == 0) x_scale[half_blk * 8 * NT + m] = e == 128 ? 4096.0f : pow2i(e - 2);
        }
        __syncthreads();
      }

      for (int i_rb = 0; i_rb < P.rb_chunk; ++i_rb) {
        const int rb = chunk0 + i_rb * gridDim.x;
        if (rb >= P.n_rb) break;
        float y[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[t][i] = 0.0f;
        uint32_t raw[2][kHeld];
        if (warp < nb) load_scales(raw, rb, b0 + warp);
        for (int blk = warp; blk < nb; blk += kWarps) {
          const int st = done % kStages;
          const bool ok = tc::wait_bounded(bars + st, (done / kStages) & 1, abort_flag, 2000000000ull, P.status, false);
          ++done;
          if (!__all_sync(0xFFFFFFFFu, ok)) break;
          float s[2][kHeld];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kHeld; ++i) s[h][i] = scale_of(raw[h][i]);
          if (blk + kWarps < nb) load_scales(raw, rb, b0 + blk + kWarps);
          const uint32_t words = word0 + st * kStageBytes;
          const int x_at = blk * 512;
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {  // 128 k
            constexpr int kPer = 1 << (GS - 5);  // chunks of 32 k in a group
            float sum[NT][4], acc[NT][4];
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
              const int c = 4 * hb + c4;
              const uint32_t a0 = lds32(words ^ (c << 4)), a1 = lds32((words ^ (c << 4)) + 1024);
              const uint32_t r0 = a0 >> 8, r1 = a1 >> 8;
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (c4 % kPer == 0) {
                  const float2 neg = *reinterpret_cast<const float2*>(neg_sum + ((blk * 8 + c) / kPer * NT + t) * 8 + 2 * q);
                  acc[t][0] = acc[t][2] = neg.x;
                  acc[t][1] = acc[t][3] = neg.y;
                }
                const uint4 x = lds128(x_lane[t] + x_at + 64 * c);
                mma(acc[t], a0 & 0x000F000Fu, a1 & 0x000F000Fu, a0 & 0x00F000F0u, a1 & 0x00F000F0u, x.x, x.y);
                mma(acc[t], r0 & 0x000F000Fu, r1 & 0x000F000Fu, r0 & 0x00F000F0u, r1 & 0x00F000F0u, x.z, x.w);
              }
              if (c4 % kPer == kPer - 1) {  // the group's scales, from the lane that loaded them
                const int g = c / kPer;
                const float s0 = __shfl_sync(0xFFFFFFFFu, s[0][g >> 2], (lane & ~3) | (g & 3));
                const float s1 = __shfl_sync(0xFFFFFFFFu, s[1][g >> 2], (lane & ~3) | (g & 3));
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float f = i < 2 ? s0 : s1;
                    sum[t][i] = c4 == kPer - 1 ? acc[t][i] * f : fmaf(acc[t][i], f, sum[t][i]);
                  }
              }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float2 f = *reinterpret_cast<const float2*>(x_scale + ((blk * 2 + hb) * NT + t) * 8 + 2 * q);
#pragma unroll
              for (int i = 0; i < 4; ++i) y[t][i] = fmaf(sum[t][i], i & 1 ? f.y : f.x, y[t][i]);
            }
          }
          __syncwarp();  // every lane has read the stage
          fetch();
        }
        // ---- add the warps' sums: [warp][token][row]
        if (C::kBuffers == 1) __syncthreads();  // the last ones are read
        float* buf = reduce + parity * kWarps * C::kSum;
        if (C::kBuffers == 2) parity ^= 1;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            buf[warp * C::kSum + (8 * t + 2 * q + (i & 1)) * 16 + n + 8 * (i >> 1)] = y[t][i];
        __syncthreads();
        const int o = threadIdx.x;  // output: token o / 16, row o % 16
        if (o < C::kSum && (o >> 4) < P.M) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += buf[w * C::kSum + o];
          if (slices) {
            float* kept = acc_kept + i_rb * C::kSum + o;
            if (b0 > 0) v += *kept;
            *kept = v;
          }
          const int row = 16 * rb + (o & 15);
          if (b0 + nb == P.blocks && row < P.N) static_cast<T*>(P.Y)[int64_t(o >> 4) * P.N + row] = from_f32<T>(v);
        }
      }
    }
  }
  // after a timeout: let the copies in flight land before the shared memory goes
  for (; done < issued; ++done)
    tc::wait_bounded(bars + done % kStages, (done / kStages) & 1, abort_flag, 2000000000ull, P.status, true);
}

template <typename T, int NT, int GS>
static cudaError_t launch(Params P, int num_sms, cudaStream_t stream) {
  using C = Cfg<NT>;
  P.n_rb = (P.N + 15) / 16;
  P.blocks = (P.K + kBlockK - 1) / kBlockK;
  const int grid = P.n_rb < C::kCtas * num_sms ? P.n_rb : C::kCtas * num_sms;
  const int per_cta = (P.n_rb + grid - 1) / grid;
  // a slice: whole rounds of the warps, as many as fit
  const int fit = (C::kXBytes / P.M - 64) / (kBlockK * 2) / C::kWarps * C::kWarps;
  const bool slices = P.blocks > fit;
  P.slice_blocks = slices ? fit : P.blocks;
  P.rb_chunk = slices && per_cta > C::kAccBytes / (C::kSum * 4) ? C::kAccBytes / (C::kSum * 4) : per_cta;
  const Layout L = layout<NT, GS>(P.M, P.slice_blocks, P.rb_chunk, slices);
  auto kernel = gemm4_kernel<T, NT, GS>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L.bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(unsigned(grid)), dim3(C::kThreads), size_t(L.bytes), stream, P);
}

template <typename T, int NT>
static cudaError_t launch_group(const Params& P, int group, int num_sms, cudaStream_t stream) {
  if (group == 32) return launch<T, NT, 5>(P, num_sms, stream);
  if (group == 64) return launch<T, NT, 6>(P, num_sms, stream);
  return launch<T, NT, 7>(P, num_sms, stream);
}

}  // namespace g4

cudaError_t launch_gemm4(const void* X, int M, int dtype, const patch_weight4& W, void* Y, int32_t* status,
                         int num_sms, cudaStream_t stream) {
  g4::Params P = {};
  P.X = X;
  P.scales = W.scales;
  P.Y = Y;
  P.status = status;
  P.N = int(W.N);
  P.K = int(W.K);
  P.M = M;
  P.scale_dtype = W.scale_dtype;
  if (!make_map_rows_u8(&P.codes, W.codes, W.K / 2, W.N, 128, 16)) return cudaErrorInvalidValue;
  using BF = __nv_bfloat16;
  if (dtype == PATCH_DTYPE_BF16)
    return M <= 8 ? g4::launch_group<BF, 1>(P, W.group, num_sms, stream) : g4::launch_group<BF, 2>(P, W.group, num_sms, stream);
  return M <= 8 ? g4::launch_group<__half, 1>(P, W.group, num_sms, stream)
                : g4::launch_group<__half, 2>(P, W.group, num_sms, stream);
}

}  // namespace patch
