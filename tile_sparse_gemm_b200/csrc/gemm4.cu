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
    float s;
    if (sdtype == PATCH_DTYPE_BF16) {
      const __nv_bfloat16 r = __float2bfloat16_rn(s0);
      s = to_f32(r);
      if (lead) static_cast<__nv_bfloat16*>(scales)[gi] = r;
    } else {
      const __half r = __float2half_rn(fminf(s0, 65504.0f));  // fp16's largest: an infinite scale has no codes
      s = to_f32(r);
      if (lead) static_cast<__half*>(scales)[gi] = r;
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
// off in the accumulator, which starts at -8 2^-24 sum x of its group: the same
// product with the code -8 everywhere, taken once per CTA.
//
// X is put in shared memory as fp16 in operand order (per 8 k: the pairs (0,4)
// (1,5) (2,6) (3,7)), every 128 elements of a token divided by a power of two
// that brings their largest into [2^14, 2^15): bf16 and fp16 values down to 2^-24 of
// it stay exact, smaller ones are off by at most 2^-35 of it (2^-39 where the partner
// is not divided by 16).
//
// A CTA has an equal share of the row tiles of 16 and takes two at a time (a row
// group); its warps take the group's blocks of 256 k in turn, 128 bytes of each
// row, fetched by TMA into a ring of the warp's own (no registers held while bytes
// are on their way), and their sums are added in shared memory in warp order
// (deterministic).  A lane reads 4 bytes at a time, so that the four lanes of a
// row hold a quarter each of every group of 32.  Up to 8 tokens: 8 warps, each
// with both tiles (an operand of X serves two), two CTAs per SM where their shared
// memory allows it and that is faster.  Up to 16: 8 warps for either tile, one CTA
// per SM.  K beyond what X's place holds is taken in slices, the sums of four row
// groups kept meanwhile by the threads that add them.
//
// Every CTA prepares all of X that it needs, which for few rows or many tokens takes
// longer than the products.  So up to 8 CTAs may form a cluster: they share row groups,
// each has its part of K (and of X), and their sums are added through distributed shared
// memory, in the order of the parts.
//
// Measured: 128000 x 4096, 1 token, group 32: 68 us (codes and scales, 295 MB, at 4.4
// TB/s; fetching alone takes 46 us, the rest is what the integer and tensor instructions
// of a block take beyond that; 63 us in a row of launches); 14336 x 4096, 16 tokens: 23 us, of which 5 prepare X in
// every CTA and 11 are the products; 4096 x 4096, 1 token: 5.0 us, mostly latency.
namespace g4 {

constexpr int kBlockK = 256, kBoxBytes = 16 * 128;

struct Params {
  CUtensorMap codes;
  const void *X, *scales;
  void* Y;
  int32_t* status;
  int N, K, M, dtype;
  int blocks, slice_blocks, tiles, chunk;  // 256-k blocks of K and of a slice; row tiles; row groups of a CTA at a time
  int parts;                               // of K: CTAs of a cluster
};

constexpr int kKWarps = 8;  // warps that share a row tile's blocks of k
constexpr int kGroupRows = 32;
constexpr int kMaxParts = 8;  // the portable size of a cluster
constexpr int kSmemOfSm = 228 * 1024, kSmemReserved = 1024;  // shared memory; what each CTA takes beside its own
constexpr int kMostBlocks = kSmemOfSm / (kBlockK * 2);  // of X in an SM, of one token
constexpr int kKept = 4;  // row groups whose sums are kept over slices, in registers

template <int NT>
struct Cfg {
  static constexpr int kRowWarps = NT, kWarps = kKWarps * kRowWarps, kThreads = 32 * kWarps, kCtas = NT == 1 ? 2 : 1;
  static constexpr int MT = 2 / kRowWarps;                // row tiles of a warp
  static constexpr int kStages = 2;
  static constexpr int kStageBytes = MT * kBoxBytes;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
};

// Behind the ring: X [M][slice_blocks * 32] units of 16 bytes, sums per group, scales per 128 k, the warps' sums
// [warp][token][row of the group], a ring of scales beside that of codes.
struct Layout {
  int x, x_row, neg_sum, x_scale, reduce, scales, bars, bytes;
};
template <int NT, int GS>
__host__ __device__ inline Layout layout(int M, int slice_blocks) {
  using C = Cfg<NT>;
  Layout l;
  l.x = C::kRing;
  l.x_row = slice_blocks * 32;
  l.neg_sum = l.x + M * l.x_row * 16;
  l.x_scale = l.neg_sum + slice_blocks * (kBlockK >> GS) * 8 * NT * 4;
  l.reduce = l.x_scale + slice_blocks * 2 * 8 * NT * 4;
  l.scales = l.reduce + kKWarps * M * kGroupRows * 4;
  l.bars = l.scales + C::kWarps * C::kStages * C::MT * 16 * (kBlockK >> GS) * 2;
  l.bytes = l.bars + C::kWarps * C::kStages * 8 + 16;
  return l;
}

__device__ __forceinline__ void store_y(uint16_t* at, float v, int dtype) {
  *at = dtype == PATCH_DTYPE_BF16 ? f32_to_bf16_rne(v) : __half_as_ushort(__float2half_rn(v));
}
// d = a b + c
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float load_of_cta(uint32_t addr, int rank) {  // the word at this shared address of a cluster's CTA
  uint32_t there;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
  return v;
}
// S: type of the scales; NT: 8-token tiles; GS: log2 of the group; kParts: K is split over a cluster; kVec: K is a
// multiple of kBlockK, so that a block's scales of a row are one aligned piece.  The last two are kernels of their own:
// in a row of launches 128000 x 4096 takes 63 us, with kVec's checks in one kernel for both 64, with kParts' 66.
template <typename S, int NT, int GS, bool kParts, bool kVec>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, Cfg<NT>::kCtas) gemm4_kernel(const __grid_constant__ Params P) {
  using C = Cfg<NT>;
  constexpr int kWarps = C::kWarps, kStages = C::kStages, MT = C::MT;
  constexpr int kGroups = kBlockK >> GS;  // of a block: 8, 4, 2
  constexpr int kScaleRow = 2 * kGroups;  // bytes of their scales
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, q = lane & 3;
  const int kw = warp % kKWarps, rw = warp / kKWarps;
  const int parts = kParts ? P.parts : 1, part = kParts ? int(blockIdx.x) % parts : 0;  // clusters are CTAs in a row
  const int kb0 = int(int64_t(P.blocks) * part / parts);                     // this CTA's blocks of K: kb0 on
  const int blocks = int(int64_t(P.blocks) * (part + 1) / parts) - kb0;
  const bool slices = !kParts && P.slice_blocks < blocks;
  const Layout L = layout<NT, GS>(P.M, P.slice_blocks);
  uint4* xs = reinterpret_cast<uint4*>(smem + L.x);
  float* neg_sum = reinterpret_cast<float*>(smem + L.neg_sum);
  float* x_scale = reinterpret_cast<float*>(smem + L.x_scale);
  float* reduce = reinterpret_cast<float*>(smem + L.reduce);
  uint8_t* scales = smem + L.scales + warp * kStages * MT * 16 * kScaleRow;
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

  // This CTA's row tiles are tile0 .. tile1 - 1, two of them a row group, `chunk` groups at a
  // time; for these, slice after slice, the warp's blocks are kw, kw + kKWarps, ... of the
  // slice.  The cursor of what is fetched next runs ahead through the same order.
  const int n_shares = int(gridDim.x) / parts, share = int(blockIdx.x) / parts;
  const int tile0 = int(int64_t(P.tiles) * share / n_shares);
  const int tile1 = int(int64_t(P.tiles) * (share + 1) / n_shares);
  const int groups = (tile1 - tile0 + 1) / 2;
  auto nb_of = [&](int b0) { return min(P.slice_blocks, blocks - b0); };
  const int row_groups = P.K >> GS;
  struct {
    int chunk0, b0, i, blk;  // first group of the chunk, first block of the slice, group of the chunk, block of the slice
    int nb, tile, boxes;     // blocks of the slice, the warp's first tile and how many it has
    const S* src;            // this lane's row's scales of block b0
  } fet = {0, 0, 0, kw, 0, 0, 0, nullptr};
  auto settle = [&](bool next) {  // the first place with a block for this warp, from here or from the next group on
    for (;; next = true) {
      if (next) {
        fet.blk = kw;
        // the common case: the next group, of two whole tiles (and a warp that has blocks: else no place is set)
        if (kw < fet.nb && !slices && fet.chunk0 + fet.i + 2 < groups) {
          ++fet.i;
          fet.tile += 2;
          fet.src += int64_t(2 * 16) * row_groups;
          return;
        }
        if (++fet.i >= P.chunk || fet.chunk0 + fet.i >= groups) {
          fet.i = 0;
          fet.b0 += P.slice_blocks;
          if (fet.b0 >= blocks) {
            fet.b0 = 0;
            fet.chunk0 += P.chunk;
          }
        }
      }
      if (fet.chunk0 >= groups) return;
      fet.nb = nb_of(fet.b0);
      if (fet.blk < fet.nb) break;
    }
    fet.tile = tile0 + (fet.chunk0 + fet.i) * 2 + rw;
    fet.boxes = max(min(MT, tile1 - fet.tile), 0);  // a last group may have one tile only: the other's sums are not stored
    fet.src = static_cast<const S*>(P.scales) + int64_t(min(16 * fet.tile + lane, P.N - 1)) * row_groups + (kb0 + fet.b0) * kGroups;
  };
  settle(false);
  int issued = 0, done = 0;  // done: blocks that have come and been used
  bool lost = false;
  auto fetch = [&]() {  // the whole warp; one group of asynchronous copies a call, on every lane
    if (fet.chunk0 < groups) {
      const int st = issued % kStages;
      if (lane == 0) {
        if (fet.boxes > 0)
          tc::mbar_expect_tx(bars + st, uint32_t(fet.boxes * kBoxBytes));
        else
          tc::mbar_arrive(bars + st);
        uint8_t* dst = smem + (warp * kStages + st) * C::kStageBytes;
        const int x = (kb0 + fet.b0 + fet.blk) * 128;
        if (fet.boxes > 0) tc::tma_load_2d(dst, &P.codes, bars + st, x, fet.tile * 16);
        if (fet.boxes > 1) tc::tma_load_2d(dst + kBoxBytes, &P.codes, bars + st, x, fet.tile * 16 + 16);
      }
      if (lane < 16 * MT) {  // a row's scales each
        const S* src = fet.src + fet.blk * kGroups;
        S* dst = reinterpret_cast<S*>(scales + (st * MT * 16 + lane) * kScaleRow);
        if constexpr (kVec) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "n"(kScaleRow)
                       : "memory");
        } else {
          const int left = row_groups - (kb0 + fet.b0 + fet.blk) * kGroups;
          if (row_groups % 2 == 0) {  // rows of whole words: asynchronous as well, zeros behind K (29573 x 9600, 12 tokens: 112 -> 93 us)
#pragma unroll
            for (int g = 0; g < kGroups; g += 2)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst + g)),
                           "l"(g < left ? src + g : fet.src), "r"(g < left ? 4 : 0)
                           : "memory");
          } else {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) dst[g] = g < left ? src[g] : from_f32<S>(0.0f);
          }
        }
      }
      ++issued;
      fet.blk += kKWarps;
      if (fet.blk >= fet.nb) settle(true);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int s = 0; s < kStages; ++s) fetch();

  const uint4* x_lane[NT][2];  // of even and odd chunks; tokens beyond M read the last one's, their columns are not stored
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = min(8 * t + n, P.M - 1);
    x_lane[t][0] = xs + m * L.x_row + q + (m & 1) * 4;
    x_lane[t][1] = x_lane[t][0] - (m & 1) * 8;
  }
  // the lane's words: row n, chunk c of 16 bytes at c ^ n (128-byte swizzle); row n + 8 is 1024 bytes on
  const uint32_t word0 = n * 128 + n * 16 + 4 * q;

  float kept[kKept] = {};
  for (int chunk0 = 0; chunk0 < groups; chunk0 += P.chunk) {
    for (int b0 = 0; b0 < blocks; b0 += P.slice_blocks) {
      const int nb = nb_of(b0);
      // ---- X of the slice: 16 threads per token and 128 k
      if (slices || chunk0 == 0) {
        __syncthreads();  // the last slice's is read
        constexpr int kAhead = 4;  // units of 8 elements a thread has under way
        const int row_units = nb * 32;
        int m = 0, at = threadIdx.x;  // token and unit of it
        while (at >= row_units && m < P.M) at -= row_units, ++m;
        while (m < P.M) {
          uint4 raw[kAhead];
          int ms[kAhead], us[kAhead];
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            ms[j] = m;
            us[j] = at;
            const int k = (kb0 + b0) * kBlockK + at * 8;
            raw[j] = make_uint4(0, 0, 0, 0);
            if (m < P.M && k < P.K)
              raw[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.X) + int64_t(m) * P.K + k);
            at += C::kThreads;
            while (at >= row_units && m < P.M) at -= row_units, ++m;
          }
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            if (ms[j] >= P.M) break;  // all 16 threads of a token's 128 k together
            float x[8];
            if (P.dtype == PATCH_DTYPE_BF16)
              load16(reinterpret_cast<const __nv_bfloat16*>(&raw[j]), x);
            else
              load16(reinterpret_cast<const __half*>(&raw[j]), x);
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
            const unsigned half = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
            for (int d = 8; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, d));
            const int e = max(int(__float_as_uint(amax) >> 23) - 127, -113);
            const float f = e == 128 ? 1.0f : pow2i(14 - e), f16 = f * 0.0625f;
            // odd tokens have the halves of 128 bytes exchanged: 8 tokens' pieces lie in different banks
            xs[ms[j] * L.x_row + (us[j] ^ ((ms[j] & 1) << 2))] =
                make_uint4(pack_f16(x[0] * f, x[4] * f), pack_f16(x[1] * f16, x[5] * f16), pack_f16(x[2] * f, x[6] * f),
                           pack_f16(x[3] * f16, x[7] * f16));
            if ((threadIdx.x & 15) == 0) x_scale[(us[j] >> 4) * 8 * NT + ms[j]] = e == 128 ? 4096.0f : pow2i(e - 2);
          }
        }
        __syncthreads();
        // -8 times the sums of X over each group, as the products will take them
        for (int grp = warp; grp < nb * kGroups * NT; grp += kWarps) {
          const int t = grp % NT, g0 = grp / NT;  // token tile, group of the slice
          constexpr int kPer = 1 << (GS - 5);
          float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int c = g0 * kPer + i;
            const uint4 x = *(t == 0 ? x_lane[0][c & 1] + c * 4 : x_lane[NT - 1][c & 1] + c * 4);
            mma(acc, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, x.x, x.y, acc);
            mma(acc, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, x.z, x.w, acc);
          }
          if (n == 0) *reinterpret_cast<float2*>(neg_sum + grp * 8 + 2 * q) = make_float2(acc[0], acc[1]);
        }
        __syncthreads();
      }

      const int n_here = min(P.chunk, groups - chunk0);
      for (int i = 0; i < n_here; ++i) {
        const int row0 = 16 * (tile0 + (chunk0 + i) * 2);
        float y[MT][NT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[t][u][k] = 0.0f;
        for (int blk = kw; !lost && blk < nb; blk += kKWarps) {
          const int st = done % kStages;
          const bool ok = tc::wait_bounded(bars + st, (done / kStages) & 1, abort_flag, 2000000000ull, P.status, false);
          lost = !__all_sync(0xFFFFFFFFu, ok);
          if (lost) break;
          ++done;
          asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");  // this stage's scales
          __syncwarp();
          alignas(16) S sc[MT][2][kGroups];  // of rows n and n + 8
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint8_t* at = scales + ((st * MT + t) * 16 + n + 8 * h) * kScaleRow;
              if constexpr (kScaleRow == 16) *reinterpret_cast<uint4*>(sc[t][h]) = *reinterpret_cast<const uint4*>(at);
              if constexpr (kScaleRow == 8) *reinterpret_cast<uint2*>(sc[t][h]) = *reinterpret_cast<const uint2*>(at);
              if constexpr (kScaleRow == 4) *reinterpret_cast<uint32_t*>(sc[t][h]) = *reinterpret_cast<const uint32_t*>(at);
            }
          const uint8_t* words = smem + (warp * kStages + st) * C::kStageBytes;
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {  // 128 k
            constexpr int kPer = 1 << (GS - 5);  // chunks of 32 k in a group
            float sum[MT][NT][4], acc[MT][NT][4];
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
              const int c = 4 * hb + c4;
              uint4 x[NT];
              float neg[NT][4];
#pragma unroll
              for (int u = 0; u < NT; ++u) {
                x[u] = x_lane[u][c & 1][(blk * 8 + c) * 4];
                if (c4 % kPer == 0) {
                  const float2 v = *reinterpret_cast<const float2*>(neg_sum + ((blk * 8 + c) / kPer * NT + u) * 8 + 2 * q);
                  neg[u][0] = neg[u][2] = v.x;
                  neg[u][1] = neg[u][3] = v.y;
                }
              }
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                const uint8_t* at = words + (word0 ^ (c << 4)) + t * kBoxBytes;
                const uint32_t a0 = *reinterpret_cast<const uint32_t*>(at), a1 = *reinterpret_cast<const uint32_t*>(at + 1024);
                const uint32_t r0 = a0 >> 8, r1 = a1 >> 8;
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                  mma(acc[t][u], a0 & 0x000F000Fu, a1 & 0x000F000Fu, a0 & 0x00F000F0u, a1 & 0x00F000F0u, x[u].x, x[u].y,
                      c4 % kPer == 0 ? neg[u] : acc[t][u]);
                  mma(acc[t][u], r0 & 0x000F000Fu, r1 & 0x000F000Fu, r0 & 0x00F000F0u, r1 & 0x00F000F0u, x[u].z, x[u].w,
                      acc[t][u]);
                }
                if (c4 % kPer == kPer - 1) {
                  const int g = c / kPer;
                  const float s0 = to_f32(sc[t][0][g]), s1 = to_f32(sc[t][1][g]);
#pragma unroll
                  for (int u = 0; u < NT; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      const float f = k < 2 ? s0 : s1;
                      sum[t][u][k] = c4 == kPer - 1 ? acc[t][u][k] * f : fmaf(acc[t][u][k], f, sum[t][u][k]);
                    }
                }
              }
            }
#pragma unroll
            for (int u = 0; u < NT; ++u) {
              const float2 f = *reinterpret_cast<const float2*>(x_scale + ((blk * 2 + hb) * NT + u) * 8 + 2 * q);
#pragma unroll
              for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) y[t][u][k] = fmaf(sum[t][u][k], k & 1 ? f.y : f.x, y[t][u][k]);
            }
          }
          __syncwarp();  // every lane has read the stage
          fetch();
        }
        // ---- add the warps' sums: [kw][token][row of the group]
        const int outs = P.M * kGroupRows;
        if (!kParts)
          __syncthreads();  // the last ones are read
        else if (chunk0 + i > 0)
          cluster_wait();  // by the cluster's other CTAs too
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int m = 8 * u + 2 * q + (k & 1);
            if (m < P.M)
#pragma unroll
              for (int t = 0; t < MT; ++t)
                reduce[kw * outs + m * kGroupRows + 16 * (rw + t) + n + 8 * (k >> 1)] = y[t][u][k];
          }
        __syncthreads();
        const int o = threadIdx.x;  // outs <= threads
        if (o < outs) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kKWarps; ++w) v += reduce[w * outs + o];
          if (b0 > 0) v += kept[0];
#pragma unroll
          for (int j = 0; j + 1 < kKept; ++j) kept[j] = kept[j + 1];  // with slices, a chunk is kKept groups at most:
          kept[kKept - 1] = v;                                       // the next slice finds this one's sum first
          const int row = row0 + o % kGroupRows;
          if (kParts)
            reduce[o] = v;  // this thread alone has read the word
          else if (b0 + nb == blocks && row < P.N && row < 16 * tile1)
            store_y(static_cast<uint16_t*>(P.Y) + int64_t(o / kGroupRows) * P.N + row, v * 4096.0f, P.dtype);
        }
        if (kParts) {  // no slices then: each CTA adds and stores its share of the group's outputs
          __syncwarp();
          cluster_arrive();
          cluster_wait();
          const int o1 = outs * (part + 1) / parts, ox = outs * part / parts + int(threadIdx.x);
          if (ox < o1) {
            float v = 0.0f;
            for (int r = 0; r < parts; ++r) v += load_of_cta(tc::smem_u32(reduce + ox), r);
            const int row = row0 + ox % kGroupRows;
            if (row < P.N && row < 16 * tile1)
              store_y(static_cast<uint16_t*>(P.Y) + int64_t(ox / kGroupRows) * P.N + row, v * 4096.0f, P.dtype);
          }
          __syncwarp();
          cluster_arrive();
        }
      }
      for (int i = n_here; i < kKept; ++i) {  // turn a shorter chunk's sums round as well
        const float v = kept[0];
#pragma unroll
        for (int j = 0; j + 1 < kKept; ++j) kept[j] = kept[j + 1];
        kept[kKept - 1] = v;
      }
    }
  }
  // after a timeout: let the copies in flight land before the shared memory goes
  for (; done < issued; ++done)
    tc::wait_bounded(bars + done % kStages, (done / kStages) & 1, abort_flag, tc::kDrainNs, P.status, true);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  if (kParts) cluster_wait();  // the others have read this CTA's sums
}

template <typename S, int NT, int GS>
static cudaError_t launch(Params P, int num_sms, cudaStream_t stream) {
  using C = Cfg<NT>;
  P.tiles = (P.N + 15) / 16;
  P.blocks = (P.K + kBlockK - 1) / kBlockK;
  // Parts of K, and one or two CTAs an SM (which have to fit: X, its sums and the scales grow with tokens, K and finer
  // groups), by an estimate of a CTA's time in ns: X of a block and token 20 (again for every chunk of row groups where
  // K is taken in slices), a row group's products of a block 165 (both tiles' warps), 180 (8 warps alone on their SM)
  // or 300 (two CTAs an SM), its sums 300, 1500 with each slice, or 2200 through the cluster.
  // Measured, two CTAs an SM and one: 128000 x 4096, group 128, 1 token 50 us, 58; 6 tokens 84, 65; 9000 x 11008,
  // group 32, 4 tokens 38, 25; where two do not fit, 8 tokens and group 32, 128000 x 4096 142 as two waves, 81.
  // Measured in a row of launches with one part and with the chosen: 577 x 11072, 14 tokens 31 us, 12 (4 parts);
  // 4096 x 14336, 8 tokens 26, 21, 16 tokens 38, 26; 256 x 14336, 1 token 12.1, 6.0 (8); 29573 x 9600, 12 tokens
  // 93, 77 (2).  One part stays where the others lose, with two: 4096 x 4096, 1 token 6.0, 7.2, 16 tokens 11.9, 12.6;
  // 14336 x 4096, 16 tokens 24, 28; 128000 x 4096, 1 token 63, 104.
  float best = 0.0f;
  int grid = 0;
  for (int ctas = C::kCtas; ctas >= 1; --ctas) {
    auto fits = [&](int x_blocks) {
      return x_blocks <= kMostBlocks && layout<NT, GS>(P.M, x_blocks).bytes <= kSmemOfSm / ctas - kSmemReserved;
    };
    // of a slice: whole rounds of the warps, as many as fit
    int slice = (P.blocks > kMostBlocks ? kMostBlocks : P.blocks - 1) / kKWarps * kKWarps;
    while (slice > 0 && !fits(slice)) slice -= kKWarps;
    for (int parts = 1; parts <= kMaxParts && parts <= P.blocks; parts *= 2) {
      const int local = (P.blocks + parts - 1) / parts;
      // clusters that run at once: they lie in one of the GPU's parts of 16 to 20 SMs each (33 of 4, 15 of 8 on 148 SMs)
      const int most = ctas * num_sms * (parts <= 2 ? 16 : parts == 4 ? 14 : 13) / 16 / parts;
      const bool slices = !fits(local);
      if (most < 1 || (slices && (parts > 1 || slice == 0))) continue;
      const int shares = P.tiles < most ? P.tiles : most, groups = ((P.tiles + shares - 1) / shares + 1) / 2;
      const float times = slices ? float((groups + kKept - 1) / kKept) : 1.0f;
      const float sums = parts > 1 ? 2200.0f : slices ? 300.0f + 1500.0f * float((local + slice - 1) / slice) : 300.0f;
      const float ns = 20.0f * float(P.M) * float(local) * times +
                       float(groups) * ((ctas == 2 ? 300.0f : NT == 1 ? 180.0f : 165.0f) * float(local) + sums);
      if (grid && ns >= best) continue;
      best = ns;
      grid = shares * parts;
      P.parts = parts;
      P.slice_blocks = slices ? slice : local;
      P.chunk = slices && groups > kKept ? kKept : groups;
    }
  }
  const Layout L = layout<NT, GS>(P.M, P.slice_blocks);
  const bool vec = P.K % kBlockK == 0;
  auto kernel = P.parts > 1 ? vec ? gemm4_kernel<S, NT, GS, true, true> : gemm4_kernel<S, NT, GS, true, false>
                : vec       ? gemm4_kernel<S, NT, GS, false, true>
                            : gemm4_kernel<S, NT, GS, false, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L.bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid_dim{unsigned(grid)}, block_dim{C::kThreads};
  return P.parts == 1 ? launch_pdl(kernel, grid_dim, block_dim, size_t(L.bytes), stream, P)
                      : launch_pdl_cluster(kernel, grid_dim, block_dim, size_t(L.bytes), stream, unsigned(P.parts), P);
}

template <typename S, int NT>
static cudaError_t launch_group(const Params& P, int group, int num_sms, cudaStream_t stream) {
  if (group == 32) return launch<S, NT, 5>(P, num_sms, stream);
  if (group == 64) return launch<S, NT, 6>(P, num_sms, stream);
  return launch<S, NT, 7>(P, num_sms, stream);
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
  P.dtype = dtype;
  if (!make_map_rows_u8(&P.codes, W.codes, W.K / 2, W.N, 128, 16)) return cudaErrorInvalidValue;
  using BF = __nv_bfloat16;
  if (W.scale_dtype == PATCH_DTYPE_BF16)
    return M <= 8 ? g4::launch_group<BF, 1>(P, W.group, num_sms, stream) : g4::launch_group<BF, 2>(P, W.group, num_sms, stream);
  return M <= 8 ? g4::launch_group<__half, 1>(P, W.group, num_sms, stream)
                : g4::launch_group<__half, 2>(P, W.group, num_sms, stream);
}

}  // namespace patch
