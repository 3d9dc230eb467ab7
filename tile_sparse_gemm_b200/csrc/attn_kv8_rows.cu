// Attention over the paged 8-bit cache for sequences with many new tokens
// (chunks of a prompt): tiles of 128 query rows on tcgen05 (include/patch.h:
// patch_attn_kv8; attn_kv8.cu has the form for few rows and the mathematics).
//
// What bounds it: with 128 rows to a tile every cached byte meets 128 rows, so it is
// bound by computing.  A block of 128 tokens is two products of 128 x 128 x D (2 x 524
// tensor-core cycles of an SM at D = 128), 16384 exponentials (1024 cycles of the
// special-function units) and some 700 cycles of other softmax instructions, and
// the conversion of the values.  The roles run side by side, one CTA per SM (its tensor
// memory holds two blocks of scores and the sums, its registers 14 warps of 128):
//   warps 0-7   softmax, two threads per row with half of a block's scores each: scores
//               from tensor memory, the row's maximum exchanged between the two,
//               probabilities as fp16 back into the place of the scores, where the second
//               product takes them.  The sum of the values stays in tensor memory and is
//               rescaled only when a row's maximum grows by more than 2^8 (probabilities
//               are at most 2^8 then, well inside fp16; sums are fp32);
//   warps 8-11  convert the e4m3 values that TMA has brought to fp16, transposed (tokens
//               in a row), in the 128-byte swizzle that the tensor cores read;
//   warp 12     one thread issues the products: S = Q K^T for block g into one of two
//               places once O += P V of block g - 2, which held that place, is done;
//   warp 13     fetches: block table, scales, TMA.
// The keys are multiplied as they lie in the cache, e4m3 by e4m3 (kind::f8f6f4, twice
// fp16's rate): a query element, scaled so that its row's largest is in [2^7, 2^8), is the
// sum of two (bf16) or three (fp16) e4m3 numbers, each the rounding of what the ones before
// leave.  bf16 has 8 bits and fp16 11, an e4m3 number takes off at least 4 of them, so the
// sum is exact but for what lies below e4m3's smallest step, 2^-10 or 2^-17 of the row's
// largest.  Two terms take as long as one fp16 product, and the keys need no conversion.
// The value scales weigh the probabilities, in units 2^5 below the first block's largest: up to 2^7 units
// fp16 holds the weighted probabilities with no fewer bits than the plain ones; where a larger scale comes the
// unit is raised.  A block with a smaller one takes bf16 instead, whose range holds every scale, on
// the values' side, and its probabilities as sums of two numbers in two products.
//
// Measured: 4 prompts of 1024 queries over 4000 tokens, 32 heads over 8 of 128: 325 us,
// 722 TFLOP/s; 512 queries over 8000: 98 us, 663 TFLOP/s (value scales apart in every block,
// each 2^-30 to 2^30: 696 and 201 us).  A block takes a CTA about 2600
// cycles: the softmax warps' 1350 for exponentials and probabilities, 220 for the maximum,
// 210 to exchange it, 390 to read and mask, and their waits; a tile costs 8000 more.
// Work is shared out as in attn_kv8.cu: equal runs of blocks for all CTAs, wherever
// tiles begin and end; a tile cut between CTAs is finished by the last to arrive.
#include <type_traits>

#include "attn_kv8.cuh"

namespace patch {
namespace attn {

struct RowsParams {
  CUtensorMap k_map, v_map;
  AttnParams a;
  uint32_t* counters;  // one per CTA
  float* parts;        // two tile states per CTA
  uint64_t limit_ns;
  int page_shift, box_shift;
};

// TERMS: e4m3 numbers whose sum stands for a query element.
template <int D, int N_TERMS>
struct RowsCfg {
  static constexpr int TERMS = N_TERMS, CH = 128, R = 128;  // tokens of a block, rows of a tile
  static constexpr int SL = CH / 16;       // slices of 16 tokens, the least page
  static constexpr int kWarps = 14, kThreads = 32 * kWarps;
  static constexpr int kRawBytes = CH * D;
  static constexpr int kQ = 0;                        // [TERMS][128 rows][D bytes], swizzled like the cache's
  static constexpr int kV = kQ + TERMS * R * D;       // 2 x [CH / 64][D][64 tokens]
  static constexpr int kRawK = kV + 2 * CH * D * 2;   // 2 x e4m3 as in the cache
  static constexpr int kRawV = kRawK + 2 * kRawBytes;
  static constexpr int kNan = kRawV + 2 * kRawBytes;    // 4 x [CH tokens][4 words]: elements of a token that are NaN
  static constexpr int kScales = kNan + 4 * CH * 16;  // 8 x [SL] (key, value) scales
  static constexpr int kBars = kScales + 8 * SL * 8;
  static constexpr int kXch = kBars + 256;            // between a row's two threads: maxima [2][2][128], sums, query maxima
  static constexpr int kMisc = kXch + 8 * R * 4;
  static constexpr int kSmem = kMisc + 256;
  static constexpr int kStateFloats = R * D + 2 * R;       // o (in groups of 4 columns), m, l
  static constexpr uint32_t kTmemCols = 512, kO = 2 * CH;  // S and P at 0 and CH, then O
};

constexpr float kLeast = 1.0e-37f;  // of a score's factor: not 0, hidden scores are -inf times it
constexpr float kGrow = 8.0f;  // log2 of what a maximum may grow by before O is rescaled
// Value scales, in units of the tile's sums, of up to 2^7 weigh the probabilities: 2^15 at most, and none loses bits.
constexpr float kUnits = 128.0f;

// fp32 sums of fp16 (kind::f16) or of e4m3 (kind::f8f6f4): type codes 0 both
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N) {
  return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_8cols(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_64cols(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
      "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
      "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
      "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
      "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]),
      "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]), "=r"(v[41]), "=r"(v[42]),
      "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]), "=r"(v[48]), "=r"(v[49]),
      "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]), "=r"(v[56]),
      "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr)
      : "memory");
}
// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// the A operand in tensor memory: lane = row, a column holds two neighbouring fp16 of k
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {  // saturating, NaN stays NaN
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma_a_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// For a block whose value scales are apart, kept out of the loops that every block goes through: calls in them keep
// the compiler from taking the next loads ahead, and products take a longer way (4 prompts of 1024 queries
// over 4000 tokens: 366 us, 326 so).  The softmax warps, which wait for the scales anyway, do all of it: with
// another wait in the warps that convert, 2048 queries of each of 4 prompts in fp16 take 336 us, 323 so.
// A row's probabilities as sums of two bf16 numbers each, exactly: fp16 has 11 bits.
template <int kCols>
__device__ __noinline__ void split_probabilities(uint32_t s_at) {
#pragma unroll 1
  for (int i = 0; i < kCols / 2; i += 16) {
    uint32_t w[16], rest[16];
    tc::tmem_ld_16cols(s_at + i, w);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      w[j] = pack_bf16(p.x, p.y);
      rest[j] = pack_bf16(p.x - __uint_as_float(w[j] << 16), p.y - __uint_as_float(w[j] & 0xFFFF0000u));
    }
    tmem_st_16cols(s_at + i, w);
    tmem_st_16cols(s_at + kCols / 2 + i, rest);
  }
}

// The converted values of a block in bf16, times their pages' scales, by the threads of the softmax.
template <int CH, int D>
__device__ __noinline__ void widen_values(uint8_t* v_at, const float2* scales) {
#pragma unroll 8
  for (int i = threadIdx.x; i < CH * D / 2; i += 256) {
    const int pair = i & 31, row = (i >> 5) % D, atom = (i >> 5) / D;  // two tokens, element, 64 tokens
    const float weight = scales[4 * atom + (pair >> 3)].y;
    uint32_t* at = reinterpret_cast<uint32_t*>(v_at + atom * (D * 128) + row * 128 + (((pair >> 2) ^ (row & 7)) << 4) + (pair & 3) * 4);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(at));
    *at = pack_bf16(f.x * weight, f.y * weight);
  }
  tc::fence_proxy_async_smem();
}

// Both terms of the probabilities times the values.
template <int CH, int R, int D>
__device__ __noinline__ void products_apart(uint32_t o_at, uint32_t p_at, uint64_t v_desc, bool fresh) {
  constexpr int N = CH / 16;
#pragma unroll 16
  for (int i = 0; i < 2 * N; ++i) {
    const int k = i % N;
    mma_a_tmem(o_at, p_at + CH / 2 * (k / (N / 2)) + CH / 4 * (i / N) + 8 * (k % (N / 2)),
               v_desc + (k >> 2) * (D * 128 / 16) + 2 * (k & 3), tc::idesc_bf16(R, D, false), !fresh || i > 0);
  }
}

// A slice of a page outside the pool, unless the slice lies before the window.
__device__ __noinline__ void report_page(int32_t* status, int tok, int lo) {
  if (tok + 16 > lo) set_status(status, PATCH_DEV_BOUNDS);
}

template <typename T, int D>
using RowsOf = RowsCfg<D, std::is_same<T, __half>::value ? 3 : 2>;

template <typename T, int D>
__global__ void __launch_bounds__(RowsOf<T, D>::kThreads, 1) attn_kv8_rows_kernel(const __grid_constant__ RowsParams P) {
  using C = RowsOf<T, D>;
  constexpr int CH = C::CH, R = C::R, SL = C::SL, TERMS = C::TERMS, kCols = CH / 2;  // kCols: scores of a block that a thread has
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnParams& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.heads / a.kv_heads;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  // Barriers of the pipeline.  Those with two or more places take blocks in turn, so that no
  // waiter is ever two phases behind.
  uint64_t* raw_k = bars;                                   // [2] key bytes landed
  uint64_t *raw_v = bars + 2, *raw_v_free = bars + 4;       // [2] value bytes landed, read
  uint64_t* v_full = bars + 7;                              // [2] values converted
  uint64_t* s_full = bars + 9;                              // [2] scores done (the keys' place is free)
  uint64_t* p_full = bars + 11;                             // [2] probabilities written
  uint64_t* o_done = bars + 13;                             // [2] O += P V done
  uint64_t *q_full = bars + 15, *drain = bars + 16;
  uint64_t* scales_full = bars + 17;                        // [8]
  float2* scales = reinterpret_cast<float2*>(smem + C::kScales);
  int64_t* misc = reinterpret_cast<int64_t*>(smem + C::kMisc);  // of make_share: 16 words
  int* abort_flag = reinterpret_cast<int*>(misc + 20);
  int* last_flag = abort_flag + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(abort_flag + 2);
  int* nan_block = abort_flag + 4;  // [4] 1 + number of the block whose NaN masks are valid
  // [8] the unit of the values' sums from a block on, negative where the block's value scales are apart (kUnits)
  volatile float* v_unit = reinterpret_cast<float*>(misc + 24);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 25; ++i)  // arrivals: of the converting warps, of the softmax warps, or one
      tc::mbar_init(bars + i, i == 4 || i == 5 || i == 7 || i == 8 ? 4 : i == 11 || i == 12 || i == 15 ? 8 : 1);
    tc::fence_barrier_init();
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) nan_block[i] = 0;
    tc::prefetch_tensormap(&P.k_map);
    tc::prefetch_tensormap(&P.v_map);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Share sh;
  if (!make_share<CH, R, C::kWarps, 1>(a, G, misc, sh)) return;
  if (warp == 12) tc::tmem_alloc(tmem_at, C::kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_at;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return tc::wait_bounded(bar, parity & 1, abort_flag, P.limit_ns, a.status, false);
  };
  // every role walks the same blocks: g counts them over the CTA's whole share
  Cursor cur{};
  cur.start<CH, R>(a, G, misc + C::kWarps, sh.u0, sh.u0 + sh.u_n);
  const int64_t v1 = sh.u0 + sh.u_n;

  if (warp < 8) {
    // ================= softmax: two threads a row of the tile
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + C::kXch);
    // what the row's other thread has written at the same place (both behind one barrier of the two warps)
    auto exchange = [&](int place, float x) {
      xch[(2 * place + half) * R + row] = x;
      tc::named_bar_sync(3 + (warp & 3), 64);
      return xch[(2 * place + (half ^ 1)) * R + row];
    };
    int g = 0;
    for (; cur.c < cur.c_end; cur.next<CH, R>(a, G)) {
      const Tile& t = cur.t;
      // ---- half of this row's query, divided by a power of two, to shared memory
      const int r = t.rt * R + row;
      const bool live = r < t.m * G;
      float row_scale;
      {
        const T* src = static_cast<const T*>(a.q) + int64_t(t.row0 + r / G) * a.q_ts + int64_t(t.h * G + r % G) * a.q_hs +
                       half * (D / 2);
        uint4 raw[D / 16];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          raw[i] = make_uint4(0, 0, 0, 0);
          if (live) raw[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          float x[8];
          load16(reinterpret_cast<const T*>(&raw[i]), x);
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
        }
        amax = fmaxf(amax, exchange(3, amax));
        // the largest to [2^7, 2^8); an infinity becomes NaN, which all its scores would be
        const int e = min(134 - int(__float_as_uint(amax) >> 23), 126);
        // a negative scale turns the query round, so that maxima of products are maxima of scores
        const float down = pow2i(e) * (a.scale < 0.0f ? -1.0f : 1.0f);
        row_scale = pow2i(-e) * (fabsf(a.scale) * kLog2e);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {  // pieces of 16 elements
          float x[16];
          load16(reinterpret_cast<const T*>(&raw[2 * i]), x);
          load16(reinterpret_cast<const T*>(&raw[2 * i + 1]), x + 8);
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = amax < INFINITY ? x[j] * down : __int_as_float(0x7FC00000);
          const int p = half * (D / 32) + i;
          uint8_t* dst = smem + C::kQ + row * D + ((p ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4);
#pragma unroll
          for (int term = 0; term < TERMS; ++term) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              w[j] = pack_e4m3(x[4 * j], x[4 * j + 1]) | pack_e4m3(x[4 * j + 2], x[4 * j + 3]) << 16;
              uint32_t taken[2];
              cvt4(w[j], taken[0], taken[1]);
#pragma unroll
              for (int k = 0; k < 2; ++k) {  // what is left, exactly
                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&taken[k]));
                x[4 * j + 2 * k] -= y.x;
                x[4 * j + 2 * k + 1] -= y.y;
              }
            }
            *reinterpret_cast<uint4*>(dst + term * (R * D)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(q_full);
      const int pos = t.len - t.m + r / G;
      const int see_hi = live ? (a.causal ? min(t.len, pos + 1) : t.len) : 0;
      const int see_lo = a.window > 0 ? int(max(int64_t(0), pos - a.window + 1)) : 0;
      const int all_hi = a.causal ? t.len - t.m + t.rt * R / G + 1 : t.len;
      const int last_row = min(t.m - 1, (t.rt * R + R - 1) / G);
      const int all_lo = a.window > 0 ? int(max(int64_t(0), t.len - t.m + last_row - a.window + 1)) : 0;

      float m = -INFINITY, l = 0.0f, v_ref = 0.0f;  // l: of this thread's scores; v_ref: the unit of O
      // elements half * D / 2 on of the row that a NaN value reaches
      uint32_t nan_row[D / 64];
#pragma unroll
      for (int i = 0; i < D / 64; ++i) nan_row[i] = 0;
      // what a block's NaN values mean for this row (once the block's values have been converted)
      auto see_nan = [&](int c, int g_of) {
        if (nan_block[g_of & 3] != g_of + 1) return;
        const uint32_t* mask = reinterpret_cast<const uint32_t*>(smem + C::kNan + (g_of & 3) * CH * 16) + half * (D / 64);
        const int t0 = (t.chunk0 + c) * CH;
        for (int k = max(0, see_lo - t0); k < min(CH, see_hi - t0); ++k)
#pragma unroll
          for (int i = 0; i < D / 64; ++i) nan_row[i] |= mask[4 * k + i];
      };
      // A wait that runs out does not end the loops: what follows is of no use then, but every warp still
      // goes through the barriers that it shares with others.
      for (int c = cur.c; c < cur.c_end; ++c, ++g) {
        const bool first = c == cur.c;
        wait(scales_full + (g & 7), g >> 3);
        wait(s_full + (g & 1), g >> 1);
        __syncwarp();
        tc::tc_fence_after();
        if (c - 2 >= cur.c) see_nan(c - 2, g - 2);  // these scores have taken the place of its probabilities
        const int t0 = (t.chunk0 + c) * CH + kCols * half;  // of this thread's tokens
        const uint32_t s_at = lanes + (g & 1) * CH + kCols * half;
        // the slices' key scales (times the row's), read before the scores so that their latency is hidden
        const float2* sc = scales + SL * (g & 7) + SL / 2 * half;
        float kf[SL / 2];
#pragma unroll
        for (int i = 0; i < SL / 2; ++i) kf[i] = fmaxf(sc[i].x * row_scale, kLeast);
        const float unit = v_unit[g & 7], v_new = fabsf(unit);
        float s[kCols];  // products; hidden ones -inf
        tmem_ld_64cols(s_at, reinterpret_cast<uint32_t(&)[64]>(s));
        // Below, a score is not rounded before the maximum, which is, is taken off; from 2^24 on it could lie far
        // above it.  Where scores may be that large, round them here.
        constexpr float kWild = float(16777216.0 / (448.0 * 256.0 * D));
        float most = kf[0];
#pragma unroll
        for (int i = 1; i < SL / 2; ++i) most = fmaxf(most, kf[i]);
        if (t0 + kCols > all_hi || t0 < all_lo || most >= kWild) {
          const int hi = see_hi - t0, lo = see_lo - t0;
          const bool wild = most >= kWild;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            if (wild) s[j] = __fmul_rn(s[j], kf[j / 16]);
            if (j >= hi || j < lo) s[j] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < SL / 2; ++i) kf[i] = wild ? 1.0f : kf[i];
        }
        float mx = m;
#pragma unroll
        for (int i = 0; i < SL / 2; ++i) {
          const float* x = s + 16 * i;
          float top[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = max3(x[4 * j], x[4 * j + 1], fmaxf(x[4 * j + 2], x[4 * j + 3]));
          mx = fmaxf(mx, fmaxf(max3(top[0], top[1], top[2]), top[3]) * kf[i]);
        }
        mx = fmaxf(mx, exchange(g & 1, mx));  // two places in turn: a thread is at most one barrier ahead
        const bool grow = mx > m + kGrow || (m == -INFINITY && mx > m);
        if (__any_sync(0xFFFFFFFFu, grow || v_new != v_ref)) {
          const float f = grow ? ex2(m - mx) : 1.0f;  // 0 for a row's first scores
          if (grow) m = mx;
          l *= f;
          const float fo = v_new != v_ref ? f * (v_ref * per_unit(v_new)) : f;
          v_ref = v_new;
          if (!first) {  // O is these threads' once the block before has been added
            wait(o_done + ((g - 1) & 1), (g - 1) >> 1);
            __syncwarp();
            tc::tc_fence_after();
#pragma unroll 1
            for (int j = half * (D / 2); j < (half + 1) * (D / 2); j += 16) {
              uint32_t o[16];
              tc::tmem_ld_16cols(lanes + C::kO + j, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fo);
              tmem_st_16cols(lanes + C::kO + j, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.0f : m;
        const uint64_t base2 = pack2(-base, -base);
        uint64_t sum[2] = {0, 0};  // of even and odd scores, in turn
#pragma unroll
        for (int i = 0; i < SL / 2; ++i) {
          const float vr = unit < 0.0f ? 1.0f : sc[i].y;
          const uint64_t k2 = pack2(kf[i], kf[i]), vr2 = pack2(vr, vr);
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 e = unpack2(fma2(pack2(s[16 * i + 2 * j], s[16 * i + 2 * j + 1]), k2, base2));
            const uint64_t p2 = pack2(ex2(e.x), ex2(e.y));
            sum[j & 1] = add2(sum[j & 1], p2);
            const float2 p = unpack2(mul2(p2, vr2));
            w[j] = pack_f16(p.x, p.y);
          }
          tmem_st_8cols(s_at + 8 * i, w);  // over scores that this thread has read
        }
        const float2 both = unpack2(add2(sum[0], sum[1]));
        l += both.x + both.y;
        tc::tmem_wait_st();
        if (unit < 0.0f) {
          split_probabilities<kCols>(s_at);
          tc::tmem_wait_st();
          wait(v_full + (g & 1), g >> 1);
          widen_values<CH, D>(smem + C::kV + (g & 1) * (CH * D * 2), scales + SL * (g & 7));
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + (g & 1));
      }
      // ---- the tile's sums over this CTA's blocks
      wait(o_done + ((g - 1) & 1), (g - 1) >> 1);
      __syncwarp();
      tc::tc_fence_after();
      if (cur.c_end - 2 >= cur.c) see_nan(cur.c_end - 2, g - 2);
      see_nan(cur.c_end - 1, g - 1);
      l += exchange(2, l);
      const bool whole = cur.c == 0 && cur.c_end == t.chunks;
      const int64_t at = t.row0 + r / G;
      const int head = t.h * G + r % G;
      float* part = P.parts + (2 * blockIdx.x + (cur.c == 0 ? 1 : 0)) * int64_t(C::kStateFloats);
      T* dst = static_cast<T*>(a.out) + at * a.o_ts + head * a.o_hs;
      auto write_lse = [&](float m_, float l_) {
        if (a.lse && live && half == 0)
          a.lse[at * a.heads + head] = m_ == -INFINITY && l_ == 0.0f ? -INFINITY : (m_ + log2f(l_)) / kLog2e;
      };
      const float inv = m == -INFINITY && l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
      for (int j = 0; j < D / 2; j += 16) {
        const int d = half * (D / 2) + j;
        uint32_t raw[16];
        tc::tmem_ld_16cols(lanes + C::kO + d, raw);
        float o[16];
        uint32_t bad = nan_row[0];
        if (D == 128 && j >= 32) bad = nan_row[D / 64 - 1];
        bad >>= j & 31;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          o[k] = __uint_as_float(raw[k]) * v_ref;
          if (whole) o[k] *= inv;
          if (bad >> k & 1) o[k] = __int_as_float(0x7FC00000);
        }
        if (whole) {
          if (live) {
            store16(dst + d, o);
            store16(dst + d + 8, o + 8);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4*>(part + ((d + k) / 4 * R + row) * 4) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      tc::tc_fence_before();
      if (whole) {
        write_lse(m, l);
      } else {
        if (half == 0) {
          part[R * D + row] = m;
          part[R * D + R + row] = l;
        }
        const int64_t unit0 = v1 - cur.left;
        const int64_t c0 = sh.owner(unit0 + tile_units<R>()), c1 = sh.owner(unit0 + tile_units<R>() + t.chunks - 1);
        tc::named_bar_sync(1, 256);
        if (threadIdx.x == 0) {  // releases what the barrier has brought before it, and takes in what the others did
          uint32_t arrived;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(arrived) : "l"(P.counters + c0) : "memory");
          if (arrived == uint32_t(c1 - c0)) P.counters[c0] = 0;
          *last_flag = arrived == uint32_t(c1 - c0);
        }
        tc::named_bar_sync(1, 256);
        if (*last_flag) {  // the last to arrive joins the parts, in CTA order
          auto part_of = [&](int64_t i) { return P.parts + (2 * i + (i == c0 ? 1 : 0)) * int64_t(C::kStateFloats); };
          m = -INFINITY;
          for (int64_t i = c0; i <= c1; ++i) m = fmaxf(m, __ldcg(part_of(i) + R * D + row));
          const float base = m == -INFINITY ? 0.0f : m;
          l = 0.0f;
          for (int64_t i = c0; i <= c1; ++i)
            l += __ldcg(part_of(i) + R * D + R + row) * ex2(__ldcg(part_of(i) + R * D + row) - base);
          const float inv_all = m == -INFINITY && l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
          for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 16) {
            float o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0.0f;
            for (int64_t i = c0; i <= c1; ++i) {
              const float* p = part_of(i);
              const float f = ex2(__ldcg(p + R * D + row) - base);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(p + ((d + k) / 4 * R + row) * 4));
                o[k] += x.x * f;
                o[k + 1] += x.y * f;
                o[k + 2] += x.z * f;
                o[k + 3] += x.w * f;
              }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= inv_all;
            if (live) {
              store16(dst + d, o);
              store16(dst + d + 8, o + 8);
            }
          }
          write_lse(m, l);
        }
        tc::named_bar_sync(1, 256);  // the flag is read before the next cut tile writes it
      }
    }
  } else if (warp < 12) {
    // ================= conversion of values
    const int w = warp - 8;
    // Values of block g: lane = two neighbouring tokens, 16 elements of each at a time.  A NaN must
    // not reach the rows that do not see its token (0 x NaN): it is taken out and kept as a bit, in a
    // mask for every token and piece; `dirty`: the places in which this thread has left bits.
    uint32_t dirty = 0;
    for (int i = threadIdx.x - 256; i < 4 * CH; i += 128) reinterpret_cast<uint4*>(smem + C::kNan)[i] = make_uint4(0, 0, 0, 0);
    tc::named_bar_sync(2, 128);
    auto convert_v = [&](int g, int behind) {  // behind: tokens of the block before what no row sees
      bool ok = wait(raw_v + (g & 1), g >> 1);
      if (ok && g > 1) ok = wait(o_done + (g & 1), (g - 2) >> 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) return false;
      uint32_t had = 0;
#pragma unroll 2
      for (int i = 0; i < CH / 64 * (D / 64); ++i) {
        const int atom = i / (D / 64), p = w * (D / 64) + i % (D / 64);  // 64 tokens, 16-byte piece
        uint32_t x[2][4], nan = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int tok = 64 * atom + 2 * lane + k;
          const uint4 v = *reinterpret_cast<const uint4*>(smem + C::kRawV + (g & 1) * C::kRawBytes + tok * D +
                                                          ((p ^ (D == 128 ? tok & 7 : (tok >> 1) & 3)) << 4));
          const bool in = tok < behind;  // behind them anything may lie
          x[k][0] = in ? v.x : 0, x[k][1] = in ? v.y : 0, x[k][2] = in ? v.z : 0, x[k][3] = in ? v.w : 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) nan |= (x[k][j] & 0x7F7F7F7Fu) + 0x01010101u;  // bit 7 of a byte: 0x7F, 0xFF
        }
        nan &= 0x80808080u;
        had |= nan;
        if (nan != 0 || (dirty >> (g & 3) & 1)) {
          uint16_t* mask = reinterpret_cast<uint16_t*>(smem + C::kNan + (g & 3) * CH * 16) + (64 * atom + 2 * lane) * 8 + p;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t bits = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t is = ((x[k][j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
              x[k][j] &= ~(is | (is - (is >> 7)));  // whole bytes
              bits |= ((is >> 7) * 0x01020408u >> 24 & 15u) << (4 * j);
            }
            mask[8 * k] = uint16_t(bits);
          }
        }
        uint8_t* dst = smem + C::kV + (g & 1) * (CH * D * 2) + atom * (D * 128) + 16 * p * 128 + (lane & 3) * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t e[4];  // elements 4 j .. 4 j + 3 of the piece, of both tokens
          cvt4(__byte_perm(x[0][j], x[1][j], 0x5140), e[0], e[1]);
          cvt4(__byte_perm(x[0][j], x[1][j], 0x7362), e[2], e[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint32_t*>(dst + (4 * j + k) * 128 + (((lane >> 2) ^ ((4 * j + k) & 7)) << 4)) = e[k];
        }
      }
      dirty = (dirty & ~(1u << (g & 3))) | uint32_t(had != 0) << (g & 3);
      if (had) nan_block[g & 3] = g + 1;
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(v_full + (g & 1));
        tc::mbar_arrive(raw_v_free + (g & 1));
      }
      return true;
    };
    int g = 0;
    for (bool ok = true; ok && cur.c < cur.c_end; cur.next<CH, R>(a, G))
      for (int c = cur.c; ok && c < cur.c_end; ++c, ++g)
        ok = convert_v(g, cur.t.hi - (cur.t.chunk0 + c) * CH);
  } else if (warp == 13) {
    // ================= loads: lane i < SL has the 16-token slice i of a block
    const uint32_t raw_k_at = tc::smem_u32(smem + C::kRawK), raw_v_at = tc::smem_u32(smem + C::kRawV);
    int g = 0, ahead = 0;  // blocks whose copies have been issued; 1: the next one's keys as well
    bool ok = true;
    for (; ok && cur.c < cur.c_end; cur.next<CH, R>(a, G)) {
      const Tile& t = cur.t;
      auto page_of = [&](int c) {
        const int tok = (t.chunk0 + c) * CH + 16 * (lane & (SL - 1));
        return lane < SL && tok < t.hi ? a.block_table[t.b * a.max_pages + (tok >> P.page_shift)] : -1;
      };
      auto in_pool = [&](int phys) { return phys >= 0 && phys < a.n_pages; };
      // of a lane's slice: (key, value) scales; (1, 0) where no row sees it or it reads as zeros
      auto scales_of = [&](int c, int phys) {
        const int tok = (t.chunk0 + c) * CH + 16 * (lane & (SL - 1));
        if (lane >= SL || tok >= t.hi || !in_pool(phys)) return make_float2(1.0f, 0.0f);
        const int blk = phys * a.kv_heads + t.h;
        return make_float2(a.k_scale[blk], tok + 16 > t.lo ? a.v_scale[blk] : 0.0f);
      };
      // page ids are read two blocks ahead, scales one: their latency is hidden behind the waits
      int phys = page_of(cur.c), next = cur.c + 1 < cur.c_end ? page_of(cur.c + 1) : -1;
      float2 sc = scales_of(cur.c, phys);
      float unit = 0.0f, inverse = 0.0f;  // of the tile's values, and its reciprocal
      for (int c = cur.c; c < cur.c_end; ++c, ++g) {
        const int t0 = (t.chunk0 + c) * CH, tok = t0 + 16 * (lane & (SL - 1));
        const int box = 1 << P.box_shift;
        const int n_box = max(min(CH >> P.box_shift, (t.hi - t0 + box - 1) >> P.box_shift), 0);
        const uint32_t bytes = uint32_t(n_box * D) << P.box_shift;
        const bool in = in_pool(phys), wanted = lane < SL && tok < t.hi;
        if (wanted && !in) report_page(a.status, tok, t.lo);
        const int blk = in ? phys * a.kv_heads + t.h : int(a.n_pages) * a.kv_heads;  // behind the end: reads zeros
        const bool leads = wanted && (16 * lane & (box - 1)) == 0;
        auto issue = [&](const CUtensorMap* map, uint32_t dst, uint64_t* bar) {
          if (lane == 0) {
            if (n_box > 0)
              tc::mbar_expect_tx(bar, bytes);
            else
              tc::mbar_arrive(bar);
          }
          __syncwarp();
          if (leads) tma_load_3d(dst + 16 * lane * D, map, tc::smem_u32(bar), 0, tok & (a.page - 1), blk);
        };
        ok = g < 2 || wait(s_full + (g & 1), (g - 2) >> 1);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        issue(&P.k_map, raw_k_at + (g & 1) * C::kRawBytes, raw_k + (g & 1));
        ok = g < 2 || wait(raw_v_free + (g & 1), (g - 2) >> 1);
        ahead = !__all_sync(0xFFFFFFFFu, ok);
        if (ahead) break;
        issue(&P.v_map, raw_v_at + (g & 1) * C::kRawBytes, raw_v + (g & 1));
        // the largest value scale and the smallest but 0 (none is negative: their order is that of their bits)
        const float most = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(sc.y)));
        const float least = __uint_as_float(__reduce_min_sync(0xFFFFFFFFu, __float_as_uint(sc.y > 0.0f ? sc.y : INFINITY)));
        if (most > kUnits * unit) {
          unit = value_unit(unit, most, most * 0x1p-5f);
          inverse = per_unit(unit);
        }
        if (lane < SL) scales[SL * (g & 7) + lane] = make_float2(sc.x, sc.y * inverse);
        if (lane == 0) v_unit[g & 7] = most > kUnits * unit || least < unit ? -unit : unit;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(scales_full + (g & 7));
        if (c + 1 < cur.c_end) {
          phys = next;
          sc = scales_of(c + 1, phys);
          if (c + 2 < cur.c_end) next = page_of(c + 2);
        }
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
    }
    // Let the copies in flight land: one of each ring place at most is not awaited yet.  After a timeout, this
    // warp's or another's, nobody else waits for them.
    for (int i = 1; i <= 2; ++i) {
      const int k = g + ahead - i, v = g - i;
      if (k >= 0) tc::wait_bounded(raw_k + (k & 1), (k >> 1) & 1, abort_flag, tc::kDrainNs, a.status, true);
      if (v >= 0) tc::wait_bounded(raw_v + (v & 1), (v >> 1) & 1, abort_flag, tc::kDrainNs, a.status, true);
    }
  } else if (lane == 0) {
    // ================= the products
    const uint32_t q_at = tc::smem_u32(smem + C::kQ), k_at = tc::smem_u32(smem + C::kRawK);
    const uint64_t q_desc = D == 128 ? tc::sw128_desc(q_at) : tc::sw64_desc(q_at);
    const uint64_t k_desc = D == 128 ? tc::sw128_desc(k_at) : tc::sw64_desc(k_at);
    const uint64_t v_desc = tc::sw128_desc(tc::smem_u32(smem + C::kV));
    uint32_t first_bits = 0;  // bit g & 31: block g is the first of its tile here
    int pv = 0;               // the next block whose values are added
    auto product_pv = [&]() {
      const int g = pv++;
      if (!wait(v_full + (g & 1), g >> 1) || !wait(p_full + (g & 1), g >> 1)) return false;
      tc::tc_fence_after();
      const bool fresh = first_bits >> (g & 31) & 1;
      if (v_unit[g & 7] < 0.0f) {
        products_apart<CH, R, D>(tmem + C::kO, tmem + (g & 1) * CH, v_desc + (g & 1) * (CH * D * 2 / 16), fresh);
      } else {
#pragma unroll
        for (int k = 0; k < CH / 16; ++k)  // 16 tokens: 8 columns of P (in its half), 32 bytes of a row of V
          mma_a_tmem(tmem + C::kO, tmem + (g & 1) * CH + kCols * (k / (SL / 2)) + 8 * (k % (SL / 2)),
                     v_desc + (g & 1) * (CH * D * 2 / 16) + (k >> 2) * (D * 128 / 16) + 2 * (k & 3), idesc_f32(R, D),
                     !fresh || k > 0);
      }
      tc::tc_commit(o_done + (g & 1));
      return true;
    };
    int g = 0, tiles = 0;
    bool ok = true;
    for (; ok && cur.c < cur.c_end; cur.next<CH, R>(a, G), ++tiles) {
      for (int c = cur.c; ok && c < cur.c_end; ++c, ++g) {
        const bool first = c == cur.c;
        first_bits = (first_bits & ~(1u << (g & 31))) | uint32_t(first) << (g & 31);
        // the place of these scores was block g - 2's; at a tile's end everything is added before Q changes
        const int upto = first ? g - 1 : g - 2;
        while (ok && pv <= upto) ok = product_pv();
        if (ok && upto >= 0) ok = wait(o_done + (upto & 1), upto >> 1);
        ok = ok && wait(raw_k + (g & 1), g >> 1) && (!first || wait(q_full, tiles));
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < TERMS * (D / 32); ++k)  // 32 bytes of a row at a time, term after term
          mma_e4m3(tmem + (g & 1) * CH, q_desc + (k / (D / 32)) * (R * D / 16) + 2 * (k % (D / 32)),
                   k_desc + (g & 1) * (C::kRawBytes / 16) + 2 * (k % (D / 32)), idesc_f32(R, CH), k > 0);
        tc::tc_commit(s_full + (g & 1));
      }
    }
    while (ok && pv < g) ok = product_pv();
    tc::tc_commit(drain);  // nothing in flight when the memory goes
    tc::wait_bounded(drain, 0, abort_flag, tc::kDrainNs, a.status, true);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 12) tc::tmem_dealloc(tmem, C::kTmemCols);
}

template <typename T, int D>
static cudaError_t launch_rows(const RowsParams& P, int ctas, cudaStream_t stream) {
  using C = RowsOf<T, D>;
  constexpr int kSmem = C::kSmem;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  auto kernel = attn_kv8_rows_kernel<T, D>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(unsigned(ctas)), dim3(C::kThreads), kSmem, stream, P);
}

}  // namespace attn

// Counters (where attn_kv8.cu has its own), then two tile states for each CTA, of which every SM has one.
static size_t rows_counter_bytes(int num_sms) { return (size_t(num_sms) * 4 + 255) / 256 * 256; }
static size_t rows_state_bytes(int64_t head_dim) {
  return 2 * 4 * size_t(head_dim == 128 ? attn::RowsCfg<128, 2>::kStateFloats : attn::RowsCfg<64, 2>::kStateFloats);
}
size_t attn_kv8_rows_workspace_bytes(int64_t head_dim, int num_sms) {
  return rows_counter_bytes(num_sms) + num_sms * rows_state_bytes(head_dim);
}

cudaError_t launch_attn_kv8_rows(const AttnParams& a, int head_dim, int dtype, void* workspace,
                                 int num_sms, uint64_t limit_ns, cudaStream_t stream) {
  attn::RowsParams P = {};
  P.a = a;
  P.counters = static_cast<uint32_t*>(workspace);
  P.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + rows_counter_bytes(num_sms));
  P.limit_ns = limit_ns;
  const int box = int(a.page);  // up to a whole block
  for (P.page_shift = 4; (1 << P.page_shift) < a.page;) ++P.page_shift;
  for (P.box_shift = 4; (1 << P.box_shift) < box;) ++P.box_shift;
  if (!make_map_pages_u8(&P.k_map, a.k, head_dim, a.page, a.n_pages * a.kv_heads, box) ||
      !make_map_pages_u8(&P.v_map, a.v, head_dim, a.page, a.n_pages * a.kv_heads, box))
    return cudaErrorInvalidValue;
  if (dtype == PATCH_DTYPE_BF16)
    return head_dim == 128 ? attn::launch_rows<__nv_bfloat16, 128>(P, num_sms, stream)
                           : attn::launch_rows<__nv_bfloat16, 64>(P, num_sms, stream);
  return head_dim == 128 ? attn::launch_rows<__half, 128>(P, num_sms, stream)
                         : attn::launch_rows<__half, 64>(P, num_sms, stream);
}

}  // namespace patch
