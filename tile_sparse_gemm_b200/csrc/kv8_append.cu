// New keys and values into the paged 8-bit cache, keys rotated on the way
// (include/patch.h: patch_kv8_append).
//
// A page, head and tensor (k or v) belongs to one CTA, which finds its new tokens'
// largest magnitude, takes the scale and rounds them.  The scale is a power of
// two: e4m3 keeps its relative precision under any scale, scaling is exact, and a
// page whose scale grows as tokens arrive is stored again without a second rounding.
//
// Prompts are bound by bandwidth (2 bytes in, 1 out): a thread holds one unit of 16
// elements of a page in registers between the two passes, each input is read once
// and each output written once; the CTA takes several heads, the next one's loads
// under way meanwhile, and reads the angles of the page's tokens once for all of
// them.  8 prompts of 4096 tokens, 8 heads of 128: 47 us, 4.3 TB/s; what is lost is
// mostly each CTA's start (its sequence, block and angles: four loads in a row) and a
// barrier a head.  Loads two heads ahead do not help (50 us).  Decode steps (a token
// or a few per page) are bound by latency: small CTAs, one head each, that read their
// tokens twice; 64 sequences of one token 3.9 us.
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

// A touched page: the tokens begin .. begin + count - 1 of a sequence are rows row .. of k and v.
struct Touched {
  int64_t row, begin, phys;
  int off, count;
};

// Item -> (sequence, page of it).  Sequence b owns the items from cu[b] / page + 2 b
// on: at least as many as the pages its tokens touch.  count == 0: none.
__device__ __forceinline__ Touched touched(const AppendParams& P, int64_t item) {
  Touched t = {};
  int b, j = 0;
  int64_t row0, n = 1;
  if (P.cu_new) {
    const int32_t* cu = P.cu_new;
    const int page = P.page;
    b = warp_find(P.batch, item, [&](int i) { return int64_t(cu[i] / page) + 2 * i; });
    if (b >= P.batch) return t;
    row0 = cu[b];
    n = min(int64_t(cu[b + 1]), int64_t(P.n_tokens)) - row0;
    if (row0 < 0) return t;
    j = int(item - (row0 / page + 2 * b));
  } else {
    b = int(item);
    row0 = b;
  }
  const int past = P.past_lens[b];
  const bool bad = past < 0;  // none of its tokens is stored; its first item says so
  const int64_t page_no = max(past, 0) / P.page + j;
  const int64_t begin = max(int64_t(past), page_no * P.page), end = min(past + n, (page_no + 1) * P.page);
  if (begin >= end && (!bad || j > 0 || n <= 0)) return t;
  t.begin = begin;
  t.count = max(int(end - begin), 1);
  t.off = int(begin - page_no * P.page);
  t.row = bad ? row0 : row0 + begin - past;
  t.phys = !bad && page_no < P.max_pages ? P.block_table[b * P.max_pages + page_no] : -1;
  return t;
}

// Where a unit of 16 elements lies in a head: a rotated unit is 8 pairs (two
// 8-element pieces), one behind the rotated part 16 elements in a row.
template <bool kInterleaved>
struct Unit {
  int tok, unit, d0, d1;
  bool pair;
  __device__ __forceinline__ Unit(int idx, int per_token, bool turn, int rot_units) {
    tok = idx / per_token;
    unit = idx % per_token;
    pair = turn && unit < rot_units;
    d0 = pair && !kInterleaved ? 8 * unit : 16 * unit;
    d1 = pair && !kInterleaved ? d0 + 8 * rot_units : d0 + 8;
  }
  __device__ __forceinline__ void angles(const AppendParams& P, int64_t begin, float (&cs)[16]) const {
    const float4* tab = reinterpret_cast<const float4*>(P.table + (begin + tok) * (16 * P.rot_units) + 16 * unit);
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(cs + 4 * i) = __ldg(tab + i);
  }
};

// the larger of amax and the unit's magnitudes (NaN left out by fmaxf)
__device__ __forceinline__ float magnitude(const float (&x)[16], float amax) {
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  return amax;
}
// the same without infinities, which do not set the scale either
__device__ __forceinline__ float finite_magnitude(const float (&x)[16], float amax) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (fabsf(x[i]) < INFINITY) amax = fmaxf(amax, fabsf(x[i]));
  return amax;
}

// 1 / scale, exact for a power of two of the cache's range
__device__ __forceinline__ float inverse(float scale) {
  const uint32_t b = __float_as_uint(scale);
  return (b & 0x7FFFFFu) == 0 ? __uint_as_float((254u << 23) - b) : 1.0f / scale;
}

__device__ __forceinline__ void store_unit(uint8_t* row, int d0, int d1, const float (&x)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_e4m3x4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
  *reinterpret_cast<uint2*>(row + d0) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(row + d1) = make_uint2(w[2], w[3]);
}

// the CTA's largest value (none below 0: their order is that of their bits), on every thread; one barrier
template <int kThreads>
__device__ __forceinline__ float cta_max(float v, uint32_t* part) {
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, lane < kThreads / 32 ? part[lane] : 0u));
}

// The page's scale, given the new tokens' largest magnitude and (off > 0) its present one; the
// tokens that the page holds are stored again if it grows.
template <int D, int kThreads>
__device__ __forceinline__ float settle_scale(float amax, float held, int off, float* scale_at, uint8_t* page) {
  const float scale = fmaxf(pow2i(scale_exponent(__float_as_uint(amax))), held);
  if (threadIdx.x == 0) *scale_at = scale;
  if (off > 0 && scale > held) {
    const float f = held / scale;  // exact: powers of two
    for (int i = threadIdx.x; i < off * (D / 16); i += kThreads) {
      uint4 w = reinterpret_cast<uint4*>(page)[i];
      uint32_t* e = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        e[q] = pack_e4m3x4(e4m3_to_f32(e[q] & 255) * f, e4m3_to_f32((e[q] >> 8) & 255) * f,
                           e4m3_to_f32((e[q] >> 16) & 255) * f, e4m3_to_f32(e[q] >> 24) * f);
      reinterpret_cast<uint4*>(page)[i] = w;
    }
  }
  return scale;
}

// kThreads = page * D / 16: one unit of a full page each.
template <typename T, int D, bool kInterleaved, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) kv8_append_kernel(const __grid_constant__ AppendParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Touched t = touched(P, blockIdx.x);
  if (t.count == 0) return;
  const int which = blockIdx.z;
  const bool turn = which == 0 && P.rot_units > 0;
  const int h0 = blockIdx.y * P.heads_per_cta, h1 = min(h0 + P.heads_per_cta, P.kv_heads);
  const Unit<kInterleaved> u(threadIdx.x, D / 16, turn, P.rot_units);
  const bool live = u.tok < t.count;
  const T* src = static_cast<const T*>(P.x[which]) + (t.row + u.tok) * P.ts[which] + h0 * P.hs[which];
  uint4 raw0 = {}, raw1 = {};
  if (live) {
    raw0 = *reinterpret_cast<const uint4*>(src + u.d0);
    raw1 = *reinterpret_cast<const uint4*>(src + u.d1);
  }
  if (t.phys < 0 || t.phys >= P.n_pages || (P.rot_units > 0 && t.begin + t.count > P.n_pos)) {
    if (threadIdx.x == 0) set_status(P.status, PATCH_DEV_BOUNDS);
    return;
  }
  float cs[16];
  if (u.pair && live) u.angles(P, t.begin, cs);
  __shared__ uint32_t part[3][kThreads / 32];
  for (int h = h0; h < h1; ++h) {
    float x[16];
    load16(reinterpret_cast<const T*>(&raw0), x);
    load16(reinterpret_cast<const T*>(&raw1), x + 8);
    if (u.pair && live) rotate_unit<8, kInterleaved>(x, cs, 1.0f);
    if (h + 1 < h1 && live) {
      src += P.hs[which];
      raw0 = *reinterpret_cast<const uint4*>(src + u.d0);
      raw1 = *reinterpret_cast<const uint4*>(src + u.d1);
    }
    float* scale_at = P.scale[which] + t.phys * P.kv_heads + h;
    const float held = t.off > 0 ? *scale_at : 0.0f;
    // two buffers in turn: a thread is at most one barrier ahead
    float amax = cta_max<kThreads>(magnitude(x, 0.0f), part[h & 1]);
    if (amax == INFINITY) amax = cta_max<kThreads>(finite_magnitude(x, 0.0f), part[2]);
    uint8_t* page = P.cache[which] + (t.phys * P.kv_heads + h) * (int64_t(P.page) * D);
    const float scale = settle_scale<D, kThreads>(amax, held, t.off, scale_at, page);
    if (live) store_unit(page + (t.off + u.tok) * D, u.d0, u.d1, x, inverse(scale));
  }
}

// Any number of tokens with few threads: a unit is read again for the second pass.
template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(64) kv8_append_few_kernel(const __grid_constant__ AppendParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Touched t = touched(P, blockIdx.x);
  if (t.count == 0) return;
  const int which = blockIdx.z, h = blockIdx.y;
  const bool turn = which == 0 && P.rot_units > 0;
  const T* src = static_cast<const T*>(P.x[which]) + t.row * P.ts[which] + h * P.hs[which];
  if (t.phys < 0 || t.phys >= P.n_pages || (P.rot_units > 0 && t.begin + t.count > P.n_pos)) {
    if (threadIdx.x == 0) set_status(P.status, PATCH_DEV_BOUNDS);
    return;
  }
  auto load = [&](const Unit<kInterleaved>& u, float (&x)[16]) {
    const T* row = src + u.tok * P.ts[which];
    load16(row + u.d0, x);
    load16(row + u.d1, x + 8);
    if (u.pair) {
      float cs[16];
      u.angles(P, t.begin, cs);
      rotate_unit<8, kInterleaved>(x, cs, 1.0f);
    }
  };
  float* scale_at = P.scale[which] + t.phys * P.kv_heads + h;
  const float held = t.off > 0 ? *scale_at : 0.0f;
  const int units = t.count * (D / 16);
  float amax = 0.0f;
  for (int i = threadIdx.x; i < units; i += 64) {
    float x[16];
    load(Unit<kInterleaved>(i, D / 16, turn, P.rot_units), x);
    amax = magnitude(x, amax);
  }
  __shared__ uint32_t part[2][2];
  amax = cta_max<64>(amax, part[0]);
  if (amax == INFINITY) {
    amax = 0.0f;
    for (int i = threadIdx.x; i < units; i += 64) {
      float x[16];
      load(Unit<kInterleaved>(i, D / 16, turn, P.rot_units), x);
      amax = finite_magnitude(x, amax);
    }
    amax = cta_max<64>(amax, part[1]);
  }
  uint8_t* page = P.cache[which] + (t.phys * P.kv_heads + h) * (int64_t(P.page) * D);
  const float scale = settle_scale<D, 64>(amax, held, t.off, scale_at, page);
  for (int i = threadIdx.x; i < units; i += 64) {
    const Unit<kInterleaved> u(i, D / 16, turn, P.rot_units);
    float x[16];
    load(u, x);
    store_unit(page + (t.off + u.tok) * D, u.d0, u.d1, x, inverse(scale));
  }
}

template <typename T, int D, bool kInterleaved>
static cudaError_t launch_append(AppendParams P, int num_sms, cudaStream_t stream) {
  const int64_t items = P.cu_new ? P.n_tokens / P.page + 2 * int64_t(P.batch) : P.batch;
  const int units = P.page * (D / 16);  // of a full page: 64 ... 1024
  const int64_t ctas = items * P.kv_heads * 2, at_once = int64_t(num_sms) * (1024 / units);  // 1024 threads an SM
  // Up to half a page per sequence, and more page-wide CTAs than run at once: the small ones (8 heads of 128,
  // page 64; 64 sequences of 1 token 3.9 us against 9.4, of 32 tokens 8.2 against 10.8, of 64 tokens 13.1
  // against 13.9, of 128 17.3 against 14.9; one sequence of 1 token 2.7 against 2.6, of 32 tokens 5.1 against 2.9).
  if (ctas > at_once && int64_t(P.n_tokens) * 2 <= int64_t(P.batch) * P.page)
    return launch_pdl(kv8_append_few_kernel<T, D, kInterleaved>, dim3(unsigned(items), unsigned(P.kv_heads), 2),
                      dim3(64), 0, stream, P);
  // Heads of a CTA: as many as let all CTAs run at once, a third or more of which find no page (two spare items
  // a sequence).  1, 2, 4, 8 heads: 8 x 1024 tokens 22.5, 17.0, 14.5, 12.7 us; 1 x 2048 6.9, 5.2, 5.6, 8.6;
  // 1 x 512 3.9, 4.0, 5.5, 8.5.
  P.heads_per_cta = int(ctas >= 8 * at_once ? 8 : (ctas + at_once - 1) / at_once);
  const dim3 grid(unsigned(items), unsigned((P.kv_heads + P.heads_per_cta - 1) / P.heads_per_cta), 2);
  if (units == 64) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 64>, grid, dim3(64), 0, stream, P);
  if (units == 128) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 128>, grid, dim3(128), 0, stream, P);
  if (units == 256) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 256>, grid, dim3(256), 0, stream, P);
  if (units == 512) return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 512>, grid, dim3(512), 0, stream, P);
  return launch_pdl(kv8_append_kernel<T, D, kInterleaved, 1024>, grid, dim3(1024), 0, stream, P);
}

cudaError_t launch_kv8_append(AppendParams P, int head_dim, int dtype, int layout, int num_sms, cudaStream_t stream) {
  const bool il = layout == PATCH_ROPE_INTERLEAVED && P.rot_units > 0;
  if (dtype == PATCH_DTYPE_BF16) {
    if (head_dim == 128)
      return il ? launch_append<__nv_bfloat16, 128, true>(P, num_sms, stream) : launch_append<__nv_bfloat16, 128, false>(P, num_sms, stream);
    return il ? launch_append<__nv_bfloat16, 64, true>(P, num_sms, stream) : launch_append<__nv_bfloat16, 64, false>(P, num_sms, stream);
  }
  if (head_dim == 128) return il ? launch_append<__half, 128, true>(P, num_sms, stream) : launch_append<__half, 128, false>(P, num_sms, stream);
  return il ? launch_append<__half, 64, true>(P, num_sms, stream) : launch_append<__half, 64, false>(P, num_sms, stream);
}

}  // namespace patch
