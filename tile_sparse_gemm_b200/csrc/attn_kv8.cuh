// Shared by the kernels of attention over the paged 8-bit cache: row tiles,
// their chunks of tokens, and equal shares of all chunks for the CTAs.
#pragma once

#include "common.cuh"
#include "decoder.cuh"
#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace patch {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

// four e4m3 bytes to two fp16 pairs (exact)
__device__ __forceinline__ void cvt4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// The unit of a tile's sums of values: a power of two, not far from the value scales that its tokens have, since what
// enters the tensor cores is fp16.  `most`: the largest scale of the tokens that come next; `to`: the unit wanted
// for it.  A unit only grows, and by at most 2^100 unless `most` is out of fp32's reach under it, so that sums
// under the old one keep their bits whatever becomes of the new tokens; 2^19 is enough for any scale.
__device__ __forceinline__ float value_unit(float unit, float most, float to) {
  float u = fminf(to, 0x1p19f);
  if (unit > 0.0f) u = fmaxf(fmaxf(unit, fminf(u, unit * 0x1p100f)), most * 0x1p-100f);
  return __uint_as_float(__float_as_uint(u) & 0xFF800000u);
}
// 1 / unit, exact (2^-119 .. 2^125 for a unit of 2^-108 .. 2^19); anything finite for 0
__device__ __forceinline__ float per_unit(float unit) { return __uint_as_float((254u << 23) - __float_as_uint(unit)); }

__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

// A row tile of one sequence and head: which tokens its rows see.
struct Tile {
  int b, h, rt;
  int len, m, row0;    // the sequence's tokens, queries, first row of q
  int chunk0, chunks;  // its run of chunks (at least one, so that every tile is written)
  int lo, hi;          // tokens before lo, and from hi on, are seen by no row
};

__device__ __forceinline__ void sequence(const AttnParams& a, int b, int& len, int& m, int& row0) {
  if (a.cu_q) {
    row0 = min(max(a.cu_q[b], 0), a.n_tokens);
    m = min(max(a.cu_q[b + 1], row0), a.n_tokens) - row0;
  } else {
    row0 = b;
    m = 1;
  }
  len = int(min(int64_t(max(a.kv_lens[b], 0)), a.max_pages * a.page));
}

// x / G, the rows of a token: a shift for powers of two (a division's latency is most of what a tile costs
// in the sums below)
__device__ __forceinline__ int by_group(int x, int G) {
  return (G & (G - 1)) == 0 ? x >> (31 - __clz(G)) : x / G;
}

template <int CH, int R>
__device__ __forceinline__ void set_rows(const AttnParams& a, int G, Tile& t) {
  int hi = t.len, lo = 0;
  if (a.causal) hi = max(0, min(t.len, t.len - t.m + min(t.m - 1, by_group(t.rt * R + R - 1, G)) + 1));
  if (a.window > 0) lo = int(max(int64_t(0), int64_t(t.len) - t.m + by_group(t.rt * R, G) - a.window + 1));
  t.lo = lo;
  t.hi = hi;
  t.chunk0 = lo / CH;
  t.chunks = max(1, (hi + CH - 1) / CH - t.chunk0);
}
template <int R>
__device__ __forceinline__ int row_tiles(int m, int G) {
  return (m * G + R - 1) / R;
}

// Shares are equal in units: a chunk is one, and a tile's own cost (its queries, its output) is
// tile_units in front of its chunks: about half a chunk's time in a warp with 8 or 16 rows, 8000
// cycles against a block's 2600 with 128 (four prompts of 100 to 512 tokens over up to 8000: 218 us with
// one unit, 205 with two, 200 with four or six; 64 single tokens over up to 8000, 8 rows: 95 us with one, 101 with two).
template <int R>
constexpr int tile_units() {
  return R == 128 ? 4 : 1;
}

// units of all of a sequence's tiles of one head
template <int CH, int R>
__device__ __forceinline__ int64_t units_per_head(const AttnParams& a, int G, Tile& t) {
  const int n = row_tiles<R>(t.m, G);
  if (n == 0) return 0;
  if (!a.causal) {
    t.rt = 0;
    set_rows<CH, R>(a, G, t);
    return int64_t(n) * (t.chunks + tile_units<R>());
  }
  int64_t s = 0;
#pragma unroll 4
  for (t.rt = 0; t.rt < n; ++t.rt) {
    set_rows<CH, R>(a, G, t);
    s += t.chunks + tile_units<R>();
  }
  return s;
}
// to the next tile, in the order (sequence, head, row tile)
template <int CH, int R>
__device__ __forceinline__ void next_tile(const AttnParams& a, int G, Tile& t) {
  if (++t.rt >= row_tiles<R>(t.m, G)) {
    t.rt = 0;
    if (++t.h == a.kv_heads) {
      t.h = 0;
      do {
        if (++t.b >= a.batch) return;
        sequence(a, t.b, t.len, t.m, t.row0);
      } while (t.m == 0);
    }
  }
  set_rows<CH, R>(a, G, t);
}

// A warp's place in its share: chunks c .. c_end - 1 of tile t are next, `left`
// units of the share count from the tile's first on.  c == c_end: done.
struct Cursor {
  Tile t;
  int c, c_end;
  int64_t left;

  template <int R>
  __device__ __forceinline__ void clip() {
    c_end = int(min(int64_t(t.chunks), max(left - tile_units<R>(), int64_t(0))));
  }
  // The part [v0, v1) of all units; at: the sequence that v0 lies in and the units before it (make_share).
  template <int CH, int R>
  __device__ __forceinline__ void start(const AttnParams& a, int G, const int64_t* at, int64_t v0, int64_t v1);
  template <int CH, int R>
  __device__ __forceinline__ void next(const AttnParams& a, int G) {
    left -= t.chunks + tile_units<R>();
    c = c_end = 0;
    if (left <= tile_units<R>()) return;
    next_tile<CH, R>(a, G, t);
    clip<R>();
  }
};

__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? int64_t(uint32_t(x) / uint32_t(y)) : x / y;
}

// A CTA's share [u0, u0 + u_n) of all W units: the first `more` CTAs take per + 1, the others per.
struct Share {
  int64_t u0, u_n, per, more;
  __device__ __forceinline__ int64_t start(int i, int n) const { return u0 + u_n * i / n; }  // of n equal parts
  __device__ __forceinline__ int64_t owner(int64_t u) const {                                // CTA of a unit
    const int64_t cut = more * (per + 1);
    return u < cut ? quotient(u, per + 1) : more + quotient(u - cut, per);
  }
};

// The whole CTA of kWarps warps.  misc: kWarps words, then for each of kStarts equal parts
// of the share the sequence it begins in and the units before that.  A share has kStarts units
// where all together are fewer than that a CTA.  false: no work for this CTA.
template <int CH, int R, int kWarps, int kStarts>
__device__ __forceinline__ bool make_share(const AttnParams& a, int G, int64_t* misc, Share& s) {
  constexpr int kThreads = 32 * kWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto units_of = [&](int b) -> int64_t {
    if (b >= a.batch) return 0;
    Tile t;
    sequence(a, b, t.len, t.m, t.row0);
    return units_per_head<CH, R>(a, G, t) * a.kv_heads;
  };
  auto warp_scan = [&](int64_t v) {  // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v += y;
    }
    return v;
  };
  const int64_t mine = units_of(threadIdx.x);  // the only sequences unless there are more than threads
  int64_t rest = 0;
  for (int b = threadIdx.x + kThreads; b < a.batch; b += kThreads) rest += units_of(b);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
      const int len = a.kv_lens[b];
      if (len < 0 || len > a.max_pages * a.page) set_status(a.status, PATCH_DEV_BOUNDS);
    }
  int64_t in = warp_scan(mine), W = 0;
  {
    const int64_t all = a.batch > kThreads ? warp_scan(mine + rest) : in;
    if (lane == 31) misc[warp] = all;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) W += misc[w];
  }
  const int64_t n_cta = min(int64_t(gridDim.x), (W + kStarts - 1) / kStarts);
  if (blockIdx.x >= n_cta) return false;
  s.per = quotient(W, n_cta);
  s.more = W - s.per * n_cta;
  s.u0 = s.per * blockIdx.x + min(int64_t(blockIdx.x), s.more);
  s.u_n = s.per + (blockIdx.x < s.more ? 1 : 0);
  int64_t before = 0;
  for (int base = 0; base < a.batch; base += kThreads) {
    const int64_t v = base ? units_of(base + threadIdx.x) : mine;
    if (base || a.batch > kThreads) {
      if (base) in = warp_scan(v);
      __syncthreads();
      if (lane == 31) misc[warp] = in;
      __syncthreads();
    }
    int64_t ex = before + in - v;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) ex += misc[w];
      before += misc[w];
    }
#pragma unroll
    for (int i = 0; i < kStarts; ++i) {
      const int64_t u = s.start(i, kStarts);
      if (ex <= u && u < ex + v) {
        misc[kWarps + 2 * i] = base + threadIdx.x;
        misc[kWarps + 2 * i + 1] = ex;
      }
    }
    if (before >= s.u0 + s.u_n) break;
  }
  __syncthreads();
  return true;
}

template <int CH, int R>
__device__ __forceinline__ void Cursor::start(const AttnParams& a, int G, const int64_t* at, int64_t v0, int64_t v1) {
  t.b = int(at[0]);
  sequence(a, t.b, t.len, t.m, t.row0);
  int64_t off = v0 - at[1];
  const int64_t per_head = units_per_head<CH, R>(a, G, t);
  t.h = int(quotient(off, per_head));
  off -= per_head * t.h;
  t.rt = 0;
  set_rows<CH, R>(a, G, t);
  while (off >= t.chunks + tile_units<R>()) {
    off -= t.chunks + tile_units<R>();
    ++t.rt;
    set_rows<CH, R>(a, G, t);
  }
  left = v1 - (v0 - off);
  c = int(max(off - tile_units<R>(), int64_t(0)));
  clip<R>();
}

}  // namespace attn
}  // namespace patch
