// Attention of new tokens over the paged 8-bit cache (include/patch.h:
// patch_attn_kv8).
//
// Mathematics.  For a tile of query rows (the queries of one sequence that
// share a key/value head, R = 8 or 16 at a time) the cache is read once with
// the running maximum m and sum l of the softmax,
//   m' = max(m, s),  l' = l 2^(m - m') + 2^(s - m'),  o' = o 2^(m - m') + 2^(s - m') v,
// scores in units of log 2.  States (m, l, o) of parts of the keys join the
// same way, so the keys of a tile can be cut anywhere.
//
// What bounds it: bytes of the cache (2 D a token and head) for few rows.  So
// the work is cut by bytes: every (sequence, head, row tile) is a run of chunks
// of 32 (D = 128) or 64 (D = 64) tokens, 8 KiB of keys and values each, and
// every warp of every CTA (8 warps, one CTA per SM) takes an equal share of all
// chunks in a row, wherever tiles begin and end; the sequences' lengths are read
// on the device.  A warp fetches its chunks by TMA into a ring of its own and
// waits for no other warp until its share is done.  A tile that lies in one
// warp's share is written by it; the pieces of the others are joined through
// shared memory, and of a tile cut between CTAs by the last CTA to arrive, in
// the order of the pieces (deterministic).
//
// Tensor cores (mma.sync m16n8k16, fp16 in, fp32 out): tokens are the 16 rows,
// queries the 8 columns, S^T = K Q^T and O^T = V^T P^T, since a decode step has
// 1 to 8 query rows per key/value head and tcgen05's smallest M of 64 would be
// filled with padding; here one instruction takes 256 cached values.  e4m3 is
// a subset of fp16, so keys and values are converted exactly (one cvt for two)
// on their way from shared memory to the operand registers.  The contracted
// index of a product may run in any order: each lane's 16-byte pieces of a
// cache row serve directly as its operands, and values are transposed by a
// byte permute of two tokens' words.  A page's key scale multiplies the scores,
// its value scale (in units of a power of two near the tile's first) the probabilities;
// what fp16 cannot hold with all its bits there is weighed in fp32 (`apart` below).
//
// Measured (32 heads over 8 of 128): 64 sequences of up to 8000 tokens, 502 MB, 95 us
// (5.3 TB/s; the loop itself runs at 7); one sequence of 131000, 268 MB, 57 us (4.7 TB/s).
// One of 1500, 32 heads over 32, 12 us: about 5 us until the first bytes are there
// (launch, lengths, block table, TMA), 2 to work, 3 to join.
#include <type_traits>

#include "attn_kv8.cuh"

namespace patch {
namespace attn {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunkBytes = 4096;  // of keys, and of values
constexpr float kUnits = 32768.0f;  // of value scales: 2^15, times a probability within fp16

struct Params {
  CUtensorMap k_map, v_map;
  AttnParams a;
  uint32_t* counters;  // one per CTA: arrivals at the tile that begins in it and goes on
  float* parts;        // two tile states per CTA
  uint64_t limit_ns;
  int page_shift, box_shift;  // log2 of a page's and a TMA box's tokens
};

template <int D, int NT>
struct Cfg {
  static constexpr int CH = kChunkBytes / D;  // tokens of a chunk
  static constexpr int SL = CH / 16;          // slices of 16 tokens
  static constexpr int KS = D / 16;           // k steps of S, row tiles of O
  static constexpr int R = 8 * NT;            // query rows of a tile
  static constexpr int STAGES = NT == 1 ? 3 : 2;
  static constexpr int kStateFloats = R * D + 2 * R;  // o, m, l of a tile
  static constexpr int kStateBytes = kStateFloats * 4;
  static constexpr int kRingBytes = STAGES * 2 * kChunkBytes;  // of a warp
  static constexpr int kHeads = kWarps * kRingBytes;           // a state for each warp: the tile it entered in the middle
  static constexpr int kBars = kHeads + kWarps * kStateBytes;  // full barriers
  static constexpr int kScales = kBars + kWarps * STAGES * 8;  // ring of scales: up to 4 boxes x (k, v)
  static constexpr int kPieces = kScales + kWarps * STAGES * 32;
  static constexpr int kMisc = kPieces + 2 * kWarps * 48;
  static constexpr int kSmem = kMisc + 256;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint4 lds128(const uint8_t* a) { return *reinterpret_cast<const uint4*>(a); }
__device__ __forceinline__ uint2 lds64(const uint8_t* a) { return *reinterpret_cast<const uint2*>(a); }
// A piece of a tile that one warp did not do alone.
struct Piece {
  int valid, ends;  // ends: it holds the tile's last chunk
  int row0, m, rt, h, chunks, pad;
  int64_t unit0;    // of the tile
  int64_t pad2;
};
static_assert(sizeof(Piece) == 48, "kPieces");

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) attn_kv8_kernel(const __grid_constant__ Params P) {
  using C = Cfg<D, NT>;
  constexpr int CH = C::CH, SL = C::SL, KS = C::KS, R = C::R, STAGES = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  const AttnParams& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, q4 = lane & 3;
  const int G = a.heads / a.kv_heads;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars) + warp * STAGES;
  float* scales = reinterpret_cast<float*>(smem + C::kScales) + warp * STAGES * 8;
  Piece* pieces = reinterpret_cast<Piece*>(smem + C::kPieces);
  int64_t* misc = reinterpret_cast<int64_t*>(smem + C::kMisc);  // of make_share: 24 words
  int* abort_flag = reinterpret_cast<int*>(misc + 24);
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) tc::mbar_init(bars + s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pieces[2 * warp].valid = pieces[2 * warp + 1].valid = 0;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.k_map)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.v_map)) : "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // queries, lengths and cache come from earlier kernels

  // ---- this CTA's share of all units, and each warp's first sequence
  Share sh;
  if (!make_share<CH, R, kWarps, kWarps>(a, G, misc, sh)) return;

  // ---- this warp's share
  Cursor cur{};
  cur.start<CH, R>(a, G, misc + kWarps + 2 * warp, sh.start(warp, kWarps), sh.start(warp + 1, kWarps));

  // ---- a second cursor runs ahead and fetches
  const uint32_t ring = tc::smem_u32(smem) + warp * C::kRingBytes;
  Cursor fet = cur;
  int issued = 0;
  auto fetch = [&]() {  // the whole warp
    if (fet.c < fet.c_end) {
      const int st = issued % STAGES;
      const int t0 = (fet.t.chunk0 + fet.c) * CH;
      const int box = 1 << P.box_shift;
      const int n_box = min(CH >> P.box_shift, (fet.t.hi - t0 + box - 1) >> P.box_shift);  // < 1: a tile that sees nothing
      const uint32_t bar = tc::smem_u32(bars + st);
      if (lane == 0) {
        if (n_box > 0)
          tc::mbar_expect_tx(bars + st, uint32_t(n_box) * uint32_t(2 * D) << P.box_shift);
        else
          tc::mbar_arrive(bars + st);
      }
      __syncwarp();
      if (lane < n_box) {
        const int tok = t0 + (lane << P.box_shift), in_page = tok & (a.page - 1);
        const int phys = a.block_table[fet.t.b * a.max_pages + (tok >> P.page_shift)];
        const bool ok = phys >= 0 && phys < a.n_pages;
        if (!ok && tok + box > fet.t.lo) set_status(a.status, PATCH_DEV_BOUNDS);  // else before the window
        const int blk = ok ? phys * a.kv_heads + fet.t.h : int(a.n_pages) * a.kv_heads;  // behind the end: reads zeros
        const uint32_t dst = ring + st * 2 * kChunkBytes + lane * (D << P.box_shift);
        tma_load_3d(dst, &P.k_map, bar, 0, in_page, blk);
        tma_load_3d(dst + kChunkBytes, &P.v_map, bar, 0, in_page, blk);
        // a box's scales, asynchronously too (a page outside the pool reads as zeros under any scale)
        const int sc = ok ? blk : 0;
        cp_async4(scales + st * 8 + 2 * lane, a.k_scale + sc);
        cp_async4(scales + st * 8 + 2 * lane + 1, a.v_scale + sc);
      }
      ++issued;
      if (++fet.c == fet.c_end) fet.next<CH, R>(a, G);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");  // one group a call, on every lane
  };
  for (int s = 0; s < STAGES; ++s) fetch();

  int done = 0;  // chunks that have come and been used
  bool lost = false;
  for (; cur.c < cur.c_end; cur.next<CH, R>(a, G)) {
    const Tile& t = cur.t;
    // ---- the rows' queries as operands, each row divided by a power of two
    uint32_t qf[NT][KS][2];
    float row_scale[NT][2];  // of this lane's accumulator columns 2 q4, 2 q4 + 1
    int see_lo[NT][2], see_hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = t.rt * R + 8 * nt + n;
      const bool live = row < t.m * G;
      float x[D / 4];
      float amax = 0.0f;
      const T* src = static_cast<const T*>(a.q) + int64_t(t.row0 + row / G) * a.q_ts +
                     int64_t(t.h * G + row % G) * a.q_hs + (D / 4) * q4;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        if (live) {
          load16(src + 8 * i, x + 8 * i);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[8 * i + j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[8 * i + j]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // `up`: 2^x with amax in [2^x, 2^(x+1)), x from -126 to 126 so that 1 / up is normal as well; an infinity stays one
      const uint32_t ex = __float_as_uint(amax) >> 23, fit = min(max(ex, 1u), 253u);
      const float down = ex == 255 ? 1.0f : __uint_as_float((254 - fit) << 23);
      const float up = ex == 255 ? 1.0f : __uint_as_float(fit << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[nt][s][0] = pack_f16(x[4 * s] * down, x[4 * s + 1] * down);
        qf[nt][s][1] = pack_f16(x[4 * s + 2] * down, x[4 * s + 3] * down);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = t.rt * R + 8 * nt + 2 * q4 + e;
        row_scale[nt][e] = __shfl_sync(0xFFFFFFFFu, up, 4 * (2 * q4 + e)) * (a.scale * kLog2e);
        const int pos = t.len - t.m + r / G;
        see_hi[nt][e] = r < t.m * G ? (a.causal ? min(t.len, pos + 1) : t.len) : 0;
        see_lo[nt][e] = a.window > 0 ? int(max(int64_t(0), pos - a.window + 1)) : 0;
      }
    }
    const int all_hi = a.causal ? t.len - t.m + t.rt * R / G + 1 : t.len;  // every row sees the tokens before it ...
    const int last_row = min(t.m - 1, (t.rt * R + R - 1) / G);
    const int all_lo = a.window > 0 ? int(max(int64_t(0), t.len - t.m + last_row - a.window + 1)) : 0;  // ... from here on

    // The softmax state in the layout of the O^T accumulators: rows 8 nt + 2 q4 + e
    // of the tile; elements 16 n + 2 j + {0, 1} (D = 64: 8 n + 2 j + {0, 1}) in o[j][nt][2 {0, 1} + e].
    float o[KS][NT][4], m[NT][2], l[NT][2], v_ref = 0.0f, v_inv = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][nt][i] = 0.0f;
    }

    for (int c = cur.c; c < cur.c_end; ++c) {
      const int st = done % STAGES;
      const bool ok = tc::wait_bounded(bars + st, (done / STAGES) & 1, abort_flag, P.limit_ns, a.status, false);
      lost = !__all_sync(0xFFFFFFFFu, ok);
      if (lost) break;
      ++done;
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");  // this stage's scales
      __syncwarp();
      const uint8_t *ks_at = smem + warp * C::kRingBytes + st * 2 * kChunkBytes, *vs_at = ks_at + kChunkBytes;
      const int t0 = (t.chunk0 + c) * CH;
      // ---- scores
      float s[SL][NT][4];
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[sl][nt][i] = 0.0f;
        const int r0 = 16 * sl + n, r1 = r0 + 8;
        uint32_t w0[KS], w1[KS];
        if constexpr (D == 128) {  // 128-byte swizzle: piece p of row r lies at p ^ (r & 7)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t p = uint32_t((2 * q4 + i) ^ n) * 16;
            const uint4 x = lds128(ks_at + r0 * 128 + p), y = lds128(ks_at + r1 * 128 + p);
            w0[4 * i] = x.x, w0[4 * i + 1] = x.y, w0[4 * i + 2] = x.z, w0[4 * i + 3] = x.w;
            w1[4 * i] = y.x, w1[4 * i + 1] = y.y, w1[4 * i + 2] = y.z, w1[4 * i + 3] = y.w;
          }
        } else {  // 64-byte swizzle: p ^ ((r >> 1) & 3)
          const uint32_t p = uint32_t(q4 ^ ((n >> 1) & 3)) * 16;
          const uint4 x = lds128(ks_at + r0 * 64 + p), y = lds128(ks_at + r1 * 64 + p);
          w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
          w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t a0, a1, a2, a3;
          cvt4(w0[k], a0, a2);
          cvt4(w1[k], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(s[sl][nt], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
        }
      }
      // ---- softmax
      const bool some_hidden = t0 + CH > all_hi || t0 < all_lo;
      float mx[NT][2], vs[SL], v_hi = 0.0f, v_lo = INFINITY;  // value scales; the largest, and the smallest but 0
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx[nt][0] = m[nt][0], mx[nt][1] = m[nt][1];
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
        const float2 sc = *reinterpret_cast<const float2*>(scales + st * 8 + 2 * ((16 * sl) >> P.box_shift));
        vs[sl] = sc.y;
        // seen by no row, perhaps not fetched
        if (some_hidden && (t0 + 16 * sl >= t.hi || t0 + 16 * sl + 16 <= t.lo)) vs[sl] = 0.0f;
        v_hi = fmaxf(v_hi, vs[sl]);
        if (vs[sl] > 0.0f) v_lo = fminf(v_lo, vs[sl]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[sl][nt][i] *= sc.x * row_scale[nt][i & 1];
      }
      if (some_hidden) {
#pragma unroll
        for (int sl = 0; sl < SL; ++sl)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = t0 + 16 * sl + n + 8 * (i >> 1);
              if (tok >= see_hi[nt][i & 1] || tok < see_lo[nt][i & 1]) s[sl][nt][i] = -INFINITY;
            }
      }
#pragma unroll
      for (int sl = 0; sl < SL; ++sl)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[nt][i & 1] = fmaxf(mx[nt][i & 1], s[sl][nt][i]);
      // O is in units of v_ref, 2^8 below the first scale.  Where a chunk's scales lie in 1 .. 2^15 units they weigh the
      // probabilities: p vs / v_ref is 65504 at most and no smaller than p.  Where not (`apart`), each slice's product
      // is taken with the probabilities alone and weighed in fp32.
      const float v_new = v_hi > kUnits * v_ref ? value_unit(v_ref, v_hi, v_hi * 0x1p-8f) : v_ref;
      const bool apart = v_lo < v_new || v_hi > kUnits * v_new;
      bool grew = v_new != v_ref;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xFFFFFFFFu, mx[nt][e], d));
          grew |= mx[nt][e] != m[nt][e];
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {
        if (v_new != v_ref) v_inv = per_unit(v_new);
        const float fv = v_ref * v_inv;  // of the values summed so far
        v_ref = v_new;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = mx[nt][e] == -INFINITY ? 1.0f : ex2(m[nt][e] - mx[nt][e]);
            m[nt][e] = mx[nt][e];
            l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[j][nt][e] *= f * fv;
              o[j][nt][2 + e] *= f * fv;
            }
          }
      }
      uint32_t pb[SL][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
        for (int sl = 0; sl < SL; ++sl) {
          const float vr = apart ? 1.0f : vs[sl] * v_inv;
          const float p0 = ex2(s[sl][nt][0] - m0), p1 = ex2(s[sl][nt][1] - m1);
          const float p2 = ex2(s[sl][nt][2] - m0), p3 = ex2(s[sl][nt][3] - m1);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          // fp16 probabilities: 11 bits against the 4 of the values they weigh
          pb[sl][nt][0] = transpose8x8(pack_f16(p0 * vr, p1 * vr));
          pb[sl][nt][1] = transpose8x8(pack_f16(p2 * vr, p3 * vr));
        }
      }
      // ---- values
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
        constexpr int NW = D / 32;  // words of a lane's piece of a row
        uint32_t w[4][NW];          // tokens 2 q4, 2 q4 + 1, 2 q4 + 8, 2 q4 + 9 of the slice
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 16 * sl + 2 * q4 + (k & 1) + 8 * (k >> 1);
          if constexpr (D == 128) {
            const uint4 x = lds128(vs_at + r * 128 + uint32_t(n ^ (r & 7)) * 16);
            w[k][0] = x.x, w[k][1] = x.y, w[k][2] = x.z, w[k][3] = x.w;
          } else {
            const uint2 x = lds64(vs_at + r * 64 + uint32_t((n >> 1) ^ ((r >> 1) & 3)) * 16 + (n & 1) * 8);
            w[k][0] = x.x, w[k][1] = x.y;
          }
        }
        const float weight = vs[sl] * v_inv;  // where the slices are apart
        if (some_hidden) {
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool behind = t0 + 16 * sl + 2 * q4 + (k & 1) + 8 * (k >> 1) >= t.hi;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
              if (behind) w[k][i] = 0;  // behind the tokens anything may lie
              bad |= __vcmpeq4(w[k][i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
            }
          }
          // A NaN value must not reach a row that does not see its token (0 x NaN): take
          // it out here and put it back where it is seen, by counting with the tensor cores.
          if (__any_sync(0xFFFFFFFFu, bad)) {
            uint32_t seen[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const int tok = t0 + 16 * sl + n + 8 * hf;
                seen[nt][hf] = transpose8x8(pack_f16(tok < see_hi[nt][0] && tok >= see_lo[nt][0] ? 1.0f : 0.0f,
                                                     tok < see_hi[nt][1] && tok >= see_lo[nt][1] ? 1.0f : 0.0f));
              }
#pragma unroll
            for (int i = 0; i < NW; ++i) {
              uint32_t z[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t is = __vcmpeq4(w[k][i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                w[k][i] &= ~is;
                z[k] = is & 0x38383838u;  // e4m3 1.0
              }
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                uint32_t a0, a1, a2, a3;
                cvt4(__byte_perm(z[0], z[1], p ? 0x7362 : 0x5140), a0, a1);
                cvt4(__byte_perm(z[2], z[3], p ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma_f16(cnt, a0, a1, a2, a3, seen[nt][0], seen[nt][1]);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (cnt[k] > 0.0f) o[2 * i + p][nt][k] = __int_as_float(0x7FC00000);
                }
              }
            }
          }
        }
        auto products = [&](auto alone) {
#pragma unroll
          for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              uint32_t a0, a1, a2, a3;
              cvt4(__byte_perm(w[0][i], w[1][i], p ? 0x7362 : 0x5140), a0, a1);
              cvt4(__byte_perm(w[2][i], w[3][i], p ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float(&sum)[4] = o[2 * i + p][nt];
                if constexpr (decltype(alone)::value) {
                  float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma_f16(part, a0, a1, a2, a3, pb[sl][nt][0], pb[sl][nt][1]);
#pragma unroll
                  for (int k = 0; k < 4; ++k) sum[k] = fmaf(part[k], weight, sum[k]);
                } else {
                  mma_f16(sum, a0, a1, a2, a3, pb[sl][nt][0], pb[sl][nt][1]);
                }
              }
            }
        };
        if (apart)
          products(std::true_type());
        else
          products(std::false_type());
      }
      __syncwarp();  // every lane has read the stage
      fetch();
    }

    if (lost) break;  // nothing goes where copies may still land

    // ---- the tile's state over this warp's chunks: out, or kept as a piece
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], d);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          o[j][nt][e] *= v_ref;
          o[j][nt][2 + e] *= v_ref;
        }
      }
    const bool begins = cur.c == 0, ends = cur.c_end == t.chunks;
    constexpr int kStep = D / 8;  // elements of a lane in a row
    if (begins && ends) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = t.rt * R + 8 * nt + 2 * q4 + e;
          if (r >= t.m * G) continue;
          const int64_t row = t.row0 + r / G;
          const int head = t.h * G + r % G;
          const bool none = m[nt][e] == -INFINITY && l[nt][e] == 0.0f;
          const float inv = none ? 0.0f : 1.0f / l[nt][e];
          T* dst = static_cast<T*>(a.out) + row * a.o_ts + head * a.o_hs + kStep * n;
          float x[kStep];
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            x[2 * j] = o[j][nt][e] * inv;
            x[2 * j + 1] = o[j][nt][2 + e] * inv;
          }
#pragma unroll
          for (int j = 0; j < kStep / 8; ++j) store16(dst + 8 * j, x + 8 * j);
          if (a.lse && n == 0) a.lse[row * a.heads + head] = none ? -INFINITY : (m[nt][e] + log2f(l[nt][e])) / kLog2e;
        }
    } else {
      // Entered in the middle: its own place, work goes on.  Left in the middle: the share is
      // done, and the state takes the place of the ring.
      float* keep = reinterpret_cast<float*>(begins ? smem + warp * C::kRingBytes : smem + C::kHeads + warp * C::kStateBytes);
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (n == 0) {
            keep[R * D + 8 * nt + 2 * q4 + e] = m[nt][e];
            keep[R * D + R + 8 * nt + 2 * q4 + e] = l[nt][e];
          }
#pragma unroll
          for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) keep[((j * NT + nt) * 4 + 2 * x + e) * 32 + lane] = o[j][nt][2 * x + e];
        }
      if (lane == 0) pieces[2 * warp + begins] = Piece{1, ends, t.row0, t.m, t.rt, t.h, t.chunks, 0, sh.start(warp + 1, kWarps) - cur.left, 0};
    }
  }
  // after a timeout: let the copies in flight land before their memory is used again
  for (; done < issued; ++done)
    tc::wait_bounded(bars + done % STAGES, (done / STAGES) & 1, abort_flag, tc::kDrainNs, a.status, true);
  asm volatile("cp.async.wait_all;" ::: "memory");

  // ---- join the pieces: a run of one tile's pieces is the one that begins it (or comes in from the
  // CTA before) and the following warps' that entered it in the middle.  Every thread joins kEl
  // elements in a row of one of the tile's rows.
  __syncthreads();
  constexpr int kPerRow = kThreads / R, kEl = D / kPerRow;
  const int row = threadIdx.x / kPerRow, d0 = (threadIdx.x % kPerRow) * kEl;
  auto piece_at = [&](int i) {
    return reinterpret_cast<const float*>((i & 1) ? smem + (i >> 1) * C::kRingBytes : smem + C::kHeads + (i >> 1) * C::kStateBytes);
  };
  auto element = [&](int i) {  // place of element d0 + i of the row in a piece
    constexpr int kStep = D / 8;
    const int d = d0 + i, j = (d % kStep) >> 1;
    return ((j * NT + (row >> 3)) * 4 + 2 * (d & 1) + (row & 1)) * 32 + 4 * (d / kStep) + ((row & 7) >> 1);
  };
  // x, m, l joined with the states that at(j) gives places of (m, l, elements from d0 on), kBatch of
  // them under way together
  float x[kEl], m, l;
  auto join = [&](auto batch, int64_t count, auto at) {
    constexpr int kBatch = decltype(batch)::value;
    m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int k = 0; k < kEl; ++k) x[k] = 0.0f;
    for (int64_t j0 = 0; j0 < count; j0 += kBatch) {
      float pm[kBatch], pl[kBatch], px[kBatch][kEl];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        pm[j] = -INFINITY, pl[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < kEl; ++k) px[j][k] = 0.0f;
        if (j0 + j < count) at(j0 + j, pm[j], pl[j], px[j]);
      }
      float mn = m;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, pm[j]);
      const float base = mn == -INFINITY ? 0.0f : mn, f0 = ex2(m - base);
      m = mn;
      l *= f0;
#pragma unroll
      for (int k = 0; k < kEl; ++k) x[k] *= f0;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float f = ex2(pm[j] - base);
        l += pl[j] * f;
#pragma unroll
        for (int k = 0; k < kEl; ++k) x[k] += px[j][k] * f;
      }
    }
  };
  // bit 2 w + begins of what each warp has kept
  const bool kept = lane < 2 * kWarps && pieces[lane & (2 * kWarps - 1)].valid;
  const uint32_t valid = __ballot_sync(0xFFFFFFFFu, kept);
  const uint32_t last = __ballot_sync(0xFFFFFFFFu, kept && pieces[lane & (2 * kWarps - 1)].ends);
  for (uint32_t todo = valid; todo;) {
    const int i = __ffs(todo) - 1;
    const uint32_t from = ~0u << i, stop = last & from, begun = valid & 0xAAAAAAAAu & (from << 1);
    int behind = stop ? __ffs(stop) : 2 * kWarps;  // of the run: its tile ends or the next one begins
    if (begun) behind = min(behind, __ffs(begun) - 1);
    const bool comes_in = (i & 1) == 0, ends = last >> (behind - 1) & 1;
    uint32_t run = todo & ((1u << behind) - 1);
    todo &= ~run;
    const Piece first = pieces[i];
    join(std::integral_constant<int, 4>(), __popc(run), [&](int64_t, float& pm, float& pl, float (&px)[kEl]) {
      const float* p = piece_at(__ffs(run) - 1);
      run &= run - 1;
      pm = p[R * D + row];
      pl = p[R * D + R + row];
#pragma unroll
      for (int k = 0; k < kEl; ++k) px[k] = p[element(k)];
    });
    bool write = true;
    if (comes_in || !ends) {  // cut between CTAs
      const int64_t c0 = sh.owner(first.unit0 + tile_units<R>()), c1 = sh.owner(first.unit0 + tile_units<R>() + first.chunks - 1);
      float* part = P.parts + (2 * blockIdx.x + (comes_in ? 0 : 1)) * int64_t(C::kStateFloats);
#pragma unroll
      for (int k = 0; k < kEl; k += 2) *reinterpret_cast<float2*>(part + row * D + d0 + k) = make_float2(x[k], x[k + 1]);
      if (d0 == 0) {
        part[R * D + row] = m;
        part[R * D + R + row] = l;
      }
      __syncthreads();
      if (threadIdx.x == 0) {  // releases what the barrier has brought before it, and takes in what the others did
        uint32_t arrived;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(arrived) : "l"(P.counters + c0) : "memory");
        if (arrived == uint32_t(c1 - c0)) P.counters[c0] = 0;
        abort_flag[1] = arrived == uint32_t(c1 - c0);
      }
      __syncthreads();
      write = abort_flag[1] != 0;
      if (write)  // the last to arrive joins the parts, in CTA order
        join(std::integral_constant<int, 8>(), c1 - c0 + 1, [&](int64_t j, float& pm, float& pl, float (&px)[kEl]) {
          const float* p = P.parts + (2 * (c0 + j) + (j == 0 ? 1 : 0)) * int64_t(C::kStateFloats);
          pm = __ldcg(p + R * D + row);
          pl = __ldcg(p + R * D + R + row);
#pragma unroll
          for (int k = 0; k < kEl; k += 2) {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(p + row * D + d0 + k));
            px[k] = y.x, px[k + 1] = y.y;
          }
        });
    }
    const int r = first.rt * R + row;
    if (write && r < first.m * G) {
      const int64_t at = first.row0 + r / G;
      const int head = first.h * G + r % G;
      const bool none = m == -INFINITY && l == 0.0f;
      const float inv = none ? 0.0f : 1.0f / l;
      T* dst = static_cast<T*>(a.out) + at * a.o_ts + head * a.o_hs + d0;
#pragma unroll
      for (int k = 0; k < kEl; ++k) dst[k] = from_f32<T>(x[k] * inv);
      if (a.lse && d0 == 0) a.lse[at * a.heads + head] = none ? -INFINITY : (m + log2f(l)) / kLog2e;
    }
  }
}

template <typename T, int D, int NT>
static cudaError_t launch(const Params& P, int num_sms, cudaStream_t stream) {
  constexpr int kSmem = Cfg<D, NT>::kSmem;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  auto kernel = attn_kv8_kernel<T, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(unsigned(num_sms)), dim3(kThreads), kSmem, stream, P);
}

}  // namespace attn

// Counters first (the same place for both kernels, one per CTA, left zero), then two tile states per CTA.
static size_t attn_counter_bytes(int num_sms) { return (size_t(num_sms) * 4 + 255) / 256 * 256; }

// Tiles of 128 rows (attn_kv8_rows.cu) where a sequence and head have 64 query rows or more on average.
// Few-row kernel against the other, 8 sequences of 2000 tokens, 32 heads over 8 of 128: 32 rows 27 us, 33;
// 48 rows 34, 34; 64 rows 39, 34; 128 rows 63, 35.  One of 16000: 64 rows 40, 54; 128 rows 62, 55.  64 of 500,
// 16 over 4 of 64: 48 rows 30, 29; 64 rows 38, 28; 96 rows 49, 29.  One prompt among 63 single tokens over 2048
// tokens each: 256 queries (20 rows on average) 115, 133; 1000 (66 rows) 235, 171.
static bool many_rows(int64_t n_tokens, int64_t batch, int64_t q_heads, int64_t kv_heads) {
  return n_tokens * (q_heads / kv_heads) >= 64 * batch;
}

size_t attn_kv8_workspace_bytes(int64_t n_tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                int num_sms) {
  if (many_rows(n_tokens, batch, q_heads, kv_heads)) return attn_kv8_rows_workspace_bytes(head_dim, num_sms);
  const size_t state = head_dim == 128 ? attn::Cfg<128, 2>::kStateBytes : attn::Cfg<64, 2>::kStateBytes;
  return attn_counter_bytes(num_sms) + 2 * size_t(num_sms) * state;
}

cudaError_t launch_attn_kv8(const AttnParams& a, int head_dim, int dtype, void* workspace, int num_sms,
                            uint64_t limit_ns, cudaStream_t stream) {
  if (many_rows(a.n_tokens, a.batch, a.heads, a.kv_heads))
    return launch_attn_kv8_rows(a, head_dim, dtype, workspace, num_sms, limit_ns, stream);
  attn::Params P = {};
  P.a = a;
  P.counters = static_cast<uint32_t*>(workspace);
  P.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attn_counter_bytes(num_sms));
  P.limit_ns = limit_ns;
  const int ch = attn::kChunkBytes / head_dim, box = a.page < ch ? a.page : ch;
  for (P.page_shift = 4; (1 << P.page_shift) < a.page;) ++P.page_shift;
  for (P.box_shift = 4; (1 << P.box_shift) < box;) ++P.box_shift;
  if (!make_map_pages_u8(&P.k_map, a.k, head_dim, a.page, a.n_pages * a.kv_heads, box) ||
      !make_map_pages_u8(&P.v_map, a.v, head_dim, a.page, a.n_pages * a.kv_heads, box))
    return cudaErrorInvalidValue;
  // rows of a tile: 8, or 16 where the queries of a sequence and head usually fill more than 8 (8 sequences of
  // 2000 tokens, 8 heads of 128: 8 rows 17.8 us, 22.5 with 16; 12 rows 21.7, 22.5; 32 rows 30.4, 27.4)
  const bool wide = int64_t(a.n_tokens) * (a.heads / a.kv_heads) > 8 * int64_t(a.batch);
  using BF = __nv_bfloat16;
  if (dtype == PATCH_DTYPE_BF16) {
    if (head_dim == 128) return wide ? attn::launch<BF, 128, 2>(P, num_sms, stream) : attn::launch<BF, 128, 1>(P, num_sms, stream);
    return wide ? attn::launch<BF, 64, 2>(P, num_sms, stream) : attn::launch<BF, 64, 1>(P, num_sms, stream);
  }
  if (head_dim == 128) return wide ? attn::launch<__half, 128, 2>(P, num_sms, stream) : attn::launch<__half, 128, 1>(P, num_sms, stream);
  return wide ? attn::launch<__half, 64, 2>(P, num_sms, stream) : attn::launch<__half, 64, 1>(P, num_sms, stream);
}

}  // namespace patch
