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
// every CTA (one per SM) takes an equal share of all chunks, wherever tiles
// begin and end; the sequences' lengths are read on the device.  Each of a
// CTA's 8 warps fetches its own chunks (every eighth) by TMA into a ring of its
// own, so no warp waits for another until a tile ends; then the warps' states
// are joined in a tree.  A tile cut between CTAs is finished by the last of
// them, which joins the parts in CTA order (deterministic).
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
// its value scale (relative to the largest so far) the probabilities.
#include "common.cuh"
#include "decoder.cuh"
#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace patch {
namespace attn {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunkBytes = 4096;  // of keys, and of values
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  CUtensorMap k_map, v_map;
  AttnParams a;
  uint32_t* counters;  // one per CTA: arrivals at the tile that begins in it and goes on
  float* parts;        // two tile states per CTA
  uint64_t limit_ns;
};

template <int D, int NT>
struct Cfg {
  static constexpr int CH = kChunkBytes / D;        // tokens of a chunk
  static constexpr int SL = CH / 16;                // slices of 16 tokens
  static constexpr int KS = D / 16;                 // k steps of S, row tiles of O
  static constexpr int R = 8 * NT;                  // query rows of a tile
  static constexpr int STAGES = NT == 1 ? 3 : 2;
  static constexpr int kStateRegs = 4 * KS * NT + 4 * NT;  // o, m, l of a warp, per lane
  static constexpr int kStateBytes = kStateRegs * 128;
  static constexpr int kRing = kWarps * STAGES * 2 * kChunkBytes;
  static constexpr int kBars = kRing;                                  // full barriers
  static constexpr int kScales = kBars + kWarps * STAGES * 8;          // ring of scales: 4 slices x (k, v)
  static constexpr int kSlots = kScales + kWarps * STAGES * 32;        // tree: 7 states
  static constexpr int kMisc = kSlots + 7 * kStateBytes;
  static constexpr int kSmem = kMisc + 128 + 1024;                     // and alignment
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// four e4m3 bytes to two fp16 pairs (exact)
__device__ __forceinline__ void cvt4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A row tile of one sequence and head: which tokens its rows see.
struct Tile {
  int b, h, rt;
  int len, m, row0;     // the sequence's tokens, queries, first row of q
  int chunk0, chunks;   // its run of chunks (at least one, so that every tile is written)
  int hi;               // tokens from here on are seen by no row
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

template <int CH, int R>
__device__ __forceinline__ void set_rows(const AttnParams& a, int G, Tile& t) {
  const int i0 = t.rt * R / G, i1 = min(t.m - 1, (t.rt * R + R - 1) / G);
  int hi = t.len, lo = 0;
  if (a.causal) hi = max(0, min(t.len, t.len - t.m + i1 + 1));
  if (a.window > 0) lo = int(max(int64_t(0), int64_t(t.len) - t.m + i0 - a.window + 1));
  t.hi = hi;
  t.chunk0 = lo / CH;
  t.chunks = max(1, (hi + CH - 1) / CH - t.chunk0);
}
template <int R>
__device__ __forceinline__ int row_tiles(int m, int G) {
  return (m * G + R - 1) / R;
}
// chunks of all of a sequence's tiles of one head
template <int CH, int R>
__device__ __forceinline__ int64_t chunks_per_head(const AttnParams& a, int G, int b) {
  Tile t;
  sequence(a, b, t.len, t.m, t.row0);
  const int n = row_tiles<R>(t.m, G);
  if (n == 0) return 0;
  if (!a.causal) {
    t.rt = 0;
    set_rows<CH, R>(a, G, t);
    return int64_t(n) * t.chunks;
  }
  int64_t s = 0;
  for (t.rt = 0; t.rt < n; ++t.rt) {
    set_rows<CH, R>(a, G, t);
    s += t.chunks;
  }
  return s;
}
// to the next tile, in the order (sequence, head, row tile); past the last one b == batch
template <int CH, int R>
__device__ __forceinline__ void next_tile(const AttnParams& a, int G, Tile& t) {
  if (++t.rt < row_tiles<R>(t.m, G)) {
    set_rows<CH, R>(a, G, t);
    return;
  }
  t.rt = 0;
  if (++t.h == a.kv_heads) {
    t.h = 0;
    do {
      if (++t.b >= a.batch) return;
      sequence(a, t.b, t.len, t.m, t.row0);
    } while (t.m == 0);
  }
  set_rows<CH, R>(a, G, t);
}

// A warp's softmax state of a tile, in the layout of the O^T accumulators:
// lane (n = lane / 4, q = lane % 4) holds rows 8 nt + 2q + e of the tile and,
// of D = 128, elements 16 n + 2 j + {0, 1} (8 n + 2 j + {0, 1} of D = 64) in
// o[j][nt][2 * which + e].
template <int D, int NT>
struct State {
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][nt][i] = 0.0f;
    }
  }
  // p: 32-lane columns of floats, this lane's column
  __device__ __forceinline__ void store(float* p) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        p[(4 * nt + e) * 32] = m[nt][e];
        p[(4 * nt + 2 + e) * 32] = l[nt][e];
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[(4 * NT + (j * NT + nt) * 4 + i) * 32] = o[j][nt][i];
    }
  }
  // join with a stored state; kGlobal: written by another CTA (read past L1)
  template <bool kGlobal>
  __device__ __forceinline__ void join(const float* p) {
    auto get = [&](int i) { return kGlobal ? __ldcg(p + i * 32) : p[i * 32]; };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float fa[2], fb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mb = get(4 * nt + e), lb = get(4 * nt + 2 + e);
        const float mx = fmaxf(m[nt][e], mb), base = mx == -INFINITY ? 0.0f : mx;
        fa[e] = ex2(m[nt][e] - base);
        fb[e] = ex2(mb - base);
        m[nt][e] = mx;
        l[nt][e] = l[nt][e] * fa[e] + lb * fb[e];
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[j][nt][i] = o[j][nt][i] * fa[i & 1] + get(4 * NT + (j * NT + nt) * 4 + i) * fb[i & 1];
    }
  }
};

// Join the 8 warps' states into warp 0's.  Three rounds over slots of their
// own (0-3, 4-5, 6): a slot is written again only behind a barrier that its
// reader has passed.
template <int D, int NT>
__device__ __forceinline__ void tree(State<D, NT>& s, uint8_t* slots, int warp, int lane) {
  constexpr int kBytes = Cfg<D, NT>::kStateBytes;
  auto slot = [&](int i) { return reinterpret_cast<float*>(slots + i * kBytes) + lane; };
  if (warp >= 4) s.store(slot(warp - 4));
  __syncthreads();
  if (warp < 4) s.template join<false>(slot(warp));
  if (warp == 2 || warp == 3) s.store(slot(warp + 2));
  __syncthreads();
  if (warp < 2) s.template join<false>(slot(warp + 4));
  if (warp == 1) s.store(slot(6));
  __syncthreads();
  if (warp == 0) s.template join<false>(slot(6));
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) attn_kv8_kernel(const __grid_constant__ Params P) {
  using C = Cfg<D, NT>;
  constexpr int CH = C::CH, SL = C::SL, KS = C::KS, R = C::R, STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const AttnParams& a = P.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, q4 = lane & 3;
  const int G = a.heads / a.kv_heads;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars) + warp * STAGES;
  float* scales = reinterpret_cast<float*>(smem + C::kScales) + warp * STAGES * 8;
  int64_t* misc = reinterpret_cast<int64_t*>(smem + C::kMisc);  // 8 words of scan, abort flag
  int* abort_flag = reinterpret_cast<int*>(misc + 12);
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) tc::mbar_init(bars + s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.k_map)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.v_map)) : "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // queries, lengths and cache come from earlier kernels

  // This CTA's share of all chunks: [u0, u1) of W.
  int64_t part = 0;
  for (int b = threadIdx.x; b < a.batch; b += kThreads) {
    part += chunks_per_head<CH, R>(a, G, b);
    const int len = a.kv_lens[b];
    if (blockIdx.x == 0 && (len < 0 || len > a.max_pages * a.page)) set_status(a.status, PATCH_DEV_BOUNDS);
  }
  auto warp_scan = [&](int64_t v) {  // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v += y;
    }
    return v;
  };
  const int64_t sum = warp_scan(part);
  if (lane == 31) misc[warp] = sum;
  __syncthreads();
  int64_t W = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) W += misc[w];
  W *= a.kv_heads;
  const int64_t n_cta = min(int64_t(gridDim.x), W);
  if (blockIdx.x >= n_cta) return;
  const int64_t u0 = W * blockIdx.x / n_cta, u1 = W * (blockIdx.x + 1) / n_cta;
  // the sequence that chunk u0 lies in, and the chunks before it
  int64_t before = 0;
  for (int base = 0; base < a.batch; base += kThreads) {
    const int b = base + threadIdx.x;
    const int64_t v = b < a.batch ? chunks_per_head<CH, R>(a, G, b) * a.kv_heads : 0;
    const int64_t in = warp_scan(v);
    __syncthreads();
    if (lane == 31) misc[warp] = in;
    __syncthreads();
    int64_t ex = before + in - v;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) ex += misc[w];
      before += misc[w];
    }
    if (ex <= u0 && u0 < ex + v) {
      misc[8] = b;
      misc[9] = ex;
    }
    if (before > u0) break;
  }
  __syncthreads();
  Tile t;
  t.b = int(misc[8]);
  int64_t c_seg;  // the first chunk of this CTA's part of tile t
  {
    sequence(a, t.b, t.len, t.m, t.row0);
    const int64_t off = u0 - misc[9], per_head = chunks_per_head<CH, R>(a, G, t.b);
    t.h = int(off / per_head);
    c_seg = off % per_head;
    t.rt = 0;
    set_rows<CH, R>(a, G, t);
    while (c_seg >= t.chunks) {
      c_seg -= t.chunks;
      ++t.rt;
      set_rows<CH, R>(a, G, t);
    }
  }

  // This warp's chunks are u0 + warp, u0 + warp + 8, ...: a cursor runs ahead of the work and fetches.
  const uint32_t ring = tc::smem_u32(smem) + warp * STAGES * 2 * kChunkBytes;
  const int box = min(a.page, CH), boxes = CH / box;
  Tile ft = t;
  int64_t fc = c_seg + warp, fu = u0 + warp;
  int issued = 0;
  auto fetch = [&]() {  // the whole warp
    if (fu >= u1) return;
    while (fc >= ft.chunks) {
      fc -= ft.chunks;
      next_tile<CH, R>(a, G, ft);
    }
    const int st = issued % STAGES;
    const int t0 = (ft.chunk0 + int(fc)) * CH;
    const int n_box = min(boxes, (ft.hi - t0 + box - 1) / box);  // none in a tile that sees nothing
    const uint32_t bar = tc::smem_u32(bars + st);
    if (lane == 0) {
      if (n_box > 0)
        tc::mbar_expect_tx(bars + st, uint32_t(n_box * box * D * 2));
      else
        tc::mbar_arrive(bars + st);
    }
    __syncwarp();
    if (lane < n_box) {
      const int tok = t0 + lane * box;
      const int64_t phys = a.block_table[ft.b * a.max_pages + tok / a.page];
      const bool ok = phys >= 0 && phys < a.n_pages;
      if (!ok) set_status(a.status, PATCH_DEV_BOUNDS);
      const int64_t blk = ok ? phys * a.kv_heads + ft.h : a.n_pages * a.kv_heads;  // behind the end: reads zeros
      const uint32_t dst = ring + st * 2 * kChunkBytes + lane * box * D;
      tma_load_3d(dst, &P.k_map, bar, 0, tok % a.page, int(blk));
      tma_load_3d(dst + kChunkBytes, &P.v_map, bar, 0, tok % a.page, int(blk));
      const float ks = ok ? a.k_scale[blk] : 1.0f, vs = ok ? a.v_scale[blk] : 1.0f;
      for (int i = 0; i < box / 16; ++i) {
        scales[st * 8 + 2 * (lane * (box / 16) + i)] = ks;
        scales[st * 8 + 2 * (lane * (box / 16) + i) + 1] = vs;
      }
    }
    __syncwarp();  // the scales are for the whole warp
    ++issued;
    fu += kWarps;
    fc += kWarps;
  };
  for (int s = 0; s < STAGES; ++s) fetch();

  int done = 0;
  State<D, NT> S;
  for (int64_t u = u0; u < u1;) {
    // ---- this CTA's chunks c_seg .. c_end - 1 of tile t
    const int64_t tile_u0 = u - c_seg;
    const int64_t c_end = min(int64_t(t.chunks), c_seg + (u1 - u));
    // the rows' queries as operands, each row divided by a power of two
    uint32_t qf[NT][KS][2];
    float row_scale[NT][2];   // of this lane's accumulator columns 2 q4, 2 q4 + 1
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
      // 2^x with amax in [2^x, 2^(x+1)); 1 for zeros, subnormals and infinities
      const uint32_t ex = __float_as_uint(amax) >> 23;
      const bool plain = ex == 0 || ex >= 254;
      const float down = plain ? 1.0f : __uint_as_float((254 - ex) << 23), up = plain ? 1.0f : __uint_as_float(ex << 23);
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
    S.clear();
    float v_ref = 0.0f;

    for (int64_t c = c_seg + (((u0 + warp - u) % kWarps) + kWarps) % kWarps; c < c_end; c += kWarps) {
      const int st = done % STAGES;
      const bool ok = tc::wait_bounded(bars + st, (done / STAGES) & 1, abort_flag, P.limit_ns, a.status, false);
      ++done;
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const uint32_t ks_at = ring + st * 2 * kChunkBytes, vs_at = ks_at + kChunkBytes;
      const int t0 = (t.chunk0 + int(c)) * CH;
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
      float v_new = v_ref;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx[nt][0] = S.m[nt][0], mx[nt][1] = S.m[nt][1];
      const bool some_hidden = t0 + CH > all_hi || t0 < all_lo;
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
        const float ks = scales[st * 8 + 2 * sl];
        // a slice that no row sees may not have been fetched: its scale is left out
        if (t0 + 16 * sl < t.hi) v_new = fmaxf(v_new, scales[st * 8 + 2 * sl + 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = i & 1, tok = t0 + 16 * sl + n + 8 * (i >> 1);
            float x = s[sl][nt][i] * (ks * row_scale[nt][e]);
            if (some_hidden && (tok >= see_hi[nt][e] || tok < see_lo[nt][e])) x = -INFINITY;
            s[sl][nt][i] = x;
            mx[nt][e] = fmaxf(mx[nt][e], x);
          }
      }
      bool grew = v_new != v_ref;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xFFFFFFFFu, mx[nt][e], d));
          grew |= mx[nt][e] != S.m[nt][e];
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {
        const float fv = v_new > 0.0f ? __fdiv_rn(v_ref, v_new) : 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = mx[nt][e] == -INFINITY ? 1.0f : ex2(S.m[nt][e] - mx[nt][e]);
            S.m[nt][e] = mx[nt][e];
            S.l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              S.o[j][nt][e] *= f * fv;
              S.o[j][nt][2 + e] *= f * fv;
            }
          }
        v_ref = v_new;
      }
      uint32_t pb[SL][NT][2];
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
        const float vr = t0 + 16 * sl < t.hi && v_ref > 0.0f ? __fdiv_rn(scales[st * 8 + 2 * sl + 1], v_ref) : 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float m = S.m[nt][i & 1];
            p[i] = ex2(s[sl][nt][i] - (m == -INFINITY ? 0.0f : m));
            S.l[nt][i & 1] += p[i];
          }
          // fp16 probabilities: 11 bits against the 4 of the values they weigh
          pb[sl][nt][0] = transpose8x8(pack_f16(p[0] * vr, p[1] * vr));
          pb[sl][nt][1] = transpose8x8(pack_f16(p[2] * vr, p[3] * vr));
        }
      }
      // ---- values
#pragma unroll
      for (int sl = 0; sl < SL; ++sl) {
        constexpr int NW = D / 32;   // words of a lane's piece of a row
        uint32_t w[4][NW];           // tokens 2 q4, 2 q4 + 1, 2 q4 + 8, 2 q4 + 9 of the slice
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
          if (some_hidden && t0 + r >= t.hi)  // behind the tokens: anything may lie there
#pragma unroll
            for (int i = 0; i < NW; ++i) w[k][i] = 0;
        }
        if (some_hidden) {
          // A NaN value must not reach a row that does not see its token (0 x NaN): take
          // it out here and put it back where it is seen, by counting with the tensor cores.
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < NW; ++i) bad |= __vcmpeq4(w[k][i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
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
                    if (cnt[k] > 0.0f) S.o[2 * i + p][nt][k] = __int_as_float(0x7FC00000);
                }
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t a0, a1, a2, a3;
            cvt4(__byte_perm(w[0][i], w[1][i], p ? 0x7362 : 0x5140), a0, a1);
            cvt4(__byte_perm(w[2][i], w[3][i], p ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(S.o[2 * i + p][nt], a0, a1, a2, a3, pb[sl][nt][0], pb[sl][nt][1]);
          }
      }
      __syncwarp();  // every lane has read the stage
      fetch();
    }

    // ---- the tile's state over this CTA's chunks, in warp 0
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) S.l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, S.l[nt][e], d);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          S.o[j][nt][e] *= v_ref;
          S.o[j][nt][2 + e] *= v_ref;
        }
      }
    tree<D, NT>(S, smem + C::kSlots, warp, lane);
    bool write = warp == 0;
    if (c_seg > 0 || c_end < t.chunks) {  // a cut tile
      const int64_t first = ((tile_u0 + 1) * n_cta - 1) / W, last = ((tile_u0 + t.chunks) * n_cta - 1) / W;
      constexpr int64_t kState = C::kStateRegs * 32;
      int* flag = abort_flag + 1;
      if (warp == 0) {
        S.store(P.parts + (2 * blockIdx.x + (blockIdx.x == first ? 1 : 0)) * kState + lane);
        __threadfence();
        __syncwarp();
        if (lane == 0) *flag = atomicAdd(P.counters + first, 1u) == uint32_t(last - first);
      }
      __syncthreads();
      const bool is_last = *flag != 0;
      write = false;
      if (is_last) {  // the last to arrive joins the parts, in CTA order
        __threadfence();
        S.clear();
        for (int64_t i = first + warp; i <= last; i += kWarps)
          S.template join<true>(P.parts + (2 * i + (i == first ? 1 : 0)) * kState + lane);
        tree<D, NT>(S, smem + C::kSlots, warp, lane);
        write = warp == 0;
        if (threadIdx.x == 0) P.counters[first] = 0;
      }
      __syncthreads();  // the flag is read before the next cut tile writes it
    }
    if (write) {
      constexpr int kStep = D / 8;  // elements of a lane
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = t.rt * R + 8 * nt + 2 * q4 + e;
          if (r >= t.m * G) continue;
          const int64_t row = t.row0 + r / G;
          const int head = t.h * G + r % G;
          const float inv = S.m[nt][e] == -INFINITY && S.l[nt][e] == 0.0f ? 0.0f : 1.0f / S.l[nt][e];
          T* dst = static_cast<T*>(a.out) + row * a.o_ts + head * a.o_hs + kStep * n;
          float x[kStep];
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            x[2 * j] = S.o[j][nt][e] * inv;
            x[2 * j + 1] = S.o[j][nt][2 + e] * inv;
          }
#pragma unroll
          for (int j = 0; j < kStep / 8; ++j) store16(dst + 8 * j, x + 8 * j);
          if (a.lse && n == 0)
            a.lse[row * a.heads + head] =
                S.m[nt][e] == -INFINITY && S.l[nt][e] == 0.0f ? -INFINITY : (S.m[nt][e] + log2f(S.l[nt][e])) / kLog2e;
        }
    }
    u += c_end - c_seg;
    c_seg = 0;
    next_tile<CH, R>(a, G, t);
  }
  // after a timeout: let the copies in flight land before the shared memory goes
  for (; done < issued; ++done)
    tc::wait_bounded(bars + done % STAGES, (done / STAGES) & 1, abort_flag, P.limit_ns, a.status, true);
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

// Counters first (one per CTA, left zero), then two tile states of up to 16 rows per CTA.
static size_t attn_counter_bytes(int num_sms) { return (size_t(num_sms) * 4 + 255) / 256 * 256; }

size_t attn_kv8_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t head_dim, int num_sms) {
  const size_t state = head_dim == 128 ? attn::Cfg<128, 2>::kStateBytes : attn::Cfg<64, 2>::kStateBytes;
  return attn_counter_bytes(num_sms) + 2 * size_t(num_sms) * state;
}

cudaError_t launch_attn_kv8(const AttnParams& a, int head_dim, int dtype, void* workspace, int num_sms,
                            uint64_t limit_ns, cudaStream_t stream) {
  attn::Params P = {};
  P.a = a;
  P.counters = static_cast<uint32_t*>(workspace);
  P.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attn_counter_bytes(num_sms));
  P.limit_ns = limit_ns;
  const int ch = attn::kChunkBytes / head_dim, box = a.page < ch ? a.page : ch;
  if (!make_map_pages_u8(&P.k_map, a.k, head_dim, a.page, a.n_pages * a.kv_heads, box) ||
      !make_map_pages_u8(&P.v_map, a.v, head_dim, a.page, a.n_pages * a.kv_heads, box))
    return cudaErrorInvalidValue;
  // rows of a tile: 8, or 16 where the queries of a sequence and head usually fill more than 8
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
