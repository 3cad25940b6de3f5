// kvq_window.cuh -- decode attention over the first positions and a sliding
// window of the compressed cache.
//
// For the token at position p and query head hq of KV head h = hq / g:
//   s_t = scale q . k_hat_t  for t <= p with t < n_sink or t > p - window,
//   out = sum softmax(s) v_hat,  lse = ln sum e^s   (no position: out 0, lse -inf).
//
// A unit is a (sequence, KV head) and up to 8 NT of its (token, query head)
// columns.  The rows that its tokens attend, [0, n_sink) and [lo, len), are cut
// into blocks of 16 or 32 rows of one kind (bf16 text, visual), which the warps
// of the unit's CTAs take in turn: text blocks first, so that a warp's
// accumulator changes to packed rows once.  A thread-block cluster holds the CTAs
// of one or more units: units of heads that keep bf16 rows get more of them than
// those of packed heads.  Every warp streams its blocks through a ring of its own
// in shared memory (cp.async, K and V rows as separate pieces, so that V and the
// next K are under way while a block's scores are made), and runs an online softmax
// of its own.  The warps meet in shared memory, the CTAs in distributed shared
// memory: one launch, no workspace.  (Asynchronous stores on barriers in place of
// the cluster barrier there: 0.1 us less of 5.3 and of 6.5, not kept.)
//
//   QK: S[t][c] = K[t] . q[c]   (mma.sync m16n8k16, positions = M, columns = N)
//   PV: O[d][c] += V[t][d] P[t][c]   (d = M)
// Packed rows enter as exact fp16 subnormals with their scales and zero points
// applied as in the attention mass (K) and the split kernel (V).  bf16 rows stay
// bf16; the weights meet bf16 V rows as a high and a low bf16 part (2^-17), and
// packed ones as fp16, also times their scales (2^-11 each).  So that a faint
// weight (a long window next to a first position that takes most of the mass)
// keeps its digits in fp16, the score that sets a column's reference weighs
// 2^(top - kSlack); the reference moves when a weight would pass 2^top, top = kTop, or
// less where a V scale s is so large that s 2^top would pass fp16.  Sums of bf16 V
// rows from some 2^100 on may leave fp32 with such weights (and would from 2^128 / T on
// with any that are not made small for it): output elements where that happened
// are made again, row by row.
//
// mma.sync and not tcgen05: a decode step has few columns, and a unit's rows are
// a few thousand at most, spread over the SMs; 128 positions take 1.2 us of an SM
// with 16 columns (a tile of the tree kernel 1.6, whatever its columns).
//
// Bound by instruction issue and latency (530 instructions a block of 32 packed
// rows and 8 columns, half of the issue slots used at 12 to 16 warps an SM), small
// calls by their start, a block and the two meetings.  Measured (GB300): 2,078
// positions of a LLaVA-OneVision layer 6.2 us; a window of 8K of 32K x 8 in 2 bits
// (80 MB) 21.6 us, 3.7 TB/s; 16 tokens over 1,103 positions x 32 x 40 heads (281
// MB, 11.6 GFLOP) 85 us.  Steps: units split by the rows they hold (24 us where
// equal shares took 31), unpacked codes shared by two column tiles and three CTAs
// of 168 registers an SM (91 us, before 137 with one of eight warps), a loop for
// each kind of rows (85, before 88), the first rows asked for while the previous
// kernel ends (6.1 and 21.6 us, before 6.5 and 22.4), the check for sums past fp32 (6.2,
// 21.6 and 85.1 us, before 6.1, 21.5 and 84.5).
#pragma once

#include <cstddef>
#include <type_traits>

#include "kvq_split.cuh"

#include "kvq_geom.cuh"
#include "kvq_qk.cuh"

namespace kvq {
namespace win {

constexpr int kPiece = 4096;  // bytes of a ring slot: 16 bf16 rows
constexpr int kSlots = 3;
constexpr int kMaxRanks = 16;
constexpr int kTop = 14, kSlack = 3;  // weights are at most 2^top, and 2^(top - kSlack) where the reference was set
constexpr int kPitch = kD + 4;  // of a column's o row in the warps' meeting

struct Args {
  Geom c;
  const uint16_t* q;  // [B][n_q][Hq][D]
  const int32_t* seq_len;
  int32_t T, n_q, n_sink, window;
  float scale_log2;
  uint16_t* out;
  float* lse;
  int32_t nblk;  // column blocks of a (sequence, KV head)
  // Units of class k (0 both bf16, 1 K bf16, 2 packed): U[k], of 2^lg[k] CTAs
  // each; the grid's CTAs from first[k] on, whole clusters.
  int32_t U[3], lg[3], first[3], cluster;
  uint8_t head[KVQ_MAX_HEADS];  // heads of the classes in order
  uint8_t head0[3];             // where a class begins among them
};

// W warps a CTA, NT tiles of 8 columns.
template <int NT, int W>
struct Smem {
  alignas(128) uint8_t ring[W][kSlots * kPiece];
  Columns<NT> col;
  int32_t at[NT * 8];  // position of a column's token (-1: none)
  float ml[W][NT * 8][2];
  // (units of several CTAs only)
  float4 recv[NT * 256];                        // [rank][its share of the unit's 8 NT x D outputs]
  float2 recv_ml[kMaxRanks][NT * 8];
};

// 16-byte chunk c of row r of a piece of bf16 rows sits at chunk c ^ swizzle:
// the rows of an ldmatrix (V) or of a quarter-warp's loads (K) spread over the banks.
__device__ __forceinline__ int swz_k(int r) { return (r & 1) << 2; }
__device__ __forceinline__ int swz_v(int r) { return r & 7; }

// bytes of global memory at src into shared memory, or zeros.
template <int N>
__device__ __forceinline__ void cp_async_or_zero(void* dst, const void* src, bool live) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(N), "r"(live ? N : 0) : "memory");
}

// rows [0, n) of 16 bf16 rows from `src` on into a piece, the others zero.
template <bool kValue>
__device__ __forceinline__ void copy_bf16(uint8_t* to, const uint8_t* src, int n, int lane) {
  const int hi = lane >> 4, c = lane & 15;
  src += lane * 16;
  auto at = [&](int k) {  // of chunk c of row 2 k + hi
    const int r = 2 * k + hi;
    return to + r * kRowBytes + ((c ^ (kValue ? swz_v(r) : swz_k(r))) << 4);
  };
  if (n == 16) {
#pragma unroll
    for (int k = 0; k < 8; ++k) cp_async16(at(k), src + k * 2 * kRowBytes);
  } else {
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const bool live = 2 * k + hi < n;
      cp_async_or_zero<16>(at(k), live ? src + k * 2 * kRowBytes : src - hi * kRowBytes, live);
    }
  }
}

// rows [0, n) of RB packed rows of BITS bits and their scale/zero rows.
template <int BITS, int G, int RB>
__device__ __forceinline__ void copy_packed(uint8_t* to, const uint8_t* codes, const uint8_t* sz, int n, int lane) {
  constexpr int kSz = 4 * kD / G;
  const bool row = lane < n;
  if (n == RB) {
#pragma unroll
    for (int x = 0; x < RB * BITS; x += 32) cp_async16(to + 16 * (x + lane), codes + 16 * (x + lane));
  } else {
#pragma unroll 1
    for (int x = lane; x < RB * BITS; x += 32) {
      const bool live = x < n * BITS;
      cp_async_or_zero<16>(to + 16 * x, codes + 16 * (live ? x : 0), live);
    }
  }
  if (lane < RB) cp_async_or_zero<kSz>(to + RB * BITS * 16 + kSz * lane, sz + kSz * (row ? lane : 0), row);
}

// PV of 16 bf16 rows of a piece: the weights of a column as high and low bf16.
template <int NT, typename Weights>
__device__ __forceinline__ void pv_bf16(const uint8_t* vc, Weights&& P, int lane, Acc (&acc)[NT]) {
  uint32_t b[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float* w = P(t);
    const uint32_t h0 = pack_bf16x2(w[0], w[1]), h1 = pack_bf16x2(w[2], w[3]);
    b[t][0] = movmatrix_trans(h0);
    b[t][1] = movmatrix_trans(h1);
    b[t][2] = movmatrix_trans(pack_bf16x2(w[0] - bf16_lo(h0), w[1] - bf16_hi(h0)));
    b[t][3] = movmatrix_trans(pack_bf16x2(w[2] - bf16_lo(h1), w[3] - bf16_hi(h1)));
  }
  const int row = (lane & 7) + ((lane >> 4) & 1) * 8, chunk = (lane >> 3) & 1;
  const uint8_t* base = vc + row * kRowBytes;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    uint32_t A[4];
    ldsm_x4_trans(base + (((2 * m + chunk) ^ swz_v(row)) << 4), A);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mma_bf16(acc[t].o[m], A, b[t][0], b[t][1]);
      mma_bf16(acc[t].o[m], A, b[t][2], b[t][3]);
    }
  }
}

// PV of 16 packed rows (pv_packed of the split kernel, the unpacked codes
// shared by the tiles): per group the scales meet the weights, the zero points
// have an MMA of their own.
template <int VB, int G, int NT, typename Weights>
__device__ __forceinline__ void pv_packed_rows(const uint8_t* vc, const uint8_t* vsz, int r0, Weights&& P, int gid, int tig, Acc (&acc)[NT]) {
  constexpr int kRow = 16 * VB, kSlice = 2 * VB, NG = kD / G, kSz = 4 * NG;
  const int row[4] = {r0 + 2 * tig, r0 + 2 * tig + 1, r0 + 2 * tig + 8, r0 + 2 * tig + 9};
  uint32_t sz[4][(2 * NG + 1) / 2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* p = vsz + row[i] * kSz;
    if constexpr (NG == 4) {
      const uint4 a = lds128(p);
      sz[i][0] = a.x, sz[i][1] = a.y, sz[i][2] = a.z, sz[i][3] = a.w;
    } else if constexpr (NG == 2) {
      const uint2 a = lds64(p);
      sz[i][0] = a.x, sz[i][1] = a.y;
    } else {
      sz[i][0] = lds32(p);
    }
  }
  // fp16 halves: z_g at half g, s_g at half NG + g
  auto half_of = [](int h) { return (h & 1) ? 0x7632u : 0x5410u; };
  uint32_t b0[NT][NG], b1[NT][NG], pb[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float* w = P(t);
    pb[t][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
    pb[t][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int hs = NG + g;
    const uint32_t sa = prmt(sz[0][hs >> 1], sz[1][hs >> 1], half_of(hs)), sc = prmt(sz[2][hs >> 1], sz[3][hs >> 1], half_of(hs));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      b0[t][g] = hmul2_u(pb[t][0], sa);
      b1[t][g] = hmul2_u(pb[t][1], sc);
    }
  }
  {  // zero points: rows = groups
    uint32_t za = 0u, zc = 0u;
    if (gid < NG) {
      const bool up = NG == 4 && gid >= 2;
      za = prmt(up ? sz[0][NG / 4] : sz[0][0], up ? sz[1][NG / 4] : sz[1][0], half_of(gid));
      zc = prmt(up ? sz[2][NG / 4] : sz[2][0], up ? sz[3][NG / 4] : sz[3][0], half_of(gid));
    }
    const uint32_t Z[4] = {za, 0u, zc, 0u};
#pragma unroll
    for (int t = 0; t < NT; ++t) mma_f16(acc[t].zo, Z, pb[t][0], pb[t][1]);
  }
  constexpr int kWords = VB / 2;  // of a lane's slice
  uint32_t cw[4][kWords];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* p = vc + row[i] * kRow + kSlice * gid;
    if constexpr (VB == 2) {
      cw[i][0] = lds32(p);
    } else if constexpr (VB == 4) {
      const uint2 a = lds64(p);
      cw[i][0] = a.x, cw[i][1] = a.y;
    } else {
      const uint4 a = lds128(p);
      cw[i][0] = a.x, cw[i][1] = a.y, cw[i][2] = a.z, cw[i][3] = a.w;
    }
  }
  constexpr int kTiles = 8 / VB;  // m-tiles of a half-word (one of 8 bits)
#pragma unroll
  for (int h = 0; h < VB; ++h) {  // half-words of the slice
    const uint32_t xa = prmt(cw[0][h >> 1], cw[1][h >> 1], half_of(h)), xc = prmt(cw[2][h >> 1], cw[3][h >> 1], half_of(h));
    const uint32_t ya = VB == 2 ? (xa >> 6) : (xa >> 8), yc = VB == 2 ? (xc >> 6) : (xc >> 8);
#pragma unroll
    for (int mm = 0; mm < kTiles; ++mm) {
      const int m = h * kTiles + mm;
      uint32_t A[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int c = 2 * mm + r;  // code of the half-word
        const bool hi = VB == 2 ? (c >= 5) : (VB == 4 ? (c >= 2) : (c >= 1));
        const uint32_t mask = (VB == 2 ? 0x00030003u : (VB == 4 ? 0x000F000Fu : 0x00FF00FFu)) << kVShift<VB>(m, r);
        A[r] = (hi ? ya : xa) & mask;
        A[2 + r] = (hi ? yc : xc) & mask;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_f16(acc[t].o[m], A, b0[t][(16 * m) / G], b1[t][(16 * m) / G]);
    }
  }
}

// A block of rows of one kind.
struct Block {
  int t, n;       // position of its first row, rows
  int64_t row;    // first row among the rows of its kind
  bool visual;
};

// Elements 4 lane .. 4 lane + 3 of cache row t of K (kKey) or V, in fp32.
template <bool kKey>
__device__ __forceinline__ float4 elements_of(const Geom& p, const HeadRows& hr, int t, int lane) {
  const bool visual = t >= p.vs && t < p.ve;
  const int64_t at = visual ? t - p.vs : (t < p.vs ? t : t - p.Tv);
  const uint8_t* row = kKey ? (visual ? hr.vis_k : hr.text_k) : (visual ? hr.vis_v : hr.text_v);
  if (!visual || !(kKey ? hr.k_packed : hr.v_packed)) {
    const uint2 w = reinterpret_cast<const uint2*>(row + at * kRowBytes)[lane];
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  }
  const int bits = kKey ? p.kb : p.vb, szrow = kKey ? p.kszrow : p.vszrow, groups = szrow / 4, g = 4 * lane * groups / kD;
  row += at * (kKey ? p.krow : p.vrow);
  const __half* sz = reinterpret_cast<const __half*>((kKey ? hr.vis_ksz : hr.vis_vsz) + at * szrow);
  const float z = __half2float(sz[g]), s = __half2float(sz[groups + g]);
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int slot;  // (kvq.h)
    if (kKey) {
      const int P = lane >> 3, tt = (lane >> 1) & 3, e = lane & 1, odd = i & 1;
      slot = 32 * tt + (bits == 2   ? 16 * (i >> 1) + 8 * e + (P < 3 ? 4 - P + 3 * odd : odd)
                        : bits == 4 ? 8 * i + 4 * e + P
                                    : 4 * (2 * P + (i >> 1)) + 2 * e + odd);
    } else {
      const int d = 4 * lane + i;
      slot = 16 * (d & 7) + 2 * (d >> 4) + ((d >> 3) & 1);
    }
    const int bit = bits * slot;
    x[i] = fmaf(static_cast<float>((row[bit >> 3] >> (bit & 7)) & ((1 << bits) - 1)), s, z);
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

// Output elements 4 lane .. 4 lane + 3 of the token at position pos for one query
// column (of Columns::qb), row by row in fp32: with weights that its lse (`ref`, in
// log2 units) makes add up to 1/4, no sum of finite values leaves fp32.  Called by a
// whole warp where a sum of the fast way did.
static __device__ __noinline__ float4 attend_again(const Args& a, int b, int h, const uint4* column, int pos, float ref) {
  const int lane = threadIdx.x & 31;
  const HeadRows hr = head_rows(a.c, b, h);
  const uint2 w = reinterpret_cast<const uint2*>(column + (lane >> 3) * 32 + ((lane >> 1) & 3))[lane & 1];
  const float4 q = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  const int first = min(a.n_sink, pos + 1), next = max(first, pos - a.window + 1);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 2
  for (int i = 0; i < first + pos + 1 - next; ++i) {
    const int t = i < first ? i : i - first + next;
    const float4 k = elements_of<true>(a.c, hr, t, lane), v = elements_of<false>(a.c, hr, t, lane);
    float x = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float p = ex2(fmaf(x, a.scale_log2, -ref) - 2.f);
    l += p;
    o.x = fmaf(p, v.x, o.x), o.y = fmaf(p, v.y, o.y), o.z = fmaf(p, v.z, o.z), o.w = fmaf(p, v.w, o.w);
  }
  const float inv = 1.f / l;
  return make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

template <int KB, int VB, int G, int NT, int W>
__global__ void __launch_bounds__(32 * W, NT == 1 ? 16 / W : 12 / W) window_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<NT, W>& sm = *reinterpret_cast<Smem<NT, W>*>(smem_raw);
  constexpr int kWarps = W, kThreads = 32 * W;
  const Geom& p = a.c;
  constexpr int kKRow = KB < 16 ? 16 * KB : kRowBytes, kVRow = VB < 16 ? 16 * VB : kRowBytes;
  constexpr int kKSz = KB < 16 ? 4 * kD / G : 0, kVSz = VB < 16 ? 4 * kD / G : 0;
  // rows of a block whose K and V are both packed
  constexpr int kRB = 32 * (kKRow + kKSz) <= kPiece && 32 * (kVRow + kVSz) <= kPiece ? 32 : 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int cta = blockIdx.x, cls = cta >= a.first[2] ? 2 : (cta >= a.first[1] ? 1 : 0);
  const int lg = a.lg[cls], ranks = 1 << lg, unit = (cta - a.first[cls]) >> lg, rank = (cta - a.first[cls]) & (ranks - 1);
  const bool idle = unit >= a.U[cls];  // (fills a cluster)
  const int hb = a.nblk == 1 ? unit : unit / a.nblk, cb = unit - hb * a.nblk;
  const int hi = p.B == 1 ? hb : hb / p.B, b = hb - hi * p.B;
  const int h = idle ? 0 : a.head[a.head0[cls] + hi];
  cluster_arrive();  // waited for before the first store to another CTA
  if (a.seq_len) pdl_wait();
  int len = a.seq_len ? a.seq_len[b] : a.T;
  if (len < 0 || len > a.T || idle) len = 0;
  const int p0 = len - a.n_q;  // position of token 0
  const HeadRows hr = head_rows(p, b, h);
  const bool kpk = KB < 16 && hr.k_packed, vpk = VB < 16 && hr.v_packed;
  const int vrb = kpk && vpk ? kRB : 16;  // rows of a visual block

  // Runs of rows of one kind, one a lane: text before the visual block (of the
  // first positions, of the window), text behind it, visual rows.
  int run_t, run_n, run_end, run_first;
  {
    int a1 = min(a.n_sink, len), b0 = max(a1, p0 - a.window + 1);
    if (b0 <= a1) a1 = b0 = 0;
    const int x0 = lane & 1 ? b0 : 0, x1 = lane & 1 ? len : a1, kind = lane >> 1;
    const int k0 = kind == 0 ? 0 : (kind == 1 ? p.ve : p.vs), k1 = kind == 0 ? p.vs : (kind == 1 ? len : p.ve);
    run_t = max(x0, k0);
    run_n = kind < 3 ? max(0, min(x1, k1) - run_t) : 0;
    const int rb = kind == 2 ? vrb : 16;
    const int nb = (run_n + rb - 1) / rb;
    run_end = nb;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run_end, o);
      if (lane >= o) run_end += y;
    }
    run_first = run_end - nb;
  }
  const int blocks = __shfl_sync(0xffffffffu, run_end, 5);
  auto block_of = [&](int i) {
    const int r = __popc(__ballot_sync(0xffffffffu, lane < 6 && i >= run_end));
    const int t = __shfl_sync(0xffffffffu, run_t, r), n = __shfl_sync(0xffffffffu, run_n, r);
    const int off = (i - __shfl_sync(0xffffffffu, run_first, r)) * (r >= 4 ? vrb : 16);
    Block k;
    k.visual = r >= 4;
    k.t = t + off;
    k.n = min(n - off, k.visual ? vrb : 16);
    k.row = r < 2 ? k.t : (r < 4 ? k.t - p.Tv : k.t - p.vs);
    return k;
  };
  uint8_t* const ring = sm.ring[warp];
  auto issue_k = [&](const Block& k, uint8_t* to) {
    if (KB < 16 && k.visual && kpk) {
      const uint8_t* src = hr.vis_k + k.row * kKRow;
      const uint8_t* sz = hr.vis_ksz + k.row * kKSz;
      if constexpr (KB < 16) {
        if (kRB == 16 || vrb == 16) copy_packed<KB, G, 16>(to, src, sz, k.n, lane);
        else copy_packed<KB, G, kRB>(to, src, sz, k.n, lane);
      }
    } else {
      copy_bf16<false>(to, (k.visual ? hr.vis_k : hr.text_k) + k.row * kRowBytes, k.n, lane);
    }
  };
  auto issue_v = [&](const Block& k, uint8_t* to) {
    if (VB < 16 && k.visual && vpk) {
      const uint8_t* src = hr.vis_v + k.row * kVRow;
      const uint8_t* sz = hr.vis_vsz + k.row * kVSz;
      if constexpr (VB < 16) {
        if (kRB == 16 || vrb == 16) copy_packed<VB, G, 16>(to, src, sz, k.n, lane);
        else copy_packed<VB, G, kRB>(to, src, sz, k.n, lane);
      }
    } else {
      copy_bf16<true>(to, (k.visual ? hr.vis_v : hr.text_v) + k.row * kRowBytes, k.n, lane);
    }
  };

  const int step = ranks * kWarps;
  int i = rank * kWarps + warp;
  Block now = {}, then = {};
  if (i < blocks) now = block_of(i);
  if (!a.seq_len) {
    // Lengths known: the warp's first rows into L2 while the previous kernel ends
    // (what it still writes of them replaces the lines there).
    if (i < blocks && lane < 4) {
      const bool value = lane & 1, packed = now.visual && (value ? vpk : kpk), sz = lane >= 2;
      const uint8_t* at = value ? (now.visual ? hr.vis_v : hr.text_v) : (now.visual ? hr.vis_k : hr.text_k);
      int bytes = packed ? (value ? kVRow : kKRow) : kRowBytes;
      if (sz) at = value ? hr.vis_vsz : hr.vis_ksz, bytes = value ? kVSz : kKSz;
      if (!sz || packed) prefetch_bytes(at + now.row * bytes, now.n * bytes);
    }
    pdl_wait();
  }
  if (threadIdx.x == 0) pdl_launch_dependents();  // this kernel writes no cache row
  if (i < blocks) {
    issue_k(now, ring);
    cp_async_commit();
    issue_v(now, ring + kPiece);
  }
  cp_async_commit();

  // the queries, while the first rows are under way
  load_columns<KB, G, NT, kThreads>(sm.col, p.Hq, p.g, a.q, a.n_q, b, h, cb * NT * 8, a.scale_log2);
  if (threadIdx.x < NT * 8) {
    const int tok = (cb * NT * 8 + threadIdx.x) / p.g;
    sm.at[threadIdx.x] = tok < a.n_q ? p0 + tok : -1;
  }
  __syncthreads();

  Acc acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    acc[t].m[0] = acc[t].m[1] = -INFINITY;
    acc[t].l[0] = acc[t].l[1] = 0.f;
#pragma unroll
    for (int m = 0; m < 8; ++m) acc[t].o[m][0] = acc[t].o[m][1] = acc[t].o[m][2] = acc[t].o[m][3] = 0.f;
    acc[t].zo[0] = acc[t].zo[1] = acc[t].zo[2] = acc[t].zo[3] = 0.f;
  }
  float top = kTop, most_scale = ex2(15.9f - kTop);
  int slot = 0;  // of the block's K piece
  // The warp's next blocks, up to the first visual one where `text` is set; kK,
  // kV: their K and V rows are packed.
  auto blocks_of = [&](bool text, auto k_packed, auto v_packed) {
    constexpr bool kK = decltype(k_packed)::value, kV = decltype(v_packed)::value;
    constexpr int RB = kK && kV ? kRB : 16;
#pragma unroll 1
    for (; i < blocks && !(text && now.visual); i += step) {
      const bool more = i + step < blocks;
      const int slot_v = slot == kSlots - 1 ? 0 : slot + 1, slot_n = slot_v == kSlots - 1 ? 0 : slot_v + 1;
      cp_async_wait<1>();
      __syncwarp();
      if (more) {
        then = block_of(i + step);
        issue_k(then, ring + slot_n * kPiece);
      }
      cp_async_commit();
      const uint8_t* kc = ring + slot * kPiece;
      float S[NT][RB / 16][4];
#pragma unroll
      for (int hf = 0; hf < RB / 16; ++hf) {
        auto put_scores = [&](int t, const float (&x)[4]) {
#pragma unroll
          for (int e = 0; e < 4; ++e) S[t][hf][e] = x[e];
        };
        if constexpr (kK) {
          qk_packed_rows<KB, G, NT>(kc, kc + RB * kKRow, 16 * hf, sm.col, lane, put_scores);
        } else {
          const uint8_t* r0 = kc + gid * kRowBytes;
          qk_bf16_rows<NT>([&](int P, uint4& f0, uint4& f1) {
            const int c = (4 * P + tig) ^ swz_k(gid);
            f0 = *reinterpret_cast<const uint4*>(r0 + (c << 4));
            f1 = *reinterpret_cast<const uint4*>(r0 + 8 * kRowBytes + (c << 4));
          }, sm.col, a.scale_log2, lane, put_scores);
        }
      }
      // What the columns' tokens do not see: rows past the block's last, later
      // positions, positions between the first ones and a token's window.
      const int last = now.t + now.n - 1;
      if (now.n < RB || last > p0 || (last >= a.n_sink && now.t <= len - 1 - a.window)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int2 at = *reinterpret_cast<const int2*>(&sm.at[8 * t + 2 * tig]);
#pragma unroll
          for (int hf = 0; hf < RB / 16; ++hf)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = now.t + 16 * hf + gid + (e >> 1) * 8, pos = e & 1 ? at.y : at.x;
              if (x > last || x > pos || (x >= a.n_sink && x <= pos - a.window)) S[t][hf][e] = -INFINITY;
            }
        }
      }
      // the softmax of the warp's columns; the reference moves in few blocks
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        Acc& A = acc[t];
        float mx0 = fmaxf(S[t][0][0], S[t][0][2]), mx1 = fmaxf(S[t][0][1], S[t][0][3]);
#pragma unroll
        for (int hf = 1; hf < RB / 16; ++hf) {
          mx0 = fmaxf(mx0, fmaxf(S[t][hf][0], S[t][hf][2]));
          mx1 = fmaxf(mx1, fmaxf(S[t][hf][1], S[t][hf][3]));
        }
        if (__any_sync(0xffffffffu, mx0 > A.m[0] + top || mx1 > A.m[1] + top)) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
          }
          mx0 = mx0 > A.m[0] + top ? mx0 - (top - kSlack) : A.m[0];
          mx1 = mx1 > A.m[1] + top ? mx1 - (top - kSlack) : A.m[1];
          const float c0 = ex2(A.m[0] - (mx0 == -INFINITY ? 0.f : mx0)), c1 = ex2(A.m[1] - (mx1 == -INFINITY ? 0.f : mx1));
          A.m[0] = mx0;
          A.m[1] = mx1;
          A.l[0] *= c0;
          A.l[1] *= c1;
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            A.o[m][0] *= c0;
            A.o[m][1] *= c1;
            A.o[m][2] *= c0;
            A.o[m][3] *= c1;
          }
          A.zo[0] *= c0;
          A.zo[1] *= c1;
          A.zo[2] *= c0;
          A.zo[3] *= c1;
        }
        const uint64_t ref = pair_of(A.m[0] == -INFINITY ? 0.f : -A.m[0], A.m[1] == -INFINITY ? 0.f : -A.m[1]);
        uint64_t l = pair_of(A.l[0], A.l[1]);
#pragma unroll
        for (int hf = 0; hf < RB / 16; ++hf)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            unpair(add_pair(pair_of(S[t][hf][e], S[t][hf][e + 1]), ref), S[t][hf][e], S[t][hf][e + 1]);
            S[t][hf][e] = ex2(S[t][hf][e]);
            S[t][hf][e + 1] = ex2(S[t][hf][e + 1]);
            l = add_pair(l, pair_of(S[t][hf][e], S[t][hf][e + 1]));
          }
        unpair(l, A.l[0], A.l[1]);
      }
      cp_async_wait<1>();
      __syncwarp();  // V is here; the K piece's slot is free
      if (more) issue_v(then, ring + slot * kPiece);
      cp_async_commit();
      const uint8_t* vc = ring + slot_v * kPiece;
      if constexpr (kV) {
        // a row's largest scale (a lane a row): times a weight it must stay below 2^16
        float big = 0.f;
        if (lane < RB) {
          const __half* z = reinterpret_cast<const __half*>(vc + RB * kVRow + kVSz * lane);
#pragma unroll
          for (int g = 0; g < kD / G; ++g) big = fmaxf(big, __half2float(z[kD / G + g]));
        }
        if (__any_sync(0xffffffffu, big >= most_scale)) {  // rare
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          const float to = floorf(15.9f - log2f(big)), f = ex2(to - top);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              acc[t].m[e] += top - to;
              acc[t].l[e] *= f;
            }
#pragma unroll
            for (int m = 0; m < 8; ++m) acc[t].o[m][0] *= f, acc[t].o[m][1] *= f, acc[t].o[m][2] *= f, acc[t].o[m][3] *= f;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t].zo[e] *= f;
#pragma unroll
            for (int hf = 0; hf < RB / 16; ++hf)
#pragma unroll
              for (int e = 0; e < 4; ++e) S[t][hf][e] *= f;
          }
          top = to;
          most_scale = ex2(15.9f - top);
        }
#pragma unroll
        for (int hf = 0; hf < RB / 16; ++hf)
          pv_packed_rows<VB, G, NT>(vc, vc + RB * kVRow, 16 * hf, [&](int t) { return S[t][hf]; }, gid, tig, acc);
      } else {
        pv_bf16<NT>(vc, [&](int t) { return S[t][0]; }, lane, acc);
      }
      now = then;
      slot = slot_n;
    }
  };
  constexpr std::true_type kYes;
  constexpr std::false_type kNo;
  blocks_of(kpk || vpk, kNo, kNo);  // bf16 rows
  if (i < blocks) {
    if constexpr (VB < 16) {
      if (vpk) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc_to_packed<VB>(acc[t]);
      }
    }
    if (kpk && vpk) {
      if constexpr (KB < 16 && VB < 16) blocks_of(false, kYes, kYes);
    } else if (vpk) {
      if constexpr (VB < 16) blocks_of(false, kNo, kYes);
    } else {
      if constexpr (KB < 16) blocks_of(false, kYes, kNo);
    }
    if constexpr (VB < 16) {
      if (vpk) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc_to_true<VB, G>(acc[t], tig);
      }
    }
  }
  cp_async_wait<0>();

  // The warps meet: m and l of every column, then the o rows over the CTA's m.
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = acc[t].l[e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (gid == 0) {
        sm.ml[warp][8 * t + 2 * tig + e][0] = acc[t].m[e];
        sm.ml[warp][8 * t + 2 * tig + e][1] = l;
      }
    }
  }
  __syncthreads();
  // a column's reference and sum over the CTA's warps
  auto cta_ml = [&](int c) {
    float M = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][c][0]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l += sm.ml[w][c][1] * ex2(sm.ml[w][c][0] - (M == -INFINITY ? 0.f : M));
    return make_float2(M, l);
  };
  // (the warp's lanes all have quads of one column; those that are `mine` write)
  auto put = [&](int t, int c, int d4, float4 o, float M, float l, bool mine) {
    const int cg = (cb * NT + t) * 8 + c, tok = cg / p.g;
    if (idle || tok >= a.n_q) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing attended: 0 (NaN stays)
    const int64_t row = (static_cast<int64_t>(b) * a.n_q + tok) * p.Hq + h * p.g + (cg - tok * p.g);
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    // bf16 V rows from some 2^100 on may have taken a sum past fp32
    const bool past = l < INFINITY && !(o.x * 0.f + o.y * 0.f + o.z * 0.f + o.w * 0.f == 0.f);
    if (__builtin_expect(__any_sync(0xffffffffu, past), 0)) {
      const float4 x = attend_again(a, b, h, &sm.col.qb[t][0][4 * c], p0 + tok, M + log2f(l));
      const float4 y = make_float4(__shfl_sync(0xffffffffu, x.x, d4), __shfl_sync(0xffffffffu, x.y, d4), __shfl_sync(0xffffffffu, x.z, d4),
                                   __shfl_sync(0xffffffffu, x.w, d4));
      if (past) o = y;
    }
    if (!mine) return;
    reinterpret_cast<uint2*>(a.out + row * kD)[d4] = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    if (d4 == 0 && a.lse) a.lse[row] = 0.69314718055994531f * (M + log2f(l));
  };
  const uint32_t base = cluster_ctarank() - rank;  // of the unit's CTAs in the cluster
#pragma unroll 1
  for (int t = 0; t < NT; ++t) {  // (a warp's ring holds one tile's rows)
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      if (u != t) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 8 * u + 2 * tig + e;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][c][0]);
        const float f = ex2(acc[u].m[e] - (M == -INFINITY ? 0.f : M));
        float* o = mine + (2 * tig + e) * kPitch + gid;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          o[16 * m] = acc[u].o[m][e] * f;
          o[16 * m + 8] = acc[u].o[m][2 + e] * f;
        }
      }
    }
    __syncthreads();
    // (column, quad of d) of the CTA: written here, or sent to the rank that writes it
#pragma unroll
    for (int quad = threadIdx.x; quad < 256; quad += kThreads) {
      const int c = quad >> 5, d4 = quad & 31;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w]) + c * kPitch + 4 * d4);
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
      }
      if (ranks == 1) {
        const float2 ml = cta_ml(8 * t + c);
        put(t, c, d4, s, ml.x, ml.y, true);
      } else {
        // outputs of a tile are shared out over the ranks: 256 / ranks quads each
        if (t == 0 && quad == static_cast<int>(threadIdx.x)) cluster_wait();  // every CTA of the cluster has started
        const int share = 256 >> lg, to = quad >> (8 - lg), at = quad & (share - 1);
        const uint32_t addr = dsmem_addr(&sm.recv[t * 256 + rank * share + at], base + to);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(s.x), "f"(s.y), "f"(s.z), "f"(s.w) : "memory");
      }
    }
    if (t + 1 < NT) __syncthreads();  // the rings are written anew
  }
  if (ranks == 1) {
    cluster_wait();
    if (a.cluster > 1) cluster_sync();  // (other units' CTAs meet there)
    return;
  }
#pragma unroll
  for (int x = threadIdx.x; x < NT * 8 * ranks; x += kThreads) {
    const int to = x / (NT * 8), c = x - to * (NT * 8);
    const float2 ml = cta_ml(c);
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dsmem_addr(&sm.recv_ml[rank][c], base + to)), "f"(ml.x), "f"(ml.y) : "memory");
  }
  cluster_sync();
  // lane r of a group of `ranks` has rank r's part of a quad
  const int share = 256 >> lg, src = threadIdx.x & (ranks - 1);
#pragma unroll
  for (int t = 0; t < NT; ++t)
    for (int at = threadIdx.x >> lg; at < share; at += kThreads >> lg) {
      const int quad = rank * share + at, c = quad >> 5, d4 = quad & 31;
      const float2 ml = sm.recv_ml[src][8 * t + c];
      float4 o = sm.recv[t * 256 + src * share + at];
      float M = ml.x;
      for (int x = 1; x < ranks; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      const float f = ex2(ml.x - (M == -INFINITY ? 0.f : M));
      float l = ml.y * f;
      o.x *= f, o.y *= f, o.z *= f, o.w *= f;
      for (int x = 1; x < ranks; x <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, x);
        o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
      }
      put(t, c, d4, o, M, l, src == 0);
    }
}

struct Kernel {
  const void* fn;
  int smem, alone;  // alone: shared memory of units of one CTA
};
struct Form {
  int nt, warps;  // tiles of 8 columns (1 or 2); warps a CTA (4 or 8; 4 with two tiles)
};
template <int KB, int VB, int G, int NT, int W>
Kernel kernel_with() {
  using S = Smem<NT, W>;
  return {reinterpret_cast<const void*>(&window_kernel<KB, VB, G, NT, W>), static_cast<int>(sizeof(S)), static_cast<int>(offsetof(S, recv))};
}
template <int KB, int VB, int G>
Kernel kernel_of(Form f) {
  return f.nt == 2 ? kernel_with<KB, VB, G, 2, 4>() : (f.warps == 4 ? kernel_with<KB, VB, G, 1, 4>() : kernel_with<KB, VB, G, 1, 8>());
}
template <int KB, int VB>
Kernel kernel_of(int G, Form f) {
  if constexpr (KB == 16 && VB == 16) return kernel_of<16, 16, 128>(f);
  switch (G) {
    case 32: return kernel_of<KB, VB, 32>(f);
    case 64: return kernel_of<KB, VB, 64>(f);
    case 128: return kernel_of<KB, VB, 128>(f);
  }
  return {nullptr, 0, 0};
}
template <int KB>
Kernel kernel_of(int vb, int G, Form f) {
  switch (vb) {
    case 2: return kernel_of<KB, 2>(G, f);
    case 4: return kernel_of<KB, 4>(G, f);
    case 8: return kernel_of<KB, 8>(G, f);
    case 16: return kernel_of<KB, 16>(G, f);
  }
  return {nullptr, 0, 0};
}
// The kernel for (k_bits, v_bits, G): one translation unit for each width of K.
Kernel window_kernel_k2(int vb, int G, Form f);
Kernel window_kernel_k4(int vb, int G, Form f);
Kernel window_kernel_k8(int vb, int G, Form f);
Kernel window_kernel_k16(int vb, int G, Form f);

}  // namespace win
}  // namespace kvq
