// kvq_mass.cu -- kvq_attention_mass: the attention weight that each cache
// position has received, accumulated per KV head.
//
//   mass[b, h, t] = decay mass_in[b, h, t]
//                 + sum_k sum_{hq of h} e^(scale q_k,hq . k_hat_t - lse_k,hq)
// over the tokens k = 0 .. n - 1 taken from sequence b, token k reaching the
// positions t < len - n + 1 + k.
//
// Positions are independent once lse is known, so a call is one pass over K:
// a warp takes 16 positions at a time (M = 16 of mma.sync m16n8k16) against
// the KV head's (query head, token) columns, 8 at a time (N), adds the weights
// of all columns in registers and touches each mass once.  Packed codes enter
// as exact fp16 subnormals (one AND per operand register) with the group
// scales applied in fp32 and the zero points as one more K step (z against the
// high and low fp16 parts of the query's group sums), as in the split kernel;
// bf16 rows and queries go to the bf16 MMA as they are stored.  The fp16 queries
// have a power of two of their own per column, by which the largest element
// lands in [2^8, 2^9) (128 of them sum to 65280 at most): elements are exact
// down to 2^-25 of it and off by 2^-33 of it below, and so are the group sums.
// The scale of a column undoes it (one scale for all columns: 172 us in place
// of 176 with 32 columns, the same with 4; scale and lse in one 16-byte load: 179).
//
// With few columns the pass would be bound by the K bytes, with many by the MMA
// rate (9 MMAs of 8 cycles per 16 positions and 8 columns), so the operands of
// a 16-row block stay in registers over all columns.  mma.sync and not tcgen05:
// a decode step has at most 8 columns a KV head in most models, the weights are
// wanted per position, where their fragments already are, and at 32 columns
// 128 positions take 1.0 us of an SM (the tree kernel's tile, V included, 1.6).
//
// Measured (GB300): 32K positions x 8 after a decode step (172 MB) 54 us, 3.2
// TB/s; 32 tokens over 2,972 positions x 32 x 40 heads (421 MB, 31 GFLOP) 176
// us; a LLaVA-OneVision layer 4.9 us.  Bound by instruction issue and latency
// (about 250 instructions a block and tile of columns).  A warp's packed blocks
// come through shared memory, two under way (three or five take the same): one
// ahead in registers, behind prefetches into L2, took 70 and 199 us.  fp32
// arithmetic in pairs was 3% of the first, 0 of the second; 3 CTAs of 80
// registers an SM instead of 2 took 54 and 165 (all with one scale for all columns).
#include "kvq_split.cuh"

#include "kvq_geom.cuh"
#include "kvq_qk.cuh"

#include <algorithm>
#include <cmath>

namespace kvq {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;        // positions of a block
constexpr int kMaxTiles = 8;     // 8-column tiles handled in one pass over the rows
constexpr int kCtasPerSm = 2;    // resident CTAs (registers)
constexpr int kAhead = 4;        // blocks of a warp that its L2 prefetch runs ahead

struct MassArgs {
  Geom c;
  const uint16_t* q;   // [B][n_q][Hq][D]
  const float* lse;    // [B][n_q][Hq]
  const int32_t *seq_len, *path, *path_len;
  int32_t T, n_q, max_path;
  float scale_log2, decay;
  const float* mass_in;  // [B][Hkv][T_cap] or null
  float* mass;
  // (sequence, KV head) pairs of class k (0 bf16 K rows, 1 packed) number U[k]
  // and are split over S[k] CTAs each; heads of the classes in order in head[]
  int32_t U[2], S[2], n_bf16;
  uint8_t head[KVQ_MAX_HEADS];
};

struct MassSmem {
  uint4 qh[kMaxTiles][4][32];   // fp16 operand: [tile][32-element block][lane], see q_factor
  uint4 qb[kMaxTiles][4][32];   // bf16 operand
  uint32_t zb[kMaxTiles][32];   // group sums, high then low
  // columns 2 tig, 2 tig + 1: minus lse in log2 units; what takes S to log2 units
  float2 lse2[kMaxTiles][4], scl[kMaxTiles][4];
  int2 lim[kMaxTiles][4];       // those columns see the positions below
  float qs[kMaxTiles * 8][4];
};

// The columns [col0, col0 + 8 tiles) of (b, h): token k of the n taken is
// column k g + j.  Columns that add nothing get q = 0 and lse = +inf.
template <int KB, int G>
__device__ __forceinline__ void load_columns(const MassArgs& a, MassSmem& sm, int b, int h, int len, int n, int col0,
                                             int tiles) {
  const Geom& p = a.c;
  constexpr int NG = kD / G;
  for (int x = threadIdx.x; x < tiles * 8 * 16; x += kWarps * 32) {
    const int tig = x & 3, P = (x >> 2) & 3, c = x >> 4, cg = col0 + c;
    const int k = cg / p.g, j = cg - k * p.g;
    int tok = -1;
    if (k < n) tok = a.path ? a.path[static_cast<int64_t>(b) * a.max_path + k] : k;
    float l = INFINITY;
    int64_t row = 0;
    if (tok >= 0 && tok < a.n_q) {
      row = (static_cast<int64_t>(b) * a.n_q + tok) * p.Hq + h * p.g + j;
      l = a.lse[row];
      if (l == -INFINITY) l = INFINITY;  // a row that attended nothing
    }
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (l != INFINITY) r = __ldcg(reinterpret_cast<const uint4*>(a.q + row * kD) + 4 * P + tig);
    const int t = c >> 3, lane = 4 * (c & 7) + tig;
    sm.qb[t][P][lane] = r;
    // the column's power of two 2^e (its 16 threads are neighbours); 2^e and
    // 2^-e are fp32 for every bf16
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = i == 0 ? r.x : (i == 1 ? r.y : (i == 2 ? r.z : r.w));
      top = max(top, max(v & 0x7fffu, (v >> 16) & 0x7fffu));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = min(100, kQueryExponent + 127 - static_cast<int>(top >> 7));
    const float norm = __int_as_float((127 + e) << 23);
    auto pair = [&](uint32_t lo, uint32_t hi, bool upper) {
      return pack_f16x2(norm * (upper ? bf16_hi(lo) : bf16_lo(lo)), norm * (upper ? bf16_hi(hi) : bf16_lo(hi)));
    };
    const uint32_t y[4] = {pair(r.x, r.z, false), pair(r.x, r.z, true), pair(r.y, r.w, false), pair(r.y, r.w, true)};
    const float f = q_factor<KB>(P);
    const uint32_t f2 = pack_f16x2(f, f);
    sm.qh[t][P][lane] = make_uint4(hmul2_u(y[0], f2), hmul2_u(y[1], f2), hmul2_u(y[2], f2), hmul2_u(y[3], f2));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u, v;
      h2_to_f2(y[i], u, v);
      sum += u + v;
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (tig == 0) {
      sm.qs[c][P] = sum;
      if (P == 0) {
        reinterpret_cast<float*>(&sm.lse2[t][0])[c & 7] = -l * 1.4426950408889634f;
        reinterpret_cast<float*>(&sm.scl[t][0])[c & 7] = a.scale_log2 * __int_as_float((127 - e) << 23);
        reinterpret_cast<int*>(&sm.lim[t][0])[c & 7] = len - n + 1 + k;
      }
    }
  }
  __syncthreads();
  // K index 2 tig, 2 tig + 1: high parts of groups 0 .. 3, then the low parts
  for (int x = threadIdx.x; x < tiles * 32; x += kWarps * 32) {
    const int tig = x & 3, c = x >> 2;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int g = 2 * (tig & 1) + e;
      if (g < NG) {
#pragma unroll
        for (int i = 0; i < 4 / NG; ++i) s[e] += sm.qs[c][g * (4 / NG) + i];
      }
    }
    uint32_t z = pack_f16x2(s[0], s[1]);
    if (tig >= 2) {
      float h0, h1;
      h2_to_f2(z, h0, h1);
      z = pack_f16x2(s[0] - h0, s[1] - h1);
    }
    sm.zb[c >> 3][4 * (c & 7) + tig] = z;
  }
  __syncthreads();
}

// A warp's blocks of packed rows on their way through shared memory.
template <int KB, int G>
struct Ring {
  static constexpr int kCodes = kRows * kD / 8 * KB, kSz = kRows * (kD / G) * 4;  // bytes of a block
  static constexpr int kStage = kCodes + kSz + kRows * 4, kStages = 3;
  static constexpr int kBytes = kStages * kStage;
};

template <int KB, int G>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) mass_kernel(const __grid_constant__ MassArgs a) {
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ MassSmem sm;
  const Geom& p = a.c;
  constexpr int NG = kD / G;
  constexpr int PPG = G / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  // the CTA's (sequence, KV head) and strip of its rows
  int v = blockIdx.x, cls = 0;
  if (v >= a.U[0] * a.S[0]) {
    v -= a.U[0] * a.S[0];
    cls = 1;
  }
  const int S = cls ? a.S[1] : a.S[0];
  const int unit = v / S, strip = v - unit * S;
  const int h = a.head[(cls ? a.n_bf16 : 0) + unit / p.B], b = unit - (unit / p.B) * p.B;
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();  // past the dependency wait; this kernel writes no cache row
  const int len = a.seq_len ? a.seq_len[b] : a.T;
  const int n = a.path ? a.path_len[b] : a.n_q;
  if (len < 1 || len > a.T || n < 0 || n > (a.path ? a.max_path : a.n_q) || n > len) return;
  const HeadRows hr = head_rows(p, b, h);
  // blocks of the text prefix, the visual block, the text behind it
  const int n_pre = min(len, p.vs), n_vis = max(0, min(len, p.ve) - p.vs), n_suf = max(0, len - p.ve);
  const int b1 = (n_pre + kRows - 1) / kRows, b2 = b1 + (n_vis + kRows - 1) / kRows;
  const int nb = b2 + (n_suf + kRows - 1) / kRows;
  const int first = static_cast<int>(static_cast<int64_t>(nb) * strip / S);
  const int last = static_cast<int>(static_cast<int64_t>(nb) * (strip + 1) / S);
  const int64_t base = (static_cast<int64_t>(b) * p.Hkv + h) * p.T_cap;
  const int cols = p.g * n;
  const int reach = len - n + 1;  // every column sees the positions below
  // one pass over the rows for every 64 columns (at least one: the decay)
  for (int col0 = 0; col0 == 0 || col0 < cols; col0 += 8 * kMaxTiles) {
    const int tiles = min(kMaxTiles, (cols - col0 + 7) / 8);
    if (col0 > 0) __syncthreads();
    load_columns<KB, G>(a, sm, b, h, len, n, col0, tiles);
    // what the sums are added to: lanes tig 0 have row gid, tig 1 row gid + 8
    const int my = tig == 0 ? gid : gid + 8;
    auto fetch_mass = [&](int t0, int m) {
      if (tig >= 2 || my >= m) return 0.f;
      if (col0 > 0) return a.mass[base + t0 + my];
      return a.mass_in ? a.decay * a.mass_in[base + t0 + my] : 0.f;
    };
    const bool in_ring = a.mass_in && col0 == 0;
    // weights of rows gid, gid + 8 of the block, those of even and odd columns
    uint64_t w0 = 0ull, w1 = 0ull;
    auto add = [&](int t, uint64_t x0, uint64_t x1, int t0, bool late) {
      float e0, e1, e2, e3;
      unpair(x0, e0, e1);
      unpair(x1, e2, e3);
      e0 = ex2(e0), e1 = ex2(e1), e2 = ex2(e2), e3 = ex2(e3);
      if (late) {
        const int2 lim = sm.lim[t][tig];
        const int ta = t0 + gid, tb = ta + 8;
        if (ta >= lim.x) e0 = 0.f;
        if (ta >= lim.y) e1 = 0.f;
        if (tb >= lim.x) e2 = 0.f;
        if (tb >= lim.y) e3 = 0.f;
      }
      w0 = add_pair(w0, pair_of(e0, e1));
      w1 = add_pair(w1, pair_of(e2, e3));
    };
    auto store = [&](int t0, int m, float m_in) {  // lanes tig 0 and 2 end up with row gid, 1 and 3 with gid + 8
      float a0, a1, b0, b1;
      unpair(w0, a0, a1);
      unpair(w1, b0, b1);
      a0 += a1;
      b0 += b1;
      float w = (tig & 1 ? b0 : a0) + __shfl_xor_sync(0xffffffffu, tig & 1 ? a0 : b0, 1);
      w += __shfl_xor_sync(0xffffffffu, w, 2);
      if (tig < 2 && my < m) a.mass[base + t0 + my] = m_in + w;
    };
    // A warp's blocks of a run of `rows` rows from position t_base on: the
    // blocks lo + warp, lo + warp + 8, .. below hi.  Rows past the last are
    // read from it and not stored.
    auto run_bf16 = [&](const uint8_t* rows_at, int rows, int t_base, int lo, int hi) {
      auto prefetch = [&](int i) {
        if (i >= hi) return;
        const int m = min(kRows, rows - i * kRows);
        prefetch_bytes(rows_at + static_cast<int64_t>(i) * kRows * kRowBytes, m * kRowBytes);
        if (a.mass_in) prefetch_bytes(a.mass_in + base + t_base + i * kRows, 4 * m);
      };
      if (lane == 0 && col0 == 0)
        for (int k = 0; k < kAhead; ++k) prefetch(lo + warp + k * kWarps);
#pragma unroll 1
      for (int i = lo + warp; i < hi; i += kWarps) {
        const int m = min(kRows, rows - i * kRows), t0 = t_base + i * kRows;
        const uint8_t* at = rows_at + static_cast<int64_t>(i) * kRows * kRowBytes + 16 * tig;
        uint4 f0[4], f1[4];
#pragma unroll
        for (int P = 0; P < 4; ++P) {
          f0[P] = *reinterpret_cast<const uint4*>(at + min(gid, m - 1) * kRowBytes + 64 * P);
          f1[P] = *reinterpret_cast<const uint4*>(at + min(gid + 8, m - 1) * kRowBytes + 64 * P);
        }
        const float m_in = fetch_mass(t0, m);
        if (lane == 0 && col0 == 0) prefetch(i + kAhead * kWarps);
        const bool late = t0 + m > reach;
        w0 = w1 = 0ull;
#pragma unroll 2
        for (int t = 0; t < tiles; ++t) {
          float C[2][4];
#pragma unroll
          for (int P = 0; P < 4; ++P) {
            const uint4 q = sm.qb[t][P][lane];
            const uint32_t A0[4] = {f0[P].x, f1[P].x, f0[P].y, f1[P].y};
            const uint32_t A1[4] = {f0[P].z, f1[P].z, f0[P].w, f1[P].w};
            if (P == 0) {
              mma_bf16_new(C[0], A0, q.x, q.y);
              mma_bf16_new(C[1], A1, q.z, q.w);
            } else {
              mma_bf16(C[0], A0, q.x, q.y);
              mma_bf16(C[1], A1, q.z, q.w);
            }
          }
          const uint64_t l2 = *reinterpret_cast<const uint64_t*>(&sm.lse2[t][tig]);
          const uint64_t s2 = pair_of(a.scale_log2, a.scale_log2);
          add(t, fma_pair(add_pair(pair_of(C[0][0], C[0][1]), pair_of(C[1][0], C[1][1])), s2, l2),
              fma_pair(add_pair(pair_of(C[0][2], C[0][3]), pair_of(C[1][2], C[1][3])), s2, l2), t0, late);
        }
        store(t0, m, m_in);
      }
    };
    // Packed rows: a warp has a contiguous run of blocks, kStages - 1 of them
    // (rows, scale/zero rows, masses) under way into its part of shared memory.
    // A block past the last row reads on into the segment's padding (whole
    // blocks of 16 rows).
    auto run_packed = [&](int lo, int hi) {
      if constexpr (KB < 16) {
        using R = Ring<KB, G>;
        const int w_lo = lo + (hi - lo) * warp / kWarps, w_hi = lo + (hi - lo) * (warp + 1) / kWarps;
        if (w_lo >= w_hi) return;
        uint8_t* const ring = ring_smem + warp * R::kBytes;
        auto issue = [&](int i, uint8_t* to) {
          if (i < w_hi) {
            const uint8_t* k = hr.vis_k + static_cast<int64_t>(i) * R::kCodes;
#pragma unroll
            for (int c = 0; c < R::kCodes / 512; ++c) cp_async16(to + 512 * c + 16 * lane, k + 512 * c + 16 * lane);
            if (lane < R::kSz / 16)
              cp_async16(to + R::kCodes + 16 * lane, hr.vis_ksz + static_cast<int64_t>(i) * R::kSz + 16 * lane);
            if (in_ring && lane >= kRows && lane - kRows < n_vis - i * kRows)
              cp_async4(to + R::kCodes + R::kSz + 4 * (lane - kRows),
                        a.mass_in + base + p.vs + static_cast<int64_t>(i) * kRows + lane - kRows);
          }
          cp_async_commit();
        };
        __syncwarp();
#pragma unroll
        for (int k = 0; k < R::kStages - 1; ++k) issue(w_lo + k, ring + k * R::kStage);
        uint8_t* at = ring;                                       // block i
        uint8_t* into = ring + (R::kStages - 1) * R::kStage;      // block i + kStages - 1, where i - 1 was
        auto step = [&](uint8_t* x) { return x == ring + (R::kStages - 1) * R::kStage ? ring : x + R::kStage; };
#pragma unroll 1
        for (int i = w_lo; i < w_hi; ++i) {
          const int m = n_vis - i * kRows, t0 = p.vs + i * kRows;
          cp_async_wait<R::kStages - 2>();
          __syncwarp();
          issue(i + R::kStages - 1, into);
          into = step(into);
          RawRow<KB> r0, r1;
          load_packed<KB, G>(at + gid * (R::kCodes / kRows), at + R::kCodes + gid * (R::kSz / kRows), tig, r0);
          load_packed<KB, G>(at + (gid + 8) * (R::kCodes / kRows), at + R::kCodes + (gid + 8) * (R::kSz / kRows), tig, r1);
          float m_in = 0.f;
          if (in_ring) m_in = a.decay * *reinterpret_cast<const float*>(at + R::kCodes + R::kSz + 4 * my);
          else if (col0 > 0) m_in = fetch_mass(t0, m);
          at = step(at);
          uint32_t f0[4][4], f1[4][4];
          slice_regs<KB>(r0, f0);
          slice_regs<KB>(r1, f1);
          // the zero points (halves 2 (tig & 1), + 1) and the scales
          uint32_t za = 0u, zc = 0u;
          float s0[NG], s1[NG];
          if constexpr (NG == 4) {
            za = (tig & 1) ? r0.sz.y : r0.sz.x;
            zc = (tig & 1) ? r1.sz.y : r1.sz.x;
            h2_to_f2(r0.sz.z, s0[0], s0[1]);
            h2_to_f2(r0.sz.w, s0[2], s0[3]);
            h2_to_f2(r1.sz.z, s1[0], s1[1]);
            h2_to_f2(r1.sz.w, s1[2], s1[3]);
          } else if constexpr (NG == 2) {
            if (!(tig & 1)) za = r0.sz.x, zc = r1.sz.x;
            h2_to_f2(r0.sz.y, s0[0], s0[1]);
            h2_to_f2(r1.sz.y, s1[0], s1[1]);
          } else {
            if (!(tig & 1)) za = r0.sz.x & 0xffffu, zc = r1.sz.x & 0xffffu;
            float z;
            h2_to_f2(r0.sz.x, z, s0[0]);
            h2_to_f2(r1.sz.x, z, s1[0]);
          }
          const float kf = pow2i(24 - kLiftQ - k_first_shift<KB>());
          uint64_t s0p[NG], s1p[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            s0p[g] = pair_of(s0[g] * kf, s0[g] * kf);
            s1p[g] = pair_of(s1[g] * kf, s1[g] * kf);
          }
          const bool late = t0 + kRows > reach;
          w0 = w1 = 0ull;
#pragma unroll 2
          for (int t = 0; t < tiles; ++t) {
            float C[NG][4], x[4];
#pragma unroll
            for (int P = 0; P < 4; ++P) {
              const uint4 q = sm.qh[t][P][lane];
              const uint32_t A0[4] = {f0[P][0], f1[P][0], f0[P][1], f1[P][1]};
              const uint32_t A1[4] = {f0[P][2], f1[P][2], f0[P][3], f1[P][3]};
              if (P % PPG == 0) mma_f16_new(C[P / PPG], A0, q.x, q.y);
              else mma_f16(C[P / PPG], A0, q.x, q.y);
              mma_f16(C[P / PPG], A1, q.z, q.w);
            }
            const uint32_t Z[4] = {za, zc, 0u, 0u};
            mma_f16_new(x, Z, sm.zb[t][lane], 0u);
            uint64_t x0 = pair_of(x[0], x[1]), x1 = pair_of(x[2], x[3]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              x0 = fma_pair(s0p[g], pair_of(C[g][0], C[g][1]), x0);
              x1 = fma_pair(s1p[g], pair_of(C[g][2], C[g][3]), x1);
            }
            const uint64_t l2 = *reinterpret_cast<const uint64_t*>(&sm.lse2[t][tig]);
            const uint64_t s2 = *reinterpret_cast<const uint64_t*>(&sm.scl[t][tig]);
            add(t, fma_pair(x0, s2, l2), fma_pair(x1, s2, l2), t0, late);
          }
          store(t0, m, m_in);
        }
      }
    };
    const int e0 = min(last, b1), s1_ = max(first, b1), e1 = min(last, b2), s2_ = max(first, b2);
    if (first < e0) run_bf16(hr.text_k, n_pre, 0, first, e0);
    if (s1_ < e1) {
      if (KB < 16 && hr.k_packed) run_packed(s1_ - b1, e1 - b1);
      else run_bf16(hr.vis_k, n_vis, p.vs, s1_ - b1, e1 - b1);
    }
    if (s2_ < last)
      run_bf16(hr.text_k + static_cast<int64_t>(p.vs) * kRowBytes, n_suf, p.ve, s2_ - b2, last - b2);
  }
}

struct Kernel {
  const void* fn;
  int smem;
};
template <int KB, int G>
Kernel kernel_of() {
  return {reinterpret_cast<const void*>(&mass_kernel<KB, G>), KB < 16 ? kWarps * Ring<KB, G>::kBytes : 0};
}
template <int KB>
Kernel kernel_for(int G) {
  if constexpr (KB == 16) return kernel_of<16, 128>();
  switch (G) {
    case 32: return kernel_of<KB, 32>();
    case 64: return kernel_of<KB, 64>();
    case 128: return kernel_of<KB, 128>();
  }
  return {nullptr, 0};
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_attention_mass(const kvq_layout* L, const void* cache, const void* q_bf16, const float* lse,
                                         int32_t n_q, const int32_t* seq_len, int32_t T, const int32_t* path,
                                         int32_t max_path, const int32_t* path_len, float softmax_scale,
                                         const float* mass_in, float decay, float* mass, void* stream) {
  kvq_status st = kvq_check_layout(L);
  if (st != KVQ_OK) return st;
  if (!cache || !q_bf16 || !lse || !mass) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cache) % 256 || reinterpret_cast<uintptr_t>(q_bf16) % 16 ||
      reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(mass) % 4 ||
      reinterpret_cast<uintptr_t>(mass_in) % 4 || reinterpret_cast<uintptr_t>(seq_len) % 4 ||
      reinterpret_cast<uintptr_t>(path) % 4 || reinterpret_cast<uintptr_t>(path_len) % 4)
    return KVQ_ERR_INVALID_ARG;
  if (n_q < 1 || n_q > KVQ_MAX_QUERY_TOKENS || T < 1 || T > L->d.T_cap) return KVQ_ERR_INVALID_ARG;
  if (T > kvq::kMaxLen) return KVQ_ERR_UNSUPPORTED;
  if (!path != !path_len) return KVQ_ERR_INVALID_ARG;
  if (path ? (max_path < 1 || max_path > KVQ_MAX_QUERY_TOKENS) : (!seq_len && n_q > T)) return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !std::isfinite(decay)) return KVQ_ERR_INVALID_ARG;
  const int64_t bytes = 4 * static_cast<int64_t>(L->d.B) * L->d.H_kv * L->d.T_cap;
  if (mass_in != mass && kvq::ranges_meet(mass_in, bytes, mass, bytes)) return KVQ_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(L->d.B) * L->d.H_kv;
  if (units > 0x3fffffffLL || static_cast<int64_t>(L->g) * KVQ_MAX_QUERY_TOKENS > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  const kvq::Kernel k = L->d.k_bits == 2   ? kvq::kernel_for<2>(L->d.group_size)
                        : L->d.k_bits == 4 ? kvq::kernel_for<4>(L->d.group_size)
                        : L->d.k_bits == 8 ? kvq::kernel_for<8>(L->d.group_size)
                                           : kvq::kernel_for<16>(L->d.group_size);
  if (!k.fn) return KVQ_ERR_UNSUPPORTED;
  st = kvq_allow_smem(k.fn, k.smem);
  if (st != KVQ_OK) return st;
  kvq::MassArgs a;
  kvq::fill_geom(L, cache, &a.c);
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.lse = lse;
  a.seq_len = seq_len;
  a.path = path;
  a.path_len = path_len;
  a.T = T;
  a.n_q = n_q;
  a.max_path = max_path;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.decay = decay;
  a.mass_in = mass_in;
  a.mass = mass;
  // CTAs per (sequence, KV head): one wave of resident CTAs (several when
  // there are many pairs), the pairs with bf16 K rows split finer (a bf16
  // block takes about twice as long), but no CTA below a block for each of
  // its warps.
  int h = 0;
  for (int k = 0; k < L->n_prot; ++k) a.head[h++] = L->prot_head[k];
  for (int k = 0; k < L->n_konly; ++k) a.head[h++] = L->konly_head[k];
  a.n_bf16 = h;
  for (int k = 0; k < L->n_packed; ++k) a.head[h++] = L->packed_head[k];
  a.U[0] = L->d.B * a.n_bf16;
  a.U[1] = L->d.B * L->n_packed;
  const double cost[2] = {2.0, 1.0};
  const int64_t wave = static_cast<int64_t>(kvq::kCtasPerSm) * n_sm;
  const int64_t cap = units <= wave / 2 ? wave : 6 * wave;  // many pairs: several waves, for an even end
  const int most = std::max(1, T / ((units <= wave / 2 ? 1 : 4) * kvq::kRows * kvq::kWarps));
  a.S[0] = a.S[1] = 1;
  for (;;) {
    int worst = -1;
    for (int k = 0; k < 2; ++k)
      if (a.U[k] && a.S[k] < most && (worst < 0 || cost[k] / a.S[k] > cost[worst] / a.S[worst])) worst = k;
    const int64_t used = static_cast<int64_t>(a.U[0]) * a.S[0] + static_cast<int64_t>(a.U[1]) * a.S[1];
    if (worst < 0 || used + a.U[worst] > cap) break;
    ++a.S[worst];
  }
  return kvq::launch_dependent(k.fn, dim3(a.U[0] * a.S[0] + a.U[1] * a.S[1]), kvq::kWarps * 32, k.smem, stream, &a);
}
