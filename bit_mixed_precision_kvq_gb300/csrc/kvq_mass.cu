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
// bf16 rows and queries go to the bf16 MMA as they are stored.
//
// With few columns the pass is bound by the K bytes, with many by the MMA rate
// (9 MMAs of 8 cycles per 16 positions and 8 columns), so the operands of a
// 16-row block stay in registers over all columns.  mma.sync and not tcgen05:
// the contraction is at most 64 columns thin between unpacking and exponential,
// and the weights are wanted per position, where their fragments already are.
#include "kvq_split.cuh"

#include "kvq_geom.cuh"

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
  int32_t strips;                // CTAs per (sequence, KV head)
  uint8_t head[KVQ_MAX_HEADS];   // heads, those with the longest rows first
};

struct MassSmem {
  uint4 qh[kMaxTiles][4][32];   // fp16 operand: [tile][32-element block][lane]
  uint4 qb[kMaxTiles][4][32];   // bf16 operand
  uint32_t zb[kMaxTiles][32];   // group sums, high then low
  float2 lse2[kMaxTiles][4];    // lse in log2 units of columns 2 tig, 2 tig + 1
  int2 lim[kMaxTiles][4];       // those columns see the positions below
  float qs[kMaxTiles * 8][4];
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The columns [col0, col0 + 8 tiles) of (b, h): token k of the n taken is
// column k g + j.  Columns that add nothing get q = 0 and lse = +inf.
template <int G>
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
    const uint32_t y[4] = {bf16pair_f16(r.x, false, r.z, false), bf16pair_f16(r.x, true, r.z, true),
                           bf16pair_f16(r.y, false, r.w, false), bf16pair_f16(r.y, true, r.w, true)};
    sm.qh[t][P][lane] = make_uint4(y[0], y[1], y[2], y[3]);
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
        float* l2 = reinterpret_cast<float*>(&sm.lse2[t][0]);
        int* lm = reinterpret_cast<int*>(&sm.lim[t][0]);
        l2[c & 7] = l * 1.4426950408889634f;
        lm[c & 7] = len - n + 1 + k;
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
        s[e] *= a.scale_log2 / kZbScale;
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

// A block of up to 16 positions of one kind.
struct Block {
  const uint8_t *row, *sz;  // first row
  int t0, n;
  bool packed;
};

template <int KB>
struct RawRow {
  uint32_t w[KB < 16 ? KB : 16];  // a lane's slice (4 KB bytes), or 4 x 16 bytes of a bf16 row
  uint4 sz;
};

template <int KB, int G>
__device__ __forceinline__ void load_packed(const uint8_t* row, const uint8_t* sz, int tig, RawRow<KB>& r) {
  if constexpr (KB == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(row + 8 * tig);
    r.w[0] = x.x;
    r.w[1] = x.y;
  } else if constexpr (KB < 16) {
#pragma unroll
    for (int i = 0; i < KB / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(row + 4 * KB * tig)[i];
      r.w[4 * i] = x.x;
      r.w[4 * i + 1] = x.y;
      r.w[4 * i + 2] = x.z;
      r.w[4 * i + 3] = x.w;
    }
  }
  if constexpr (G == 32) {
    r.sz = *reinterpret_cast<const uint4*>(sz);
  } else if constexpr (G == 64) {
    const uint2 x = *reinterpret_cast<const uint2*>(sz);
    r.sz.x = x.x;
    r.sz.y = x.y;
  } else {
    r.sz.x = *reinterpret_cast<const uint32_t*>(sz);
  }
}

// Operand registers f[P][i] (pair P, register i) of a lane's slice: codes at
// bit kKShift(P) of each half (kvq_split.cuh).
template <int KB>
__device__ __forceinline__ void slice_regs(const RawRow<KB>& r, uint32_t (&f)[4][4]) {
  if constexpr (KB == 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t x = r.w[h], y = x >> 6, z = x << 2;
      f[0][2 * h] = x & 0x03000300u;
      f[0][2 * h + 1] = y & 0x03000300u;
      f[1][2 * h] = x & 0x00C000C0u;
      f[1][2 * h + 1] = y & 0x00C000C0u;
      f[2][2 * h] = x & 0x00300030u;
      f[2][2 * h + 1] = y & 0x00300030u;
      f[3][2 * h] = z & 0x000C000Cu;
      f[3][2 * h + 1] = x & 0x000C000Cu;
    }
  } else if constexpr (KB == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = r.w[i] >> 8;
      f[0][i] = r.w[i] & 0x000F000Fu;
      f[1][i] = r.w[i] & 0x00F000F0u;
      f[2][i] = y & 0x000F000Fu;
      f[3][i] = y & 0x00F000F0u;
    }
  } else if constexpr (KB == 8) {
#pragma unroll
    for (int P = 0; P < 4; ++P)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = r.w[2 * P + (i >> 1)];
        f[P][i] = ((i & 1) ? (v >> 8) : v) & 0x00FF00FFu;
      }
  }
}

template <int KB, int G>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) mass_kernel(const __grid_constant__ MassArgs a) {
  __shared__ MassSmem sm;
  const Geom& p = a.c;
  constexpr int NG = kD / G;
  constexpr int PPG = G / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int unit = blockIdx.x / a.strips, strip = blockIdx.x - unit * a.strips;
  const int h = a.head[unit / p.B], b = unit - (unit / p.B) * p.B;
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
  const int first = static_cast<int>(static_cast<int64_t>(nb) * strip / a.strips);
  const int last = static_cast<int>(static_cast<int64_t>(nb) * (strip + 1) / a.strips);
  auto block = [&](int i) {
    Block x;
    x.sz = nullptr;
    x.packed = false;
    if (i >= b1 && i < b2) {
      const int r = (i - b1) * kRows;
      x.t0 = p.vs + r;
      x.n = min(kRows, n_vis - r);
      x.packed = hr.k_packed;
      x.row = hr.vis_k + static_cast<int64_t>(r) * (hr.k_packed ? p.krow : kRowBytes);
      if (hr.k_packed) x.sz = hr.vis_ksz + static_cast<int64_t>(r) * p.kszrow;
    } else {
      const int r = (i < b1 ? i : i - b2) * kRows;
      x.t0 = i < b1 ? r : p.ve + r;
      x.n = min(kRows, (i < b1 ? n_pre : n_suf) - r);
      x.row = hr.text_k + static_cast<int64_t>(i < b1 ? r : p.vs + r) * kRowBytes;
    }
    return x;
  };
  const int64_t base = (static_cast<int64_t>(b) * p.Hkv + h) * p.T_cap;
  const int cols = p.g * n;
  // a block's rows into L2, ahead of the loads (one lane)
  auto prefetch = [&](int i) {
    if (i >= last) return;
    const Block x = block(i);
    prefetch_bytes(x.row, x.n * (x.packed ? p.krow : kRowBytes));
    if (x.packed) prefetch_bytes(x.sz, x.n * p.kszrow);
    if (a.mass_in) prefetch_bytes(a.mass_in + base + x.t0, 4 * x.n);
  };
  if (lane == 0)
    for (int k = 0; k < kAhead; ++k) prefetch(first + warp + k * kWarps);
  // one pass over the rows for every 64 columns (at least one: the decay)
  for (int col0 = 0; col0 == 0 || col0 < cols; col0 += 8 * kMaxTiles) {
    const int tiles = min(kMaxTiles, (cols - col0 + 7) / 8);
    if (col0 > 0) __syncthreads();
    load_columns<G>(a, sm, b, h, len, n, col0, tiles);
    RawRow<KB> r0, r1;
    auto fetch = [&](const Block& x) {
      if constexpr (KB < 16) {
        if (x.packed) {  // rows past the last are read from it
          const int i0 = min(gid, x.n - 1), i1 = min(gid + 8, x.n - 1);
          load_packed<KB, G>(x.row + i0 * p.krow, x.sz + i0 * p.kszrow, tig, r0);
          load_packed<KB, G>(x.row + i1 * p.krow, x.sz + i1 * p.kszrow, tig, r1);
        }
      }
    };
    // the mass that the block's sum is added to: lanes tig 0 have row gid, tig 1 row gid + 8
    const int my = tig == 0 ? gid : gid + 8;
    auto fetch_mass = [&](const Block& x) {
      if (tig >= 2 || my >= x.n) return 0.f;
      if (col0 > 0) return a.mass[base + x.t0 + my];
      return a.mass_in ? a.decay * a.mass_in[base + x.t0 + my] : 0.f;
    };
    Block cur;
    float cur_mass = 0.f;
    if (first + warp < last) {
      cur = block(first + warp);
      cur_mass = fetch_mass(cur);
      fetch(cur);
    }
#pragma unroll 1
    for (int i = first + warp; i < last; i += kWarps) {
      const Block x = cur;
      const float m_in = cur_mass;
      if (lane == 0 && col0 == 0) prefetch(i + kAhead * kWarps);
      const bool late = x.t0 + x.n > len - n + 1;  // some column does not reach the last rows
      float w0 = 0.f, w1 = 0.f;                    // weights of rows gid, gid + 8
      auto add = [&](int t, float (&S)[4]) {
        const float2 l2 = sm.lse2[t][tig];
        float e0 = ex2(S[0] - l2.x), e1 = ex2(S[1] - l2.y), e2 = ex2(S[2] - l2.x), e3 = ex2(S[3] - l2.y);
        if (late) {
          const int2 lim = sm.lim[t][tig];
          const int ta = x.t0 + gid, tb = ta + 8;
          if (ta >= lim.x) e0 = 0.f;
          if (ta >= lim.y) e1 = 0.f;
          if (tb >= lim.x) e2 = 0.f;
          if (tb >= lim.y) e3 = 0.f;
        }
        w0 += e0 + e1;
        w1 += e2 + e3;
      };
      if (KB < 16 && x.packed) {
        if constexpr (KB < 16) {
          uint32_t f0[4][4], f1[4][4];
          slice_regs<KB>(r0, f0);
          slice_regs<KB>(r1, f1);
          const uint4 sz0 = r0.sz, sz1 = r1.sz;
          if (i + kWarps < last) {
            cur = block(i + kWarps);
            cur_mass = fetch_mass(cur);
            fetch(cur);
          }
          uint32_t za = 0u, zc = 0u;  // z halves 2 (tig & 1), + 1
          float s0[NG], s1[NG];
          if constexpr (NG == 4) {
            za = (tig & 1) ? sz0.y : sz0.x;
            zc = (tig & 1) ? sz1.y : sz1.x;
            h2_to_f2(sz0.z, s0[0], s0[1]);
            h2_to_f2(sz0.w, s0[2], s0[3]);
            h2_to_f2(sz1.z, s1[0], s1[1]);
            h2_to_f2(sz1.w, s1[2], s1[3]);
          } else if constexpr (NG == 2) {
            if (!(tig & 1)) za = sz0.x, zc = sz1.x;
            h2_to_f2(sz0.y, s0[0], s0[1]);
            h2_to_f2(sz1.y, s1[0], s1[1]);
          } else {
            if (!(tig & 1)) za = sz0.x & 0xffffu, zc = sz1.x & 0xffffu;
            float z;
            h2_to_f2(sz0.x, z, s0[0]);
            h2_to_f2(sz1.x, z, s1[0]);
          }
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float kf = a.scale_log2 * kKFactor<KB>(g * PPG);
            s0[g] *= kf;
            s1[g] *= kf;
          }
#pragma unroll 1
          for (int t = 0; t < tiles; ++t) {
            float C[4][4];
#pragma unroll
            for (int P = 0; P < 4; ++P) {
              C[P][0] = C[P][1] = C[P][2] = C[P][3] = 0.f;
              const uint4 q = sm.qh[t][P][lane];
              const uint32_t A0[4] = {f0[P][0], f1[P][0], f0[P][1], f1[P][1]};
              const uint32_t A1[4] = {f0[P][2], f1[P][2], f0[P][3], f1[P][3]};
              mma_f16(C[P], A0, q.x, q.y);
              mma_f16(C[P], A1, q.z, q.w);
            }
            float S[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t Z[4] = {za, zc, 0u, 0u};
            mma_f16(S, Z, sm.zb[t][lane], 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k) S[k] *= kZbScale;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float v = C[g * PPG][k];
#pragma unroll
                for (int e = 1; e < PPG; ++e)
                  v = fmaf(C[g * PPG + e][k], kKFactor<KB>(g * PPG + e) / kKFactor<KB>(g * PPG), v);
                S[k] = fmaf(k < 2 ? s0[g] : s1[g], v, S[k]);
              }
            add(t, S);
          }
        }
      } else {
        uint4 f0[4], f1[4];
#pragma unroll
        for (int P = 0; P < 4; ++P) {
          const int off = 64 * P + 16 * tig;
          f0[P] = *reinterpret_cast<const uint4*>(x.row + min(gid, x.n - 1) * kRowBytes + off);
          f1[P] = *reinterpret_cast<const uint4*>(x.row + min(gid + 8, x.n - 1) * kRowBytes + off);
        }
        if (i + kWarps < last) {
          cur = block(i + kWarps);
          cur_mass = fetch_mass(cur);
          fetch(cur);
        }
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
          float C[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int P = 0; P < 4; ++P) {
            const uint4 q = sm.qb[t][P][lane];
            const uint32_t A0[4] = {f0[P].x, f1[P].x, f0[P].y, f1[P].y};
            const uint32_t A1[4] = {f0[P].z, f1[P].z, f0[P].w, f1[P].w};
            mma_bf16(C[0], A0, q.x, q.y);
            mma_bf16(C[1], A1, q.z, q.w);
          }
          float S[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) S[k] = (C[0][k] + C[1][k]) * a.scale_log2;
          add(t, S);
        }
      }
      w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
      w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
      w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
      w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
      if (tig < 2 && my < x.n) a.mass[base + x.t0 + my] = m_in + (tig == 0 ? w0 : w1);
    }
  }
}

template <int KB>
const void* mass_kernel_for(int G) {
  if constexpr (KB == 16) return reinterpret_cast<const void*>(&mass_kernel<16, 128>);
  switch (G) {
    case 32: return reinterpret_cast<const void*>(&mass_kernel<KB, 32>);
    case 64: return reinterpret_cast<const void*>(&mass_kernel<KB, 64>);
    case 128: return reinterpret_cast<const void*>(&mass_kernel<KB, 128>);
  }
  return nullptr;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_attention_mass(const kvq_layout* L, const void* cache, const void* q_bf16, const float* lse,
                                         int32_t n_q, const int32_t* seq_len, int32_t T, const int32_t* path,
                                         int32_t max_path, const int32_t* path_len, float softmax_scale,
                                         const float* mass_in, float decay, float* mass, void* stream) {
  const kvq_status st = kvq_check_layout(L);
  if (st != KVQ_OK) return st;
  if (!cache || !q_bf16 || !lse || !mass) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cache) % 256 || reinterpret_cast<uintptr_t>(q_bf16) % 16 ||
      reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(mass) % 4 ||
      reinterpret_cast<uintptr_t>(mass_in) % 4 || reinterpret_cast<uintptr_t>(seq_len) % 4 ||
      reinterpret_cast<uintptr_t>(path) % 4 || reinterpret_cast<uintptr_t>(path_len) % 4)
    return KVQ_ERR_INVALID_ARG;
  if (n_q < 1 || n_q > KVQ_MAX_QUERY_TOKENS || T < 1 || T > L->d.T_cap) return KVQ_ERR_INVALID_ARG;
  if (!path != !path_len) return KVQ_ERR_INVALID_ARG;
  if (path ? (max_path < 1 || max_path > KVQ_MAX_QUERY_TOKENS) : (!seq_len && n_q > T)) return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !std::isfinite(decay)) return KVQ_ERR_INVALID_ARG;
  const int64_t bytes = 4 * static_cast<int64_t>(L->d.B) * L->d.H_kv * L->d.T_cap;
  if (mass_in != mass && kvq::ranges_meet(mass_in, bytes, mass, bytes)) return KVQ_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(L->d.B) * L->d.H_kv;
  // CTAs per (sequence, KV head): enough for several waves of resident CTAs,
  // so that heads with bf16 rows (up to 10 times the bytes) even out, but at
  // least a block for every warp of a CTA.
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  const int64_t want = (4 * kvq::kCtasPerSm * static_cast<int64_t>(n_sm) + units - 1) / units;
  const int64_t most = std::max<int64_t>(1, T / (kvq::kRows * kvq::kWarps));
  const int64_t strips = std::max<int64_t>(1, std::min(want, most));
  if (units * strips > 0x7fffffffLL || static_cast<int64_t>(L->g) * KVQ_MAX_QUERY_TOKENS > 0x7fffffffLL)
    return KVQ_ERR_UNSUPPORTED;
  const void* fn = L->d.k_bits == 2   ? kvq::mass_kernel_for<2>(L->d.group_size)
                   : L->d.k_bits == 4 ? kvq::mass_kernel_for<4>(L->d.group_size)
                   : L->d.k_bits == 8 ? kvq::mass_kernel_for<8>(L->d.group_size)
                                      : kvq::mass_kernel_for<16>(L->d.group_size);
  if (!fn) return KVQ_ERR_UNSUPPORTED;
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
  a.strips = static_cast<int32_t>(strips);
  int h = 0;
  for (int k = 0; k < L->n_prot; ++k) a.head[h++] = L->prot_head[k];
  for (int k = 0; k < L->n_konly; ++k) a.head[h++] = L->konly_head[k];
  for (int k = 0; k < L->n_packed; ++k) a.head[h++] = L->packed_head[k];
  return kvq::launch_dependent(fn, dim3(static_cast<unsigned>(units * strips)), kvq::kWarps * 32, 0, stream, &a);
}
