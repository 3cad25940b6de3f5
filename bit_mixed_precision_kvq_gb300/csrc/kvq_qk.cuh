// kvq_qk.cuh -- scores of cache rows against query columns on mma.sync, as the
// attention mass and windowed decode kernels form them: 16 positions (M)
// against 8 columns (N), packed codes as exact fp16 subnormals, bf16 rows and
// queries as they are stored.
#pragma once

#include "kvq_split.cuh"

namespace kvq {

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A code of block P sits at bit kKShift(P) of its half, i.e. is 2^(p - 24) c;
// the fp16 query elements of the block carry 2^(6 + p0 - p), p0 the smallest p,
// so that the blocks of a group share one accumulator (and 2^6, so that the
// factor is 1 or more and costs small elements nothing: 2^15 at most).
constexpr int kQueryExponent = 8;  // a column's largest |q| lands in [2^8, 2^9)
constexpr int kLiftQ = 6;
template <int KB>
__device__ __forceinline__ constexpr int k_first_shift() {
  return KB == 2 ? 2 : 0;
}
template <int KB>
__device__ __forceinline__ float q_factor(int P) {
  const int p = KB == 2 ? 8 - 2 * P : (KB == 4 ? 4 * (P & 1) : 0);
  return __int_as_float((127 + kLiftQ + k_first_shift<KB>() - p) << 23);
}

// D = A * B (a fresh accumulator).
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

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

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 8 NT query columns as MMA operands: fp16 with a power of two of each
// column's own (its largest element lands in [2^8, 2^9), so that the others are
// exact down to 2^-25 of it), and bf16 as stored.
template <int NT>
struct Columns {
  uint4 qh[NT][4][32];   // fp16 operand: [tile][32-element block][lane], see q_factor
  uint4 qb[NT][4][32];   // bf16 operand
  uint32_t zb[NT][32];   // group sums, high then low
  float2 scl[NT][4];     // columns 2 tig, 2 tig + 1: what takes packed scores to log2 units
  float qs[NT * 8][4];
};

// The columns from col0 on of KV head h of sequence b, column k g + j being
// query head j of token k; those past the last token are zero.  Called by all
// kThreads threads; the caller synchronises before use.
template <int KB, int G, int NT, int kThreads>
__device__ __forceinline__ void load_columns(Columns<NT>& sm, int Hq, int g, const uint16_t* q, int n_q, int b, int h, int col0,
                                             float scale_log2) {
  constexpr int NG = kD / G;
  for (int x = threadIdx.x; x < NT * 8 * 16; x += kThreads) {
    const int tig = x & 3, P = (x >> 2) & 3, c = x >> 4, cg = col0 + c;
    const int k = cg / g, j = cg - k * g;
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (k < n_q)
      r = __ldcg(reinterpret_cast<const uint4*>(q + ((static_cast<int64_t>(b) * n_q + k) * Hq + h * g + j) * kD) + 4 * P + tig);
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
      if (P == 0) reinterpret_cast<float*>(&sm.scl[t][0])[c & 7] = scale_log2 * __int_as_float((127 - e) << 23);
    }
  }
  __syncthreads();
  // K index 2 tig, 2 tig + 1: high parts of groups 0 .. 3, then the low parts
  for (int x = threadIdx.x; x < NT * 32; x += kThreads) {
    const int tig = x & 3, c = x >> 2;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int g0 = 2 * (tig & 1) + e;
      if (g0 < NG) {
#pragma unroll
        for (int i = 0; i < 4 / NG; ++i) s[e] += sm.qs[c][g0 * (4 / NG) + i];
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
}

// Scores, in log2 units, of packed rows r0 + gid, r0 + gid + 8 of a staged
// block (codes at kc, scale/zero rows at ksz): f(tile, S) with S as an MMA
// accumulator holds them.
template <int KB, int G, int NT, typename F>
__device__ __forceinline__ void qk_packed_rows(const uint8_t* kc, const uint8_t* ksz, int r0, const Columns<NT>& sm, int lane, F&& f) {
  constexpr int NG = kD / G, PPG = G / 32, kRow = 16 * KB, kSz = 4 * NG;
  const int gid = lane >> 2, tig = lane & 3;
  RawRow<KB> a, b;
  load_packed<KB, G>(kc + (r0 + gid) * kRow, ksz + (r0 + gid) * kSz, tig, a);
  load_packed<KB, G>(kc + (r0 + gid + 8) * kRow, ksz + (r0 + gid + 8) * kSz, tig, b);
  uint32_t f0[4][4], f1[4][4];
  slice_regs<KB>(a, f0);
  slice_regs<KB>(b, f1);
  // the zero points (halves 2 (tig & 1), + 1) and the scales
  uint32_t za = 0u, zc = 0u;
  float s0[NG], s1[NG];
  if constexpr (NG == 4) {
    za = (tig & 1) ? a.sz.y : a.sz.x;
    zc = (tig & 1) ? b.sz.y : b.sz.x;
    h2_to_f2(a.sz.z, s0[0], s0[1]);
    h2_to_f2(a.sz.w, s0[2], s0[3]);
    h2_to_f2(b.sz.z, s1[0], s1[1]);
    h2_to_f2(b.sz.w, s1[2], s1[3]);
  } else if constexpr (NG == 2) {
    if (!(tig & 1)) za = a.sz.x, zc = b.sz.x;
    h2_to_f2(a.sz.y, s0[0], s0[1]);
    h2_to_f2(b.sz.y, s1[0], s1[1]);
  } else {
    if (!(tig & 1)) za = a.sz.x & 0xffffu, zc = b.sz.x & 0xffffu;
    float z;
    h2_to_f2(a.sz.x, z, s0[0]);
    h2_to_f2(b.sz.x, z, s1[0]);
  }
  const float kf = pow2i(24 - kLiftQ - k_first_shift<KB>());
  uint64_t s0p[NG], s1p[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    s0p[g] = pair_of(s0[g] * kf, s0[g] * kf);
    s1p[g] = pair_of(s1[g] * kf, s1[g] * kf);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float C[NG][4], S[4];
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
    mma_f16_new(S, Z, sm.zb[t][lane], 0u);
    uint64_t x0 = pair_of(S[0], S[1]), x1 = pair_of(S[2], S[3]);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      x0 = fma_pair(s0p[g], pair_of(C[g][0], C[g][1]), x0);
      x1 = fma_pair(s1p[g], pair_of(C[g][2], C[g][3]), x1);
    }
    const uint64_t scl = *reinterpret_cast<const uint64_t*>(&sm.scl[t][tig]);
    unpair(mul_pair(x0, scl), S[0], S[1]);
    unpair(mul_pair(x1, scl), S[2], S[3]);
    f(t, S);
  }
}

// The same of 16 bf16 rows: load(P, x, y) gives elements 32 P + 8 tig .. + 7 of
// rows gid and gid + 8.
template <int NT, typename Load, typename F>
__device__ __forceinline__ void qk_bf16_rows(Load&& load, const Columns<NT>& sm, float scale_log2, int lane, F&& f) {
  uint4 x[4], y[4];
#pragma unroll
  for (int P = 0; P < 4; ++P) load(P, x[P], y[P]);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float C[2][4];
#pragma unroll
    for (int P = 0; P < 4; ++P) {
      const uint4 q = sm.qb[t][P][lane];
      const uint32_t A0[4] = {x[P].x, y[P].x, x[P].y, y[P].y};
      const uint32_t A1[4] = {x[P].z, y[P].z, x[P].w, y[P].w};
      if (P == 0) {
        mma_bf16_new(C[0], A0, q.x, q.y);
        mma_bf16_new(C[1], A1, q.z, q.w);
      } else {
        mma_bf16(C[0], A0, q.x, q.y);
        mma_bf16(C[1], A1, q.z, q.w);
      }
    }
    float S[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) S[i] = (C[0][i] + C[1][i]) * scale_log2;
    f(t, S);
  }
}

}  // namespace kvq
