// kvq_simple.cuh -- one element of a stored row, by the storage order of
// kvq.h: the direct form that the first tree and mass kernels read rows with.
#pragma once

#include "kvq_geom.cuh"

namespace kvq {

__device__ __forceinline__ int k_slot(int bits, int d) {
  const int P = d >> 5, t = (d >> 3) & 3, e = (d >> 2) & 1, i = d & 3;
  if (bits == 2) {
    const int c = (i & 1) ? (P == 3 ? 1 : 7 - P) : (P == 3 ? 0 : 4 - P);
    return 32 * t + 16 * (i >> 1) + 8 * e + c;
  }
  return bits == 4 ? 32 * t + 8 * i + 4 * e + P : 32 * t + 4 * (2 * P + (i >> 1)) + 2 * e + (i & 1);
}
__device__ __forceinline__ int v_slot(int d) { return 16 * (d & 7) + 2 * (d >> 4) + ((d >> 3) & 1); }

// Elements d0 .. d0 + 3 of a row: bf16 (sz null) or codes with their
// scale/zero row.
__device__ __forceinline__ float4 row4(const uint8_t* row, const uint8_t* sz, int bits, int G, bool key, int d0) {
  float x[4];
  if (!sz) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + 2 * d0);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  }
  const __half* h = reinterpret_cast<const __half*>(sz);
  const int grp = d0 / G;
  const float z = __half2float(h[grp]), s = __half2float(h[kD / G + grp]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int bit = bits * (key ? k_slot(bits, d0 + i) : v_slot(d0 + i));
    const int code = (row[bit >> 3] >> (bit & 7)) & ((1 << bits) - 1);
    x[i] = fmaf(static_cast<float>(code), s, z);
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ float4 k_row4(const Geom& p, const HeadRows& r, int t, int d0) {
  if (t >= p.vs && t < p.ve) {
    const int64_t i = t - p.vs;
    if (r.k_packed) return row4(r.vis_k + i * p.krow, r.vis_ksz + i * p.kszrow, p.kb, p.G, true, d0);
    return row4(r.vis_k + i * kRowBytes, nullptr, 16, p.G, true, d0);
  }
  return row4(r.text_k + static_cast<int64_t>(t < p.vs ? t : t - p.Tv) * kRowBytes, nullptr, 16, p.G, true, d0);
}
__device__ __forceinline__ float4 v_row4(const Geom& p, const HeadRows& r, int t, int d0) {
  if (t >= p.vs && t < p.ve) {
    const int64_t i = t - p.vs;
    if (r.v_packed) return row4(r.vis_v + i * p.vrow, r.vis_vsz + i * p.vszrow, p.vb, p.G, false, d0);
    return row4(r.vis_v + i * kRowBytes, nullptr, 16, p.G, false, d0);
  }
  return row4(r.text_v + static_cast<int64_t>(t < p.vs ? t : t - p.Tv) * kRowBytes, nullptr, 16, p.G, false, d0);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

}  // namespace kvq
