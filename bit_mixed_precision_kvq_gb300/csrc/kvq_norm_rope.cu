// kvq_norm_rope.cu -- kvq_norm_rope: the rows of query and key heads normed
// and rotated by positions of several axes, in one pass.
//
//   y = x / sqrt(mean_d x_d^2 + eps) * w        (y = x without a weight)
//   pair i of the first rot_dim elements turns by the angle
//   a_i = pos[axis_i] * inv_freq_i:
//     (y_p, y_q) -> (y_p cos a_i - y_q sin a_i, y_q cos a_i + y_p sin a_i)
//
// Every row is read once and written once (512 bytes), with some 55 instructions
// a lane in between: bound by memory once there are enough rows.  16 lanes hold a
// row of 128, each the elements of 4 pairs (8 beyond the rotated part), so that a
// pair never crosses lanes and the mean takes 4 shuffles.  A lane's angles depend
// on the token alone: 16 lanes take up to 8 heads of one token, load all their
// rows at once, make the weights times cosines and sines meanwhile, and end
// (short-lived CTAs overlap their phases; a CTA that went from token to token
// with 4 rows under way took 234 us where this takes 162).
//
// Angles.  A position may be large (a product with a frequency near 1 loses
// all its digits in fp32 from 2^24 on), so the turn is taken modulo 1 in
// integers: inv_freq / 2 pi modulo 1 as a 64-bit binary fraction, times the
// position modulo 2^64.  Its top 32 bits, rounded to fp32, are the angle to
// 2^-25 of a turn, and the fast sine and cosine of it are off by 2^-21.  The rest
// is fp32, in pairs, rounded once to bf16.  Squares leave fp32 for elements outside
// some 2^-63 .. 2^63: a row whose mean + eps is not in [2^-100, 2^128) is not stored but
// made again at the end, scaled by a power of two.
//
// Measured (GB300): 8 x 2940 tokens, 40 + 40 heads with norms (963 MB) 167 us (162
// without the look at the means' range), 5.8 TB/s, 0.85 of a copy; 16 x 26 tokens, 32 +
// 32 heads 5.1 us; one token 2.0 us.
#include "kvq_geom.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace kvq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRowLanes = 16;

struct RopeSide {
  const uint16_t* in;  // element (b, h, t, d) at b sb + h sh + t st + d
  uint16_t* out;
  int64_t sb, sh, st, ob, oh, ot;
  const uint16_t* weight;  // bf16 [D] or null: no norm
  int32_t H, groups;       // heads, and groups of them
};

struct RopeArgs {
  RopeSide side[2];  // q, k
  const int32_t* pos;  // [n_axes][B][n]
  int64_t pos_axis, pos_b;
  const float* freq;  // [rot / 2]
  float eps;
  int32_t n, tokens, rot;  // tokens: B n
  uint8_t axis[kD / 2];
};

// Pairs of fp32 from four bf16 and back.
__device__ __forceinline__ void wide(uint2 w, uint64_t& x, uint64_t& y) {
  x = pair_of(bf16_lo(w.x), bf16_hi(w.x));
  y = pair_of(bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ uint32_t narrow(uint64_t x) {
  float u, v;
  unpair(x, u, v);
  return pack_bf16x2(u, v);
}
__device__ __forceinline__ uint64_t neg_pair(uint64_t x) { return x ^ 0x8000000080000000ull; }

// A row's two chunks of 4 as (first, second) elements of its pairs: they are
// the chunks themselves when pairs lie apart, else neighbours.
template <bool kNeighbours>
__device__ __forceinline__ void split(uint64_t& x0, uint64_t& x1, uint64_t& y0, uint64_t& y1) {
  if constexpr (kNeighbours) {
    float a, b, c, d, e, f, g, h;
    unpair(x0, a, b);
    unpair(x1, c, d);
    unpair(y0, e, f);
    unpair(y1, g, h);
    x0 = pair_of(a, c);
    x1 = pair_of(e, g);
    y0 = pair_of(b, d);
    y1 = pair_of(f, h);
  }
}
template <bool kNeighbours>
__device__ __forceinline__ void join(uint64_t& x0, uint64_t& x1, uint64_t& y0, uint64_t& y1) {
  if constexpr (kNeighbours) {
    float a, b, c, d, e, f, g, h;
    unpair(x0, a, b);
    unpair(x1, c, d);
    unpair(y0, e, f);
    unpair(y1, g, h);
    x0 = pair_of(a, e);
    x1 = pair_of(b, f);
    y0 = pair_of(c, g);
    y1 = pair_of(d, h);
  }
}

constexpr uint32_t kLeastMean = 27u << 23;  // 2^-100: squares that underflowed are 2^-43 of it at most

// The power of two that takes a row's largest element to [1, 2), or to where its
// square is far from fp32's ends.  Called by whole warps, 16 lanes a row (the caller
// takes the rows that want it).
__device__ __forceinline__ float to_one(uint2 x, uint2 y) {
  uint32_t top = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu));
  top = max(top & 0xffffu, top >> 16);
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  return __int_as_float((127 - max(-100, min(100, static_cast<int>(top >> 7) - 127))) << 23);
}

// f / 2 pi modulo 1 in units of 2^-64, to 2 of them for every finite f: the 24 bits
// m of f times the bits of 1 / 2 pi that do not make whole turns (reduction as
// published by Payne and Hanek, 1983).
__device__ __forceinline__ uint64_t turn_of(float f) {
  constexpr uint64_t kInv = 0x28be60db9391054aull;  // 2^64 / 2 pi
  const uint32_t u = __float_as_uint(f), e = (u >> 23) & 0xff;
  uint64_t t;
  if (e <= 127) {  // m 2^(e - 150) / 2 pi: one product by the first 64 bits of 1 / 2 pi
    const uint32_t m = e ? (u & 0x7fffffu) | 0x800000u : (u & 0x7fffffu) << 1;
    const uint64_t lo = static_cast<uint64_t>(m) * static_cast<uint32_t>(kInv), hi = static_cast<uint64_t>(m) * static_cast<uint32_t>(kInv >> 32) + (lo >> 32);
    const int s = 150 - static_cast<int>(e);  // 23 and more; the product is hi 2^32 + low half of lo
    t = s < 32 ? (hi << (32 - s)) | (static_cast<uint32_t>(lo) >> s) : (s < 96 ? hi >> (s - 32) : 0ull);
  } else {  // |f| >= 2: m times the 128 bits of 1 / 2 pi behind its first e - 150
    constexpr uint64_t k1 = 0x7f09d5f47d4d3770ull, k2 = 0x36d8a5664f10e410ull, k3 = 0x7f9458eaf7aef158ull;  // its next bits
    const uint64_t m = (u & 0x7fffffu) | 0x800000u;
    const int o = static_cast<int>(e) - 150 + 64, r = o & 63;  // 42 .. 169, from 64 zero bits before the first on
    const uint64_t x = o < 64 ? 0ull : (o < 128 ? kInv : k1), y = o < 64 ? kInv : (o < 128 ? k1 : k2), z = o < 64 ? k1 : (o < 128 ? k2 : k3);
    const uint64_t w0 = r ? (x << r) | (y >> (64 - r)) : x, w1 = r ? (y << r) | (z >> (64 - r)) : y;
    t = m * w0 + __umul64hi(m, w1);
  }
  return u >> 31 ? 0ull - t : t;
}

// blockIdx.y: the group of at most kHeads heads; 16 lanes take them for one
// token, all rows loaded before any is used.
template <int kHeads, bool kNeighbours>
__global__ void __launch_bounds__(kRopeThreads, kHeads == 8 ? 3 : 4) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  const int j = threadIdx.x & (kRowLanes - 1);
  const bool turns = 8 * j < a.rot;
  // first elements of the lane's two chunks of 4
  const bool apart = turns && !kNeighbours;
  const int e0 = apart ? 4 * j : 8 * j, gap = apart ? a.rot / 2 : 4;
  const bool key = static_cast<int>(blockIdx.y) >= a.side[0].groups;
  const RopeSide& s = a.side[key];
  const int h0 = (static_cast<int>(blockIdx.y) - (key ? a.side[0].groups : 0)) * kHeads, rows = min(kHeads, s.H - h0);
  const int token = static_cast<int>(blockIdx.x) * (kRopeThreads / kRowLanes) + static_cast<int>(threadIdx.x) / kRowLanes;
  const bool live = token < a.tokens;  // (the other half of the warp may be)
  const int b = live ? token / a.n : 0, t = live ? token - b * a.n : 0;
  const uint16_t* from = s.in + b * s.sb + t * s.st + h0 * s.sh + e0;
  // No pdl_launch_dependents: K may be written where it stays, into the text rows
  // of a cache, and the next kernel may read cache rows before its own dependency
  // wait.  It launches when this one has finished (behind a fence and a barrier of
  // every CTA: 190 us in place of 163 for the large case, 2.4 of 2.0 for one token).
  pdl_wait();
  uint2 x[kHeads], y[kHeads];
  {
    const int64_t sh = s.sh;
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      x[k] = y[k] = make_uint2(0u, 0u);
      if (live && k < rows) {
        x[k] = *reinterpret_cast<const uint2*>(from);
        y[k] = *reinterpret_cast<const uint2*>(from + gap);
      }
      from += sh;
    }
  }
  const bool norm = s.weight != nullptr;
  const uint64_t one = pair_of(1.f, 1.f);
  uint64_t p0 = one, p1 = one, q0 = one, q1 = one;  // the weight's elements of the pairs
  if (norm) {
    wide(*reinterpret_cast<const uint2*>(s.weight + e0), p0, p1);
    wide(*reinterpret_cast<const uint2*>(s.weight + e0 + gap), q0, q1);
    if (turns) split<kNeighbours>(p0, p1, q0, q1);
  }
  // (first, second) -> (first A - second B, second C + first D) times the row's norm
  uint64_t A0 = p0, A1 = p1, B0 = 0, B1 = 0, C0 = q0, C1 = q1, D0 = 0, D1 = 0;
  if (turns) {
    const int32_t* pos = a.pos + b * a.pos_b + t;
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = pos[a.axis[4 * j + i] * a.pos_axis];
      const int32_t frac = static_cast<int32_t>((static_cast<uint64_t>(at) * turn_of(a.freq[4 * j + i])) >> 32);
      // radians in [-pi, pi): the fast functions are off by 2^-21 there
      __sincosf(static_cast<float>(frac) * 1.46291807926715968e-9f, &sn[i], &cs[i]);  // pi / 2^31
    }
    const uint64_t c0 = pair_of(cs[0], cs[1]), c1 = pair_of(cs[2], cs[3]), s0 = pair_of(sn[0], sn[1]), s1 = pair_of(sn[2], sn[3]);
    A0 = mul_pair(p0, c0), A1 = mul_pair(p1, c1);
    B0 = neg_pair(mul_pair(q0, s0)), B1 = neg_pair(mul_pair(q1, s1));
    C0 = mul_pair(q0, c0), C1 = mul_pair(q1, c1);
    D0 = mul_pair(p0, s0), D1 = mul_pair(p1, s1);
  }
  uint16_t* to = s.out + b * s.ob + t * s.ot + h0 * s.oh + e0;
  const int64_t oh = s.oh;
  // A row's two chunks times r to its output: where `mine` is set, and unless its squares
  // leave fp32 (returns that they do, once r is 1).
  auto put = [&](uint2 xk, uint2 yk, auto scaled, float r, uint16_t* at, bool mine) {
    bool far = false;
    uint64_t u0, u1, v0, v1;
    wide(xk, u0, u1);
    wide(yk, v0, v1);
    if (norm) {
      if constexpr (decltype(scaled)::value) {
        const uint64_t rr = pair_of(r, r);
        u0 = mul_pair(u0, rr), u1 = mul_pair(u1, rr), v0 = mul_pair(v0, rr), v1 = mul_pair(v1, rr);
      }
      float lo, hi;
      unpair(fma_pair(u0, u0, fma_pair(u1, u1, fma_pair(v0, v0, mul_pair(v1, v1)))), lo, hi);
      float sum = lo + hi;
#pragma unroll
      for (int o = 1; o < kRowLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float mean = fmaf(sum, 1.f / kD, decltype(scaled)::value ? a.eps * r * r : a.eps);
      if constexpr (!decltype(scaled)::value)  // not in [2^-100, infinity)
        far = mine && __float_as_uint(mean) - kLeastMean >= 0x7f800000u - kLeastMean;
      const float f = rsqrtf(mean);
      const uint64_t ff = pair_of(f, f);
      u0 = mul_pair(u0, ff), u1 = mul_pair(u1, ff), v0 = mul_pair(v0, ff), v1 = mul_pair(v1, ff);
    }
    if (turns) {
      split<kNeighbours>(u0, u1, v0, v1);
      const uint64_t w0 = fma_pair(u0, A0, mul_pair(v0, B0)), w1 = fma_pair(u1, A1, mul_pair(v1, B1));
      v0 = fma_pair(v0, C0, mul_pair(u0, D0)), v1 = fma_pair(v1, C1, mul_pair(u1, D1));
      u0 = w0, u1 = w1;
      join<kNeighbours>(u0, u1, v0, v1);
    } else if (norm) {
      u0 = mul_pair(u0, p0), u1 = mul_pair(u1, p1), v0 = mul_pair(v0, q0), v1 = mul_pair(v1, q1);
    }
    if (mine && !far) {
      *reinterpret_cast<uint2*>(at) = make_uint2(narrow(u0), narrow(u1));
      *reinterpret_cast<uint2*>(at + gap) = make_uint2(narrow(v0), narrow(v1));
    }
    return far;
  };
  uint32_t again = 0;
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (put(x[k], y[k], std::false_type(), 1.f, to, live && k < rows)) again |= 1u << k;
    to += oh;
  }
  const uint32_t any = __reduce_or_sync(0xffffffffu, again);
  if (__builtin_expect(any != 0, 0)) {  // those rows' inputs are as they were
    const uint16_t* const row0 = s.in + b * s.sb + t * s.st + h0 * s.sh + e0;
    to -= kHeads * oh;
#pragma unroll 1
    for (int k = 0; k < kHeads; ++k) {
      if (!(any >> k & 1)) continue;
      const bool mine = again >> k & 1;
      uint2 xk = make_uint2(0u, 0u), yk = xk;
      if (mine) xk = *reinterpret_cast<const uint2*>(row0 + k * s.sh), yk = *reinterpret_cast<const uint2*>(row0 + k * s.sh + gap);
      put(xk, yk, std::true_type(), to_one(xk, yk), to + k * oh, mine);
    }
  }
}

// Host: [B][H][n] rows at 16-byte boundaries whose span stays below 2^62 bytes.
bool rows_ok(const kvq_rows& r, int64_t B, int64_t H, int64_t n) {
  constexpr int64_t kMaxStride = int64_t{1} << 58;
  if (!r.data || reinterpret_cast<uintptr_t>(r.data) % 16) return false;
  if (r.stride_b < 0 || r.stride_h < 0 || r.stride_t < 0 || r.stride_b % 8 || r.stride_h % 8 || r.stride_t % 8) return false;
  return r.stride_b <= kMaxStride / B && r.stride_h <= kMaxStride / H && r.stride_t <= kMaxStride / n;
}
int64_t span_bytes(const kvq_rows& r, int64_t B, int64_t H, int64_t n) {
  return 2 * ((B - 1) * r.stride_b + (H - 1) * r.stride_h + (n - 1) * r.stride_t + kD);
}
// Host: every row has memory of its own: each dimension steps over all that
// the dimensions of smaller strides span.
bool rows_apart(const kvq_rows& r, int64_t B, int64_t H, int64_t n) {
  int64_t s[3] = {r.stride_b, r.stride_h, r.stride_t}, m[3] = {B, H, n}, span = kD;
  for (int i = 0; i < 3; ++i) {
    int k = i;  // the smallest stride left (dimensions of one entry have none to speak of)
    for (int q = i; q < 3; ++q)
      if ((m[q] > 1 ? s[q] : 0) < (m[k] > 1 ? s[k] : 0)) k = q;
    const int64_t ts = s[k], tm = m[k];
    s[k] = s[i], m[k] = m[i], s[i] = ts, m[i] = tm;
    if (tm == 1) continue;
    if (ts < span) return false;
    span += (tm - 1) * ts;
  }
  return true;
}

// Host: may rows of x (Hx heads) and of y (Hy) share an element?  Not when
// their spans lie apart, nor when they are parts of one buffer that repeats
// every M elements (the tokens of a fused projection, the sequences of a
// batch), each in its own part of the M.
bool rows_meet(const kvq_rows& x, int64_t Hx, const kvq_rows& y, int64_t Hy, int64_t B, int64_t n) {
  if (!ranges_meet(x.data, span_bytes(x, B, Hx, n), y.data, span_bytes(y, B, Hy, n))) return false;
  const int64_t sx[3] = {x.stride_b, x.stride_h, x.stride_t}, sy[3] = {y.stride_b, y.stride_h, y.stride_t};
  const int64_t mx[3] = {B, Hx, n}, my[3] = {B, Hy, n};
  const int64_t d = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(y.data)) -
                     static_cast<int64_t>(reinterpret_cast<uintptr_t>(x.data))) / 2;
  for (int64_t M : sx) {
    if (M <= 0) continue;
    int64_t wx = kD, wy = kD;
    bool repeats = true;
    for (int i = 0; i < 3; ++i) {
      if (mx[i] > 1) sx[i] >= M ? void(repeats = repeats && sx[i] % M == 0) : void(wx += (mx[i] - 1) * sx[i]);
      if (my[i] > 1) sy[i] >= M ? void(repeats = repeats && sy[i] % M == 0) : void(wy += (my[i] - 1) * sy[i]);
    }
    const int64_t at = (d % M + M) % M;
    if (repeats && wx <= at && at + wy <= M) return false;
  }
  return true;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_norm_rope(const kvq_layout* L, const kvq_rope_desc* R, const kvq_rows* q, const kvq_rows* k,
                                    int32_t n_tok, const int32_t* pos, int64_t pos_stride_axis, int64_t pos_stride_b,
                                    const float* inv_freq, const void* q_weight, const void* k_weight, float eps,
                                    const kvq_rows* q_out, const kvq_rows* k_out, void* stream) {
  kvq_status st = kvq_check_layout(L);
  if (st != KVQ_OK) return st;
  if (!R || !pos || !inv_freq || (!q && !k) || !q != !q_out || !k != !k_out) return KVQ_ERR_INVALID_ARG;
  if (R->rot_dim < 8 || R->rot_dim > kvq::kD || R->rot_dim % 8 || (R->interleaved != 0 && R->interleaved != 1) ||
      R->n_axes < 1 || R->n_axes > KVQ_MAX_ROPE_AXES)
    return KVQ_ERR_INVALID_ARG;
  for (int i = 0; i < R->rot_dim / 2; ++i)
    if (R->axis[i] >= R->n_axes) return KVQ_ERR_INVALID_ARG;
  if (n_tok < 0 || !std::isfinite(eps) || eps < 0.f) return KVQ_ERR_INVALID_ARG;
  if (n_tok == 0) return KVQ_OK;
  const int64_t B = L->d.B;
  if (pos_stride_axis < 0 || pos_stride_b < 0 || pos_stride_axis > (int64_t{1} << 58) / KVQ_MAX_ROPE_AXES ||
      pos_stride_b > (int64_t{1} << 58) / B)
    return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(pos) % 4 || reinterpret_cast<uintptr_t>(inv_freq) % 4 ||
      reinterpret_cast<uintptr_t>(q_weight) % 16 || reinterpret_cast<uintptr_t>(k_weight) % 16)
    return KVQ_ERR_INVALID_ARG;
  kvq::RopeArgs a = {};
  const kvq_rows* in[2] = {q, k};
  const kvq_rows* out[2] = {q_out, k_out};
  const int32_t H[2] = {q ? L->d.H_q : 0, k ? L->d.H_kv : 0};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    if (!kvq::rows_ok(*in[i], B, H[i], n_tok) || !kvq::rows_ok(*out[i], B, H[i], n_tok) ||
        !kvq::rows_apart(*out[i], B, H[i], n_tok))
      return KVQ_ERR_INVALID_ARG;
    const bool in_place = in[i]->data == out[i]->data && (B == 1 || in[i]->stride_b == out[i]->stride_b) &&
                          (H[i] == 1 || in[i]->stride_h == out[i]->stride_h) &&
                          (n_tok == 1 || in[i]->stride_t == out[i]->stride_t);
    if (!in_place && kvq::ranges_meet(in[i]->data, kvq::span_bytes(*in[i], B, H[i], n_tok), out[i]->data,
                                      kvq::span_bytes(*out[i], B, H[i], n_tok)))
      return KVQ_ERR_INVALID_ARG;
  }
  if (q && k && (kvq::rows_meet(*q_out, H[0], *k, H[1], B, n_tok) || kvq::rows_meet(*q, H[0], *k_out, H[1], B, n_tok) ||
                 kvq::rows_meet(*q_out, H[0], *k_out, H[1], B, n_tok)))
    return KVQ_ERR_INVALID_ARG;
  // what every row is made with must not lie under the outputs
  const int64_t n_pos = (R->n_axes - 1) * pos_stride_axis + (B - 1) * pos_stride_b + n_tok;
  for (int i = 0; i < 2; ++i) {
    if (!out[i]) continue;
    const int64_t span = kvq::span_bytes(*out[i], B, H[i], n_tok);
    if (kvq::ranges_meet(out[i]->data, span, pos, 4 * n_pos) || kvq::ranges_meet(out[i]->data, span, inv_freq, 2 * R->rot_dim) ||
        kvq::ranges_meet(out[i]->data, span, q_weight, kvq::kRowBytes) ||
        kvq::ranges_meet(out[i]->data, span, k_weight, kvq::kRowBytes))
      return KVQ_ERR_INVALID_ARG;
  }
  if (B * n_tok > 0x7ff00000LL) return KVQ_ERR_UNSUPPORTED;  // (past the last token by a stride of the grid)
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  a.pos = pos;
  a.pos_axis = pos_stride_axis;
  a.pos_b = pos_stride_b;
  a.freq = inv_freq;
  a.eps = eps;
  a.n = n_tok;
  a.tokens = static_cast<int32_t>(B * n_tok);
  a.rot = R->rot_dim;
  for (int i = 0; i < R->rot_dim / 2; ++i) a.axis[i] = R->axis[i];
  // Heads a lane group: one when there are few rows, for latency (one token of 32
  // heads 2.1 us, 2.8 with 8), else 8 to share the angles (16 x 26 tokens of 64
  // heads 5.0 us, 5.4 with 4, 8.6 with 1; 8 x 2940 of 80: 162, 184, 549).
  const int64_t rows = static_cast<int64_t>(a.tokens) * (H[0] + H[1]);
  const int64_t resident = static_cast<int64_t>(n_sm) * 1024 / kvq::kRowLanes;
  const int heads = rows <= resident ? 1 : (rows <= 2 * resident ? 4 : 8);
  const void* weights[2] = {q_weight, k_weight};
  for (int i = 0; i < 2; ++i) {
    kvq::RopeSide& s = a.side[i];
    if (!in[i]) continue;
    s = {static_cast<const uint16_t*>(in[i]->data), static_cast<uint16_t*>(out[i]->data),
         in[i]->stride_b, in[i]->stride_h, in[i]->stride_t, out[i]->stride_b, out[i]->stride_h, out[i]->stride_t,
         static_cast<const uint16_t*>(weights[i]), H[i], (H[i] + heads - 1) / heads};
  }
  const int groups = a.side[0].groups + a.side[1].groups;
  if (groups > 65535) return KVQ_ERR_UNSUPPORTED;
  const int64_t per = kvq::kRopeThreads / kvq::kRowLanes;
  const int64_t grid = (a.tokens + per - 1) / per;
  auto kernel = [&](auto pair) -> const void* {
    constexpr bool kPair = decltype(pair)::value;
    if (heads == 1) return reinterpret_cast<const void*>(&kvq::norm_rope_kernel<1, kPair>);
    if (heads == 4) return reinterpret_cast<const void*>(&kvq::norm_rope_kernel<4, kPair>);
    return reinterpret_cast<const void*>(&kvq::norm_rope_kernel<8, kPair>);
  };
  const void* fn = R->interleaved ? kernel(std::true_type()) : kernel(std::false_type());
  return kvq::launch_dependent(fn, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(groups)), kvq::kRopeThreads, 0, stream, &a);
}
