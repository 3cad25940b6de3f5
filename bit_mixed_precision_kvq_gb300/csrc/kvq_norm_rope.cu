// kvq_norm_rope.cu -- kvq_norm_rope: the rows of query and key heads normed
// and rotated by positions of several axes, in one pass.
//
//   y = x / sqrt(mean_d x_d^2 + eps) * w        (y = x without a weight)
//   pair i of the first rot_dim elements turns by the angle
//   a_i = pos[axis_i] * inv_freq_i:
//     (y_p, y_q) -> (y_p cos a_i - y_q sin a_i, y_q cos a_i + y_p sin a_i)
//
// Every row is read once and written once (512 bytes), with some 60 fp32
// operations a lane in between: bound by memory once there are enough rows.
// 16 lanes hold a row of 128, each the elements of 4 pairs (8 beyond the
// rotated part), so that a pair never crosses lanes and the mean takes 4
// shuffles.  A lane's angles depend on the token alone: 16 lanes take `heads`
// heads of one token, with the loads of kFlight rows issued before any is used.
//
// Angles.  A position may be large (a product with a frequency near 1 loses
// all its digits in fp32 from 2^24 on), so the turn is taken modulo 1 in
// integers: inv_freq / 2 pi modulo 1 as a 64-bit binary fraction, times the
// position modulo 2^64.  Its top 32 bits, rounded to fp32, are the angle to
// 2^-25 of a turn.  The rest is fp32, rounded once to bf16.
#include "kvq_geom.cuh"

#include <algorithm>
#include <cmath>

namespace kvq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRowLanes = 16;

struct RopeSide {
  const uint16_t* in;  // element (b, h, t, d) at b sb + h sh + t st + d
  uint16_t* out;
  int64_t sb, sh, st, ob, oh, ot;
  const uint16_t* weight;  // bf16 [D] or null: no norm
  int32_t H, groups;       // heads, and groups of `heads` of them
};

struct RopeArgs {
  RopeSide side[2];  // q, k
  const int32_t* pos;  // [n_axes][B][n]
  int64_t pos_axis, pos_b;
  const float* freq;  // [rot / 2]
  float eps;
  int32_t n, rot, heads;
  bool interleaved;
  int64_t tokens;  // B n
  uint8_t axis[kD / 2];
};

__device__ __forceinline__ void bf16x4(uint2 w, float (&x)[4]) {
  x[0] = bf16_lo(w.x);
  x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y);
  x[3] = bf16_hi(w.y);
}
__device__ __forceinline__ uint2 bf16x4_of(const float (&x)[4]) {
  return make_uint2(f32_to_bf16_bits(x[0]) | (static_cast<uint32_t>(f32_to_bf16_bits(x[1])) << 16),
                    f32_to_bf16_bits(x[2]) | (static_cast<uint32_t>(f32_to_bf16_bits(x[3])) << 16));
}

template <int kFlight>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  const int j = threadIdx.x & (kRowLanes - 1);
  const int half = a.rot / 2;
  const bool turns = 8 * j < a.rot;
  // first elements of the lane's two chunks of 4
  const bool apart = turns && !a.interleaved;
  const int e0 = apart ? 4 * j : 8 * j, e1 = apart ? half + 4 * j : 8 * j + 4;
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  uint64_t turn[4] = {};  // inv_freq / 2 pi of pairs 4j .. 4j + 3, modulo 1
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      double f = static_cast<double>(a.freq[4 * j + i]) * 0.15915494309189533577;
      f -= floor(f);
      turn[i] = f < 1.0 ? static_cast<uint64_t>(f * 18446744073709551616.0) : 0ull;
    }
  }
  const int groups = a.side[0].groups + a.side[1].groups;
  const int64_t items = a.tokens * groups;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kRopeThreads / kRowLanes);
  const int upper = threadIdx.x / kRowLanes % 2;  // which half of the warp
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / kRowLanes) + threadIdx.x / kRowLanes;
       it - upper < items; it += step) {
    const bool live = it < items;  // the lower half may have rows when the upper has none
    const int64_t token = (live ? it : 0) / groups;
    int grp = static_cast<int>((live ? it : 0) - token * groups);
    const int b = static_cast<int>(token / a.n), t = static_cast<int>(token - static_cast<int64_t>(b) * a.n);
    const bool key = grp >= a.side[0].groups;
    if (key) grp -= a.side[0].groups;
    const RopeSide& s = a.side[key];
    const int h0 = grp * a.heads, h1 = live ? min(h0 + a.heads, s.H) : h0;
    const uint16_t* in = s.in + b * s.sb + t * s.st;
    uint16_t* out = s.out + b * s.ob + t * s.ot;
    uint2 x0[kFlight], x1[kFlight];
    auto load = [&](int h) {
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        x0[k] = x1[k] = make_uint2(0u, 0u);
        if (h + k < h1) {
          x0[k] = *reinterpret_cast<const uint2*>(in + (h + k) * s.sh + e0);
          x1[k] = *reinterpret_cast<const uint2*>(in + (h + k) * s.sh + e1);
        }
      }
    };
    load(h0);
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {};
    if (turns) {
      const int32_t* pos = a.pos + b * a.pos_b + t;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t p = pos[a.axis[4 * j + i] * a.pos_axis];
        const int32_t frac = static_cast<int32_t>((static_cast<uint64_t>(p) * turn[i]) >> 32);
        sincospif(static_cast<float>(frac) * 4.656612873077392578125e-10f, &sn[i], &cs[i]);  // 2^-31: half turns
      }
    }
    float w0[4] = {1.f, 1.f, 1.f, 1.f}, w1[4] = {1.f, 1.f, 1.f, 1.f};
    if (s.weight) {
      bf16x4(*reinterpret_cast<const uint2*>(s.weight + e0), w0);
      bf16x4(*reinterpret_cast<const uint2*>(s.weight + e1), w1);
    }
    const int rounds = (a.heads + kFlight - 1) / kFlight;  // the same for both halves of a warp
    for (int r = 0; r < rounds; ++r) {
      const int h = h0 + r * kFlight;
      if (r > 0) load(h);
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        float u[4], v[4];
        bf16x4(x0[k], u);
        bf16x4(x1[k], v);
        if (a.side[0].weight || a.side[1].weight) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) sum = fmaf(u[i], u[i], fmaf(v[i], v[i], sum));
#pragma unroll
          for (int o = 1; o < kRowLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float f = s.weight ? rsqrtf(fmaf(sum, 1.f / kD, a.eps)) : 1.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] *= f * w0[i];
            v[i] *= f * w1[i];
          }
        }
        if (turns) {
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p = u[2 * i], q = u[2 * i + 1];
              u[2 * i] = p * cs[i] - q * sn[i];
              u[2 * i + 1] = q * cs[i] + p * sn[i];
              const float y = v[2 * i], z = v[2 * i + 1];
              v[2 * i] = y * cs[2 + i] - z * sn[2 + i];
              v[2 * i + 1] = z * cs[2 + i] + y * sn[2 + i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = u[i], q = v[i];
              u[i] = p * cs[i] - q * sn[i];
              v[i] = q * cs[i] + p * sn[i];
            }
          }
        }
        if (h + k < h1) {
          *reinterpret_cast<uint2*>(out + (h + k) * s.oh + e0) = bf16x4_of(u);
          *reinterpret_cast<uint2*>(out + (h + k) * s.oh + e1) = bf16x4_of(v);
        }
      }
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
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  a.pos = pos;
  a.pos_axis = pos_stride_axis;
  a.pos_b = pos_stride_b;
  a.freq = inv_freq;
  a.eps = eps;
  a.n = n_tok;
  a.rot = R->rot_dim;
  a.interleaved = R->interleaved != 0;
  a.tokens = B * n_tok;
  for (int i = 0; i < R->rot_dim / 2; ++i) a.axis[i] = R->axis[i];
  // Few rows: one a lane group, for latency; else as many as share the angles well.
  const int64_t rows = a.tokens * (H[0] + H[1]);
  const int64_t resident = static_cast<int64_t>(n_sm) * 1024 / kvq::kRowLanes;
  a.heads = rows <= resident ? 1 : (rows <= 4 * resident ? 4 : 8);
  const void* weights[2] = {q_weight, k_weight};
  for (int i = 0; i < 2; ++i) {
    kvq::RopeSide& s = a.side[i];
    if (!in[i]) continue;
    s = {static_cast<const uint16_t*>(in[i]->data), static_cast<uint16_t*>(out[i]->data),
         in[i]->stride_b, in[i]->stride_h, in[i]->stride_t, out[i]->stride_b, out[i]->stride_h, out[i]->stride_t,
         static_cast<const uint16_t*>(weights[i]), H[i], (H[i] + a.heads - 1) / a.heads};
  }
  const int64_t items = a.tokens * (a.side[0].groups + a.side[1].groups);
  const int64_t per = kvq::kRopeThreads / kvq::kRowLanes;
  const int64_t grid = std::min<int64_t>((items + per - 1) / per, static_cast<int64_t>(n_sm) * 32);
  const void* fn = a.heads == 1 ? reinterpret_cast<const void*>(&kvq::norm_rope_kernel<1>)
                                : reinterpret_cast<const void*>(&kvq::norm_rope_kernel<4>);
  return kvq::launch_dependent(fn, dim3(static_cast<unsigned>(grid)), kvq::kRopeThreads, 0, stream, &a);
}
