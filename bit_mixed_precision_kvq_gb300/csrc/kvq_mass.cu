// kvq_mass.cu -- kvq_attention_mass: the attention weight that each cache
// position has received, accumulated per KV head.
//
//   mass[b, h, t] = decay mass_in[b, h, t]
//                 + sum_k sum_{hq of h} e^(scale q_k,hq . k_hat_t - lse_k,hq)
// over the tokens k = 0 .. n - 1 taken from sequence b, token k reaching the
// positions t < len - n + 1 + k.
#include "kvq_simple.cuh"

#include <cmath>

namespace kvq {
namespace {

struct MassArgs {
  Geom c;
  const uint16_t* q;   // [B][n_q][Hq][D]
  const float* lse;    // [B][n_q][Hq]
  const int32_t *seq_len, *path, *path_len;
  int32_t T, n_q, max_path;
  float scale_log2, decay;
  const float* mass_in;  // [B][Hkv][T_cap] or null
  float* mass;
};

// The simple form: a warp per (sequence, KV head, position).
constexpr int kWarps = 8;
__global__ void __launch_bounds__(kWarps * 32) mass_kernel(const __grid_constant__ MassArgs a) {
  const Geom& p = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (a.T + kWarps - 1) / kWarps;
  const int64_t bh = blockIdx.x / chunks;
  const int t = static_cast<int>(blockIdx.x - bh * chunks) * kWarps + warp;
  const int b = static_cast<int>(bh / p.Hkv), h = static_cast<int>(bh - static_cast<int64_t>(b) * p.Hkv);
  pdl_wait();
  const int len = a.seq_len ? a.seq_len[b] : a.T;
  const int n = a.path ? a.path_len[b] : a.n_q;
  if (len < 1 || len > a.T || n < 0 || n > (a.path ? a.max_path : a.n_q) || n > len || t >= len) return;
  const float4 k = k_row4(p, head_rows(p, b, h), t, 4 * lane);
  float sum = 0.f;
  for (int i = max(0, t - len + n); i < n; ++i) {
    const int tok = a.path ? a.path[static_cast<int64_t>(b) * a.max_path + i] : i;
    if (tok < 0 || tok >= a.n_q) continue;
    for (int hq = h * p.g; hq < (h + 1) * p.g; ++hq) {
      const int64_t row = (static_cast<int64_t>(b) * a.n_q + tok) * p.Hq + hq;
      const float4 q = row4(reinterpret_cast<const uint8_t*>(a.q + row * kD), nullptr, 16, p.G, true, 4 * lane);
      const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w);
      const float lse = a.lse[row];
      if (lse != -INFINITY) sum += exp2f(fmaf(a.scale_log2, s, -1.4426950408889634f * lse));
    }
  }
  const int64_t at = bh * p.T_cap + t;
  if (lane == 0) a.mass[at] = (a.mass_in ? a.decay * a.mass_in[at] : 0.f) + sum;
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
  const int64_t blocks = static_cast<int64_t>(L->d.B) * L->d.H_kv * ((T + kvq::kWarps - 1) / kvq::kWarps);
  if (blocks > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
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
  return kvq::launch_dependent(reinterpret_cast<const void*>(&kvq::mass_kernel), dim3(static_cast<unsigned>(blocks)),
                               kvq::kWarps * 32, 0, stream, &a);
}
