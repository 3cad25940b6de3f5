// kvq_tree.cu -- kvq_decode_attention_tree: attention of a tree of drafted
// tokens over the cache and the drafts themselves.
//
// For sequence b with context [0, len), token i and query head hq of KV head
// h = hq / g:
//   s_t = scale q . k_hat_t   for t < len,
//   s_j = scale q . k_draft_j for the drafts j with bit j of mask[b, i] set,
//   out = sum softmax(s) v,  lse = ln sum e^s   (no position: out 0, lse -inf).
#include "kvq_simple.cuh"

#include <cmath>

namespace kvq {
namespace {

struct TreeArgs {
  Geom c;
  const uint16_t *q, *kd, *vd;
  int64_t sb, sh, st;  // strides of the drafts, in elements
  const uint64_t* mask;
  int64_t mask_sb;
  const int32_t* seq_len;
  int32_t T, n_q;
  float scale_log2;
  uint16_t* out;
  float* lse;
};

// The simple form: a CTA per output row, a warp per position at a time.
constexpr int kWarps = 4;
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float sm_o[kWarps][kD], sm_ml[kWarps][2];
  const Geom& p = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;  // (b * n_q + i) * Hq + hq
  const int hq = static_cast<int>(row % p.Hq), h = hq / p.g;
  const int bi = static_cast<int>(row / p.Hq), b = bi / a.n_q, i = bi - b * a.n_q;
  pdl_wait();
  const int len = a.seq_len ? a.seq_len[b] : a.T;
  const bool live = len >= 0 && len <= a.T;
  const HeadRows r = head_rows(p, b, h);
  const uint64_t mask = a.mask[b * a.mask_sb + i];
  const float4 q = row4(reinterpret_cast<const uint8_t*>(a.q + row * kD), nullptr, 16, p.G, true, 4 * lane);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t = warp; live && t < len + a.n_q; t += kWarps) {
    const int j = t - len;
    if (j >= 0 && !((mask >> j) & 1)) continue;
    const int64_t dr = b * a.sb + h * a.sh + j * a.st;
    const float4 k = j < 0 ? k_row4(p, r, t, 4 * lane)
                           : row4(reinterpret_cast<const uint8_t*>(a.kd + dr), nullptr, 16, p.G, true, 4 * lane);
    const float4 v = j < 0 ? v_row4(p, r, t, 4 * lane)
                           : row4(reinterpret_cast<const uint8_t*>(a.vd + dr), nullptr, 16, p.G, false, 4 * lane);
    const float s = a.scale_log2 * warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w);
    const float mn = fmaxf(m, s), c = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * c + w;
    o = make_float4(o.x * c + w * v.x, o.y * c + w * v.y, o.z * c + w * v.z, o.w * c + w * v.w);
  }
  *reinterpret_cast<float4*>(&sm_o[warp][4 * lane]) = o;
  if (lane == 0) {
    sm_ml[warp][0] = m;
    sm_ml[warp][1] = l;
  }
  __syncthreads();
  const int d = threadIdx.x;
  float M = -INFINITY, L = 0.f, O = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_ml[w][0]);
  for (int w = 0; w < kWarps; ++w) {
    const float f = sm_ml[w][0] == -INFINITY ? 0.f : exp2f(sm_ml[w][0] - M);
    L += f * sm_ml[w][1];
    O += f * sm_o[w][d];
  }
  a.out[row * kD + d] = f32_to_bf16_bits(L > 0.f ? O / L : 0.f);
  if (d == 0 && a.lse) a.lse[row] = 0.69314718055994531f * (M + log2f(L));
}

}  // namespace
}  // namespace kvq

// Checks of the drafted rows shared by the tree's entry points: pointers,
// strides, and that they do not lie in the cache buffer.
kvq_status kvq_check_drafts(const kvq_layout* L, const void* cache, const void* k, const void* v, int64_t sb, int64_t sh,
                            int64_t st, int32_t n_q) {
  if (!cache || !k || !v) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cache) % 256 || reinterpret_cast<uintptr_t>(k) % 16 || reinterpret_cast<uintptr_t>(v) % 16)
    return KVQ_ERR_INVALID_ARG;
  if (n_q < 1 || n_q > KVQ_MAX_QUERY_TOKENS) return KVQ_ERR_INVALID_ARG;
  // a bound that no tensor in memory reaches, so that the span below cannot overflow
  constexpr int64_t kMaxStride = int64_t{1} << 42;
  if (sb < 0 || sh < 0 || st < 0 || sb % 8 || sh % 8 || st % 8) return KVQ_ERR_INVALID_ARG;
  if (sb > kMaxStride / L->d.B || sh > kMaxStride / L->d.H_kv || st > kMaxStride / n_q) return KVQ_ERR_INVALID_ARG;
  const int64_t span = 2 * ((L->d.B - 1) * sb + (L->d.H_kv - 1) * sh + (n_q - 1) * st + kvq::kD);
  if (kvq::ranges_meet(cache, L->total_bytes, k, span) || kvq::ranges_meet(cache, L->total_bytes, v, span))
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

extern "C" size_t kvq_decode_tree_workspace_bytes(const kvq_layout* L, int32_t n_q) {
  if (kvq_check_layout(L) != KVQ_OK || n_q < 1 || n_q > KVQ_MAX_QUERY_TOKENS) return 0;
  return 256;
}

extern "C" kvq_status kvq_decode_attention_tree(const kvq_layout* L, const void* cache, const void* q_bf16,
                                                const void* k_draft_bf16, const void* v_draft_bf16, int64_t stride_b,
                                                int64_t stride_h, int64_t stride_t, int32_t n_q,
                                                const uint64_t* tree_mask, int64_t mask_stride_b,
                                                const int32_t* seq_len, int32_t T_ctx, float softmax_scale,
                                                void* out_bf16, float* lse, void* workspace, size_t ws_bytes,
                                                void* stream) {
  kvq_status st = kvq_check_layout(L);
  if (st != KVQ_OK) return st;
  st = kvq_check_drafts(L, cache, k_draft_bf16, v_draft_bf16, stride_b, stride_h, stride_t, n_q);
  if (st != KVQ_OK) return st;
  if (!q_bf16 || !out_bf16 || !tree_mask || !workspace) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(q_bf16) % 16 || reinterpret_cast<uintptr_t>(out_bf16) % 16 ||
      reinterpret_cast<uintptr_t>(workspace) % 256 || reinterpret_cast<uintptr_t>(tree_mask) % 8 ||
      reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(seq_len) % 4)
    return KVQ_ERR_INVALID_ARG;
  if (mask_stride_b != 0 && mask_stride_b < n_q) return KVQ_ERR_INVALID_ARG;
  if (T_ctx < 0 || T_ctx > L->d.T_cap || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (ws_bytes < kvq_decode_tree_workspace_bytes(L, n_q)) return KVQ_ERR_CAPACITY;
  const int64_t rows = static_cast<int64_t>(L->d.B) * n_q * L->d.H_q;
  if (rows > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  kvq::TreeArgs a;
  kvq::fill_geom(L, cache, &a.c);
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.kd = static_cast<const uint16_t*>(k_draft_bf16);
  a.vd = static_cast<const uint16_t*>(v_draft_bf16);
  a.sb = stride_b;
  a.sh = stride_h;
  a.st = stride_t;
  a.mask = tree_mask;
  a.mask_sb = mask_stride_b;
  a.seq_len = seq_len;
  a.T = T_ctx;
  a.n_q = n_q;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.lse = lse;
  return kvq::launch_dependent(reinterpret_cast<const void*>(&kvq::tree_kernel), dim3(static_cast<unsigned>(rows)),
                               kvq::kWarps * 32, 0, stream, &a);
}
