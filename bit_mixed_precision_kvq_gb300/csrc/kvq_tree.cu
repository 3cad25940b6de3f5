// kvq_tree.cu -- kvq_decode_attention_tree: attention of a tree of drafted
// tokens over the cache and the drafts themselves.
//
// For sequence b with context [0, len), token i and query head hq of KV head
// h = hq / g:
//   s_t = scale q . k_hat_t   for t < len,
//   s_j = scale q . k_draft_j for the drafts j with bit j of mask[b, i] set,
//   out = sum softmax(s) v,  lse = ln sum e^s   (no position: out 0, lse -inf).
#include "kvq_tree.cuh"

#include <algorithm>
#include <cmath>
#include <mutex>

namespace kvq {
namespace tree {
namespace {

// The outputs of units that are split over several CTAs: a CTA per output
// row, thread = d.  Partials are o (relative to the reference m), m and l;
// each is read once, coalesced (latency-bound: 448 rows of 17 to 25 partials
// in about 3 us, most of it hidden behind the last tree CTAs).
__global__ void __launch_bounds__(kD) combine_kernel(const __grid_constant__ Args a) {
  __shared__ float wgt[kMaxSplitCtas];
  __shared__ float red[4][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x;  // (b * n_q + i) * Hq + hq
  const int hq = static_cast<int>(row % a.c.Hq), h = hq / a.c.g;
  const int bi = static_cast<int>(row / a.c.Hq), b = bi / a.n_q, i = bi - b * a.n_q;
  const int cg = i * a.c.g + (hq - h * a.c.g), cb = cg / a.nb, c = cg - cb * a.nb;
  int S;
  const int cta = first_cta(a, b, h, cb, &S);
  pdl_wait();
  pdl_launch_dependents();
  if (S == 1) return;  // written by its CTA
  const int64_t pitch = static_cast<int64_t>(a.N) * (kD + 2);
  const float* slot = a.ws + cta * pitch;
  const float* ml = slot + a.N * kD + 2 * c;
  float M = -INFINITY;
  bool bad = false;
  for (int s = tid; s < S; s += kD) {
    const float m = __ldcg(ml + s * pitch);
    wgt[s] = m;
    bad |= m != m;
    M = fmaxf(M, m);
  }
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) red[warp][0] = bad ? __int_as_float(0x7fffffff) : M;
  __syncthreads();
  M = -INFINITY;
  bad = false;
  for (int k = 0; k < 4; ++k) {
    bad |= red[k][0] != red[k][0];
    M = fmaxf(M, red[k][0]);
  }
  float L = 0.f;
  for (int s = tid; s < S; s += kD) {
    const float m = wgt[s], f = m == -INFINITY || m != m ? 0.f : exp2f(m - M);
    wgt[s] = f;
    L = fmaf(f, __ldcg(ml + s * pitch + 1), L);
  }
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) red[warp][1] = L;
  __syncthreads();
  L = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
  const float* o = slot + c * kD + tid;
  float O = 0.f;
#pragma unroll 8
  for (int s = 0; s < S; ++s) O = fmaf(wgt[s], wgt[s] > 0.f ? __ldcg(o + s * pitch) : 0.f, O);
  const float nan = __int_as_float(0x7fffffff);
  a.out[row * kD + tid] = f32_to_bf16_bits(bad ? nan : (L > 0.f ? O / L : 0.f));
  if (tid == 0 && a.lse) a.lse[row] = bad ? nan : 0.69314718055994531f * (M + log2f(L));
}

// Columns of the widest unit, rounded to the MMA's granularity.
struct Columns {
  int nblk, nb, N;
};
Columns columns_of(const kvq_layout* L, int32_t n_q) {
  const int64_t cols = static_cast<int64_t>(L->g) * n_q;
  Columns c;
  c.nblk = static_cast<int>((cols + kMaxCols - 1) / kMaxCols);  // below 2^31: n_q and kMaxCols are at most 64
  c.nb = static_cast<int>((cols + c.nblk - 1) / c.nblk);
  c.N = (c.nb + 15) / 16 * 16;
  return c;
}

constexpr int64_t kWsHead = 256;
int64_t ws_bytes_of(const kvq_layout* L, int32_t n_q) {
  return kWsHead + static_cast<int64_t>(kMaxSplitCtas) * columns_of(L, n_q).N * (kD + 2) * 4;
}

const void* kernel_for(int kb, int vb, int G) {
  switch (kb) {
    case 2: return tree_kernel_k2(vb, G);
    case 4: return tree_kernel_k4(vb, G);
    case 8: return tree_kernel_k8(vb, G);
    case 16: return tree_kernel_k16(vb, G);
  }
  return nullptr;
}

}  // namespace
}  // namespace tree
}  // namespace kvq

// Once per kernel and device: `bytes` of dynamic shared memory, above the 48 KB
// that every kernel has.
kvq_status kvq_allow_smem(const void* fn, int bytes) {
  static std::mutex mu;
  static const void* done[64][64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return kvq_cuda_fail(e);
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64)
    for (const void* f : done[dev])
      if (f == fn) return KVQ_OK;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return kvq_cuda_fail(e);
  if (dev < 64)
    for (const void*& f : done[dev])
      if (!f) {
        f = fn;
        break;
      }
  return KVQ_OK;
}

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
  return static_cast<size_t>(kvq::tree::ws_bytes_of(L, n_q));
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
  if (T_ctx > kvq::kMaxLen) return KVQ_ERR_UNSUPPORTED;
  if (ws_bytes < static_cast<size_t>(kvq::tree::ws_bytes_of(L, n_q))) return KVQ_ERR_CAPACITY;
  const int64_t rows = static_cast<int64_t>(L->d.B) * n_q * L->d.H_q;
  const kvq::tree::Columns cols = kvq::tree::columns_of(L, n_q);
  const int64_t units = static_cast<int64_t>(L->d.B) * L->d.H_kv * cols.nblk;
  if (rows > 0x7fffffffLL || units > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  const void* fn = kvq::tree::kernel_for(L->d.k_bits, L->d.v_bits, L->d.group_size);
  if (!fn) return KVQ_ERR_UNSUPPORTED;
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  st = kvq_allow_smem(fn, sizeof(kvq::tree::Smem));
  if (st != KVQ_OK) return st;
  kvq::tree::Args a;
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
  a.status = static_cast<uint32_t*>(workspace);
  a.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kvq::tree::kWsHead);
  a.polls = kvq_tile_polls();
  a.nblk = cols.nblk;
  a.nb = cols.nb;
  a.N = cols.N;
  int h = 0;
  for (int k = 0; k < L->n_prot; ++k) a.head[h++] = L->prot_head[k];
  for (int k = 0; k < L->n_konly; ++k) a.head[h++] = L->konly_head[k];
  for (int k = 0; k < L->n_packed; ++k) a.head[h++] = L->packed_head[k];
  kvq::tree::plan_splits(L, cols.nblk, (T_ctx + n_q + kvq::tree::kTile - 1) / kvq::tree::kTile, n_sm, a.U, a.S, a.head0);
  const int grid = a.U[0] * a.S[0] + a.U[1] * a.S[1] + a.U[2] * a.S[2];
  st = kvq::launch_dependent(fn, dim3(grid), kvq::tree::kThreads, sizeof(kvq::tree::Smem), stream, &a);
  if (st != KVQ_OK || (a.S[0] == 1 && a.S[1] == 1 && a.S[2] == 1)) return st;
  return kvq::launch_dependent(reinterpret_cast<const void*>(&kvq::tree::combine_kernel), dim3(static_cast<unsigned>(rows)),
                               kvq::kD, 0, stream, &a);
}
