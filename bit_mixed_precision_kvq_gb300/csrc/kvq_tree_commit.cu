// kvq_tree_commit.cu -- kvq_tree_commit: the accepted path of a tree of
// drafted tokens stored behind its sequence.
//
// Text position len + k of every KV head takes draft row path[b][k], K and V,
// for k < path_len[b].  The drafts lie outside the cache, so the rows can be
// copied in any order and the same draft may be stored twice.
#include "kvq_geom.cuh"

namespace kvq {
namespace {

struct CommitArgs {
  Geom c;
  const uint16_t *kd, *vd;
  int64_t sb, sh, st;  // strides of the drafts, in elements
  const int32_t *path, *path_len, *seq_len;
  int32_t T, n_q, max_path;
  int32_t* new_len;
};

// A CTA per (sequence, KV head): 16 lanes of 16 bytes per row, the K rows
// then the V rows.  The work is a few KB per CTA: the launch and one round
// of dependent loads (lengths and path, then rows) are all of its time: 1.7 us
// for 6 rows of 4 heads, 2.2 us for 16 sequences of up to 9 rows of 32 heads
// (2.4 MB, 0.36 us of it bytes).
constexpr int kThreads = 256;
__global__ void __launch_bounds__(kThreads) commit_kernel(const __grid_constant__ CommitArgs a) {
  const Geom& p = a.c;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  __shared__ int32_t path[KVQ_MAX_QUERY_TOKENS];
  pdl_wait();
  const int len = a.seq_len ? a.seq_len[b] : a.T, n = a.path_len[b];
  bool ok = len >= 0 && len <= a.T && n >= 0 && n <= a.max_path && len <= p.T_cap - n;
  if (ok && n > 0 && p.vs < p.ve && len < p.ve && len + n > p.vs) ok = false;  // every new position is text
  bool in_range = true;
  if (ok && threadIdx.x < static_cast<unsigned>(n)) {
    const int j = a.path[static_cast<int64_t>(b) * a.max_path + threadIdx.x];
    path[threadIdx.x] = j;
    in_range = j >= 0 && j < a.n_q;
  }
  ok = __syncthreads_and(ok && in_range);
  if (a.new_len && h == 0 && threadIdx.x == 0) a.new_len[b] = ok ? len + n : -1;
  if (!ok) return;
  const HeadRows r = head_rows(p, b, h);
  const int64_t tr = len < p.ve ? len : len - p.Tv;  // text row of position len (len <= vs or len >= ve)
  const int64_t src = b * a.sb + h * a.sh;
  for (int x = threadIdx.x; x < 2 * 16 * n; x += kThreads) {
    const int lane = x & 15, row = x >> 4, k = row < n ? row : row - n;
    const uint16_t* s = (row < n ? a.kd : a.vd) + src + path[k] * a.st + 8 * lane;
    uint8_t* d = (row < n ? r.text_k : r.text_v) + (tr + k) * kRowBytes + 16 * lane;
    *reinterpret_cast<uint4*>(d) = __ldcg(reinterpret_cast<const uint4*>(s));
  }
  // No early launch of the next kernel: the rows are visible to it when this
  // grid has finished (a decode call may copy cache rows before its own wait).
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_tree_commit(const kvq_layout* L, void* cache, const void* k_draft_bf16,
                                      const void* v_draft_bf16, int64_t stride_b, int64_t stride_h, int64_t stride_t,
                                      int32_t n_q, const int32_t* path, int32_t max_path, const int32_t* path_len,
                                      const int32_t* seq_len, int32_t T_ctx, int32_t* new_len, void* stream) {
  kvq_status st = kvq_check_layout(L);
  if (st != KVQ_OK) return st;
  st = kvq_check_drafts(L, cache, k_draft_bf16, v_draft_bf16, stride_b, stride_h, stride_t, n_q);
  if (st != KVQ_OK) return st;
  if (!path || !path_len || reinterpret_cast<uintptr_t>(path) % 4 || reinterpret_cast<uintptr_t>(path_len) % 4 ||
      reinterpret_cast<uintptr_t>(seq_len) % 4 || reinterpret_cast<uintptr_t>(new_len) % 4)
    return KVQ_ERR_INVALID_ARG;
  if (max_path < 1 || max_path > KVQ_MAX_QUERY_TOKENS) return KVQ_ERR_INVALID_ARG;
  if (T_ctx < 0 || T_ctx > L->d.T_cap) return KVQ_ERR_INVALID_ARG;
  // the CTAs of a sequence read its lengths and path while one writes new_len
  const int64_t nb = 4 * static_cast<int64_t>(L->d.B);
  if (kvq::ranges_meet(new_len, nb, seq_len, nb) || kvq::ranges_meet(new_len, nb, path_len, nb) ||
      kvq::ranges_meet(new_len, nb, path, nb * max_path))
    return KVQ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(L->d.B) * L->d.H_kv > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  kvq::CommitArgs a;
  kvq::fill_geom(L, cache, &a.c);
  a.kd = static_cast<const uint16_t*>(k_draft_bf16);
  a.vd = static_cast<const uint16_t*>(v_draft_bf16);
  a.sb = stride_b;
  a.sh = stride_h;
  a.st = stride_t;
  a.path = path;
  a.path_len = path_len;
  a.seq_len = seq_len;
  a.T = T_ctx;
  a.n_q = n_q;
  a.max_path = max_path;
  a.new_len = new_len;
  return kvq::launch_dependent(reinterpret_cast<const void*>(&kvq::commit_kernel), dim3(L->d.B * L->d.H_kv), kvq::kThreads,
                               0, stream, &a);
}
