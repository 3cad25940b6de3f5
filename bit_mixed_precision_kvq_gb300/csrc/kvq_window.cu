// kvq_window.cu -- kvq_decode_attention_window: argument checks, the split and
// the launch (the kernel: kvq_window.cuh).
#include "kvq_window.cuh"

#include <algorithm>
#include <cmath>

extern "C" kvq_status kvq_decode_attention_window(const kvq_layout* L, const void* cache, const void* q_bf16, int32_t n_q,
                                                  const int32_t* seq_len, int32_t T, int32_t n_sink, int32_t window,
                                                  float softmax_scale, void* out_bf16, float* lse, void* stream) {
  kvq_status st = kvq_check_layout(L);
  if (st != KVQ_OK) return st;
  if (!cache || !q_bf16 || !out_bf16) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cache) % 256 || reinterpret_cast<uintptr_t>(q_bf16) % 16 ||
      reinterpret_cast<uintptr_t>(out_bf16) % 16 || reinterpret_cast<uintptr_t>(lse) % 4 ||
      reinterpret_cast<uintptr_t>(seq_len) % 4)
    return KVQ_ERR_INVALID_ARG;
  if (n_q < 1 || n_q > KVQ_MAX_QUERY_TOKENS || T < 1 || T > L->d.T_cap) return KVQ_ERR_INVALID_ARG;
  if (n_sink < 0 || window < 1 || !std::isfinite(softmax_scale)) return KVQ_ERR_INVALID_ARG;
  if (T > kvq::kMaxLen) return KVQ_ERR_UNSUPPORTED;
  const int64_t cols = static_cast<int64_t>(L->g) * n_q;
  const int nt = cols > 8 ? 2 : 1;
  const int64_t nblk = (cols + 8 * nt - 1) / (8 * nt);
  const int64_t units = static_cast<int64_t>(L->d.B) * L->d.H_kv * nblk;
  if (units > 0x7ffffff || cols > 0x7fffffff) return KVQ_ERR_UNSUPPORTED;  // 16 CTAs a unit at most
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  const kvq::win::Kernel k = L->d.k_bits == 2   ? kvq::win::window_kernel_k2(L->d.v_bits, L->d.group_size, nt)
                             : L->d.k_bits == 4 ? kvq::win::window_kernel_k4(L->d.v_bits, L->d.group_size, nt)
                             : L->d.k_bits == 8 ? kvq::win::window_kernel_k8(L->d.v_bits, L->d.group_size, nt)
                                                : kvq::win::window_kernel_k16(L->d.v_bits, L->d.group_size, nt);
  if (!k.fn) return KVQ_ERR_UNSUPPORTED;
  st = kvq_allow_clusters(k.fn, k.smem);
  if (st != KVQ_OK) return st;
  kvq::win::Args a;
  kvq::fill_geom(L, cache, &a.c);
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.seq_len = seq_len;
  a.T = T;
  a.n_q = n_q;
  a.n_sink = std::min(n_sink, T);
  a.window = std::min(window, T);
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.lse = lse;
  a.nblk = static_cast<int32_t>(nblk);
  int h = 0;
  for (int i = 0; i < L->n_prot; ++i) a.head[h++] = L->prot_head[i];
  for (int i = 0; i < L->n_konly; ++i) a.head[h++] = L->konly_head[i];
  for (int i = 0; i < L->n_packed; ++i) a.head[h++] = L->packed_head[i];
  // CTAs a unit: one wave of resident ones, none without a block for its warps.
  const int64_t rows = std::min<int64_t>(T, static_cast<int64_t>(a.n_sink) + a.window + n_q - 1);
  const int64_t wave = static_cast<int64_t>(n_sm) * (nt == 1 ? 2 : 1);
  int ranks = 1;
  while (ranks < kvq::win::kMaxRanks && 2 * ranks * units <= wave && ranks * kvq::win::kWarps * 16 < rows) ranks *= 2;
  return kvq::launch_clusters(k.fn, dim3(static_cast<unsigned>(units * ranks)), ranks, kvq::win::kThreads, k.smem, stream, &a);
}
