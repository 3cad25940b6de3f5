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
  const int64_t cols = static_cast<int64_t>(L->g) * n_q;
  kvq::win::Form f;
  f.nt = cols > 8 ? 2 : 1;
  const int64_t nblk = (cols + 8 * f.nt - 1) / (8 * f.nt);
  const int64_t units = static_cast<int64_t>(L->d.B) * L->d.H_kv * nblk;
  if (units > 0x3ffffff || cols > 0x7fffffff) return KVQ_ERR_UNSUPPORTED;  // 16 CTAs a unit at most
  // The outputs lie apart from one another and from the inputs; out may be q itself
  // (a unit's CTAs have read their rows of q before any of them writes).
  const int64_t rows = static_cast<int64_t>(L->d.B) * n_q * L->d.H_q, wide = rows * kvq::kRowBytes;
  const int64_t total = static_cast<int64_t>(L->total_bytes), lens = 4 * static_cast<int64_t>(L->d.B);
  if (kvq::ranges_meet(out_bf16, wide, cache, total) || kvq::ranges_meet(out_bf16, wide, seq_len, lens) ||
      kvq::ranges_meet(out_bf16, wide, lse, 4 * rows) || (out_bf16 != q_bf16 && kvq::ranges_meet(out_bf16, wide, q_bf16, wide)) ||
      kvq::ranges_meet(lse, 4 * rows, cache, total) || kvq::ranges_meet(lse, 4 * rows, seq_len, lens) ||
      kvq::ranges_meet(lse, 4 * rows, q_bf16, wide))
    return KVQ_ERR_INVALID_ARG;
  if (T > kvq::kMaxLen) return KVQ_ERR_UNSUPPORTED;
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  // Two tiles of columns unpack a row once (16 columns x 1280 units: 85 us, 104
  // as two units of one tile).  Units enough for every SM: CTAs of four warps, one a
  // unit, several an SM (512 units of 345 positions 15.3 us, 20.0 with eight warps);
  // else eight warps, for more of them a unit (64 units of 8,257 positions 21.6 us, 36
  // with four; four units of 2,078 6.2 and 7.3).
  f.warps = f.nt == 2 || units >= 2 * n_sm ? 4 : 8;
  const kvq::win::Kernel k = L->d.k_bits == 2   ? kvq::win::window_kernel_k2(L->d.v_bits, L->d.group_size, f)
                             : L->d.k_bits == 4 ? kvq::win::window_kernel_k4(L->d.v_bits, L->d.group_size, f)
                             : L->d.k_bits == 8 ? kvq::win::window_kernel_k8(L->d.v_bits, L->d.group_size, f)
                                                : kvq::win::window_kernel_k16(L->d.v_bits, L->d.group_size, f);
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
  const int n_heads[3] = {L->n_prot, L->n_konly, L->n_packed};
  const uint8_t* heads[3] = {L->prot_head, L->konly_head, L->packed_head};
  for (int k = 0; k < 3; ++k) {
    a.head0[k] = static_cast<uint8_t>(h);
    for (int i = 0; i < n_heads[k]; ++i) a.head[h++] = heads[k][i];
    a.U[k] = static_cast<int32_t>(static_cast<int64_t>(L->d.B) * n_heads[k] * nblk);
  }
  // CTAs a unit: those of the class with the longest share double while one
  // wave holds them all and no CTA is without a block for its warps.  A row costs
  // its bytes and some work (kPosCost); the longest call counts.  (Of four warps, three
  // an SM: what two column tiles leave room for.  One tile's CTAs would fit four
  // times, and GPCs that a cluster does not fill are not looked at.)
  const int64_t seen = std::min<int64_t>(T, static_cast<int64_t>(a.n_sink) + a.window + n_q - 1);
  const int64_t vis = std::min<int64_t>(seen, L->Tv), v = L->row_bytes[KVQ_SEG_V_CODES] + L->row_bytes[KVQ_SEG_V_SZ];
  const int64_t text = (seen - vis) * kvq::kBf16PosCost;
  const int64_t cost[3] = {text + vis * kvq::kBf16PosCost, text + vis * (kvq::kRowBytes + v + kvq::kPosCost),
                           text + vis * (L->row_bytes[KVQ_SEG_K_CODES] + L->row_bytes[KVQ_SEG_K_SZ] + v + kvq::kPosCost)};
  const int64_t wave = static_cast<int64_t>(n_sm) * (f.warps == 4 ? 3 : 2);
  int S[3] = {1, 1, 1};
  for (;;) {
    int worst = -1;
    for (int k = 0; k < 3; ++k)
      if (a.U[k] && (worst < 0 || cost[k] * S[worst] > cost[worst] * S[k])) worst = k;
    if (worst < 0 || S[worst] >= kvq::win::kMaxRanks || S[worst] * f.warps * 16 >= seen) break;
    int64_t used = 0;
    for (int k = 0; k < 3; ++k) used += static_cast<int64_t>(a.U[k]) * S[k] * (k == worst ? 2 : 1);
    if (used > wave) break;
    S[worst] *= 2;
  }
  a.cluster = std::max({S[0], S[1], S[2]});
  int64_t grid = 0;
  for (int k = 0; k < 3; ++k) {
    a.lg[k] = 0;
    while (1 << a.lg[k] < S[k]) ++a.lg[k];
    a.first[k] = static_cast<int32_t>(grid);
    grid += (static_cast<int64_t>(a.U[k]) * S[k] + a.cluster - 1) / a.cluster * a.cluster;
  }
  return kvq::launch_clusters(k.fn, dim3(static_cast<unsigned>(grid)), a.cluster, 32 * f.warps,
                              a.cluster > 1 ? k.smem : k.alone, stream, &a);
}
