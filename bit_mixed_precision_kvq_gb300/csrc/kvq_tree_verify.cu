// kvq_tree_verify.cu -- kvq_tree_verify: the path of a tree of drafted tokens
// that the target accepts, and the token behind it.
//
// One thread-block cluster a sequence walks the tree.  At the path's last token
// x the cluster's CTAs share out the row of logits l: one pass gives
//   m = max l,  S = sum 2^((l - m) log2(e) / T),  p(v) = 2^((l_v - m) log2(e) / T) / S
// and the lowest v of the maximum.  Then each child is held against p as kvq.h
// says; a refusal with draft probabilities is one more pass, over
//   r_k = max(r_{k-1} / Z_{k-1} - q, 0),  Z_k = sum r_k   (r_0 = p, Z_0 = 1),
// and the end one more: argmax r(v) / race(v).  Rows are read again from L1 and
// L2 in later passes; only the rows on the walk are read at all, and all CTAs of
// a cluster compute the same decisions from the same sums, so a step costs one
// exchange through distributed shared memory.  Sums run in a fixed order.
//
// Bound by the chain of dependent rows: a few microseconds each (a round trip
// to memory, a reduction, a cluster barrier), whatever the batch until its rows
// fill the memory system.
#include "kvq_geom.cuh"

#include <climits>
#include <mutex>

namespace kvq {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxRanks = 16;  // CTAs of a cluster
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

struct VerifyArgs {
  int32_t n_q, V;
  const void* logits;
  int64_t lsb, lst;
  const int32_t* tokens;
  const uint64_t* mask;
  int64_t mask_sb;
  const float* draft;
  int64_t dsb, dst;
  const float *accept, *race, *temp;
  const int32_t* tree_len;
  int32_t *path, *path_len, *next;
  float* logprob;
};

// What CTAs exchange: a row's maximum (or the best race key), a sum, an index.
struct Part {
  float m, s;
  int32_t at;
};

struct VerifySmem {
  Part slot[2][kMaxRanks];  // by exchange parity and rank
  Part warp[kVerifyWarps];
  uint64_t kids[KVQ_MAX_QUERY_TOKENS];  // children of each token
  int32_t token[KVQ_MAX_QUERY_TOKENS];
  float u[KVQ_MAX_QUERY_TOKENS];
  float kid_l[KVQ_MAX_QUERY_TOKENS], kid_q[KVQ_MAX_QUERY_TOKENS];  // logit and draft probability of x's children
  float inv_z[KVQ_MAX_QUERY_TOKENS];  // 1 / Z_k at the path's last token
  int32_t out[KVQ_MAX_QUERY_TOKENS];  // token ids refused there
  int32_t path[KVQ_MAX_QUERY_TOKENS];
  float logp[KVQ_MAX_QUERY_TOKENS];
};

__device__ __forceinline__ void st_cluster_part(uint32_t addr, const Part& p) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(p.m) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr + 4), "f"(p.s) : "memory");
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr + 8), "r"(p.at) : "memory");
}

// Softmax statistics of a and b together: 2^0 = 1 for the one whose maximum
// stays.  at: the lowest index of the maximum.
__device__ __forceinline__ Part join_rows(const Part& a, const Part& b, float sc) {
  Part r;
  r.m = fmaxf(a.m, b.m);
  const float base = r.m == -INFINITY ? 0.f : r.m;
  r.s = a.s * exp2f((a.m - base) * sc) + b.s * exp2f((b.m - base) * sc);
  r.at = a.m > b.m ? a.at : (b.m > a.m ? b.at : min(a.at, b.at));
  return r;
}
__device__ __forceinline__ Part join_sums(const Part& a, const Part& b, float) { return {0.f, a.s + b.s, 0}; }
__device__ __forceinline__ Part join_best(const Part& a, const Part& b, float) {
  return {fmaxf(a.m, b.m), 0.f, a.m > b.m ? a.at : (b.m > a.m ? b.at : min(a.at, b.at))};
}

// Every thread's part joined over the CTA and the cluster, the same to all.
template <typename Join>
__device__ __forceinline__ Part join_all(VerifySmem& sm, Part p, float sc, int rank, int ranks, uint32_t& turn, Join&& join) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Part q = {__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                    __shfl_xor_sync(0xffffffffu, p.at, o)};
    p = lane & o ? join(q, p, sc) : join(p, q, sc);  // one order for both lanes
  }
  if (lane == 0) sm.warp[warp] = p;
  __syncthreads();
  if (warp == 0) {
    p = sm.warp[lane % kVerifyWarps];
#pragma unroll
    for (int o = kVerifyWarps / 2; o > 0; o >>= 1) {
      const Part q = {__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                      __shfl_xor_sync(0xffffffffu, p.at, o)};
      p = lane & o ? join(q, p, sc) : join(p, q, sc);
    }
    if (lane < ranks) st_cluster_part(dsmem_addr(&sm.slot[turn & 1][rank], lane), p);
  }
  // Slots alternate: a rank writes these again after the next exchange, which
  // it passes only when every rank has come to it, i.e. has read them here.
  cluster_sync();
  p = sm.slot[turn & 1][0];
  for (int r = 1; r < ranks; ++r) p = join(p, sm.slot[turn & 1][r], sc);
  ++turn;
  return p;
}

// The CTA's share of a row of V elements of type X: f(v0, values, count) for
// groups of up to kGroup = 16 bytes of consecutive ones, aligned groups first
// loaded kAhead at a time.
template <typename X>
struct Row {
  static constexpr int kGroup = 16 / sizeof(X), kAhead = 4;
  static __device__ __forceinline__ void values(uint4 w, float (&x)[kGroup]) {
    if constexpr (sizeof(X) == 2) {
      x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
      x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
    } else {
      x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
  }
  static __device__ __forceinline__ float value(const X* p) {
    if constexpr (sizeof(X) == 2) return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
    else return *p;
  }
  template <typename F>
  static __device__ __forceinline__ void each(const X* row, int V, int rank, int ranks, F&& f) {
    const int head = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / sizeof(X)));
    const int n = (V - head) / kGroup, lo = static_cast<int>(static_cast<int64_t>(n) * rank / ranks),
              hi = static_cast<int>(static_cast<int64_t>(n) * (rank + 1) / ranks);
    const uint4* at = reinterpret_cast<const uint4*>(row + head);
    float x[kGroup];
    for (int i = lo + threadIdx.x; i < hi; i += kAhead * kVerifyThreads) {
      uint4 w[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i + k * kVerifyThreads < hi) w[k] = at[i + k * kVerifyThreads];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i + k * kVerifyThreads < hi) {
          values(w[k], x);
          f(head + (i + k * kVerifyThreads) * kGroup, x, kGroup);
        }
    }
    if (rank == 0) {  // what lies before the first 16-byte boundary and behind the last
      const int tail = head + n * kGroup, v = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
      if (v < V) {
        x[0] = value(row + v);
        f(v, x, 1);
      }
    }
  }
};

// count values of a row of fp32 from index v on.
template <int N>
__device__ __forceinline__ void fetch(const float* row, int v, int count, float (&x)[N]) {
  if (count == N && reinterpret_cast<uintptr_t>(row + v) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 w = reinterpret_cast<const float4*>(row + v)[i];
      x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < count ? row[v + i] : 0.f;
  }
}

template <typename X, bool kDraft>
__global__ void __launch_bounds__(kVerifyThreads, 1) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ VerifySmem sm;
  constexpr int kGroup = Row<X>::kGroup;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = static_cast<int>(cluster_nctarank());
  const int b = blockIdx.x / ranks, tid = threadIdx.x;
  pdl_wait();
  if (tid == 0) pdl_launch_dependents();
  const int n = a.tree_len ? a.tree_len[b] : a.n_q;
  const float temp = a.temp ? a.temp[b] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float sc = greedy ? kLog2e : kLog2e / temp;
  bool good = n >= 1 && n <= a.n_q;
  if (tid < KVQ_MAX_QUERY_TOKENS) sm.kids[tid] = 0ull;
  __syncthreads();
  if (good && tid < n) {
    sm.token[tid] = a.tokens[static_cast<int64_t>(b) * a.n_q + tid];
    sm.u[tid] = a.accept[static_cast<int64_t>(b) * a.n_q + tid];
    const uint64_t above = a.mask[b * a.mask_sb + tid] & ((1ull << tid) - 1ull);
    if (above) atomicOr(reinterpret_cast<unsigned long long*>(&sm.kids[63 - __clzll(above)]), 1ull << tid);
  }
  cluster_sync();  // every CTA runs (its shared memory may be written); sm is set up

  uint32_t turn = 0;
  int cur = 0, count = 1, next = -1;
  while (good) {
    const X* row = static_cast<const X*>(a.logits) + b * a.lsb + cur * a.lst;
    const float* drow = kDraft ? a.draft + b * a.dsb + cur * a.dst : nullptr;
    uint64_t kids = sm.kids[cur];
    if (tid < 64 && (kids >> tid & 1ull)) {
      const int c = sm.token[tid];
      const bool is = c >= 0 && c < a.V;
      sm.kid_l[tid] = is ? Row<X>::value(row + c) : -INFINITY;
      if (kDraft) sm.kid_q[tid] = is ? drow[c] : 0.f;
    }
    Part p = {-INFINITY, 0.f, INT_MAX};
    Row<X>::each(row, a.V, rank, ranks, [&](int v, const float (&x)[kGroup], int c) {
      float top = x[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < kGroup; ++i)
        if (i < c && x[i] > top) top = x[i], at = i;
      if (top > p.m) {
        p.s *= exp2f((p.m - top) * sc);
        p.m = top;
        p.at = v + at;
      } else if (top == p.m) {
        p.at = min(p.at, v + at);
      }
      const float base = p.m == -INFINITY ? 0.f : p.m;
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        if (i < c) p.s += exp2f((x[i] - base) * sc);
    });
    p = join_all(sm, p, sc, rank, ranks, turn, join_rows);
    const float m = p.m, inv_s = 1.f / p.s, log_s = logf(p.s);
    const int best = p.at;
    good = p.s > 0.f && p.s < INFINITY && m > -INFINITY && m < INFINITY;
    if (!good) break;
    auto prob = [&](float l) { return exp2f((l - m) * sc) * inv_s; };
    auto log_prob = [&](float l) { return (l - m) * (sc * kLn2) - log_s; };

    // the children, in index order: the same decisions in every thread
    int took = -1, refused = 0;  // refused: entries of inv_z or out
    float total = 1.f;
    while (kids) {
      const int j = __ffsll(kids) - 1;
      kids &= kids - 1ull;
      const int c = sm.token[j];
      bool ok;
      float r = prob(sm.kid_l[j]);  // 0 for an id outside the vocabulary
      if (greedy) {
        ok = c == best;
      } else if constexpr (kDraft) {
        const float q = sm.kid_q[j];
        for (int k = 0; k < refused; ++k) r = fmaxf(r * sm.inv_z[k] - q, 0.f);
        ok = sm.u[j] * total * q < r;
      } else {
        for (int k = 0; k < refused; ++k)
          if (sm.out[k] == c) r = 0.f;
        ok = sm.u[j] * total < r;
      }
      if (ok) {
        took = j;
        break;
      }
      if (greedy) continue;
      if constexpr (kDraft) {
        // r_k = max(r_{k-1} / Z_{k-1} - q, 0) with the sum of the last one
        const float inv = 1.f / total;
        __syncthreads();  // all have read the earlier entries' state of this loop
        if (tid == 0) sm.inv_z[refused] = inv;
        __syncthreads();
        Part z = {0.f, 0.f, 0};
        Row<X>::each(row, a.V, rank, ranks, [&](int v, const float (&x)[kGroup], int cnt) {
          float q[kGroup];
          fetch(drow, v, cnt, q);
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            if (i < cnt) {
              float y = prob(x[i]);
              for (int k = 0; k <= refused; ++k) y = fmaxf(y * sm.inv_z[k] - q[i], 0.f);
              z.s += y;
            }
        });
        z = join_all(sm, z, 0.f, rank, ranks, turn, join_sums);
        if (z.s > 0.f) {  // else nothing is left and r stays
          total = z.s;
          ++refused;
        }
      } else {
        if (c >= 0 && c < a.V && r > 0.f) {
          __syncthreads();
          if (tid == 0) sm.out[refused] = c;
          __syncthreads();
          total = fmaxf(total - r, 0.f);
          ++refused;
        }
      }
    }
    if (tid == 0) sm.path[count - 1] = cur;
    if (took >= 0) {
      if (tid == 0) sm.logp[count - 1] = log_prob(sm.kid_l[took]);
      cur = took;
      ++count;
      __syncthreads();  // kid_l is written anew
      continue;
    }
    // the token behind the path
    next = best;
    if (!greedy) {
      const float* race = a.race + static_cast<int64_t>(b) * a.V;
      Part w = {0.f, 0.f, INT_MAX};
      Row<X>::each(row, a.V, rank, ranks, [&](int v, const float (&x)[kGroup], int cnt) {
        float e[kGroup], q[kGroup];
        fetch(race, v, cnt, e);
        if (kDraft && refused) fetch(drow, v, cnt, q);
        bool cut = false;
        if constexpr (!kDraft)
          for (int k = 0; k < refused; ++k) cut |= sm.out[k] >= v && sm.out[k] < v + cnt;
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
          if (i < cnt) {
            float y = prob(x[i]);
            if constexpr (kDraft) {
              for (int k = 0; k < refused; ++k) y = fmaxf(y * sm.inv_z[k] - q[i], 0.f);
            } else if (cut) {
              for (int k = 0; k < refused; ++k)
                if (sm.out[k] == v + i) y = 0.f;
            }
            const float key = e[i] > 0.f ? __fdividef(y, e[i]) : 0.f;
            if (key > w.m || (key == w.m && key > 0.f && v + i < w.at)) w.m = key, w.at = v + i;
          }
      });
      w = join_all(sm, w, 0.f, rank, ranks, turn, join_best);
      if (w.m > 0.f) next = w.at;
    }
    if (tid == 0) sm.logp[count - 1] = log_prob(Row<X>::value(row + next));
    break;
  }
  if (rank != 0) return;  // the last exchange is behind every rank
  __syncthreads();
  if (tid == 0) {
    a.path_len[b] = good ? count : -1;
    a.next[b] = good ? next : -1;
  }
  if (tid < a.n_q) {
    const int64_t i = static_cast<int64_t>(b) * a.n_q + tid;
    a.path[i] = good && tid < count ? sm.path[tid] : -1;
    if (a.logprob) a.logprob[i] = good && tid < count ? sm.logp[tid] : 0.f;
  }
}

}  // namespace
}  // namespace kvq

// Once per kernel and device: clusters of up to 16 CTAs, and `bytes` of dynamic
// shared memory.
kvq_status kvq_allow_clusters(const void* fn, int bytes) {
  static std::mutex mu;
  static const void* done[64][128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return kvq_cuda_fail(e);
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64)
    for (const void* f : done[dev])
      if (f == fn) return KVQ_OK;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && bytes > 0) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return kvq_cuda_fail(e);
  if (dev < 64)
    for (const void*& f : done[dev])
      if (!f) {
        f = fn;
        break;
      }
  return KVQ_OK;
}

extern "C" kvq_status kvq_tree_verify(int32_t B, int32_t n_q, int32_t vocab, const void* logits, int32_t logits_fp32,
                                      int64_t logits_stride_b, int64_t logits_stride_t, const int32_t* tokens,
                                      const uint64_t* tree_mask, int64_t mask_stride_b, const float* draft_prob,
                                      int64_t draft_stride_b, int64_t draft_stride_t, const float* accept,
                                      const float* race, const float* temperature, const int32_t* tree_len,
                                      int32_t* path, int32_t* path_len, int32_t* next_token, float* logprob,
                                      void* stream) {
  if (B < 1 || n_q < 1 || n_q > KVQ_MAX_QUERY_TOKENS || vocab < 1 || vocab > (1 << 30)) return KVQ_ERR_INVALID_ARG;
  if (logits_fp32 != 0 && logits_fp32 != 1) return KVQ_ERR_INVALID_ARG;
  if (!logits || !tokens || !tree_mask || !accept || !race || !path || !path_len || !next_token) return KVQ_ERR_INVALID_ARG;
  const int elt = logits_fp32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % elt || reinterpret_cast<uintptr_t>(tree_mask) % 8) return KVQ_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(tokens), static_cast<const void*>(draft_prob), static_cast<const void*>(accept),
                        static_cast<const void*>(race), static_cast<const void*>(temperature), static_cast<const void*>(tree_len),
                        static_cast<const void*>(path), static_cast<const void*>(path_len), static_cast<const void*>(next_token),
                        static_cast<const void*>(logprob)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return KVQ_ERR_INVALID_ARG;
  if (mask_stride_b != 0 && mask_stride_b < n_q) return KVQ_ERR_INVALID_ARG;
  // a bound that no tensor in memory reaches, so that the spans below cannot overflow
  constexpr int64_t kMaxStride = int64_t{1} << 56;
  auto stride_ok = [&](int64_t s, int64_t m) { return s >= 0 && s <= kMaxStride / m; };
  if (!stride_ok(logits_stride_b, B) || !stride_ok(logits_stride_t, n_q) || !stride_ok(mask_stride_b, B))
    return KVQ_ERR_INVALID_ARG;
  if (draft_prob && (!stride_ok(draft_stride_b, B) || !stride_ok(draft_stride_t, n_q))) return KVQ_ERR_INVALID_ARG;
  if (B > 65535) return KVQ_ERR_UNSUPPORTED;
  const int64_t nb = 4 * static_cast<int64_t>(B), nt = nb * n_q;
  const struct {
    const void* p;
    int64_t bytes;
  } outs[4] = {{path, nt}, {path_len, nb}, {next_token, nb}, {logprob, nt}},
    ins[8] = {{logits, elt * ((B - 1) * logits_stride_b + (n_q - 1) * logits_stride_t + vocab)},
              {tokens, nt},
              {tree_mask, 8 * ((B - 1) * mask_stride_b + n_q)},
              {draft_prob, draft_prob ? 4 * ((B - 1) * draft_stride_b + (n_q - 1) * draft_stride_t + vocab) : 0},
              {accept, nt},
              {race, nb * vocab},
              {temperature, nb},
              {tree_len, nb}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (kvq::ranges_meet(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return KVQ_ERR_INVALID_ARG;
    for (const auto& x : ins)
      if (kvq::ranges_meet(outs[i].p, outs[i].bytes, x.p, x.bytes)) return KVQ_ERR_INVALID_ARG;
  }
  int n_sm = 0;
  if (kvq_device_sm_count(&n_sm) != 0) return KVQ_ERR_CUDA;
  const void* fn = logits_fp32 ? (draft_prob ? reinterpret_cast<const void*>(&kvq::verify_kernel<float, true>)
                                             : reinterpret_cast<const void*>(&kvq::verify_kernel<float, false>))
                               : (draft_prob ? reinterpret_cast<const void*>(&kvq::verify_kernel<uint16_t, true>)
                                             : reinterpret_cast<const void*>(&kvq::verify_kernel<uint16_t, false>));
  const kvq_status st = kvq_allow_clusters(fn, 0);
  if (st != KVQ_OK) return st;
  // As many CTAs a sequence as one wave holds, but none below 16 bytes a thread.
  int ranks = 1;
  while (ranks < kvq::kMaxRanks && 2 * ranks * static_cast<int64_t>(B) <= n_sm &&
         2 * ranks * 16 * kvq::kVerifyThreads <= static_cast<int64_t>(vocab) * elt)
    ranks *= 2;
  kvq::VerifyArgs a;
  a.n_q = n_q;
  a.V = vocab;
  a.logits = logits;
  a.lsb = logits_stride_b;
  a.lst = logits_stride_t;
  a.tokens = tokens;
  a.mask = tree_mask;
  a.mask_sb = mask_stride_b;
  a.draft = draft_prob;
  a.dsb = draft_stride_b;
  a.dst = draft_stride_t;
  a.accept = accept;
  a.race = race;
  a.temp = temperature;
  a.tree_len = tree_len;
  a.path = path;
  a.path_len = path_len;
  a.next = next_token;
  a.logprob = logprob;
  return kvq::launch_clusters(fn, dim3(static_cast<unsigned>(B * ranks)), ranks, kvq::kVerifyThreads, 0, stream, &a);
}
