// kvq_tree_verify.cu -- kvq_tree_verify: the path of a tree of drafted tokens
// that the target accepts, and the token behind it.
//
// One thread-block cluster a sequence walks the tree.  At the path's last token
// x the cluster's CTAs share out the row of logits l: one pass gives
//   m = max l,  s = sum 2^((l - m) log2(e) / T),  p(v) = 2^((l_v - m) log2(e) / T) / (1 + s)
// and the lowest v of the maximum, which s leaves out: ln p of a token that is
// all but certain keeps its digits as log1p(s).  Then each child is held against
// p as kvq.h says; a refusal with draft probabilities is one more pass, over
//   r_k = max(r_{k-1} / Z_{k-1} - q, 0),  Z_k = sum r_k   (r_0 = p, Z_0 = 1),
// and the end one more: argmax log2 r(v) - log2 race(v).  Only the rows on the
// walk are read, and all CTAs of a cluster compute the same decisions from the
// same sums, so a step costs one exchange through distributed shared memory.
// Sums run in a fixed order.  Everything is fp32 (bf16 logits are exact in it).
//
// Bound by the chain of dependent passes, whatever the batch until its rows fill
// the memory system: of a row of 32,000 in 8 CTAs the pass takes 1,800 cycles, the
// exchange and the decision 2,700; of 128,000 in 4 CTAs (a batch of 32) 5,000
// and 2,500, at about 100 instructions for 8 logits and half of the issue slots.
// Measured (GB300): 5 drafts, vocabulary 32,000, 1.8 rows on average 7.9 us; 16
// sampled drafts, 152,000, 4.2 rows 18 us; 32 sequences of 64 sampled drafts,
// 128,000, 4.2 rows on average and 8 or more on the longest walk 58.5 us (the rows
// that are read take 10 at the rate of a copy).  Rolled loops: unrolled over a
// thread's groups the code of a pass that runs once a call comes from L2 (130 us
// became 68).  1,024 threads a CTA, two groups a turn, draft rows asked for ahead
// of a refusal, two CTAs an SM with shorter rings (56 us, but 20 in place of 15 for
// 16 sequences) and every warp's part sent to all ranks (57 and 17) were not kept.
#include "kvq_geom.cuh"

#include <climits>
#include <mutex>

namespace kvq {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxRanks = 16;  // CTAs of a cluster
constexpr uint32_t kLeavePolls = 4096;  // of a wait for parts that have been sent (microseconds away), whatever the limit of the others
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
  uint32_t polls;  // limit of a wait for the cluster's other CTAs
};

// What CTAs exchange: a row's maximum (or the best race key), a sum, an index.
struct alignas(16) Part {
  float m, s;
  int32_t at;
};

struct VerifySmem {
  Part slot[2][kMaxRanks];  // by exchange parity and rank
  uint64_t bar[2];          // the ranks' parts have come (transaction bytes)
  int late;                 // a wait gave up
  int any_late;             // so did one in some CTA of the cluster (which stores it here)
  int sent[kMaxRanks];      // how many exchanges each rank sent its part of (stored by the rank)
  Part warp[kVerifyWarps], joined;
  uint64_t kids[KVQ_MAX_QUERY_TOKENS];  // children of each token
  int32_t token[KVQ_MAX_QUERY_TOKENS];
  float u[KVQ_MAX_QUERY_TOKENS];
  float kid_l[KVQ_MAX_QUERY_TOKENS], kid_q[KVQ_MAX_QUERY_TOKENS];  // logit and draft probability of x's children
  float inv_z[KVQ_MAX_QUERY_TOKENS];  // 1 / Z_k at the path's last token
  int32_t out[KVQ_MAX_QUERY_TOKENS];  // token ids refused there
  int32_t path[KVQ_MAX_QUERY_TOKENS];
  float logp[KVQ_MAX_QUERY_TOKENS];
};

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The parts of a warp's lanes joined, in every lane.
// Softmax statistics: s counts all but the maximum at `at` (the lowest index of
// it); the maxima of the lanes but one that has it are added.
struct JoinRows {
  float sc;
  static __device__ __forceinline__ Part none() { return {-INFINITY, 0.f, INT_MAX}; }
  __device__ __forceinline__ Part operator()(const Part& p) const {
    const float m = warp_max(p.m);
    const int lead = __ffs(__ballot_sync(0xffffffffu, p.m == m)) - 1;  // its maximum stays out
    const float others = static_cast<int>(threadIdx.x & 31) == lead ? 0.f : 1.f;
    return {m, warp_sum((p.s + others) * ex2((p.m - (m == -INFINITY ? 0.f : m)) * sc)),
            __reduce_min_sync(0xffffffffu, p.m == m ? p.at : INT_MAX)};
  }
};
struct JoinSums {
  static __device__ __forceinline__ Part none() { return {0.f, 0.f, 0}; }
  __device__ __forceinline__ Part operator()(const Part& p) const { return {0.f, warp_sum(p.s), 0}; }
};
struct JoinBest {
  static __device__ __forceinline__ Part none() { return {-INFINITY, 0.f, INT_MAX}; }
  __device__ __forceinline__ Part operator()(const Part& p) const {
    const float m = warp_max(p.m);
    return {m, 0.f, __reduce_min_sync(0xffffffffu, p.m == m ? p.at : INT_MAX)};
  }
};

// Every thread's part joined over the CTA and the cluster, the same to all.
// Exchange t: warp 0 of each rank stores its CTA's part into slot t mod 2 of every
// rank, asynchronous stores counted on that rank's barrier (a cluster barrier
// around plain stores took 1,400 to 1,800 cycles, these about half).  Slots and
// barriers alternate: a rank sends t + 2 only with every rank's t + 1 in hand,
// which those send behind arming the barrier for t + 2.  A wait that gives up sets
// sm.late, the same for the whole CTA: the walk ends there, the other ranks'
// waits give up in their turn, and `leave` sees to the parts still on their way.
struct Exchange {
  int rank, ranks;
  uint32_t polls, turn;
};
template <typename Join>
__device__ __forceinline__ Part join_all(VerifySmem& sm, Part p, Exchange& x, const Join& join) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, s = x.turn & 1;
  p = join(p);
  if (lane == 0) sm.warp[warp] = p;
  __syncthreads();
  if (x.turn == 0) cluster_wait();  // every CTA of the cluster has started and armed its barriers
  if (warp == 0) {
    p = join(lane < kVerifyWarps ? sm.warp[lane] : Join::none());
    if (lane < x.ranks)
      st_async_v4(dsmem_addr(&sm.slot[s][x.rank], lane), make_float4(p.m, p.s, __int_as_float(p.at), 0.f), dsmem_addr(&sm.bar[s], lane));
    const uint32_t parity = (x.turn >> 1) & 1;
    const bool here = x.polls == 1 ? mbar_test_cluster(&sm.bar[s], parity) : mbar_wait_cluster(&sm.bar[s], parity, x.polls);
    const bool late = __any_sync(0xffffffffu, !here);
    if (lane == 0 && !late) mbar_arrive_expect_tx(&sm.bar[s], 16 * x.ranks);
    p = join(lane < x.ranks && !late ? sm.slot[s][lane] : Join::none());
    if (lane == 0) {
      sm.joined = p;
      if (late) sm.late = 1;
    }
  }
  __syncthreads();
  ++x.turn;
  return sm.joined;
}

// The last meeting of the cluster's CTAs: no CTA ends while another's part is on
// its way to it.  A CTA that leaves with all its exchanges done has every part
// that was sent to it (no rank sends for an exchange that another has not
// reached).  One that gave up in exchange t = turn - 1 has not: parts of t and, from
// ranks that saw t complete, of t + 1 may still come, and no barrier between CTAs
// waits for them.  So the ranks tell one another how many exchanges they sent, and
// it waits on the barriers of t and t + 1 (both armed) for the bytes that were sent,
// taking the others off.  Called by every thread with the CTA's turn, behind a
// __syncthreads that made sm.late known; `between` is work before the meeting ends.
template <typename F>
__device__ __forceinline__ void leave(VerifySmem& sm, const Exchange& x, F&& between) {
  const int tid = threadIdx.x;
  if (sm.late) {
    if (tid < x.ranks) st_dsmem(dsmem_addr(&sm.any_late, tid), 1);
    __syncwarp();
    cluster_arrive();  // release: the stores come before it
  } else {
    cluster_arrive_relaxed();
  }
  between();
  cluster_wait();
  if (!*reinterpret_cast<volatile int*>(&sm.any_late)) return;  // the same in every CTA
  if (tid < x.ranks) st_dsmem(dsmem_addr(&sm.sent[x.rank], tid), static_cast<int>(x.turn));
  __syncwarp();
  cluster_sync();
  if (!sm.late || tid != 0) return;
  const volatile int* sent = sm.sent;
  for (uint32_t t = x.turn - 1; t <= x.turn; ++t) {
    uint32_t missing = 0;
    for (int r = 0; r < x.ranks; ++r) missing += sent[r] <= static_cast<int>(t);
    if (missing) mbar_complete_tx(&sm.bar[t & 1], 16 * missing);
    mbar_wait_cluster(&sm.bar[t & 1], (t >> 1) & 1, kLeavePolls);
  }
}

// Asks for the CTA's share of a row of V elements of type X, or the first
// megabyte of it, in L2 (one thread).
template <typename X>
__device__ __forceinline__ void prefetch_share(const X* row, int V, int rank, int ranks) {
  const int log = 31 - __clz(ranks);
  const X* lo = row + (static_cast<int64_t>(V) * rank >> log);
  const X* hi = row + (static_cast<int64_t>(V) * (rank + 1) >> log);
  const uintptr_t a = (reinterpret_cast<uintptr_t>(lo) + 15) & ~uintptr_t{15}, b = reinterpret_cast<uintptr_t>(hi) & ~uintptr_t{15};
  if (a < b) prefetch_l2(reinterpret_cast<const void*>(a), static_cast<uint32_t>(min(b - a, uintptr_t{1} << 20)));
}

// A thread's groups on their way through shared memory (cp.async): kAhead of them
// under way, of a row of logits (16 bytes a group) and of up to two rows of fp32.
constexpr int kAhead = 3, kRing = kAhead + 1;
template <int kBytes>  // of a group's fp32 values: 16 or 32
struct Ring {
  uint4 x[kRing][kVerifyThreads];
  uint4 e[kRing][kBytes / 16][kVerifyThreads];
  uint4 q[kRing][kBytes / 16][kVerifyThreads];  // (with draft probabilities)
};

__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
  if (bytes == 16) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A CTA's share of a row of V elements of type X: groups of kGroup = 16 bytes,
// and in rank 0, one by one, the elements before the row's first 16-byte
// boundary and behind its last.
template <typename X>
struct Share {
  static constexpr int kGroup = 16 / sizeof(X);
  using R = Ring<4 * kGroup>;
  const X* row;
  int V, from, n;       // the thread's groups: n of them, kVerifyThreads apart, the first at index `from`
  int before, behind;   // its single elements (-1: none)

  __device__ __forceinline__ Share(const X* r, int V_, int rank, int ranks) : row(r), V(V_) {
    const int tid = threadIdx.x, log = 31 - __clz(ranks);  // a power of two
    const int head = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / sizeof(X)));
    const int all = (V - head) / kGroup;
    const int lo = static_cast<int>(static_cast<int64_t>(all) * rank >> log), hi = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) >> log);
    from = head + (lo + tid) * kGroup;
    n = max(0, hi - lo - tid + kVerifyThreads - 1) / kVerifyThreads;
    before = rank == 0 && tid < head ? tid : -1;
    behind = rank == 0 && head + all * kGroup + tid < V ? head + all * kGroup + tid : -1;
  }
  __device__ __forceinline__ static float value(const X* p) {
    if constexpr (sizeof(X) == 2) return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
    else return *p;
  }
  __device__ __forceinline__ static void values(const uint4& w, float (&x)[kGroup]) {
    if constexpr (sizeof(X) == 2) {
      x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
      x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
    } else {
      x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
  }
  // one element, with -inf behind it
  __device__ __forceinline__ static uint4 single(const X* p) {
    constexpr uint32_t kNone = sizeof(X) == 2 ? 0xff80ff80u : 0xff800000u;
    uint4 w = make_uint4(kNone, kNone, kNone, kNone);
    if constexpr (sizeof(X) == 2) w.x = 0xff800000u | *reinterpret_cast<const uint16_t*>(p);
    else w.x = *reinterpret_cast<const uint32_t*>(p);
    return w;
  }
  // Asks for the thread's first groups of the row, and of a row of fp32.
  __device__ __forceinline__ void begin(R& ring) const {
#pragma unroll 1
    for (int i = 0; i < min(n, kAhead); ++i) copy_async(&ring.x[i][threadIdx.x], row + from + i * kVerifyThreads * kGroup, 16);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void begin_e(R& ring, const float* e_row) const {
#pragma unroll 1
    for (int i = 0; i < min(n, kAhead); ++i) bring(&ring.e[i][0][threadIdx.x], e_row + from + i * kVerifyThreads * kGroup);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // a group's fp32 values, in pieces kVerifyThreads apart
  __device__ __forceinline__ static void bring(uint4* to, const float* src) {
    if (reinterpret_cast<uintptr_t>(src) % 16 == 0) {
#pragma unroll
      for (int k = 0; k < kGroup / 4; ++k) copy_async(to + k * kVerifyThreads, src + 4 * k, 16);
    } else {
#pragma unroll 1
      for (int k = 0; k < kGroup; ++k) copy_async(reinterpret_cast<float*>(to + k / 4 * kVerifyThreads) + k % 4, src + k, 4);
    }
  }
  // f(v, logits, e, q) for every group of the thread in increasing order of v;
  // e and q: rows of V fp32, or null (zeros come).  x_here, e_here: begin (or a
  // pass over at most kAhead groups) has brought the row's first groups,
  // begin_e e's.
  template <bool kE, bool kQ, typename F>
  __device__ __forceinline__ void each(R& ring, bool x_here, const float* e_row, bool e_here, const float* q_row, F&& f) const {
    constexpr int kStep = kVerifyThreads * kGroup;
    const int tid = threadIdx.x;
    auto issue = [&](int i, bool with_x, bool with_e) {
      if (i < n) {
        const int s = i % kRing, v = from + i * kStep;
        if (with_x) copy_async(&ring.x[s][tid], row + v, 16);
        if (kE && with_e) bring(&ring.e[s][0][tid], e_row + v);
        if (kQ && q_row) bring(&ring.q[s][0][tid], q_row + v);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) issue(i, !x_here, !e_here);
    const int last = n + (behind >= 0 ? 1 : 0);
#pragma unroll 1
    for (int i = before >= 0 ? -1 : 0; i < last; ++i) {
      uint4 w;
      float e[kGroup] = {}, q[kGroup] = {};
      int v;
      if (i >= 0 && i < n) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const int s = i % kRing;
        v = from + i * kStep;
        w = ring.x[s][tid];
#pragma unroll
        for (int k = 0; k < kGroup / 4; ++k) {
          if (kE) reinterpret_cast<float4*>(e)[k] = reinterpret_cast<const float4&>(ring.e[s][k][tid]);
          if (kQ && q_row) reinterpret_cast<float4*>(q)[k] = reinterpret_cast<const float4&>(ring.q[s][k][tid]);
        }
        issue(i + kAhead, true, true);  // into the slot that the group before this one had
      } else {
        v = i < 0 ? before : behind;
        w = single(row + v);
        if (kE) e[0] = e_row[v];
        if (kQ && q_row) q[0] = q_row[v];
      }
      f(v, w, e, q);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
};

__device__ __forceinline__ float fast_log2(float x) {  // 2^-22 of itself; -inf for 0
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Softmax statistics of the thread's elements (begin has been called).  The sum
// of the group that holds the maximum is kept apart and taken anew without it at
// the end.
template <typename X>
__device__ __forceinline__ Part row_part(const Share<X>& row, typename Share<X>::R& ring, float sc) {
  constexpr int kGroup = Share<X>::kGroup;
  float m = -INFINITY, rest = 0.f, own = 0.f;
  int at = INT_MAX;  // first index of the group with the maximum
  uint4 best = {};   // and the group
  auto sum_of = [&](const float (&x)[kGroup], float base) {
    const uint64_t neg = pair_of(-base, -base), scale = pair_of(sc, sc);
    uint64_t sum = 0ull;
#pragma unroll
    for (int i = 0; i < kGroup; i += 2) {
      float u, v;
      unpair(mul_pair(add_pair(pair_of(x[i], x[i + 1]), neg), scale), u, v);
      sum = add_pair(sum, pair_of(ex2(u), ex2(v)));
    }
    float u, v;
    unpair(sum, u, v);
    return u + v;
  };
  row.template each<false, false>(ring, true, nullptr, false, nullptr, [&](int v, const uint4& w, const float (&)[kGroup], const float (&)[kGroup]) {
    float x[kGroup];
    Share<X>::values(w, x);
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kGroup; ++i) top = fmaxf(top, x[i]);
    const bool more = top > m;
    const float f = more ? ex2((m - top) * sc) : 1.f;
    m = more ? top : m;
    const float s = sum_of(x, m == -INFINITY ? 0.f : m);
    rest = more ? (rest + own) * f : rest + s;
    own = more ? s : own;
    at = more ? v : at;
    best.x = more ? w.x : best.x;
    best.y = more ? w.y : best.y;
    best.z = more ? w.z : best.z;
    best.w = more ? w.w : best.w;
  });
  if (m == -INFINITY) return {m, rest + own, INT_MAX};  // (NaN stays)
  float x[kGroup];
  Share<X>::values(best, x);
  int first = 0;
#pragma unroll
  for (int i = kGroup - 1; i >= 0; --i)
    if (x[i] == m) first = i;
#pragma unroll
  for (int i = 0; i < kGroup; ++i)
    if (i == first) x[i] = -INFINITY;
  return {m, rest + sum_of(x, m), at + first};
}

// -inf for the first `refused` token ids of sm.out in the group from v on.
template <int kGroup>
__device__ __forceinline__ void drop_refused(const VerifySmem& sm, int refused, int v, float (&y)[kGroup]) {
  for (int g = 0; g < refused; ++g) {
    const int d = sm.out[g] - v;
    if (d >= 0 && d < kGroup) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) y[i] = i == d ? -INFINITY : y[i];
    }
  }
}

// Sum of 2^((l - m) sc) over what of the row is not refused: a pass and an exchange
// (the caller counts it).  For the rare case that refused siblings held nearly all of a
// sum, which is known to 2^-20 of itself: subtracting them would leave its errors.
template <typename X>
__device__ __noinline__ float rest_sum(VerifySmem& sm, typename Share<X>::R& ring, const X* row_at, int V, int refused, float m, float sc,
                                       Exchange x) {
  constexpr int kGroup = Share<X>::kGroup;
  const Share<X> row(row_at, V, x.rank, x.ranks);
  Part z = JoinSums::none();
  row.template each<false, false>(ring, row.n <= kAhead, nullptr, false, nullptr, [&](int v, const uint4& w, const float (&)[kGroup], const float (&)[kGroup]) {
    float y[kGroup];
    Share<X>::values(w, y);
    drop_refused(sm, refused, v, y);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) s += ex2((y[i] - m) * sc);
    z.s += s;
  });
  return join_all(sm, z, x, JoinSums()).s;
}

// fp32 logits: two CTAs an SM (their rings are half as large), so that every cluster of
// a batch finds its place at once (16 sequences in clusters of 8: 15.4 us, 18.4 with
// 73 registers).
template <typename X, bool kDraft>
__global__ void __launch_bounds__(kVerifyThreads, sizeof(X) == 4 ? 2 : 1) verify_kernel(const __grid_constant__ VerifyArgs a) {
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ VerifySmem sm;
  typename Share<X>::R& ring = *reinterpret_cast<typename Share<X>::R*>(ring_smem);
  constexpr int kGroup = Share<X>::kGroup;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = static_cast<int>(cluster_nctarank());
  const int b = blockIdx.x / ranks, tid = threadIdx.x;
  Exchange xc = {rank, ranks, a.polls, 0u};
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&sm.bar[i], 1);
    fence_barrier_init();
    for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&sm.bar[i], 16 * ranks);
    sm.late = sm.any_late = 0;
  }
  __syncwarp();
  cluster_arrive();  // waited for at the first exchange
  if (tid < KVQ_MAX_QUERY_TOKENS) sm.kids[tid] = 0ull;
  pdl_wait();
  if (tid == 0) pdl_launch_dependents();
  const X* const rows = static_cast<const X*>(a.logits) + b * a.lsb;
  const float* const race = a.race + static_cast<int64_t>(b) * a.V;
  const int n = a.tree_len ? a.tree_len[b] : a.n_q;
  const float temp = a.temp ? a.temp[b] : 1.f;
  int32_t token = 0;
  float u = 0.f;
  uint64_t above = 0;
  if (tid < a.n_q) {
    token = a.tokens[static_cast<int64_t>(b) * a.n_q + tid];
    u = a.accept[static_cast<int64_t>(b) * a.n_q + tid];
    above = a.mask[b * a.mask_sb + tid] & ((1ull << tid) - 1ull);
  }
  Share<X> row(rows, a.V, rank, ranks);
  row.begin(ring);
  const bool greedy = !(temp > 0.f);
  const float sc = greedy ? kLog2e : fminf(kLog2e / temp, 3.4028235e38f);  // (finite for subnormal temperatures, too)
  bool good = n >= 1 && n <= a.n_q;
  __syncthreads();  // kids is zero
  if (tid < KVQ_MAX_QUERY_TOKENS) {
    sm.token[tid] = token;
    sm.u[tid] = u;
    if (above && tid < n)
      atomicOr(reinterpret_cast<unsigned long long*>(&sm.kids[63 - __clzll(above)]), 1ull << tid);
  }
  // The race row while the walk goes on: its first groups stay in the ring where
  // every row has the same groups (16-byte boundaries at the same places).
  const bool whole_race = good && !greedy && a.lst * sizeof(X) % 16 == 0;
  __syncthreads();
  if (whole_race) row.begin_e(ring, race);
  if (!good) cluster_wait();  // (no exchange comes)

  int cur = 0, count = 1, next = -1;
  while (good) {
    const float* drow = kDraft ? a.draft + b * a.dsb + cur * a.dst : nullptr;
    uint64_t kids = sm.kids[cur];
    if (kids && tid == kVerifyThreads - 1)  // what is likely to be read next
      prefetch_share(rows + (__ffsll(kids) - 1) * a.lst, a.V, rank, ranks);
    float kid_l = -INFINITY, kid_q = 0.f;  // on their way during the pass
    if (tid < 64 && (kids >> tid & 1ull)) {
      const int c = sm.token[tid];
      if (c >= 0 && c < a.V) {
        kid_l = Share<X>::value(row.row + c);
        if (kDraft) kid_q = drow[c];
      }
    }
    const Part mine = row_part(row, ring, sc);
    if (tid < 64) {
      sm.kid_l[tid] = kid_l;
      sm.kid_q[tid] = kid_q;
    }
    if (xc.turn == 0 && !greedy && tid == kVerifyThreads - 1) prefetch_share(race, a.V, rank, ranks);
    const Part p = join_all(sm, mine, xc, JoinRows{sc});
    const float m = p.m, inv_s = 1.f / (1.f + p.s), log_s = log1pf(p.s);
    const int best = p.at;
    good = !sm.late && p.s >= 0.f && p.s < INFINITY && m > -INFINITY && m < INFINITY;
    if (!good) break;
    auto prob = [&](float l) { return ex2((l - m) * sc) * inv_s; };
    auto log_prob = [&](float l) { return (l - m) * (sc * kLn2) - log_s; };
    // r_k of a group: `chain` steps of the residual
    auto residual = [&](const uint4& w, const float (&q)[kGroup], int chain, float (&y)[kGroup]) {
      float x[kGroup];
      Share<X>::values(w, x);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) y[i] = prob(x[i]);
      for (int k = 0; k < chain; ++k) {
        const float z = sm.inv_z[k];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) y[i] = fmaxf(y[i] * z - q[i], 0.f);
      }
    };

    // the children, in index order: the same decisions in every thread
    int took = -1, refused = 0;  // refused: entries of inv_z or out
    float total = 1.f;
    // without draft probabilities: the sum over what is not refused but the largest
    // logit, the same as it was last summed itself, and whether that logit is in
    float left = p.s, summed = p.s;
    bool with_best = true;
    while (kids) {
      const int j = __ffsll(kids) - 1;
      kids &= kids - 1ull;
      const int c = sm.token[j];
      bool ok;
      const float each = ex2((sm.kid_l[j] - m) * sc);  // 0 for an id outside the vocabulary
      float r = each * inv_s;
      if (greedy) {
        ok = c == best;
      } else if constexpr (kDraft) {
        const float q = sm.kid_q[j];
        for (int k = 0; k < refused; ++k) r = fmaxf(r * sm.inv_z[k] - q, 0.f);
        ok = r > 0.f && sm.u[j] * total * q < r;
      } else {
        for (int k = 0; k < refused; ++k)
          if (sm.out[k] == c) r = 0.f;
        ok = r > 0.f && sm.u[j] * total < r;
      }
      if (ok) {
        took = j;
        break;
      }
      if (greedy) continue;
      if constexpr (kDraft) {
        // r_k = max(r_{k-1} / Z_{k-1} - q, 0) with the sum of the last one
        __syncthreads();  // all have read what the last refusal wrote
        if (tid == 0) sm.inv_z[refused] = 1.f / total;
        __syncthreads();
        Part z = JoinSums::none();
        row.template each<false, true>(ring, row.n <= kAhead, nullptr, false, drow, [&](int, const uint4& w, const float (&)[kGroup], const float (&q)[kGroup]) {
          float y[kGroup];
          residual(w, q, refused + 1, y);
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < kGroup; ++i) s += y[i];
          z.s += s;
        });
        z = join_all(sm, z, xc, JoinSums());
        if (sm.late) break;
        if (z.s > 0.f) {  // else nothing is left and r stays
          total = z.s;
          ++refused;
        }
      } else if (c >= 0 && c < a.V && r > 0.f) {
        __syncthreads();
        if (tid == 0) sm.out[refused] = c;
        __syncthreads();
        ++refused;
        if (c == best) with_best = false;
        else left = fmaxf(left - each, 0.f);
        if (!with_best && left < summed * 0.03125f) {
          left = summed = rest_sum<X>(sm, ring, row.row, a.V, refused, m, sc, xc);
          ++xc.turn;
          if (sm.late) break;
        }
        total = (with_best ? 1.f + left : left) * inv_s;
      }
    }
    if (sm.late) break;
    if (tid == 0) sm.path[count - 1] = cur;
    if (took >= 0) {
      if (tid == 0) sm.logp[count - 1] = log_prob(sm.kid_l[took]);
      cur = took;
      ++count;
      row = Share<X>(rows + cur * a.lst, a.V, rank, ranks);
      row.begin(ring);
      __syncthreads();  // kid_l is written anew
      continue;
    }
    // the token behind the path
    next = best;
    if (!greedy) {
      Part k = JoinBest::none();
      row.template each<true, kDraft>(ring, row.n <= kAhead, race, whole_race, refused ? drow : nullptr, [&](int v, const uint4& w, const float (&e)[kGroup], const float (&q)[kGroup]) {
        // log2 of r / race up to a constant; -inf for what cannot be picked
        float y[kGroup];
        if (kDraft && refused) {
          residual(w, q, refused, y);
#pragma unroll
          for (int i = 0; i < kGroup; ++i) y[i] = fast_log2(y[i]);
        } else {
          Share<X>::values(w, y);
#pragma unroll
          for (int i = 0; i < kGroup; ++i) y[i] = (y[i] - m) * sc;
        }
        if constexpr (!kDraft) drop_refused(sm, refused, v, y);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const float late = y[i] - fast_log2(e[i]), key = e[i] > 0.f ? late : -INFINITY;
          k.at = key > k.m ? v + i : k.at;
          k.m = key > k.m ? key : k.m;
        }
      });
      k = join_all(sm, k, xc, JoinBest());
      if (k.m > -INFINITY) next = k.at;
    }
    if (tid == 0) sm.logp[count - 1] = log_prob(Share<X>::value(row.row + next));
    break;
  }
  // No CTA ends while a part is on its way to it, or with copies under way.
  leave(sm, xc, [&] {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // what thread 0 wrote of the path
    if (sm.late) good = false;
    if (rank == 0 && tid == 0) {
      a.path_len[b] = good ? count : -1;
      a.next[b] = good ? next : -1;
    }
    if (rank == 0 && tid < a.n_q) {
      const int64_t i = static_cast<int64_t>(b) * a.n_q + tid;
      a.path[i] = good && tid < count ? sm.path[tid] : -1;
      if (a.logprob) a.logprob[i] = good && tid < count ? sm.logp[tid] : 0.f;
    }
  });
}

}  // namespace
}  // namespace kvq

// Once per kernel and device: clusters of up to 16 CTAs, and `bytes` of dynamic
// shared memory.
kvq_status kvq_allow_clusters(const void* fn, int bytes) {
  static std::mutex mu;
  static const void* done[64][192];
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
  const int smem = logits_fp32 ? sizeof(kvq::Ring<16>) : sizeof(kvq::Ring<32>);
  const kvq_status st = kvq_allow_clusters(fn, smem);
  if (st != KVQ_OK) return st;
  // As many CTAs a sequence as the SMs hold, one each, but none below 8 bytes a
  // thread (32,000 logits of one sequence in 8 CTAs: 7.4 us when this was chosen, in 4, the
  // next below 16 bytes, 9.6).  A cluster lies within one GPC, which this does not look at:
  // with bf16 logits, whose CTAs fill an SM, the last clusters of 8 and 9, 16 to
  // 19 or 38 sequences wait for the first (two rows of 64,000: 14.2 us where 10
  // sequences take 8.3, 16.1 where 20 take 10.3, 20.0 where 39 take 14.1).
  int ranks = 1;
  while (ranks < kvq::kMaxRanks && 2 * ranks * static_cast<int64_t>(B) <= n_sm &&
         ranks * 16 * kvq::kVerifyThreads <= static_cast<int64_t>(vocab) * elt)
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
  a.polls = kvq_tile_polls();
  return kvq::launch_clusters(fn, dim3(static_cast<unsigned>(B * ranks)), ranks, kvq::kVerifyThreads, smem, stream, &a);
}
