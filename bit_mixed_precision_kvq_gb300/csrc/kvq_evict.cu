// kvq_evict.cu -- kvq_cache_evict: the cache positions that have received the
// most attention weight, moved into a smaller cache.
//
// Per (sequence b, KV head h), with L_dst holding K_vis visual rows and
// T_dst - vis_end_dst = K_text text positions behind them: the text prefix
// stays whole; of the visual block the K_vis positions of largest mass stay;
// of the text positions [vis_end, len) the last n_recent and, of the others,
// those of largest mass, K_text in all (all of them when there are fewer).
// Order of values: NaN below every number, -0 equal to +0; of equal ones the
// lowest position stays.  Kept positions keep their order, and their rows are
// copied as they are stored (codes, scales and zeros bit for bit).
//
// Two launches, selection and copy.  Measured (GB300): 32K x 8 sequences to 8K
// 62 us (172 MB read and written; selection 24, copy 38), a LLaVA-OneVision
// layer to half 12 us, a ragged batch of 16 LLaVA-1.5 chats 27 us.
#include "kvq_geom.cuh"

#include <algorithm>

namespace kvq {
namespace {

struct EvictArgs {
  Geom c, d;
  const float* mass;  // [B][Hkv][T_cap]
  const int32_t* seq_len;
  int32_t T, T_dst, n_recent;
  int32_t* keep;      // [B][Hkv][T_dst]
  float* mass_dst;    // [B][Hkv][T_cap_dst] or null
  int32_t* new_len;   // [B] or null
};

// fp32 -> uint32 in the same order; NaN lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 -> +0
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Length of sequence b, or -1 (inactive).
__device__ __forceinline__ int evict_len(const EvictArgs& a, int b) {
  const int len = a.seq_len ? a.seq_len[b] : a.T;
  return len >= a.c.ve && len <= a.T ? len : -1;
}

// ---- selection ------------------------------------------------------------------
// A CTA per range of masses (the visual block, or the text behind it, of one
// sequence and KV head).  The threshold -- the want-th largest key -- is
// found in three passes of 11, 11 and 10 bits: a histogram in shared memory of
// the keys that share the digits found so far, and the bin in which the count
// from above reaches `want`.  11 bits spread the exponents of real masses over
// enough bins that the shared-memory atomics do not queue.  A range of up to
// 32 keys a thread is read once and stays in registers; what bounds it then is
// the instructions of one SM (32,736 keys: 4 us of loads, 6 of histograms, 2 of
// bin searches, 10 of ballots and writes), as there are no more CTAs than
// ranges.  (A bisection by counting, without atomics, took 47 us there against
// 40 for this before either had its loads in flight together; a cluster of 8
// CTAs a range, histograms added up through distributed shared memory, took
// twice as long, its CTAs waiting for one another.)
//
// A CTA has as few threads as hold its keys, so that many ranges share an SM
// (1,280 pairs of sequence and head with 2,880 masses: 164 us with 512 threads and 8 keys
// each, copy included, 218 with 1,024 threads; 512 ragged ones of 576: 27 us with
// 256 threads bound to 32 registers, 36.5 without the bound), and no more than
// 8 keys a thread below 1,024 threads (32,736 keys at 512 threads: 66 us for one
// range against 25.5).
constexpr int kBins = 2048;
template <int NT>
constexpr int kMostKeys = NT == 256 ? 4 : (NT == 512 ? 8 : 32);  // keys a thread of a CTA of NT holds

template <int NT>
struct SelectSmem {
  alignas(16) uint32_t hist[kBins];
  alignas(8) uint32_t coarse[kBins / 32];  // sums of 32 bins
  uint32_t scan[NT / 32][2];
  static constexpr int kPairs = NT / 32 * kMostKeys<NT>;
  uint32_t count[kPairs];  // (round, warp): kept above the threshold | equal to it << 16
  uint2 start[kPairs];
  uint32_t digit, want;
};

// The bin in which the count from the highest one down reaches sm.want; sm.want
// becomes what is wanted of that bin.  Every thread adds up its kBins / NT
// bins, the sums of 32 bins are left to one warp, which finds the one and then
// the bin.
template <int NT>
__device__ __forceinline__ void find_bin(SelectSmem<NT>& sm) {
  constexpr int PER = kBins / NT, SHARE = PER < 32 ? 32 / PER : 1;  // threads to 32 bins
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t sum = 0;
#pragma unroll
  for (int k = 0; k < PER; k += 2) {
    const uint2 v = reinterpret_cast<const uint2*>(sm.hist)[(PER * tid + k) / 2];
    sum += v.x + v.y;
  }
#pragma unroll
  for (int o = 1; o < SHARE; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (tid % SHARE == 0) sm.coarse[tid / SHARE] = sum;
  __syncthreads();
  if (tid < 32) {
    const uint32_t want = sm.want;
    auto scan = [&](uint32_t x) {  // inclusive, over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      return x;
    };
    // lane l: the sums 63 - 2 l and 62 - 2 l, then bin 31 - l of the one found
    const uint2 c = *reinterpret_cast<const uint2*>(&sm.coarse[62 - 2 * lane]);
    const uint32_t incl = scan(c.x + c.y), above = incl - c.x - c.y;
    const bool in_hi = want <= above + c.y;
    const uint32_t from = __ffs(__ballot_sync(0xffffffffu, want <= incl)) - 1;  // there is one: want <= all keys left
    const uint32_t at = __shfl_sync(0xffffffffu, in_hi ? 63 - 2 * lane : 62 - 2 * lane, from);
    const uint32_t base = __shfl_sync(0xffffffffu, in_hi ? above : above + c.y, from);
    const uint32_t bin = 32 * at + 31 - lane, own = sm.hist[bin], over = base + scan(own) - own;
    if (over < want && want <= over + own) {
      sm.digit = bin;
      sm.want = want - over;
    }
  }
  __syncthreads();
}

// load(f) calls f(key, there is one) for every key of the thread.
template <int NT, typename F>
__device__ __forceinline__ uint32_t find_threshold(SelectSmem<NT>& sm, int want, F&& load) {
  const int tid = threadIdx.x;
  if (tid == 0) sm.want = want;
  uint32_t prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const uint32_t high = pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
    for (int k = tid; k < kBins / 4; k += NT) reinterpret_cast<uint4*>(sm.hist)[k] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    load([&](uint32_t key, bool in) {
      if (in && (key & high) == prefix) atomicAdd(&sm.hist[(key >> shift) & mask], 1u);
    });
    __syncthreads();
    find_bin(sm);
    prefix |= sm.digit << shift;
  }
  return prefix;
}

// Kept: keys above T and the first sm.want equal to it.  Counts of (round,
// warp) pairs, their exclusive scan, and the writes, in order of position.
template <int NT, int R>
__device__ void select_in_registers(SelectSmem<NT>& sm, const float* x, int n, int want, int pos0, int32_t* out,
                                    float* xout) {
  static_assert(R <= kMostKeys<NT>, "one count per (round, warp)");
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t key[R];
#pragma unroll
  for (int r = 0; r < R; ++r)  // every load before any use
    key[r] = tid + NT * r < n ? __float_as_uint(__ldcg(x + tid + NT * r)) : 0u;
#pragma unroll
  for (int r = 0; r < R; ++r) key[r] = order_key(__uint_as_float(key[r]));
  const uint32_t T = find_threshold<NT>(sm, want, [&](auto&& f) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (NT * r < n) f(key[r], tid + NT * r < n);
  });
  const uint32_t ties = sm.want;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool in = tid + NT * r < n;
    const uint32_t gt = __ballot_sync(0xffffffffu, in && key[r] > T), eq = __ballot_sync(0xffffffffu, in && key[r] == T);
    if (lane == 0) sm.count[r * NW + warp] = __popc(gt) | (__popc(eq) << 16);
  }
  __syncthreads();
  // exclusive scan of the NW * R pairs, PER of them a thread
  constexpr int PER = (NW * R + NT - 1) / NT;
  uint32_t g = 0, e = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const uint32_t c = tid * PER + k < NW * R ? sm.count[tid * PER + k] : 0u;
    g += c & 0xffffu;
    e += c >> 16;
  }
  uint32_t ig = g, ie = e;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t pg = __shfl_up_sync(0xffffffffu, ig, o), pe = __shfl_up_sync(0xffffffffu, ie, o);
    if (lane >= o) {
      ig += pg;
      ie += pe;
    }
  }
  if (lane == 31) {
    sm.scan[warp][0] = ig;
    sm.scan[warp][1] = ie;
  }
  __syncthreads();
  const bool wl = lane < warp && lane < NW;
  uint32_t g0 = __reduce_add_sync(0xffffffffu, wl ? sm.scan[lane][0] : 0u) + ig - g;
  uint32_t e0 = __reduce_add_sync(0xffffffffu, wl ? sm.scan[lane][1] : 0u) + ie - e;
#pragma unroll
  for (int k = 0; k < PER; ++k)
    if (tid * PER + k < NW * R) {
      const uint32_t c = sm.count[tid * PER + k];
      sm.start[tid * PER + k] = make_uint2(g0, e0);
      g0 += c & 0xffffu;
      e0 += c >> 16;
    }
  __syncthreads();
  const uint32_t below = (1u << lane) - 1u;
  constexpr int kBatch = R < 8 ? R : 8;  // values in flight
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += kBatch) {
    if (NT * r0 >= n) break;
    int at[kBatch];
    float v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k, i = tid + NT * r;
      const bool in = i < n;
      const uint32_t gt = __ballot_sync(0xffffffffu, in && key[r] > T), eq = __ballot_sync(0xffffffffu, in && key[r] == T);
      const uint2 s = sm.start[r * NW + warp];
      const uint32_t q = s.y + __popc(eq & below);
      const bool stays = in && (key[r] > T || (key[r] == T && q < ties));
      at[k] = stays ? static_cast<int>(s.x + __popc(gt & below) + min(q, ties)) : -1;
      v[k] = stays && xout ? __ldcg(x + i) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (at[k] >= 0) {
        out[at[k]] = pos0 + tid + NT * (r0 + k);
        if (xout) xout[at[k]] = v[k];
      }
  }
}

// Ranges that do not fit the registers: the masses are read anew in every
// pass; a warp takes a contiguous span for the writes.
template <int NT>
__device__ void select_from_memory(SelectSmem<NT>& sm, const float* x, int n, int want, int pos0, int32_t* out,
                                   float* xout) {
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t T = find_threshold<NT>(sm, want, [&](auto&& f) {
    for (int i0 = 0; i0 < n; i0 += NT) {
      const int i = i0 + tid;
      f(i < n ? order_key(__ldcg(x + i)) : 0u, i < n);
    }
  });
  const uint32_t ties = sm.want;
  const int span = (n + NW - 1) / NW;
  const int i0 = min(n, warp * span), i1 = min(n, i0 + span);
  uint32_t gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = order_key(__ldcg(x + i));
    gt += k > T;
    eq += k == T;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sm.scan[warp][0] = gt;
    sm.scan[warp][1] = eq;
  }
  __syncthreads();
  const bool wl = lane < warp && lane < NW;
  uint32_t g0 = __reduce_add_sync(0xffffffffu, wl ? sm.scan[lane][0] : 0u);
  uint32_t e0 = __reduce_add_sync(0xffffffffu, wl ? sm.scan[lane][1] : 0u);
  const uint32_t below = (1u << lane) - 1u;
  for (int base = i0; base < i1; base += 32) {
    const int i = base + lane;
    const float v = i < i1 ? __ldcg(x + i) : 0.f;
    const uint32_t k = order_key(v);
    const uint32_t mg = __ballot_sync(0xffffffffu, i < i1 && k > T), me = __ballot_sync(0xffffffffu, i < i1 && k == T);
    const uint32_t q = e0 + __popc(me & below);
    if (i < i1 && (k > T || (k == T && q < ties))) {
      const uint32_t o = g0 + __popc(mg & below) + min(q, ties);
      out[o] = pos0 + i;
      if (xout) xout[o] = v;
    }
    g0 += __popc(mg);
    e0 += __popc(me);
  }
}

// The `want` largest of x[0, n), 1 <= want <= n, in order of position:
// out[i] = pos0 + index, xout[i] = value (xout may be null).
template <int NT>
__device__ __forceinline__ void select_range(SelectSmem<NT>& sm, const float* x, int n, int want, int pos0, int32_t* out,
                                             float* xout) {
  if constexpr (NT < 1024) select_in_registers<NT, kMostKeys<NT>>(sm, x, n, want, pos0, out, xout);
  else if (n <= 8 * NT) select_in_registers<NT, 8>(sm, x, n, want, pos0, out, xout);
  else if (n <= 32 * NT) select_in_registers<NT, 32>(sm, x, n, want, pos0, out, xout);
  else select_from_memory(sm, x, n, want, pos0, out, xout);
}

// CTA (b, h, part): part 0 the text prefix and the visual block, part 1 the
// text behind it and the tails of keep and mass_dst.
template <int NT>
__global__ void __launch_bounds__(NT, NT < 1024 ? 2048 / NT : 1) select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ SelectSmem<NT> sm;
  const Geom &c = a.c, &d = a.d;
  const int part = blockIdx.x & 1;
  const int64_t bh = blockIdx.x >> 1;
  const int b = static_cast<int>(bh / c.Hkv), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.Hkv);
  pdl_wait();
  const int len = evict_len(a, b);
  int32_t* keep = a.keep + bh * a.T_dst;
  if (len < 0) {
    if (part == 1) {
      for (int i = threadIdx.x; i < a.T_dst; i += NT) keep[i] = -1;
      if (h == 0 && threadIdx.x == 0 && a.new_len) a.new_len[b] = -1;
    }
    return;
  }
  const float* x = a.mass + bh * c.T_cap;
  float* y = a.mass_dst ? a.mass_dst + bh * d.T_cap : nullptr;
  if (part == 0) {
    for (int i = threadIdx.x; i < c.vs; i += NT) {
      keep[i] = i;
      if (y) y[i] = x[i];
    }
    if (d.Tv > 0) select_range(sm, x + c.vs, c.Tv, d.Tv, c.vs, keep + c.vs, y ? y + c.vs : nullptr);
    return;
  }
  const int n_suf = len - c.ve, room = min(n_suf, a.T_dst - d.ve);
  const int last = min(a.n_recent, n_suf);             // always kept
  const int pick = room - last, n_old = n_suf - last;  // pick of the n_old before them
  if (pick > 0) select_range(sm, x + c.ve, n_old, pick, c.ve, keep + d.ve, y ? y + d.ve : nullptr);
  for (int i = threadIdx.x; i < last; i += NT) {
    const int t = len - last + i;
    keep[d.ve + pick + i] = t;
    if (y) y[d.ve + pick + i] = x[t];
  }
  const int end = d.ve + room;
  for (int i = end + threadIdx.x; i < a.T_dst; i += NT) keep[i] = -1;
  if (y)
    for (int i = end + threadIdx.x; i < d.T_cap; i += NT) y[i] = 0.f;
  if (h == 0 && threadIdx.x == 0 && a.new_len) a.new_len[b] = end;
}

// The kept rows: a CTA per (sequence, KV head, 64 rows of the new cache).
// Consecutive threads copy consecutive 16-byte granules of the destination, so
// the stores are whole lines and the loads are whole rows; a thread loads its
// scale/zero row and up to four granules of K and V before it stores any
// (short rows leave no more than that in flight, which is what bounds the
// copy: 4.0 TB/s read and written together).
constexpr int kMoveRows = 64;
constexpr int kMoveThreads = 2 * kMoveRows;
constexpr int kMoveBatch = 4;

// A scale/zero row of w = 4, 8 or 16 bytes.
__device__ __forceinline__ uint4 load_row(const uint8_t* p, int w) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (w == 16) {
    r = __ldcg(reinterpret_cast<const uint4*>(p));
  } else if (w == 8) {
    const uint2 x = __ldcg(reinterpret_cast<const uint2*>(p));
    r.x = x.x;
    r.y = x.y;
  } else {
    r.x = __ldcg(reinterpret_cast<const uint32_t*>(p));
  }
  return r;
}
__device__ __forceinline__ void store_row(uint8_t* p, int w, const uint4& r) {
  if (w == 16) *reinterpret_cast<uint4*>(p) = r;
  else if (w == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r.x, r.y);
  else *reinterpret_cast<uint32_t*>(p) = r.x;
}

// K rows of kw bytes and V rows of vw bytes (powers of two from 32 on): rows
// [0, n) at kd, vd from the rows at[i] >= 0 of ks, vs.
__device__ __forceinline__ void move_rows(uint8_t* kd, const uint8_t* ks, int kw, uint8_t* vd, const uint8_t* vs, int vw,
                                          int n, const int32_t* at) {
  const int ksh = 27 - __clz(kw), vsh = 27 - __clz(vw);  // log2 of the granules in a row
  const int nk = n << ksh, total = nk + (n << vsh);
  for (int x0 = threadIdx.x; x0 < total; x0 += kMoveThreads * kMoveBatch) {
    uint4 r[kMoveBatch];
    bool ok[kMoveBatch];
#pragma unroll
    for (int k = 0; k < kMoveBatch; ++k) {
      const int x = x0 + kMoveThreads * k;
      const bool key = x < nk;
      const int y = key ? x : x - nk, sh = key ? ksh : vsh;
      const int row = x < total ? at[y >> sh] : -1;
      ok[k] = row >= 0;
      if (ok[k])
        r[k] = __ldcg(reinterpret_cast<const uint4*>((key ? ks : vs) + (static_cast<int64_t>(row) << (sh + 4))) +
                      (y & ((1 << sh) - 1)));
    }
#pragma unroll
    for (int k = 0; k < kMoveBatch; ++k)
      if (ok[k]) {
        const int x = x0 + kMoveThreads * k;
        if (x < nk) reinterpret_cast<uint4*>(kd)[x] = r[k];
        else reinterpret_cast<uint4*>(vd)[x - nk] = r[k];
      }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 10) move_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int32_t at[2][kMoveRows];  // source rows: visual, text (-1: none)
  const Geom &c = a.c, &d = a.d;
  const int chunks = (a.T_dst + kMoveRows - 1) / kMoveRows;
  const int64_t bh = blockIdx.x / chunks;
  const int i0 = static_cast<int>(blockIdx.x - bh * chunks) * kMoveRows, n = min(kMoveRows, a.T_dst - i0);
  const int b = static_cast<int>(bh / c.Hkv), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.Hkv);
  // Rows [i0, i0 + n) of the new cache: text rows [t0, t1) (the prefix and
  // the text behind the visual block are neighbours) and visual rows [v0, v1).
  const int v0 = max(0, min(i0, d.ve) - d.vs), v1 = max(0, min(i0 + n, d.ve) - d.vs);
  const int t0 = i0 <= d.vs ? i0 : max(d.vs, i0 - d.Tv), t1 = i0 + n <= d.vs ? i0 + n : max(d.vs, i0 + n - d.Tv);
  pdl_wait();
  if (threadIdx.x < static_cast<unsigned>(n)) {
    const int i = i0 + threadIdx.x, t = a.keep[bh * a.T_dst + i];
    if (i >= d.vs && i < d.ve) at[0][i - d.vs - v0] = t < 0 ? -1 : t - c.vs;
    else at[1][(i < d.vs ? i : i - d.Tv) - t0] = t < c.ve ? t : t - c.Tv;  // -1 stays -1
  }
  __syncthreads();
  const HeadRows s = head_rows(c, b, h), r = head_rows(d, b, h);
  if (v1 > v0) {
    const int kw = s.k_packed ? c.krow : kRowBytes, vw = s.v_packed ? c.vrow : kRowBytes, m = v1 - v0;
    const int64_t o = v0;
    // the scale/zero rows: K's by the first 64 threads, V's by the others
    const bool key = threadIdx.x < kMoveRows;
    const int i = key ? threadIdx.x : threadIdx.x - kMoveRows, zw = key ? c.kszrow : c.vszrow;
    const int from = i < m && (key ? s.k_packed : s.v_packed) ? at[0][i] : -1;
    uint4 z;
    if (from >= 0) z = load_row((key ? s.vis_ksz : s.vis_vsz) + static_cast<int64_t>(from) * zw, zw);
    move_rows(r.vis_k + o * kw, s.vis_k, kw, r.vis_v + o * vw, s.vis_v, vw, m, at[0]);
    if (from >= 0) store_row((key ? r.vis_ksz : r.vis_vsz) + (o + i) * zw, zw, z);
  }
  if (t1 > t0) {
    const int64_t o = static_cast<int64_t>(t0) * kRowBytes;
    move_rows(r.text_k + o, s.text_k, kRowBytes, r.text_v + o, s.text_v, kRowBytes, t1 - t0, at[1]);
  }
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_cache_evict(const kvq_layout* L, const void* cache, const float* mass, const int32_t* seq_len,
                                      int32_t T, const kvq_layout* L_dst, void* cache_dst, int32_t T_dst,
                                      int32_t n_recent, int32_t* keep, float* mass_dst, int32_t* new_len, void* stream) {
  kvq_status st = kvq_check_layout(L);
  if (st != KVQ_OK) return st;
  st = kvq_check_layout(L_dst);
  if (st != KVQ_OK) return st;
  if (!cache || !mass || !cache_dst || !keep) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cache) % 256 || reinterpret_cast<uintptr_t>(cache_dst) % 256 ||
      reinterpret_cast<uintptr_t>(mass) % 4 || reinterpret_cast<uintptr_t>(seq_len) % 4 ||
      reinterpret_cast<uintptr_t>(keep) % 4 || reinterpret_cast<uintptr_t>(mass_dst) % 4 ||
      reinterpret_cast<uintptr_t>(new_len) % 4)
    return KVQ_ERR_INVALID_ARG;
  const kvq_layout_desc &s = L->d, &d = L_dst->d;
  if (s.B != d.B || s.H_q != d.H_q || s.H_kv != d.H_kv || s.vis_start != d.vis_start || s.k_bits != d.k_bits ||
      s.v_bits != d.v_bits || s.group_size != d.group_size)
    return KVQ_ERR_INVALID_ARG;
  for (int h = 0; h < KVQ_MAX_HEADS; ++h)
    if (s.protected_heads[h] != d.protected_heads[h]) return KVQ_ERR_INVALID_ARG;
  if (T < s.vis_end || T < 1 || T > s.T_cap) return KVQ_ERR_INVALID_ARG;
  if (L_dst->Tv > L->Tv || T_dst < d.vis_end || T_dst < 1) return KVQ_ERR_INVALID_ARG;
  if (T_dst > d.T_cap) return KVQ_ERR_CAPACITY;
  if (T > kvq::kMaxLen || d.T_cap > kvq::kMaxLen) return KVQ_ERR_UNSUPPORTED;  // the tail of mass_dst goes to T_cap
  if (n_recent < 0 || n_recent > T_dst - d.vis_end) return KVQ_ERR_INVALID_ARG;
  const int64_t bh = static_cast<int64_t>(s.B) * s.H_kv;
  // What is written shares no memory with anything else: the selection reads
  // the masses more than once, and the copy takes its rows' places from keep.
  const struct {
    const void* at;
    int64_t bytes;
  } used[] = {{cache_dst, L_dst->total_bytes}, {keep, 4 * bh * T_dst}, {mass_dst, 4 * bh * d.T_cap},
              {new_len, 4 * static_cast<int64_t>(s.B)}, {cache, L->total_bytes}, {mass, 4 * bh * s.T_cap},
              {seq_len, 4 * static_cast<int64_t>(s.B)}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 7; ++j)
      if (kvq::ranges_meet(used[i].at, used[i].bytes, used[j].at, used[j].bytes)) return KVQ_ERR_INVALID_ARG;
  const int64_t blocks = bh * ((T_dst + kvq::kMoveRows - 1) / kvq::kMoveRows);
  if (blocks > 0x7fffffffLL || 2 * bh > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  kvq::EvictArgs a;
  kvq::fill_geom(L, cache, &a.c);
  kvq::fill_geom(L_dst, cache_dst, &a.d);
  a.mass = mass;
  a.seq_len = seq_len;
  a.T = T;
  a.T_dst = T_dst;
  a.n_recent = n_recent;
  a.keep = keep;
  a.mass_dst = mass_dst;
  a.new_len = new_len;
  // The threads of a range: as few as hold its keys in registers, so that
  // several ranges share an SM.
  const int longest = std::max(L->Tv, T - s.vis_end);
  const int nt = longest <= 4 * 256 ? 256 : (longest <= 8 * 512 ? 512 : 1024);
  const void* fn = nt == 256   ? reinterpret_cast<const void*>(&kvq::select_kernel<256>)
                   : nt == 512 ? reinterpret_cast<const void*>(&kvq::select_kernel<512>)
                               : reinterpret_cast<const void*>(&kvq::select_kernel<1024>);
  st = kvq::launch_dependent(fn, dim3(static_cast<unsigned>(2 * bh)), nt, 0, stream, &a);
  if (st != KVQ_OK) return st;
  return kvq::launch_dependent(reinterpret_cast<const void*>(&kvq::move_kernel), dim3(static_cast<unsigned>(blocks)),
                               kvq::kMoveThreads, 0, stream, &a);
}
