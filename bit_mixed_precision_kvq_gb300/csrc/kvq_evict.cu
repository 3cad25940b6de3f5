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
#include "kvq_geom.cuh"

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

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

struct SelectSmem {
  uint32_t hist[256];
  uint32_t scan[kSelWarps][2];
  uint32_t count[kSelThreads];  // (round, warp): kept above the threshold | equal to it << 16
  uint2 start[kSelThreads];
  uint32_t prefix, want, equal;  // threshold so far; how many of its bin are wanted
};

// The want-th largest key of x[0, n) (1 <= want <= n), 8 bits a pass: the
// histogram of the keys that share the prefix found so far, and the bin in
// which the count from above reaches `want`.  Returns the key; *ties gets how
// many keys equal to it belong to the want largest.
__device__ uint32_t select_key(SelectSmem& sm, const float* x, int n, int want, uint32_t* ties) {
  if (threadIdx.x == 0) {
    sm.prefix = 0;
    sm.want = want;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) sm.hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t prefix = sm.prefix, high = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      const uint32_t k = order_key(x[i]);
      if ((k & high) == prefix) atomicAdd(&sm.hist[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // lane l: bins 255 - 8l .. 248 - 8l, counted from above
      uint32_t own = 0;
      for (int k = 0; k < 8; ++k) own += sm.hist[255 - 8 * threadIdx.x - k];
      uint32_t incl = own;
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (threadIdx.x >= static_cast<unsigned>(o)) incl += y;
      }
      const uint32_t w = sm.want, above = incl - own;
      __syncwarp();
      if (above < w && w <= incl) {
        uint32_t left = w - above;
        int bin = 255 - 8 * threadIdx.x;
        while (left > sm.hist[bin]) left -= sm.hist[bin--];
        sm.prefix = prefix | (static_cast<uint32_t>(bin) << shift);
        sm.want = left;
      }
    }
    __syncthreads();
  }
  *ties = sm.want;
  return sm.prefix;
}

// Positions of x[0, n) with key above `thr`, and the first `ties` equal to
// it, in order: out[i] = pos0 + index, xout[i] = value (xout may be null).
// A warp takes a span of n / 32 values, counts, and after a scan over the
// warps writes.
__device__ void write_kept(SelectSmem& sm, const float* x, int n, int pos0, uint32_t thr, uint32_t ties, int32_t* out,
                           float* xout) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int span = (n + kSelWarps - 1) / kSelWarps;
  const int i0 = min(n, warp * span), i1 = min(n, i0 + span);
  uint32_t gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = order_key(x[i]);
    gt += k > thr;
    eq += k == thr;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  __syncthreads();
  if (lane == 0) {
    sm.scan[warp][0] = gt;
    sm.scan[warp][1] = eq;
  }
  __syncthreads();
  uint32_t g0 = lane < warp ? sm.scan[lane][0] : 0, e0 = lane < warp ? sm.scan[lane][1] : 0;
  g0 = __reduce_add_sync(0xffffffffu, g0);
  e0 = __reduce_add_sync(0xffffffffu, e0);
  const uint32_t below = (1u << lane) - 1u;
  for (int base = i0; base < i1; base += 32) {
    const int i = base + lane;
    const float v = i < i1 ? x[i] : 0.f;
    const uint32_t k = order_key(v);
    const uint32_t mg = __ballot_sync(0xffffffffu, i < i1 && k > thr), me = __ballot_sync(0xffffffffu, i < i1 && k == thr);
    const uint32_t e = e0 + __popc(me & below);
    if (i < i1 && (k > thr || (k == thr && e < ties))) {
      const uint32_t at = g0 + __popc(mg & below) + min(e, ties);
      out[at] = pos0 + i;
      if (xout) xout[at] = v;
    }
    g0 += __popc(mg);
    e0 += __popc(me);
  }
}

// Selection with the keys in registers: thread k holds x[k + 1024 r], r < R.
// The threshold is found bit by bit from the highest bit in which the keys
// differ; a step counts the keys at or above a candidate (two instructions a
// key, a warp sum, one barrier) and stops once exactly `want` are.  Against
// the histogram form above this has no atomics, which a few crowded exponents
// serialise, and reads the masses once.
template <int R>
__device__ void select_in_registers(SelectSmem& sm, const float* x, int n, int want, int pos0, int32_t* out, float* xout) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t key[R];
  uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = tid + kSelThreads * r;
    // a slot past the end is never counted: 0 is below every candidate
    key[r] = i < n ? order_key(__ldcg(x + i)) : 0u;
    if (i < n) {
      lo = min(lo, key[r]);
      hi = max(hi, key[r]);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sm.scan[warp][0] = lo;
    sm.scan[warp][1] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, sm.scan[lane][0]);
  hi = __reduce_max_sync(0xffffffffu, sm.scan[lane][1]);
  // T: the largest value that at least `want` keys reach; above: keys past T
  uint32_t T = lo, above = 0;
  bool exact = false;
  if (lo != hi) {
    const int top = 31 - __clz(lo ^ hi);
    T = top == 31 ? 0u : (lo >> (top + 1)) << (top + 1);
#pragma unroll 1
    for (int bit = top; bit >= 0 && !exact; --bit) {
      const uint32_t cand = T | (1u << bit);
      uint32_t c = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) c += key[r] >= cand;
      c = __reduce_add_sync(0xffffffffu, c);
      uint32_t* row = sm.hist + 32 * (bit & 1);  // two rows: one barrier a step
      if (lane == 0) row[warp] = c;
      __syncthreads();
      c = __reduce_add_sync(0xffffffffu, row[lane]);
      if (c >= static_cast<uint32_t>(want)) {
        T = cand;
        exact = c == static_cast<uint32_t>(want);
      } else {
        above = c;
      }
    }
  }
  const uint32_t ties = exact ? 0xffffffffu : want - above;  // keys equal to T that stay
  // kept positions in order: counts of (round, warp), their scan, the writes
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool in = tid + kSelThreads * r < n;
    const uint32_t gt = __ballot_sync(0xffffffffu, in && key[r] > T), eq = __ballot_sync(0xffffffffu, in && key[r] == T);
    if (lane == 0) sm.count[r * kSelWarps + warp] = __popc(gt) | (__popc(eq) << 16);
  }
  __syncthreads();
  {
    // exclusive scan of R * 32 pairs (both counts stay below 2^16 for R <= 32)
    const uint32_t own = tid < R * kSelWarps ? sm.count[tid] : 0u;
    uint32_t g = own & 0xffffu, e = own >> 16;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t pg = __shfl_up_sync(0xffffffffu, g, o), pe = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) {
        g += pg;
        e += pe;
      }
    }
    if (lane == 31) {
      sm.scan[warp][0] = g;
      sm.scan[warp][1] = e;
    }
    __syncthreads();
    const uint32_t g0 = __reduce_add_sync(0xffffffffu, lane < warp ? sm.scan[lane][0] : 0u);
    const uint32_t e0 = __reduce_add_sync(0xffffffffu, lane < warp ? sm.scan[lane][1] : 0u);
    if (tid < R * kSelWarps) sm.start[tid] = make_uint2(g0 + g - (own & 0xffffu), e0 + e - (own >> 16));
  }
  __syncthreads();
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = tid + kSelThreads * r;
    const bool in = i < n;
    const uint32_t gt = __ballot_sync(0xffffffffu, in && key[r] > T), eq = __ballot_sync(0xffffffffu, in && key[r] == T);
    const uint2 at = sm.start[r * kSelWarps + warp];
    const uint32_t e = at.y + __popc(eq & below);
    if (in && (key[r] > T || (key[r] == T && e < ties))) {
      const uint32_t o = at.x + __popc(gt & below) + min(e, ties);
      out[o] = pos0 + i;
      if (xout) xout[o] = __ldcg(x + i);
    }
  }
}

// The `want` largest of x[0, n), in order of position: out[i] = pos0 + index,
// xout[i] = value (xout may be null).  Registers hold up to 32 keys a thread;
// longer ranges are read anew in every pass.
__device__ __forceinline__ void select_range(SelectSmem& sm, const float* x, int n, int want, int pos0, int32_t* out,
                                             float* xout) {
  if (n <= kSelThreads) {
    select_in_registers<1>(sm, x, n, want, pos0, out, xout);
  } else if (n <= 8 * kSelThreads) {
    select_in_registers<8>(sm, x, n, want, pos0, out, xout);
  } else if (n <= 32 * kSelThreads) {
    select_in_registers<32>(sm, x, n, want, pos0, out, xout);
  } else {
    uint32_t ties;
    const uint32_t thr = select_key(sm, x, n, want, &ties);
    write_kept(sm, x, n, pos0, thr, ties, out, xout);
  }
}

// CTA (b, h, part): part 0 the text prefix and the visual block, part 1 the
// text behind it and the tails of keep and mass_dst.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ SelectSmem sm;
  const Geom &c = a.c, &d = a.d;
  const int part = blockIdx.x & 1;
  const int64_t bh = blockIdx.x >> 1;
  const int b = static_cast<int>(bh / c.Hkv), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.Hkv);
  pdl_wait();
  const int len = evict_len(a, b);
  int32_t* keep = a.keep + bh * a.T_dst;
  if (len < 0) {
    if (part == 1) {
      for (int i = threadIdx.x; i < a.T_dst; i += kSelThreads) keep[i] = -1;
      if (h == 0 && threadIdx.x == 0 && a.new_len) a.new_len[b] = -1;
    }
    return;
  }
  const float* x = a.mass + bh * c.T_cap;
  float* y = a.mass_dst ? a.mass_dst + bh * d.T_cap : nullptr;
  if (part == 0) {
    for (int i = threadIdx.x; i < c.vs; i += kSelThreads) {
      keep[i] = i;
      if (y) y[i] = x[i];
    }
    if (d.Tv == 0) return;
    select_range(sm, x + c.vs, c.Tv, d.Tv, c.vs, keep + c.vs, y ? y + c.vs : nullptr);
    return;
  }
  const int n_suf = len - c.ve, room = min(n_suf, a.T_dst - d.ve);
  const int last = min(a.n_recent, n_suf);           // always kept
  const int pick = room - last, n_old = n_suf - last;  // pick of the n_old before them
  if (pick > 0) select_range(sm, x + c.ve, n_old, pick, c.ve, keep + d.ve, y ? y + d.ve : nullptr);
  for (int i = threadIdx.x; i < last; i += kSelThreads) {
    const int t = len - last + i;
    keep[d.ve + pick + i] = t;
    if (y) y[d.ve + pick + i] = x[t];
  }
  const int end = d.ve + room;
  for (int i = end + threadIdx.x; i < a.T_dst; i += kSelThreads) keep[i] = -1;
  if (y)
    for (int i = end + threadIdx.x; i < d.T_cap; i += kSelThreads) y[i] = 0.f;
  if (h == 0 && threadIdx.x == 0 && a.new_len) a.new_len[b] = end;
}

// The kept rows: a CTA per (sequence, KV head, 64 rows of the new cache).
// Consecutive threads copy consecutive granules of the destination, so the
// stores are whole lines and the loads are whole rows; a thread has up to
// eight granules in flight.
constexpr int kMoveRows = 64;
constexpr int kMoveThreads = 128;
constexpr int kMoveBatch = 8;

// Rows [0, n) of w bytes at dst from the rows at[i] >= 0 of src, in granules
// of T (w a multiple of its size).
template <typename T>
__device__ __forceinline__ void move_rows(uint8_t* dst, const uint8_t* src, int w, int n, const int32_t* at) {
  const int per = w / static_cast<int>(sizeof(T));  // a power of two
  const int sh = 31 - __clz(per), total = n << sh;
  for (int x0 = threadIdx.x; x0 < total; x0 += kMoveThreads * kMoveBatch) {
    T v[kMoveBatch];
    bool ok[kMoveBatch];
#pragma unroll
    for (int k = 0; k < kMoveBatch; ++k) {
      const int x = x0 + kMoveThreads * k;
      const int row = x < total ? at[x >> sh] : -1;
      ok[k] = row >= 0;
      if (ok[k]) v[k] = __ldcg(reinterpret_cast<const T*>(src + static_cast<int64_t>(row) * w) + (x & (per - 1)));
    }
#pragma unroll
    for (int k = 0; k < kMoveBatch; ++k)
      if (ok[k]) reinterpret_cast<T*>(dst)[x0 + kMoveThreads * k] = v[k];
  }
}
__device__ __forceinline__ void move_sz(uint8_t* dst, const uint8_t* src, int w, int n, const int32_t* at) {
  if (w == 16) move_rows<uint4>(dst, src, w, n, at);
  else if (w == 8) move_rows<uint2>(dst, src, w, n, at);
  else move_rows<uint32_t>(dst, src, w, n, at);
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a) {
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
    move_rows<uint4>(r.vis_k + o * kw, s.vis_k, kw, m, at[0]);
    move_rows<uint4>(r.vis_v + o * vw, s.vis_v, vw, m, at[0]);
    if (s.k_packed) move_sz(r.vis_ksz + o * c.kszrow, s.vis_ksz, c.kszrow, m, at[0]);
    if (s.v_packed) move_sz(r.vis_vsz + o * c.vszrow, s.vis_vsz, c.vszrow, m, at[0]);
  }
  if (t1 > t0) {
    const int64_t o = static_cast<int64_t>(t0) * kRowBytes;
    move_rows<uint4>(r.text_k + o, s.text_k, kRowBytes, t1 - t0, at[1]);
    move_rows<uint4>(r.text_v + o, s.text_v, kRowBytes, t1 - t0, at[1]);
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
  if (n_recent < 0 || n_recent > T_dst - d.vis_end) return KVQ_ERR_INVALID_ARG;
  const int64_t bh = static_cast<int64_t>(s.B) * s.H_kv;
  if (kvq::ranges_meet(cache, L->total_bytes, cache_dst, L_dst->total_bytes) ||
      kvq::ranges_meet(mass, 4 * bh * s.T_cap, mass_dst, 4 * bh * d.T_cap) ||
      kvq::ranges_meet(new_len, 4 * static_cast<int64_t>(s.B), seq_len, 4 * static_cast<int64_t>(s.B)))
    return KVQ_ERR_INVALID_ARG;
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
  st = kvq::launch_dependent(reinterpret_cast<const void*>(&kvq::select_kernel), dim3(static_cast<unsigned>(2 * bh)),
                             kvq::kSelThreads, 0, stream, &a);
  if (st != KVQ_OK) return st;
  return kvq::launch_dependent(reinterpret_cast<const void*>(&kvq::move_kernel), dim3(static_cast<unsigned>(blocks)),
                               kvq::kMoveThreads, 0, stream, &a);
}
