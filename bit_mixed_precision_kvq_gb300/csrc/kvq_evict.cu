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
    uint32_t ties;
    const uint32_t thr = select_key(sm, x + c.vs, c.Tv, d.Tv, &ties);
    write_kept(sm, x + c.vs, c.Tv, c.vs, thr, ties, keep + c.vs, y ? y + c.vs : nullptr);
    return;
  }
  const int n_suf = len - c.ve, room = min(n_suf, a.T_dst - d.ve);
  const int last = min(a.n_recent, n_suf);           // always kept
  const int pick = room - last, n_old = n_suf - last;  // pick of the n_old before them
  if (pick > 0) {
    uint32_t ties;
    const uint32_t thr = select_key(sm, x + c.ve, n_old, pick, &ties);
    write_kept(sm, x + c.ve, n_old, c.ve, thr, ties, keep + d.ve, y ? y + d.ve : nullptr);
  }
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

// Copy w bytes (a multiple of 4) with the warp's lanes, 16 bytes at a time
// where the row size allows.
__device__ __forceinline__ void copy_row(uint8_t* dst, const uint8_t* src, int w, int lane) {
  if (w % 16 == 0) {
    if (lane < w / 16) reinterpret_cast<uint4*>(dst)[lane] = __ldcg(reinterpret_cast<const uint4*>(src) + lane);
  } else if (lane < w / 4) {
    reinterpret_cast<uint32_t*>(dst)[lane] = __ldcg(reinterpret_cast<const uint32_t*>(src) + lane);
  }
}

// A warp per kept row.
constexpr int kMoveWarps = 8;
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const __grid_constant__ EvictArgs a) {
  const Geom &c = a.c, &d = a.d;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(c.B) * c.Hkv * a.T_dst) return;
  const int t = a.keep[row];
  if (t < 0) return;
  const int64_t bh = row / a.T_dst;
  const int i = static_cast<int>(row - bh * a.T_dst);
  const int b = static_cast<int>(bh / c.Hkv), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.Hkv);
  const HeadRows s = head_rows(c, b, h), r = head_rows(d, b, h);
  if (i >= d.vs && i < d.ve) {
    const int64_t x = t - c.vs, y = i - d.vs;
    const int kw = s.k_packed ? c.krow : kRowBytes, vw = s.v_packed ? c.vrow : kRowBytes;
    copy_row(r.vis_k + y * kw, s.vis_k + x * kw, kw, lane);
    copy_row(r.vis_v + y * vw, s.vis_v + x * vw, vw, lane);
    if (s.k_packed) copy_row(r.vis_ksz + y * c.kszrow, s.vis_ksz + x * c.kszrow, c.kszrow, lane);
    if (s.v_packed) copy_row(r.vis_vsz + y * c.vszrow, s.vis_vsz + x * c.vszrow, c.vszrow, lane);
  } else {
    const int64_t x = t < c.vs ? t : t - c.Tv, y = i < d.vs ? i : i - d.Tv;
    copy_row(r.text_k + y * kRowBytes, s.text_k + x * kRowBytes, kRowBytes, lane);
    copy_row(r.text_v + y * kRowBytes, s.text_v + x * kRowBytes, kRowBytes, lane);
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
  const int64_t blocks = (bh * T_dst + kvq::kMoveWarps - 1) / kvq::kMoveWarps;
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
                               kvq::kMoveWarps * 32, 0, stream, &a);
}
