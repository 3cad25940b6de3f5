// kvq_tree.cuh -- attention of a tree of drafted tokens on the fifth-
// generation tensor cores (tcgen05), for kvq_decode_attention_tree.
//
// A unit is one (sequence b, KV head h, block of up to 64 columns); a column
// is a (token i, query head of h) pair.  The unit's positions -- the context
// [0, len), then the drafts -- are taken in tiles of 128, one position per
// TMEM lane, so that a tile's MMAs cost in proportion to the columns there
// are:
//   S^T[t][c]  = k_t . q_c           M = 128 positions, N = columns, K = d
//   O^T[d][c] += sum_t v_t[d] P[t][c]  M = 128 d, N = columns, K = positions
// K rows are unpacked into TMEM (A operand: the thread that unpacks a row owns
// its lane), V rows into shared memory as fp16 (A operand, d contiguous), P
// goes to shared memory (B operand), q stays there (B operand), so that K and
// S never pass through shared memory, whose 128 B a clock the unpacking warps
// and the tensor cores share.
//
// What it measures (GB300, calls back to back): 16 drafts over 16K positions
// of 8 sequences (32/8 heads, K2/V2 G32, 161 MB, 34 GFLOP) 109 us, 1.48 TB/s
// and 318 TFLOP/s; a LLaVA-OneVision layer with 16 drafts 20 us; 26 drafts over
// a ragged batch of 16 LLaVA-1.5 chats 90 us.  A tile takes about 1.7 us, of
// which the MMAs are 0.35 (N = 64: 35 clocks an MMA from TMEM, 51 from shared
// memory) and the bytes 0.25.  The rest is instructions: some 1100 a tile and
// scheduler at 0.3 a clock, because a warp's unpacking and softmax are chains
// of dependent steps through TMEM, shared memory and mbarriers and each of
// the 17 warps walks its own code (4.3 of 14 warp-clocks an instruction wait
// on loads and barriers, 2.0 on instruction fetch).  Spills are part of those
// loads: registers are handed out to warps by fours, so that 17 warps count as
// 20, which leaves 96 a thread, and every instance spills 60 to 164 bytes (K2/V2
// G32 80, K4/V2 G64 92, K8/V4 G32 160).  16 columns instead of 64 take only 12%
// less.  Tried and not kept, on the same case: 16 softmax warps (113 us), 16
// unpack warps (114), a CTA that walks several units (119), V loaded in the same
// phase (122), the L2 prefetch 8 tiles ahead (118) or none (136).
//
// Exactness of the scores (lse is an fp32 output): a packed K value
// c s + z is held as c' s + z' with c' = c - 2^(b-1) (c - 1 for 2 bits) and
// z' = z + (c - c') s.  c' s is exact in fp16 for 2 bits and an exact
// (high, low) fp16 pair for 4 and 8 bits, two MMAs; z' goes in as one more
// K step, an fp16 (high, low) pair against the (high, low) pair of the query's
// group sums (22 bits).  K operands carry a factor 1/2, so that values up to
// 65504 do not overflow.  fp16 holds bf16's 8 bits down to 2^-17, so K is exact
// from 2^-16 up, and off by at most 2^-24 below (2^-23 with its zero point),
// which is where the stored scales and zeros, fp16 too, have their last bits.
// Every column of queries has a power of two of its own, by which its largest
// element lands in [2^8, 2^9) (128 of them sum to 65280 at most): exact down to
// 2^-25 of that element, off by 2^-33 of it at most below.  It is undone by the
// column's softmax scale.  (With one factor 2^-7 for all, queries of 5e-4 against
// keys of 2e4 gave scores off by up to 0.2; the scale per column takes 0.5% at
// 16K x 8.)
// V is dequantised to fp16 (one rounding, 2^-11 of the value, below the
// output's 2^-8; steps of 2^-24 below 2^-14), P is fp16 (2^-11), O and the
// softmax sums are fp32.
//
// Softmax: a thread owns a position (a TMEM lane) and all columns, so the
// maximum of a column would be a reduction over 128 lanes.  Instead every
// column has a reference m (log2 units, shared memory) that only moves, for
// all lanes at once, when a score's P would pass 2^15 (fp16); the score that
// moves it gets P = 2^3.  So weights are off by 2^-28 of the largest one at most
// (half a step of fp16's subnormals; with P = 1 for the largest, 2^-25, a long
// context's faint weights would be lost), and a score may pass its reference's
// by 2^12 before it moves (by 2^9, from P = 2^6: 5% more time at 16K x 8).  The
// column sums stay in the threads until the end.
//
// 128 positions a tile and not 64: M = 64 takes the tensor cores as long.  64
// columns a unit at most: their sums are registers of the softmax threads.
//
// CTA = 17 warps: 0-7 softmax (warp w: TMEM lanes 32 (w mod 4) .., half w / 4 of
// the columns), 8-15 unpack (lanes 32 (w mod 4) .., half (w - 8) / 4 of the row),
// 16 issues the MMAs.  TMEM: two K buffers (64 columns high, 64 low, 8 zero
// points), two S buffers of 64, O of 64.
#pragma once

#include "kvq_geom.cuh"
#include "kvq_tree_plan.h"
#include "kvq_umma.cuh"

namespace kvq {
namespace tree {

constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kMmaWarp = 16;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kAhead = 4;               // tiles that the L2 prefetch runs ahead
constexpr int kTile = 128;              // positions per tile (TMEM lanes)
constexpr int kMaxCols = 64;            // columns per unit (at most)
constexpr int kHalfCols = kMaxCols / 2;  // columns of a softmax thread
constexpr float kMaxGrowth = 15.f;      // log2 of the largest P (fp16)
constexpr float kLift = 3.f;            // log2 of the P of a score that sets its reference
constexpr float kUnset = -1e30f;        // reference of a column that has attended nothing
constexpr int kQueryExponent = 8;       // a column's largest |q| lands in [2^8, 2^9)

constexpr uint32_t kTmK = 0, kTmKStride = 136, kTmLo = 64, kTmZ = 128;
constexpr uint32_t kTmS = 272, kTmSStride = 64;
constexpr uint32_t kTmO = 400;
constexpr uint32_t kTmCols = 512;

struct Args {
  Geom c;
  const uint16_t *q, *kd, *vd;
  int64_t sb, sh, st;  // strides of the drafts, in elements
  const uint64_t* mask;
  int64_t mask_sb;
  const int32_t* seq_len;
  int32_t T, n_q;
  float scale_log2;  // softmax_scale * log2(e)
  uint16_t* out;
  float* lse;
  uint32_t* status;
  float* ws;          // partials: a slot per CTA, [cols][D] o, then [cols][2] (m, l)
  uint32_t polls;     // limit of a wait
  // units: class k (0 protected, 1 K-only, 2 packed heads) has U[k] of them,
  // each split over S[k] CTAs; heads of the classes in order in head[]
  int32_t U[3], S[3], head0[3];
  int32_t nblk, nb, N;  // column blocks per KV head, columns per block, columns of the MMAs (16, 32, 48, 64)
  uint8_t head[KVQ_MAX_HEADS];
};

struct Smem {
  alignas(1024) uint8_t vt[2][kTile * 256];   // V: position (row of K = t), d contiguous
  alignas(1024) uint8_t pt[2][kMaxCols * 256];  // P: position, columns contiguous
  alignas(1024) uint8_t qt[kMaxCols * 256];   // q: column, d contiguous (permuted)
  alignas(128) uint8_t qz[kMaxCols * 32];     // group sums of q: column, 16 K indexes
  uint64_t colmask[kMaxCols];
  alignas(16) float neg_m[kMaxCols];  // minus the references
  alignas(16) float scale[kMaxCols];  // what takes a column's S to its score in log2 units
  alignas(16) float fac[kMaxCols];
  float lsum[4][kMaxCols];  // per softmax warp: column maxima of a tile; at the end column sums
  float qs[kMaxCols][4];
  uint64_t k_full[2], v_full[2], s_full[2], p_full[2], pv_done[2], q_ready, drained;
  uint32_t tmem_base;
  int abort;
};

// The unit and split of a CTA.
struct Work {
  int cls, b, h, cb, s, S;
};
__device__ __forceinline__ Work work_of(const Args& a, int cta) {
  Work w;
  int i = cta, cls = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (cls == k && i >= a.U[k] * a.S[k]) {
      i -= a.U[k] * a.S[k];
      cls = k + 1;
    }
  w.cls = cls;
  w.S = cls == 0 ? a.S[0] : (cls == 1 ? a.S[1] : a.S[2]);
  const int v = i / w.S;
  w.s = i - v * w.S;
  const int nh = (cls == 0 ? a.c.n_prot : (cls == 1 ? a.c.n_konly : a.c.n_packed)) * a.nblk;
  w.b = v / nh;
  const int r = v - w.b * nh;
  const int slot = r / a.nblk;
  w.cb = r - slot * a.nblk;
  w.h = a.head[(cls == 0 ? a.head0[0] : (cls == 1 ? a.head0[1] : a.head0[2])) + slot];
  return w;
}
// First CTA of the unit (b, h, cb).
__device__ __forceinline__ int first_cta(const Args& a, int b, int h, int cb, int* S) {
  const int mode = a.c.mode[h], cls = mode == 1 ? 0 : (mode == 2 ? 1 : 2);
  const int nh = cls == 0 ? a.c.n_prot : (cls == 1 ? a.c.n_konly : a.c.n_packed);
  const int base = (cls > 0 ? a.U[0] * a.S[0] : 0) + (cls > 1 ? a.U[1] * a.S[1] : 0);
  *S = cls == 0 ? a.S[0] : (cls == 1 ? a.S[1] : a.S[2]);
  return base + ((b * nh + a.c.slot[h]) * a.nblk + cb) * *S;
}
// Context length of sequence b, -1 for an inactive one.
__device__ __forceinline__ int context_len(const Args& a, int b) {
  const int len = a.seq_len ? a.seq_len[b] : a.T;
  return len >= 0 && len <= a.T ? len : -1;
}

// A wait that gives up marks the CTA (its outputs become NaN) and the status
// word; every later wait of the CTA then polls once.  A limit of one poll asks
// without suspending: the first wait that is not over already gives up.
__device__ __forceinline__ void wait_for(const Args& a, Smem& sm, uint64_t* bar, uint32_t parity) {
  if (a.polls > 1 ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity)) return;
  if (*static_cast<volatile int*>(&sm.abort)) return;
  if (mbar_wait(bar, parity, a.polls - 1)) return;
  sm.abort = 1;
  atomicOr(a.status, KVQ_STATUS_TILE_WAIT);
}

__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

// ---- unpacking -----------------------------------------------------------------
// Half hf of a K row: lane slices t = 2 hf, 2 hf + 1 of the storage order
// (kvq.h), 8 b bytes; output pair (t & 1) * 16 + 4 P + i = elements (d0 + i,
// d0 + i + 4), d0 = 32 P + 8 t.  Half hf of a V row: elements 64 hf .. + 63 in
// order, chunk kk = elements 64 hf + 8 kk .. + 7 in registers 4 kk .. + 3.
// A masked code with the exponent of 1024 over it is the fp16 1024 + c 2^p
// for a code at bit p; one fma takes it to c - off.

__device__ __forceinline__ uint32_t h2(float x) {  // both halves
  return pack_f16x2(x, x);
}

template <int P2, int H = 0>  // code at bit P2 of each half of x -> (code - off) / 2^H
__device__ __forceinline__ uint32_t code_at(uint32_t x, uint32_t mask, float off) {
  const uint32_t v = and_or(x, mask << P2, 0x64006400u);
  if constexpr (P2 + H == 0) return hsub2_u(v, h2(1024.f + off));
  return hfma2_u(v, h2(1.f / (1 << (P2 + H))), h2(-(1024.f / (1 << P2) + off) / (1 << H)));
}

template <int KB>
__device__ __forceinline__ constexpr float k_center() {
  return KB == 2 ? 1.f : (KB == 4 ? 8.f : 128.f);
}

// c' / 2 of the 16 pairs (4 P + i) of slice t of a K row, from its words.
template <int KB>
__device__ __forceinline__ void k_codes(const uint32_t* x, uint32_t (&c)[16]) {
  constexpr float off = k_center<KB>();
  if constexpr (KB == 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w = x[h], y = w >> 6;
      uint32_t* o = c + 2 * h;  // i = 2 h, 2 h + 1
      o[0] = code_at<8, 1>(w, 0x00030003u, off);
      o[1] = code_at<8, 1>(y, 0x00030003u, off);
      o[4] = code_at<6, 1>(w, 0x00030003u, off);
      o[5] = code_at<6, 1>(y, 0x00030003u, off);
      o[8] = code_at<4, 1>(w, 0x00030003u, off);
      o[9] = code_at<4, 1>(y, 0x00030003u, off);
      o[12] = code_at<0, 1>(w, 0x00030003u, off);
      o[13] = code_at<2, 1>(w, 0x00030003u, off);
    }
  } else if constexpr (KB == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = x[i], y = w >> 8;
      c[i] = code_at<0, 1>(w, 0x000F000Fu, off);
      c[4 + i] = code_at<4, 1>(w, 0x000F000Fu, off);
      c[8 + i] = code_at<0, 1>(y, 0x000F000Fu, off);
      c[12 + i] = code_at<4, 1>(y, 0x000F000Fu, off);
    }
  } else if constexpr (KB == 8) {
#pragma unroll
    for (int P = 0; P < 4; ++P)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = x[2 * P + (i >> 1)];
        c[4 * P + i] = code_at<0, 1>((i & 1) ? w >> 8 : w, 0x00FF00FFu, off);
      }
  }
}

// Both halves of a half2 register as floats.
__device__ __forceinline__ void h2_to_f2(uint32_t w, float& lo, float& hi) {
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
}
__device__ __forceinline__ float f16_bits(uint32_t h) { return __half2float(__ushort_as_half(static_cast<uint16_t>(h))); }

// Scale and zero (twice in a word) of chunks 4 e .. 4 e + 3 of half hf of a V
// row: a group is at least 4 chunks.
template <int G>
__device__ __forceinline__ void v_scales(const uint4& sz, int hf, int e, uint32_t& s2, uint32_t& z2) {
  if constexpr (G == 32) {
    const uint32_t z = hf ? sz.y : sz.x, s = hf ? sz.w : sz.z, sel = e ? 0x3232u : 0x1010u;
    z2 = prmt(z, z, sel);
    s2 = prmt(s, s, sel);
  } else if constexpr (G == 64) {
    const uint32_t sel = hf ? 0x3232u : 0x1010u;
    z2 = prmt(sz.x, sz.x, sel);
    s2 = prmt(sz.y, sz.y, sel);
  } else {
    z2 = prmt(sz.x, sz.x, 0x1010u);
    s2 = prmt(sz.x, sz.x, 0x3232u);
  }
}
// Chunks 4 e .. 4 e + 3 of half hf of a packed V row, dequantised in order;
// w: the words loaded by load_v_packed.
template <int VB>
__device__ __forceinline__ void v_values(const uint32_t* w, int hf, int e, uint32_t s2, uint32_t z2, uint32_t (&o)[16]) {
  auto put = [&](int kk, int j, uint32_t c) { o[4 * kk + j] = hfma2_u(c, s2, z2); };
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // elements 2 j, 2 j + 1 of every chunk
    if constexpr (VB == 2) {
      const uint32_t x = prmt(w[2 * j], w[2 * j + 1], hf ? 0x7632u : 0x5410u), y = x >> 6;
      if (e == 0) {
        put(0, j, code_at<0>(x, 0x00030003u, 0.f));
        put(1, j, code_at<2>(x, 0x00030003u, 0.f));
        put(2, j, code_at<4>(x, 0x00030003u, 0.f));
        put(3, j, code_at<6>(x, 0x00030003u, 0.f));
      } else {
        put(0, j, code_at<8>(x, 0x00030003u, 0.f));
        put(1, j, code_at<4>(y, 0x00030003u, 0.f));
        put(2, j, code_at<6>(y, 0x00030003u, 0.f));
        put(3, j, code_at<8>(y, 0x00030003u, 0.f));
      }
    } else if constexpr (VB == 4) {  // words 2 n + hf
      const uint32_t a = hf ? w[4 * j + 1] : w[4 * j], b = hf ? w[4 * j + 3] : w[4 * j + 2];
      const uint32_t x = prmt(a, b, e ? 0x7632u : 0x5410u), y = x >> 8;
      put(0, j, code_at<0>(x, 0x000F000Fu, 0.f));
      put(1, j, code_at<4>(x, 0x000F000Fu, 0.f));
      put(2, j, code_at<0>(y, 0x000F000Fu, 0.f));
      put(3, j, code_at<4>(y, 0x000F000Fu, 0.f));
    } else if constexpr (VB == 8) {  // words 4 n + 2 hf, + 1, as pairs of n
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x = prmt(w[4 * j + e], w[4 * j + 2 + e], k ? 0x7632u : 0x5410u);
        put(2 * k, j, code_at<0>(x, 0x00FF00FFu, 0.f));
        put(2 * k + 1, j, code_at<0>(x >> 8, 0x00FF00FFu, 0.f));
      }
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x) { return pack_f16x2(bf16_lo(x), bf16_hi(x)); }

// Where a row's values come from.
enum RowKind { kRowNone = 0, kRowPacked = 1, kRowBf16 = 2 };
struct Row {
  int kind;
  const uint8_t *p, *sz;
};

struct Source {
  HeadRows r;
  const uint8_t *kd, *vd;  // drafts of (b, h)
  int64_t dstep;           // bytes from draft to draft
  uint64_t any;            // drafts that some token attends
  int len, end;            // context length; + n_q
};

template <bool kKey>
__device__ __forceinline__ Row row_of(const Args& a, const Source& s, int t) {
  Row w;
  w.kind = kRowNone;
  w.p = w.sz = nullptr;
  if (t < s.len) {
    const Geom& c = a.c;
    if (t >= c.vs && t < c.ve) {
      const int64_t i = t - c.vs;
      const bool packed = kKey ? s.r.k_packed : s.r.v_packed;
      w.kind = packed ? kRowPacked : kRowBf16;
      const int step = packed ? (kKey ? c.krow : c.vrow) : kRowBytes;
      w.p = (kKey ? s.r.vis_k : s.r.vis_v) + i * step;
      if (packed) w.sz = kKey ? s.r.vis_ksz + i * c.kszrow : s.r.vis_vsz + i * c.vszrow;
    } else {
      w.kind = kRowBf16;
      w.p = (kKey ? s.r.text_k : s.r.text_v) + static_cast<int64_t>(t < c.vs ? t : t - c.Tv) * kRowBytes;
    }
  } else if (t < s.end && ((s.any >> (t - s.len)) & 1)) {
    w.kind = kRowBf16;
    w.p = (kKey ? s.kd : s.vd) + (t - s.len) * s.dstep;
  }
  return w;
}

// The raw bytes of half hf of a packed row and its scale/zero row.
template <int G>
__device__ __forceinline__ void load_sz(const uint8_t* p, uint4& sz) {
  if constexpr (G == 32) {
    sz = *reinterpret_cast<const uint4*>(p);
  } else if constexpr (G == 64) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    sz.x = x.x;
    sz.y = x.y;
  } else {
    sz.x = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <int N4>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {  // N4 x 16 bytes
#pragma unroll
  for (int i = 0; i < N4; ++i) {
    const uint4 x = reinterpret_cast<const uint4*>(p)[i];
    w[4 * i] = x.x;
    w[4 * i + 1] = x.y;
    w[4 * i + 2] = x.z;
    w[4 * i + 3] = x.w;
  }
}
// Half hf of a packed K row: KB words for slice 2 hf, KB for slice 2 hf + 1.
template <int KB>
__device__ __forceinline__ void load_k_packed(const uint8_t* row, int hf, uint32_t* w) {
  load_words<KB / 2>(row + hf * 8 * KB, w);
}
// What half hf of a packed V row needs: 4 VB words (16 for VB = 8).
template <int VB>
__device__ __forceinline__ void load_v_packed(const uint8_t* row, int hf, uint32_t* w) {
  if constexpr (VB == 8) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const uint2 x = *reinterpret_cast<const uint2*>(row + 16 * n + 8 * hf);
      w[2 * n] = x.x;
      w[2 * n + 1] = x.y;
    }
  } else {
    load_words<VB>(row, w);
  }
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Both operands' majors as bits 15 (A) and 16 (B): 0 K-major, 1 MN-major.
__host__ __device__ constexpr uint32_t idesc(int n, bool a_mn, bool b_mn) {
  return umma_idesc_f16(kTile, n, b_mn) | (static_cast<uint32_t>(a_mn) << 15);
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// One lane of a converged warp; what it issues stays in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// c' / 2 -> the high (and low) fp16 parts of c' s / 2, in place and in lo.
template <int KB>
__device__ __forceinline__ void k_parts(uint32_t (&c)[16], const uint32_t (&s2)[4], uint32_t (&lo)[16]) {
#pragma unroll
  for (int P = 0; P < 4; ++P)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = c[4 * P + j], h = hmul2_u(x, s2[P]);
      c[4 * P + j] = h;
      if constexpr (KB > 2) lo[4 * P + j] = hfma2_u(x, s2[P], h ^ 0x80008000u);
    }
}

// The zero points' A row: z' / 2 as (high, low, high) of each group, groups
// in pairs (words 0-1, 2-3, 4-5).
template <int KB, int G>
__device__ __forceinline__ void z_parts(const uint4& sz, uint32_t (&zz)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) zz[j] = 0u;
#pragma unroll
  for (int w = 0; w < (G == 32 ? 2 : 1); ++w) {
    uint32_t z, t;
    if constexpr (G == 32) z = w ? sz.y : sz.x, t = w ? sz.w : sz.z;
    else if constexpr (G == 64) z = sz.x, t = sz.y;
    else z = sz.x & 0xffffu, t = sz.x >> 16;
    float z0, z1, s0, s1, h0, h1;
    h2_to_f2(z, z0, z1);
    h2_to_f2(t, s0, s1);
    z0 = fmaf(0.5f * k_center<KB>(), s0, 0.5f * z0);
    z1 = fmaf(0.5f * k_center<KB>(), s1, 0.5f * z1);
    const uint32_t h = pack_f16x2(z0, z1);
    h2_to_f2(h, h0, h1);
    zz[w] = zz[4 + w] = h;
    zz[2 + w] = pack_f16x2(z0 - h0, z1 - h1);
  }
}
// s of the four 32-element blocks, twice in a word.
template <int G>
__device__ __forceinline__ void k_scales(const uint4& sz, uint32_t (&s2)[4]) {
  if constexpr (G == 32) {
    s2[0] = prmt(sz.z, sz.z, 0x1010u);
    s2[1] = prmt(sz.z, sz.z, 0x3232u);
    s2[2] = prmt(sz.w, sz.w, 0x1010u);
    s2[3] = prmt(sz.w, sz.w, 0x3232u);
  } else if constexpr (G == 64) {
    s2[0] = s2[1] = prmt(sz.y, sz.y, 0x1010u);
    s2[2] = s2[3] = prmt(sz.y, sz.y, 0x3232u);
  } else {
    s2[0] = s2[1] = s2[2] = s2[3] = prmt(sz.x, sz.x, 0x3232u);
  }
}

// The context rows of tile i, K (key) or V, into L2.
__device__ __forceinline__ void prefetch_tile(const Geom& c, const HeadRows& r, int i, int len, bool key) {
  const int t0 = i * kTile, t1 = min(t0 + kTile, len);
  const int v0 = max(t0, c.vs), v1 = min(t1, c.ve);  // visual ones
  if (v0 < v1) {
    const int64_t x = v0 - c.vs;
    const bool packed = key ? r.k_packed : r.v_packed;
    const int w = packed ? (key ? c.krow : c.vrow) : kRowBytes, zw = key ? c.kszrow : c.vszrow;
    prefetch_bytes((key ? r.vis_k : r.vis_v) + x * w, (v1 - v0) * w);
    if (packed) prefetch_bytes((key ? r.vis_ksz : r.vis_vsz) + x * zw, (v1 - v0) * zw);
  }
  const uint8_t* text = key ? r.text_k : r.text_v;
  if (t0 < min(t1, c.vs)) prefetch_bytes(text + static_cast<int64_t>(t0) * kRowBytes, (min(t1, c.vs) - t0) * kRowBytes);
  const int s0 = max(t0, c.ve);
  if (s0 < t1) prefetch_bytes(text + static_cast<int64_t>(s0 - c.Tv) * kRowBytes, (t1 - s0) * kRowBytes);
}

template <int KB, int VB, int G>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], 8);
      mbar_init(&sm.v_full[i], 8);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kSoftmaxWarps);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.q_ready, kSoftmaxWarps);
    mbar_init(&sm.drained, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_base, kTmCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm.tmem_base;
  const int N = a.N;
  const Work w = work_of(a, blockIdx.x);
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();  // past the dependency wait; this kernel writes no cache row
  const int len = context_len(a, w.b);
  const int nt = len < 0 ? 0 : (len + a.n_q + kTile - 1) / kTile;
  const int i0 = static_cast<int>(static_cast<int64_t>(nt) * w.s / w.S);
  const int i1 = static_cast<int>(static_cast<int64_t>(nt) * (w.s + 1) / w.S);
  const int hq0 = w.h * a.c.g, col0 = w.cb * a.nb;
  const int ncols = min(a.nb, a.c.g * a.n_q - col0);
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  // packed K rows in a tile: their low parts and zero points are MMAs of their own
  const bool k_packed = KB < 16 && a.c.mode[w.h] == 0;
  auto has_packed = [&](int i) { return k_packed && i * kTile < min(a.c.ve, len) && (i + 1) * kTile > a.c.vs; };

  if (warp == kMmaWarp) {
    // ---------------- MMAs ----------------
    const uint32_t id_qk = idesc(N, false, false), id_pv = idesc(N, true, true);
    // descriptors of the first K step; a step further is so many 16-byte units
    const uint32_t lbo = 16 * N, step = 2 * lbo >> 4;
    const uint64_t dq = umma_sdesc(smem_u32(sm.qt), lbo, 128), dz = umma_sdesc(smem_u32(sm.qz), lbo, 128);
    const uint64_t dv = umma_sdesc(smem_u32(sm.vt[0]), 2048, 128), dp = umma_sdesc(smem_u32(sm.pt[0]), lbo, 128);
    auto issue_pv = [&](int n) {
      const int buf = n & 1;
      wait_for(a, sm, &sm.v_full[buf], (n >> 1) & 1);
      wait_for(a, sm, &sm.p_full[buf], (n >> 1) & 1);
      tc_fence_after();
      if (elect_one()) {
        const uint64_t v = dv + buf * (sizeof(sm.vt[0]) >> 4), p = dp + buf * (sizeof(sm.pt[0]) >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) umma_ss(tm + kTmO, v + ks * 256, p + ks * step, id_pv, n > 0 || ks > 0);
        umma_commit(&sm.pv_done[buf]);
      }
      __syncwarp();
    };
    // the rows of the tiles to come into L2: K by lane 0, V by lane 1
    const HeadRows rows = head_rows(a.c, w.b, w.h);
    if (lane < 2)
      for (int i = i0; i < min(i0 + kAhead, i1); ++i) prefetch_tile(a.c, rows, i, len, lane == 0);
    if (i1 * kTile > len)  // ... and the drafts
      for (int j = lane; j < a.n_q; j += 32) {
        const int64_t d = w.b * a.sb + w.h * a.sh + j * a.st;
        prefetch_l2(a.kd + d, kRowBytes);
        prefetch_l2(a.vd + d, kRowBytes);
      }
    if (i0 < i1) wait_for(a, sm, &sm.q_ready, 0);
    for (int i = i0; i < i1; ++i) {
      const int n = i - i0, buf = n & 1;
      wait_for(a, sm, &sm.k_full[buf], (n >> 1) & 1);
      tc_fence_after();
      // S's buffer is free: the P of tile n - 2 was waited for before its PV
      const bool packed = has_packed(i);
      if (elect_one()) {
        const uint32_t kb = tm + kTmK + buf * kTmKStride, sb = tm + kTmS + buf * kTmSStride;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) umma_ts(sb, kb + 8 * ks, dq + ks * step, id_qk, ks > 0);
        if (packed) {
          if constexpr (KB > 2) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) umma_ts(sb, kb + kTmLo + 8 * ks, dq + ks * step, id_qk, true);
          }
          umma_ts(sb, kb + kTmZ, dz, id_qk, true);
        }
        umma_commit(&sm.s_full[buf]);  // S is there, and K's buffer free
      }
      __syncwarp();
      if (lane < 2 && i + kAhead < i1) prefetch_tile(a.c, rows, i + kAhead, len, lane == 0);
      __syncwarp();
      if (n > 0) issue_pv(n - 1);
    }
    if (i0 < i1) {
      issue_pv(i1 - i0 - 1);
      // No MMA is in flight when the CTA gives its tensor memory back, also
      // where a wait above gave up (so not by the caller's limit).
      if (elect_one()) umma_commit(&sm.drained);
      __syncwarp();
      mbar_wait(&sm.drained, 0, kDefaultTilePolls);
    }
  } else if (warp >= kSoftmaxWarps) {
    // ---------------- unpack ----------------
    const int hf = (warp - kSoftmaxWarps) >> 2, pos = 32 * (warp & 3) + lane;
    const Geom& c = a.c;
    Source src;
    src.r = head_rows(c, w.b, w.h);
    src.len = max(len, 0);
    const int64_t d0 = w.b * a.sb + w.h * a.sh;
    src.kd = reinterpret_cast<const uint8_t*>(a.kd + d0);
    src.vd = reinterpret_cast<const uint8_t*>(a.vd + d0);
    src.dstep = 2 * a.st;
    src.end = src.len + a.n_q;
    {
      const uint64_t* mk = a.mask + w.b * a.mask_sb;
      const uint64_t x = (lane < a.n_q ? mk[lane] : 0) | (lane + 32 < a.n_q ? mk[lane + 32] : 0);
      src.any = static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x))) |
                (static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x >> 32))) << 32);
    }
    // All 32 rows of this warp in tile i are visual ones.
    const int first = 32 * (warp & 3), vend = min(c.ve, src.len);
    auto all_visual = [&](int i) { return i * kTile + first >= c.vs && i * kTile + first + 32 <= vend; };
    const bool kp = KB < 16 && src.r.k_packed, vp = VB < 16 && src.r.v_packed;
    // the next tile's packed half rows, loaded while this one is unpacked
    constexpr int KW = KB < 16 ? 2 * KB : 2, VW = VB == 8 ? 16 : (VB < 16 ? 4 * VB : 2);
    uint32_t kr[KW], vr[VW];
    uint4 ksz = make_uint4(0, 0, 0, 0), vsz = ksz;
    auto load_k = [&](int i) {
      if constexpr (KB < 16) {
        const int64_t x = i * kTile + pos - c.vs;
        load_k_packed<KB>(src.r.vis_k + x * c.krow, hf, kr);
        load_sz<G>(src.r.vis_ksz + x * c.kszrow, ksz);
      }
    };
    auto load_v = [&](int i) {
      if constexpr (VB < 16) {
        const int64_t x = i * kTile + pos - c.vs;
        load_v_packed<VB>(src.r.vis_v + x * c.vrow, hf, vr);
        load_sz<G>(src.r.vis_vsz + x * c.vszrow, vsz);
      }
    };
    if (i0 < i1 && all_visual(i0)) {
      if (kp) load_k(i0);
      if (vp) load_v(i0);
    }
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int n = i - i0, buf = n & 1;
      const bool vis = all_visual(i), next = i + 1 < i1 && all_visual(i + 1);
      // ---- K: registers -> TMEM ----
      const uint32_t kt = tm + lanes + kTmK + buf * kTmKStride + 32 * hf;
      if (n >= 2) {
        wait_for(a, sm, &sm.s_full[buf], ((n - 2) >> 1) & 1);  // its QK has read K's buffer
        tc_fence_after();
      }
      if (kp && vis) {
        if constexpr (KB < 16) {
          uint32_t s2[4];
          k_scales<G>(ksz, s2);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t hi[16], lo[16];
            k_codes<KB>(kr + t * KB, hi);
            k_parts<KB>(hi, s2, lo);
            tmem_st16(kt + 16 * t, hi);
            if constexpr (KB > 2) tmem_st16(kt + kTmLo + 16 * t, lo);
          }
          if (hf == 0) {
            uint32_t zz[8];
            z_parts<KB, G>(ksz, zz);
            tmem_st8(kt + kTmZ, zz);
          }
        }
      } else {
        const Row row = row_of<true>(a, src, i * kTile + pos);
        const bool packed = has_packed(i);
        uint4 sz = make_uint4(0u, 0u, 0u, 0u);
        uint32_t s2[4];
        if constexpr (KB < 16) {
          if (row.kind == kRowPacked) load_sz<G>(row.sz, sz);
          k_scales<G>(sz, s2);
        }
        // Not unrolled: this path runs once or twice a CTA of a packed head,
        // mostly from a cold instruction cache.
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          // both kinds of rows with the same loads: four 16-byte pieces of a
          // bf16 row (d = 32 P + 16 hf + 8 t .. + 7), the slice of a packed one
          uint32_t hi[16], lo[16], raw[16];
          const bool bf = row.kind == kRowBf16;
          const int pieces = bf ? 4 : (KB < 16 && row.kind == kRowPacked ? (KB + 3) / 4 : 0), step = bf ? 64 : 16;
          const uint8_t* p = row.p + (bf ? 32 * hf + 16 * t : hf * 8 * KB + (KB > 2 ? t * 4 * KB : 0));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (j < pieces) x = *reinterpret_cast<const uint4*>(p + j * step);
            raw[4 * j] = x.x;
            raw[4 * j + 1] = x.y;
            raw[4 * j + 2] = x.z;
            raw[4 * j + 3] = x.w;
          }
#pragma unroll
          for (int P = 0; P < 4; ++P) {
            const uint32_t* x = raw + 4 * P;
            hi[4 * P] = pack_f16x2(0.5f * bf16_lo(x[0]), 0.5f * bf16_lo(x[2]));
            hi[4 * P + 1] = pack_f16x2(0.5f * bf16_hi(x[0]), 0.5f * bf16_hi(x[2]));
            hi[4 * P + 2] = pack_f16x2(0.5f * bf16_lo(x[1]), 0.5f * bf16_lo(x[3]));
            hi[4 * P + 3] = pack_f16x2(0.5f * bf16_hi(x[1]), 0.5f * bf16_hi(x[3]));
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) lo[j] = 0u;
          if constexpr (KB < 16) {
            if (row.kind == kRowPacked) {
              if (KB == 2 && t) {  // the piece holds both slices
                raw[0] = raw[2];
                raw[1] = raw[3];
              }
              k_codes<KB>(raw, hi);
              k_parts<KB>(hi, s2, lo);
            }
          }
          __syncwarp();
          tmem_st16(kt + 16 * t, hi);
          if (KB > 2 && packed) tmem_st16(kt + kTmLo + 16 * t, lo);
        }
        if (packed && hf == 0) {
          uint32_t zz[8];
          if constexpr (KB < 16) z_parts<KB, G>(sz, zz);  // zeros for a bf16 row
          tmem_st8(kt + kTmZ, zz);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[buf]);
      if (kp && next) load_k(i + 1);
      // ---- V: registers -> shared memory ----
      if (n >= 2) wait_for(a, sm, &sm.pv_done[buf], ((n - 2) >> 1) & 1);
      uint8_t* vt = sm.vt[buf] + (pos >> 3) * 2048 + (pos & 7) * 16 + 1024 * hf;
      auto put_v = [&](int e, const uint32_t (&o)[16]) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          *reinterpret_cast<uint4*>(vt + 512 * e + 128 * kk) =
              make_uint4(o[4 * kk], o[4 * kk + 1], o[4 * kk + 2], o[4 * kk + 3]);
      };
      if (vp && vis) {
        if constexpr (VB < 16) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t s2, z2, o[16];
            v_scales<G>(vsz, hf, e, s2, z2);
            v_values<VB>(vr, hf, e, s2, z2, o);
            put_v(e, o);
          }
        }
      } else {
        const Row row = row_of<false>(a, src, i * kTile + pos);
        uint4 sz = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (VB < 16) {
          if (row.kind == kRowPacked) load_sz<G>(row.sz, sz);
        }
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          uint32_t o[16], raw[16];
          const bool bf = row.kind == kRowBf16;
          const int pieces = bf ? 4 : (VB < 8 && row.kind == kRowPacked ? VB : 0);
          const uint8_t* p = row.p + (bf ? 128 * hf + 64 * e : 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (j < pieces) x = *reinterpret_cast<const uint4*>(p + 16 * j);
            raw[4 * j] = x.x;
            raw[4 * j + 1] = x.y;
            raw[4 * j + 2] = x.z;
            raw[4 * j + 3] = x.w;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = bf16x2_to_f16x2(raw[j]);
          if constexpr (VB < 16) {
            if (row.kind == kRowPacked) {
              if constexpr (VB == 8) load_v_packed<VB>(row.p, hf, raw);
              uint32_t s2, z2;
              v_scales<G>(sz, hf, e, s2, z2);
              v_values<VB>(raw, hf, e, s2, z2, o);
            }
          }
          put_v(e, o);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_full[buf]);
      if (vp && next) load_v(i + 1);
    }
  } else {
    // ---------------- softmax ----------------
    const int tid = threadIdx.x;
    // q into shared memory: 16-byte chunk ch (8 d) of a column's row goes to
    // chunk 4 t + P of the permuted order; the sums of the 32-element blocks
    for (int x = tid; x < N * 4; x += kSoftmaxThreads) {
      const int c = x >> 2, P = x & 3;
      const bool ok = c < ncols;
      const int cg = col0 + c, tok = cg / a.c.g;
      const int64_t row = ok ? (static_cast<int64_t>(w.b) * a.n_q + tok) * a.c.Hq + hq0 + (cg - tok * a.c.g) : 0;
      uint4 r[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        r[t] = ok ? __ldcg(reinterpret_cast<const uint4*>(a.q + row * kD) + 4 * P + t) : make_uint4(0u, 0u, 0u, 0u);
      // The column's power of two f = 2^e, from the exponent of its largest |q|
      // (four threads have its quarters); 2^e and 2^-e are fp32 for every bf16.
      uint32_t top = 0u;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t v = j == 0 ? r[t].x : (j == 1 ? r[t].y : (j == 2 ? r[t].z : r[t].w));
          top = max(top, max(v & 0x7fffu, (v >> 16) & 0x7fffu));
        }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(100, kQueryExponent + 127 - static_cast<int>(top >> 7));
      const float f = __int_as_float((127 + e) << 23);
      if (P == 0) sm.scale[c] = 2.f * (a.scale_log2 * __int_as_float((127 - e) << 23));  // K entered halved
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t y[4] = {
            pack_f16x2(f * bf16_lo(r[t].x), f * bf16_lo(r[t].z)), pack_f16x2(f * bf16_hi(r[t].x), f * bf16_hi(r[t].z)),
            pack_f16x2(f * bf16_lo(r[t].y), f * bf16_lo(r[t].w)), pack_f16x2(f * bf16_hi(r[t].y), f * bf16_hi(r[t].w))};
        *reinterpret_cast<uint4*>(sm.qt + (4 * t + P) * (16 * N) + (c >> 3) * 128 + (c & 7) * 16) =
            make_uint4(y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += f16_bits(y[j] & 0xffffu) + f16_bits(y[j] >> 16);
      }
      sm.qs[c][P] = sum;
    }
    named_bar(1, kSoftmaxThreads);
    if (tid < N) {
      constexpr int ng = kD / G, per = 4 / ng;
      const int c = tid;
      uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (g < ng) {
          float s = 0.f;
          for (int j = 0; j < per; ++j) s += sm.qs[c][g * per + j];
          const __half sh = __float2half_rn(s);
          const uint32_t h = __half_as_ushort(sh), l = __half_as_ushort(__float2half_rn(s - __half2float(sh)));
          z[g >> 1] |= h << (16 * (g & 1));
          z[2 + (g >> 1)] |= h << (16 * (g & 1));
          z[4 + (g >> 1)] |= l << (16 * (g & 1));
        }
      uint8_t* d = sm.qz + (c >> 3) * 128 + (c & 7) * 16;
      *reinterpret_cast<uint4*>(d) = make_uint4(z[0], z[1], z[2], z[3]);
      *reinterpret_cast<uint4*>(d + 16 * N) = make_uint4(z[4], z[5], z[6], z[7]);
      sm.colmask[c] = c < ncols ? a.mask[w.b * a.mask_sb + (col0 + c) / a.c.g] : 0;
      sm.neg_m[c] = -kUnset;
    }
    fence_async_smem();  // the tensor cores read q
    named_bar(1, kSoftmaxThreads);
    if (lane == 0) mbar_arrive(&sm.q_ready);

    // this thread's position of a tile (a TMEM lane) and its columns [ch, ce)
    const int lp = 32 * (warp & 3) + lane;
    const int ch = (N / 2 + 15) / 16 * 16 * (warp >> 2), ce = warp < 4 ? min(N, (N / 2 + 15) / 16 * 16) : N;
    const uint32_t half_bar = 2 + (warp >> 2);  // barrier of the four warps that share the columns
    uint64_t l2[kHalfCols / 2];  // sums of its columns, in pairs
#pragma unroll
    for (int c = 0; c < kHalfCols / 2; ++c) l2[c] = 0ull;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int n = i - i0, buf = n & 1;
      const bool whole = (i + 1) * kTile <= len;  // every position is context
      uint32_t sees = 0xffffffffu;                // bit c - ch: column c attends this thread's position
      if (!whole) {
        const int t = i * kTile + lp;
        if (t >= len) {
          sees = 0u;
          if (t < len + a.n_q) {
#pragma unroll 1
            for (int c = ch; c < ce; ++c)
              sees |= static_cast<uint32_t>((sm.colmask[c] >> (t - len)) & 1) << (c - ch);
          }
        }
      }
      const uint32_t sb = tm + lanes + kTmS + buf * kTmSStride;
      wait_for(a, sm, &sm.s_full[buf], (n >> 1) & 1);
      tc_fence_after();
      // scores (log2 units, relative to the references if rel) of 16 columns
      auto rel16 = [&](const uint32_t (&s)[16], int c0, float (&x)[16]) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const ulonglong2 mm = *reinterpret_cast<const ulonglong2*>(&sm.neg_m[c0 + k]);
          const ulonglong2 ss = *reinterpret_cast<const ulonglong2*>(&sm.scale[c0 + k]);
          unpair(fma_pair(pair_of(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), ss.x, mm.x), x[k], x[k + 1]);
          unpair(fma_pair(pair_of(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), ss.y, mm.y), x[k + 2], x[k + 3]);
        }
      };
      auto hide16 = [&](int c0, float (&x)[16]) {
        const uint32_t b = sees >> (c0 - ch);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (!((b >> k) & 1)) x[k] = -INFINITY;
      };
      if (n >= 2) wait_for(a, sm, &sm.pv_done[buf], ((n - 2) >> 1) & 1);  // P's buffer is free
      uint8_t* pt = sm.pt[buf] + (lp >> 3) * (16 * N) + (lp & 7) * 16 + 16 * ch;
      // Weights by the references as they are; if a score of some column is
      // past its reference by more than kMaxGrowth, the references move and the
      // tile is done again (always for the first tile, which sets them).
      // (Twice settles it: no score is past the new references.  The bound is
      // for scores that a failed wait left unfinished.)
      for (int round = n == 0 ? 1 : 0; round < 4; ++round) {
        if (round > 0) {
#pragma unroll 1
          for (int c0 = ch; c0 < ce; c0 += 16) {
            uint32_t s[16];
            float x[16];
            tmem_ld16(sb + c0, s);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(s[k]) * sm.scale[c0 + k];
            if (!whole) hide16(c0, x);
            float mine = -INFINITY;  // lane k: the maximum of column c0 + k over the warp's positions
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float r = warp_max(x[k]);
              if (lane == k) mine = r;
            }
            if (lane < 16) sm.lsum[warp & 3][c0 + lane] = mine;
          }
          named_bar(half_bar, 128);
          float v = -INFINITY, old = 0.f;
          const int mine = ch + (tid & 127);  // the column whose reference this thread keeps
          if (mine < ce) {
            v = fmaxf(fmaxf(sm.lsum[0][mine], sm.lsum[1][mine]), fmaxf(sm.lsum[2][mine], sm.lsum[3][mine]));
            old = -sm.neg_m[mine];
            // 2^-100 of a sum is nothing next to the new one, which is at least 1
            sm.fac[mine] = v > old + 100.f ? 0.f : (v > old + kMaxGrowth ? ex2(old - (v - kLift)) : 1.f);
          }
          named_bar(half_bar, 128);
          if (n > 0) {
            // Undo what the tile added to the sums and rescale them; O, too,
            // once every earlier PV has landed.
            uint32_t s[16];
#pragma unroll
            for (int c0 = 0; c0 < kHalfCols; c0 += 16)
              if (ch + c0 < ce) {
                float x[16];
                tmem_ld16(sb + ch + c0, s);
                tmem_ld_wait();
                rel16(s, ch + c0, x);
                if (!whole) hide16(ch + c0, x);
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const float f0 = sm.fac[ch + c0 + k], f1 = sm.fac[ch + c0 + k + 1];
                  float u, v;
                  unpair(l2[(c0 + k) / 2], u, v);
                  l2[(c0 + k) / 2] = pair_of(f0 == 0.f ? 0.f : (u - ex2(x[k])) * f0, f1 == 0.f ? 0.f : (v - ex2(x[k + 1])) * f1);
                }
              }
            wait_for(a, sm, &sm.pv_done[buf ^ 1], ((n - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c0 = ch; c0 < ce; c0 += 16) {
              tmem_ld16(tm + lanes + kTmO + c0, s);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) * sm.fac[c0 + k]);
              tmem_st16(tm + lanes + kTmO + c0, s);
            }
            tmem_st_wait();
            named_bar(half_bar, 128);  // every thread is done with the old references
          }
          if (v > old + kMaxGrowth) sm.neg_m[mine] = kLift - v;
          named_bar(half_bar, 128);
        }
        float top = -INFINITY;
        uint32_t s[2][16];
        if (ch < ce) tmem_ld16(sb + ch, s[0]);
        if (ch + 16 < ce) tmem_ld16(sb + ch + 16, s[1]);
        tmem_ld_wait();
#pragma unroll
        for (int c0 = 0; c0 < kHalfCols; c0 += 16)
          if (ch + c0 < ce) {
            float x[16];
            rel16(s[c0 >> 4], ch + c0, x);
            if (!whole) hide16(ch + c0, x);
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              top = fmaxf(top, fmaxf(x[k], x[k + 1]));
              const float p0 = ex2(x[k]), p1 = ex2(x[k + 1]);
              l2[(c0 + k) / 2] = add_pair(l2[(c0 + k) / 2], pair_of(p0, p1));
              y[k >> 1] = pack_f16x2(p0, p1);
            }
            *reinterpret_cast<uint4*>(pt + (c0 >> 3) * 128) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(pt + (c0 >> 3) * 128 + 128) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        if (!bar_or(half_bar, 128, top > kMaxGrowth)) break;
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[buf]);  // S is free, too
    }
    // ---- the column sums over the lanes, then the outputs (thread = d) ----
    const int nd = i1 - i0;
    if (nd > 0) {
      wait_for(a, sm, &sm.pv_done[(nd - 1) & 1], ((nd - 1) >> 1) & 1);
      tc_fence_after();
    }
    named_bar(1, kSoftmaxThreads);  // lsum's last readers are done
    float l[kHalfCols];
#pragma unroll
    for (int c = 0; c < kHalfCols; c += 2) unpair(l2[c / 2], l[c], l[c + 1]);
#pragma unroll
    for (int c0 = 0; c0 < kHalfCols; c0 += 16)
      if (ch + c0 < ce) {
#pragma unroll
        for (int h = 8; h > 0; h >>= 1) {
          const bool up = lane & (2 * h);
#pragma unroll
          for (int k = 0; k < h; ++k) {
            const float give = up ? l[c0 + k] : l[c0 + k + h];
            const float got = __shfl_xor_sync(0xffffffffu, give, 2 * h);
            l[c0 + k] = (up ? l[c0 + k + h] : l[c0 + k]) + got;
          }
        }
        const float s = l[c0] + __shfl_xor_sync(0xffffffffu, l[c0], 1);
        if (!(lane & 1)) sm.lsum[warp & 3][ch + c0 + (lane >> 1)] = s;
      }
    named_bar(1, kSoftmaxThreads);
    const bool bad = sm.abort != 0;
    const float nan = __int_as_float(0x7fffffff);
    float* slot = a.ws + static_cast<int64_t>(blockIdx.x) * N * (kD + 2);
#pragma unroll 1
    for (int c0 = ch; c0 < ce; c0 += 16) {
      uint32_t o[16];
      if (nd > 0) {
        tmem_ld16(tm + lanes + kTmO + c0, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = 0u;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int c = c0 + k;
        if (c >= ncols) break;
        if (w.S > 1) {
          slot[c * kD + lp] = __uint_as_float(o[k]);
        } else {
          const float L = (sm.lsum[0][c] + sm.lsum[1][c]) + (sm.lsum[2][c] + sm.lsum[3][c]);
          const int cg = col0 + c, tok = cg / a.c.g;
          const int64_t row = (static_cast<int64_t>(w.b) * a.n_q + tok) * a.c.Hq + hq0 + (cg - tok * a.c.g);
          const float inv = bad || L != L ? nan : (L > 0.f ? 1.f / L : 0.f);
          a.out[row * kD + lp] = f32_to_bf16_bits(__uint_as_float(o[k]) * inv);
        }
      }
    }
    if (tid < ncols) {
      const int c = tid, cg = col0 + c, tok = cg / a.c.g;
      const float L = (sm.lsum[0][c] + sm.lsum[1][c]) + (sm.lsum[2][c] + sm.lsum[3][c]);
      // a sum that is NaN (a query that is) marks its row, also through the partials
      const float M = bad || L != L ? nan : (L > 0.f ? -sm.neg_m[c] : -INFINITY);
      if (w.S > 1) {
        *reinterpret_cast<float2*>(slot + N * kD + 2 * c) = make_float2(M, L);
      } else if (a.lse) {
        a.lse[(static_cast<int64_t>(w.b) * a.n_q + tok) * a.c.Hq + hq0 + (cg - tok * a.c.g)] =
            0.69314718055994531f * (M + log2f(L));
      }
    }
    tc_fence_before();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tm, kTmCols);
  }
}

const void* tree_kernel_k2(int vb, int G);
const void* tree_kernel_k4(int vb, int G);
const void* tree_kernel_k8(int vb, int G);
const void* tree_kernel_k16(int vb, int G);

}  // namespace tree
}  // namespace kvq
