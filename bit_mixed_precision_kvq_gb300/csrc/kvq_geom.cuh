// kvq_geom.cuh -- the cache of one layer as the tree, mass and eviction
// kernels see it: geometry and segment pointers by value (no work plan), and
// the rows of one (sequence, KV head).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_device.cuh"
#include "kvq_ptx.cuh"

// Lets a kernel have `bytes` of dynamic shared memory (kvq_tree.cu).
kvq_status kvq_allow_smem(const void* fn, int bytes);
// Checks of the drafted rows of the tree's entry points (kvq_tree.cu).
kvq_status kvq_check_drafts(const kvq_layout* L, const void* cache, const void* k, const void* v, int64_t sb, int64_t sh,
                            int64_t st, int32_t n_q);

namespace kvq {

constexpr int kRowBytes = 2 * kD;  // a bf16 row
// The longest sequence of the tree, mass and eviction calls: positions are
// 32-bit, and tiles, strides of a CTA and prefetches run past the last one.
constexpr int32_t kMaxLen = 0x7fffffff - 0xffff;

struct Geom {
  int32_t B, Hq, Hkv, g;
  int32_t vs, ve;              // visual range of the layout
  int32_t Tv, Tv_pad, T_text, T_cap;
  int32_t kb, vb, G;
  int32_t n_prot, n_konly, n_packed;
  int32_t krow, kszrow, vrow, vszrow;  // bytes per row of the packed segments
  uint8_t* seg[KVQ_NSEG];
  uint8_t mode[KVQ_MAX_HEADS];  // head -> protection mode (0, 1 both, 2 K only)
  uint8_t slot[KVQ_MAX_HEADS];  // head -> slot among its kind
};

// Host: fill from a checked layout.
inline void fill_geom(const kvq_layout* L, const void* cache, Geom* p) {
  const kvq_layout_desc& d = L->d;
  *p = Geom{};
  p->B = d.B;
  p->Hq = d.H_q;
  p->Hkv = d.H_kv;
  p->g = L->g;
  p->vs = d.vis_start;
  p->ve = d.vis_end;
  p->Tv = L->Tv;
  p->Tv_pad = L->Tv_pad;
  p->T_text = L->T_text;
  p->T_cap = d.T_cap;
  p->kb = d.k_bits;
  p->vb = d.v_bits;
  p->G = d.group_size;
  p->n_prot = L->n_prot;
  p->n_konly = L->n_konly;
  p->n_packed = L->n_packed;
  p->krow = static_cast<int32_t>(L->row_bytes[KVQ_SEG_K_CODES]);
  p->kszrow = static_cast<int32_t>(L->row_bytes[KVQ_SEG_K_SZ]);
  p->vrow = static_cast<int32_t>(L->row_bytes[KVQ_SEG_V_CODES]);
  p->vszrow = static_cast<int32_t>(L->row_bytes[KVQ_SEG_V_SZ]);
  uint8_t* base = static_cast<uint8_t*>(const_cast<void*>(cache));
  for (int s = 0; s < KVQ_NSEG; ++s) p->seg[s] = base + L->off[s];
  for (int h = 0; h < KVQ_MAX_HEADS; ++h) {
    p->mode[h] = d.protected_heads[h];
    p->slot[h] = static_cast<uint8_t>(L->slot[h]);
  }
}

// Host: do [a, a + na) and [b, b + nb) share a byte?
inline bool ranges_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// Host: launch with programmatic stream serialisation allowed, so that the
// kernel's CTAs may be scheduled while the previous kernel in the stream
// drains; the kernel waits (griddepcontrol.wait) before touching memory.
inline kvq_status launch_dependent(const void* fn, dim3 grid, unsigned block, size_t smem, void* stream, void* arg) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {arg};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  return e == cudaSuccess ? KVQ_OK : kvq_cuda_fail(e);
}

// The rows of one (sequence b, KV head h): text rows by text index (position
// t < vs: t, t >= ve: t - Tv), visual rows by t - vs.
struct HeadRows {
  uint8_t *text_k, *text_v;
  uint8_t *vis_k, *vis_v;    // bf16 rows, or codes
  uint8_t *vis_ksz, *vis_vsz;
  bool k_packed, v_packed;   // visual rows held as codes with scale/zero rows
};

__device__ __forceinline__ HeadRows head_rows(const Geom& p, int b, int h) {
  HeadRows r;
  const int mode = p.mode[h], s = p.slot[h];
  const int64_t text = (static_cast<int64_t>(b) * p.Hkv + h) * p.T_text * kRowBytes;
  r.text_k = p.seg[KVQ_SEG_TEXT_K] + text;
  r.text_v = p.seg[KVQ_SEG_TEXT_V] + text;
  r.vis_ksz = r.vis_vsz = nullptr;
  r.k_packed = mode == 0 && p.kb < 16;
  r.v_packed = mode != 1 && p.vb < 16;
  if (mode == 0) {
    const int64_t row = (static_cast<int64_t>(b) * p.n_packed + s) * p.Tv_pad;
    r.vis_k = p.seg[KVQ_SEG_K_CODES] + row * p.krow;
    r.vis_ksz = p.seg[KVQ_SEG_K_SZ] + row * p.kszrow;
  } else {
    const int64_t row = (static_cast<int64_t>(b) * (p.n_prot + p.n_konly) + (mode == 2 ? p.n_prot : 0) + s) * p.Tv;
    r.vis_k = p.seg[KVQ_SEG_PROT_K] + row * kRowBytes;
  }
  if (mode == 1) {
    r.vis_v = p.seg[KVQ_SEG_PROT_V] + (static_cast<int64_t>(b) * p.n_prot + s) * p.Tv * kRowBytes;
  } else {
    const int64_t row = (static_cast<int64_t>(b) * (p.n_packed + p.n_konly) + (mode == 2 ? p.n_packed : 0) + s) * p.Tv_pad;
    r.vis_v = p.seg[KVQ_SEG_V_CODES] + row * p.vrow;
    r.vis_vsz = p.seg[KVQ_SEG_V_SZ] + row * p.vszrow;
  }
  return r;
}

// Bulk prefetch into L2 of the bytes at p, in whole 16-byte granules.
__device__ __forceinline__ void prefetch_bytes(const void* p, uint32_t bytes) {
  const uint64_t p0 = reinterpret_cast<uint64_t>(p) & ~15ull;
  const uint64_t p1 = (reinterpret_cast<uint64_t>(p) + bytes + 15) & ~15ull;
  prefetch_l2(reinterpret_cast<const void*>(p0), static_cast<uint32_t>(p1 - p0));
}

}  // namespace kvq
