// kvq_tree_plan.h -- how the tree-attention call shares its units out over the
// CTAs (host code, no CUDA types).
#pragma once

#include <algorithm>
#include <cstdint>

#include "kvq.h"

namespace kvq {
namespace tree {

constexpr int kMaxSplitCtas = 160;  // CTAs of a call whose units are split (workspace slots)

// How many CTAs share a unit of each class: one wave of CTAs on the GPU's SMs
// (a CTA fills an SM), the units of a class in equal whole parts, so that the
// longest CTA is as short as such parts allow (what they leave over idles: 80
// packed units of 130 tiles take 80 of 152 SMs).
// A tile of bf16 rows takes about twice as long as a packed one where rows
// come from HBM (16K x 8: 3.6 against 1.7 us).  With more units than SMs every
// unit has one CTA, the dearest first.
constexpr int kTileCost[3] = {4, 3, 2};  // protected, K-only, packed
inline void plan_splits(const kvq_layout* L, int nblk, int tiles, int n_sm, int32_t (&U)[3], int32_t (&S)[3],
                        int32_t (&head0)[3]) {
  const int n[3] = {L->n_prot, L->n_konly, L->n_packed};
  const int cap = std::min(n_sm, kMaxSplitCtas);
  int64_t units = 0;
  for (int k = 0, h = 0; k < 3; ++k) {
    U[k] = L->d.B * n[k] * nblk;
    S[k] = 1;
    head0[k] = h;
    h += n[k];
    units += U[k];
  }
  if (units >= cap || tiles <= 1) return;
  // CTAs when no CTA of class k has more than m[k] tiles
  auto splits = [&](int m) { return (tiles + m - 1) / m; };
  auto ctas = [&](const int (&m)[3]) {
    int64_t c = 0;
    for (int k = 0; k < 3; ++k) c += static_cast<int64_t>(U[k]) * splits(m[k]);
    return c;
  };
  int lo = kTileCost[0], hi = kTileCost[0] * tiles;  // the longest CTA's time: hi always fits
  int m[3];
  auto within = [&](int x) {
    for (int k = 0; k < 3; ++k) m[k] = std::min(tiles, x / kTileCost[k]);
    return ctas(m) <= cap;
  };
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (within(mid)) hi = mid;
    else lo = mid + 1;
  }
  within(hi);
  for (bool more = true; more;) {  // what is left over: fewer tiles for any class
    more = false;
    for (int k = 2; k >= 0; --k)
      while (U[k] && m[k] > 1) {
        --m[k];
        if (ctas(m) > cap) {
          ++m[k];
          break;
        }
        more = true;
      }
  }
  for (int k = 0; k < 3; ++k)
    if (U[k]) S[k] = splits(m[k]);  // a class without units stays at 1: nothing of it is split
}

}  // namespace tree
}  // namespace kvq
