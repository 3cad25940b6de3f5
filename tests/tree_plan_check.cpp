// Host-side check of the tree call's split (kvq_tree_plan.h) over every mix of
// up to 170 units of the three classes and many lengths: a class without
// units, and every class when there are as many units as CTAs or one tile, has
// one CTA a unit; no unit has more CTAs than tiles; the CTAs fit one wave of the
// SMs; and no smaller bound on the longest CTA fits.  Prints "ok" or the first
// failure.
#include <cstdio>
#include <cstring>

#include "kvq_tree_plan.h"

int main() {
  using namespace kvq::tree;
  long long plans = 0, split = 0;
  for (int n_sm : {1, 2, 76, 148, 152, 160, 200})
    for (int nblk : {1, 2, 3})
      for (int prot = 0; prot <= 20; prot += 1 + prot / 4)
        for (int konly = 0; konly <= 12; konly += 1 + konly / 2)
          for (int packed = 0; packed <= 170; packed += 1 + packed / 16)
            for (int tiles : {0, 1, 2, 3, 7, 25, 49, 130, 1000}) {
              if (prot + konly + packed == 0 || prot + konly + packed > KVQ_MAX_HEADS) continue;
              kvq_layout L;
              std::memset(&L, 0, sizeof(L));
              L.d.B = 1;
              L.n_prot = prot;
              L.n_konly = konly;
              L.n_packed = packed;
              int32_t U[3], S[3], head0[3];
              plan_splits(&L, nblk, tiles, n_sm, U, S, head0);
              const int n[3] = {prot, konly, packed}, cap = n_sm < kMaxSplitCtas ? n_sm : kMaxSplitCtas;
              long long units = 0, ctas = 0, per_unit_longest = 0;
              bool ok = head0[0] == 0 && head0[1] == prot && head0[2] == prot + konly, any = false;
              for (int k = 0; k < 3; ++k) {
                ok &= U[k] == n[k] * nblk && S[k] >= 1 && (S[k] == 1 || S[k] <= tiles);
                ok &= U[k] > 0 || S[k] == 1;
                units += U[k];
                ctas += static_cast<long long>(U[k]) * S[k];
                any |= S[k] > 1;
                if (U[k] && tiles > 0) {
                  const long long t = static_cast<long long>(kTileCost[k]) * ((tiles + S[k] - 1) / S[k]);
                  if (t > per_unit_longest) per_unit_longest = t;
                }
              }
              if (units >= cap || tiles <= 1) ok &= !any;
              else ok &= ctas <= cap;
              // a CTA may be no longer than the best whole split allows
              if (any && per_unit_longest > 0) {
                long long need = 0;
                for (int k = 0; k < 3; ++k) {
                  const long long m = (per_unit_longest - 1) / kTileCost[k];
                  if (U[k]) need += m < 1 ? cap + 1 : U[k] * ((tiles + m - 1) / m);
                }
                ok &= need > cap;
              }
              if (!ok) {
                std::printf("SMs %d, blocks %d, units %d %d %d, tiles %d: CTAs a unit %d %d %d\n", n_sm, nblk, U[0], U[1], U[2],
                            tiles, S[0], S[1], S[2]);
                return 1;
              }
              ++plans;
              split += any;
            }
  std::printf("ok %lld plans, %lld of them split\n", plans, split);
  return 0;
}
