// Which tile, and how many parts of the key axis, prefix_attention takes for a
// shape (host code).
#pragma once
#include <stdint.h>

namespace w4a4 {

struct AttnPlan {
  int cfg;     // index of the (WQ, WK) pair
  int rpt, tiles, parts, np, ns;
  int per;     // blocks of a part
};

struct AttnShape {
  int wq, wk, bn;
  double us;   // an iteration of a workgroup, all CUs busy
};
// (WQ, WK, BN) per head width; the kernels are instantiated from it.  The
// times of D = 128 are fitted to measurements (see plan_attention); those of
// the other widths are estimates that rank the tiles of one width.  An
// iteration of the first tile of D = 256 has measured 6 us, not 3, where it
// has half the card to itself.
constexpr AttnShape kShapes[3][4] = {
    {{1, 8, 64, 2.0}, {2, 4, 64, 1.8}, {4, 2, 64, 2.0}, {8, 1, 64, 1.5}},      // D = 64
    {{1, 8, 32, 3.05}, {2, 4, 32, 2.3}, {4, 2, 64, 3.0}, {8, 1, 64, 2.0}},     // D = 128
    {{2, 2, 32, 3.0}, {4, 1, 32, 2.6}, {0, 0, 0, 0.0}, {0, 0, 0, 0.0}}};       // D = 256
constexpr int kAttnCUs = 256;

inline AttnPlan plan_attention(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t P, int64_t S, bool split) {
  const AttnShape* sh = kShapes[D == 64 ? 0 : D == 128 ? 1 : 2];
  const int64_t tg = T * (Hq / Hkv), rows = B * tg;
  AttnPlan best{};
  double best_cost = 1e300;
  for (int c = 0; c < 4; ++c) {
    if (sh[c].wq == 0) break;
    const int64_t R = 32 * sh[c].wq;
    const int64_t rpt = tg <= R ? R / tg * tg : R;
    const int64_t tiles = (rows + rpt - 1) / rpt;
    const int64_t np = (P + sh[c].bn - 1) / sh[c].bn, ns = (S + sh[c].bn - 1) / sh[c].bn;
    const int64_t nseq = tg <= R ? rpt / tg : (R + tg - 1) / tg + (R % tg != 0);
    const int64_t total = np + (nseq < B ? nseq : B) * ns;
    const int64_t units = Hkv * tiles;
    // Parts: up to one round of the card's CUs, with at least one block per
    // key group, halved as long as that is cheaper.
    const int64_t cap = (total + sh[c].wk - 1) / sh[c].wk;
    int64_t most = split && units < kAttnCUs ? kAttnCUs / units : 1;
    if (most > cap) most = cap < 1 ? 1 : cap;
    for (int64_t want = most; want >= 1; want /= 2) {
      const int64_t blocks = total < 1 ? 1 : (total + want - 1) / want;
      const int64_t parts = total < 1 ? 1 : (total + blocks - 1) / blocks;
      const int64_t iters = (blocks + sh[c].wk - 1) / sh[c].wk, rounds = (units * parts + kAttnCUs - 1) / kAttnCUs;
      // Microseconds, fitted to measurements (D = 128: a decoding batch of 64
      // over 8192 keys 40 us as planned, 46 with 32-row tiles; a chunk of 8 x
      // 50 over 2040 keys 26 as planned, 29 with 64-row tiles): iterations,
      // start and end of a workgroup, and the join's launch, parts and bytes.
      double cost = rounds * (iters * sh[c].us + 5.0);
      if (parts > 1) cost += 3.5 + 0.1 * parts + parts * Hkv * rows * (double)D * 8.0 / 4e6;
      if (cost < best_cost) {
        best_cost = cost;
        best = {c, (int)rpt, (int)tiles, (int)parts, (int)np, (int)ns, (int)blocks};
      }
    }
  }
  return best;
}

}  // namespace w4a4
