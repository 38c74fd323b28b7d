// Which kernel, tile and K split bf16_linear takes for a shape (host code).
#pragma once
#include <stdint.h>

#include "../../include/w4a4.h"

namespace w4a4 {

// Tiles, largest first.
struct TileInfo {
  int bm, bn, threads;
  double us;   // measured time of a K stage, every CU busy with one workgroup
  bool gated;
};
constexpr TileInfo kTiles[] = {{256, 320, 512, 1.95, false}, {256, 256, 512, 1.4, true}, {128, 256, 512, 0.82, true},
                               {128, 128, 512, 0.53, true},  {64, 128, 512, 0.40, true}, {32, 128, 256, 0.30, true}};
constexpr int kNumTiles = 6, kCUs = 256;

// The kernel for at most kRowsMax rows: 16 columns a workgroup.
constexpr int kRowsMax = 16, kRowsWaves = 8;

constexpr int64_t kMaxThreads = 0xFFFFFFFFll;   // of a launch

struct GemmPlan {
  bool rows;   // the kernel for few rows; the rest says what the tiles would do
  int tile, tiles_m, tiles_n, splits, pn;
};

inline GemmPlan plan_tiles(int64_t M, int64_t N, int64_t K, int act, bool split) {
  const bool gated = act == W4A4_ACT_SWIGLU;
  const int64_t stages = (K + 63) / 64;
  GemmPlan best{};
  double best_cost = 1e300;
  for (int i = 0; i < kNumTiles; ++i) {
    const TileInfo& ti = kTiles[i];
    if (gated && !ti.gated) continue;
    const int64_t bn = gated ? ti.bn / 2 : ti.bn;
    const int64_t tm = (M + ti.bm - 1) / ti.bm, tn = (N + bn - 1) / bn, tiles = tm * tn;
    if (tiles > kMaxThreads / ti.threads) continue;
    for (int64_t sp = 1; sp <= 64; sp *= 2) {
      if (sp > 1 && (!split || tiles * sp > 2 * kCUs || stages / sp < 2)) break;
      const int64_t rounds = (tiles * sp + kCUs - 1) / kCUs;
      double cost = rounds * ((stages + sp - 1) / sp * ti.us + 1.5 + ti.bm * ti.bn * 4e-5);
      if (sp > 1) cost += 3.0 + 0.1 * sp + 2.0 * sp * M * tn * ti.bn * 4.0 / 4e6;
      if (cost < best_cost) {
        best_cost = cost;
        best = {false, i, (int)tm, (int)tn, (int)sp, (int)(tn * ti.bn)};
      }
    }
  }
  return best;
}

// At most 16 rows: the kernel for few rows, or the tiles' plan `pl`.  Times in
// us in a graph, few-rows kernel / tiles, weights past the caches where they
// can be.
// * Split tiles: while K is short.  1 x 2048 x 2048 6.0 / 9.2, 16 x 2048 x 2048
//   7.4 / 9.6, 1 x 4096 x 4096 9.1 / 12.9; from there on its workgroups are
//   too few for the weights: 16 x 64 x 8192 17.3 / 10.3, 16 x 4096 x 8192
//   21.7 / 19.8, 16 x 8192 x 5120 31.9 / 22.5.
// * Unsplit tiles on less than half the card (short K, or no workspace): always.
//   16 x 2048 x 1024 5.4 / 8.4, 16 x 8192 x 1024 7.6 / 8.8, 1 x 2048 x 8192
//   12.5 / 36.0.
// * Unsplit tiles on more than that: up to four rows of more than 1024.
//   1 x 32768 x 4096 48.3 / 60.6, 1 x 32768 x 8192 91.2 / 116, 4 x 32768 x 4096
//   56.1 / 60.7; but 1 x 32768 x 1024 18.5 / 15.3, 6 x 20480 x 4096 39.7 /
//   35.5, 16 x 32768 x 8192 145 / 120, 16 x 65536 x 5120 208 / 114.  (1 x 32768
//   x 5120, 65.3 / 57.9, and 8 x 16384 x 8192 with SwiGLU, 110 / 124, go the
//   wrong way.)
inline bool rows_kernel(int64_t M, int64_t K, const GemmPlan& pl) {
  if (M > kRowsMax) return false;
  if (pl.splits > 1) return K <= 4096;
  return (int64_t)pl.tiles_m * pl.tiles_n <= kCUs / 2 || (M <= 4 && K > 1024);
}

// workspace: K may be split over workgroups.
inline GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, int act, bool workspace) {
  GemmPlan pl = plan_tiles(M, N, K, act, true);
  pl.rows = rows_kernel(M, K, pl);
  if (!pl.rows && pl.splits > 1 && !workspace) {
    pl = plan_tiles(M, N, K, act, false);
    pl.rows = rows_kernel(M, K, pl);
  }
  return pl;
}

}  // namespace w4a4
