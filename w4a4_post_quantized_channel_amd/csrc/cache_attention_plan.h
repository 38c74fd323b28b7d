// Which kernel, and how many parts of the key axis, cache_attention takes for
// a shape (host code).
#pragma once
#include <stdint.h>

namespace w4a4 {

struct CacheAttnPlan {
  int rows;      // query rows (token, head of the group) of a workgroup
  int waves;     // of a workgroup
  int tiles;     // row tiles of a sequence and KV head
  int parts;
};

constexpr int kCacheBlock = 64;   // keys of a block

// The kernels of a head width.  16 and 32 rows: every wave takes key blocks of
// its own, so an iteration covers ``waves`` blocks; more rows: the waves share a
// block.  us: an iteration, all CUs busy (fitted, see below).
struct CacheAttnShape {
  int rows, waves;
  double us;
};
constexpr int kCacheShapes = 4;
constexpr CacheAttnShape kCacheAttnShapes[3][kCacheShapes] = {
    {{16, 4, 1.6}, {16, 8, 1.3}, {32, 8, 2.2}, {256, 8, 1.1}},      // D = 64
    {{16, 4, 2.6}, {16, 8, 2.0}, {32, 8, 3.4}, {256, 8, 1.85}},     // D = 128
    {{16, 4, 5.0}, {16, 8, 4.6}, {32, 4, 4.5}, {128, 4, 2.0}}};     // D = 256
constexpr int kCacheCUs = 256;

// Microseconds, fitted to measurements (width 128, a chunk of 8 x 50, 16 heads
// over 4, 2090 keys: 24 with 32 rows a workgroup, 29 with 16, 33 with 256; width
// 64: 17, 19 and 23; width 128, 200 queries of 8 heads over 8192 keys: 25 with 32
// rows, 33 with 256; width 256, 500 queries of 8 heads over one, 4096 keys: 79
// with 32, 86 with 16, 57 with 128): iterations, start and end of a workgroup,
// and the join's launch, parts and bytes; never less than reading the caches.  A
// batch of unequal histories gains nothing from more parts (64 sequences of 4096
// to 8192 keys, 32 heads over 8: 85 us in one part, 89 in two, 92 in three, each
// with its caches cold).  Of 20 other shapes the choice was the fastest of those
// tried or within 10%, but for single tokens of width 64 over 8192 keys (66 with
// four waves, 60 with eight).
inline CacheAttnPlan plan_cache_attention(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len,
                                          bool split) {
  const CacheAttnShape* shapes = kCacheAttnShapes[D == 64 ? 0 : D == 128 ? 1 : 2];
  if (B * T * Hq > 1 << 22) split = false;                   // (the join, too, has fewer than 2^32 threads)
  const int64_t rows = T * (Hq / Hkv), blocks = (max_len + kCacheBlock - 1) / kCacheBlock;
  const double read = (double)B * Hkv * blocks * kCacheBlock * D * 1.125 / 5.3e6;   // the caches' bytes, once
  CacheAttnPlan best{};
  double best_cost = 1e300;
  for (int c = 0; c < kCacheShapes; ++c) {
    const CacheAttnShape& s = shapes[c];
    if (c > 0 && s.rows > shapes[c - 1].rows && rows <= shapes[c - 1].rows) break;   // a smaller tile holds them all
    const bool few = s.rows <= 32;
    const int64_t step = few ? s.waves : 1;                  // blocks of an iteration
    const int64_t tiles = (rows + s.rows - 1) / s.rows, units = B * Hkv * tiles;
    const int64_t slots = few && s.waves == 4 && s.rows == 16 ? 2 * kCacheCUs : kCacheCUs;
    int64_t most = split ? (blocks + step - 1) / step : 1;
    if (most > 64) most = 64;
    if (most > (1 << 20) / units) most = (1 << 20) / units;     // more rows than that fill the card by themselves
    if (most < 1) most = 1;
    for (int64_t parts = 1;; parts = parts * 2 < most ? parts * 2 : most) {
      const int64_t per = blocks < 1 ? 1 : (blocks + parts - 1) / parts;
      const int64_t iters = (per + step - 1) / step, rounds = (units * parts + slots - 1) / slots;
      const double work = rounds * iters * s.us;
      double cost = (work > read ? work : read) + rounds * 6.0;
      if (parts > 1) cost += 4.0 + 0.1 * parts + (double)parts * B * Hkv * rows * D * 8.0 / 4e6;
      if (cost < best_cost) {
        best_cost = cost;
        best = {s.rows, s.waves, (int)tiles, (int)parts};
      }
      if (parts == most) break;
    }
  }
  return best;
}

}  // namespace w4a4
