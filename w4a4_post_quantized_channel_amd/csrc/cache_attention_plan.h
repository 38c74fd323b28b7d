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

// Blocks that a plan is made for: those of max_len keys; from 1024 on in 64
// steps an octave, so that all plans up to a length can be looked at.
constexpr int64_t kEveryBlock = 1024;
inline int64_t plan_step(int64_t blocks) {                   // from ``blocks`` to the next
  int64_t step = 1;
  for (int64_t n = kEveryBlock; n <= blocks; n *= 2) step = step == 1 ? kEveryBlock / 64 : 2 * step;
  return step;
}
inline int64_t plan_blocks(int64_t max_len) {
  const int64_t blocks = (max_len + kCacheBlock - 1) / kCacheBlock, step = plan_step(blocks - 1);
  return (blocks + step - 1) / step * step;
}

// The kernels of a head width.  16 and 32 rows: every wave takes key blocks of
// its own, so an iteration covers ``waves`` blocks; more rows: the waves share a
// block.  Fitted numbers, no residencies: fit, workgroups of a CU that ``us`` is
// for (four of {16, 4} have room at width 64, three at 128, two at 256).
// Microseconds: us, an iteration with that many on all CUs; start, a workgroup's
// start and end; next, what those of the workgroups behind it add.
struct CacheAttnShape {
  int rows, waves, fit;
  double us, start, next;
};
constexpr int kCacheShapes = 4;
constexpr CacheAttnShape kCacheAttnShapes[3][kCacheShapes] = {
    {{16, 4, 2, 1.85, 6, 1}, {16, 8, 2, 3.3, 6, 3}, {32, 8, 1, 2.2, 6, 6}, {256, 8, 1, 1.1, 7.5, 7.5}},    // D = 64
    {{16, 4, 2, 2.7, 6, 1}, {16, 8, 1, 2.0, 6, 6}, {32, 8, 1, 3.4, 6, 6}, {256, 8, 1, 1.85, 7.5, 7.5}},    // D = 128
    {{16, 4, 2, 4.5, 6, 1}, {16, 8, 1, 5.0, 6, 6}, {128, 4, 1, 1.85, 12.5, 12.5}}};                        // D = 256
constexpr int kCacheCUs = 256;

// Fitted to measurements, in us; B x T queries, query heads over KV heads, keys:
//  width 128  8 x 50, 16 over 4, 2090: 24 with 32 rows a workgroup, 29 with 16, 33
//             with 256;  1 x 200, 8 over 1, 8192: 25 with 32, 33 with 256;
//             56 x 8, 40 over 5, 2: 14 with 16 rows and four waves, 27 with eight,
//             24 with 32 rows, 17 with 256
//  width 64   64 x 1, 32 over 8, 8192: 66 with four waves, 60 with eight;
//             1 x 1560, 16 over 16, 12480: 134 with 256 rows, 216 with 32
//  width 256  1 x 500, 8 over 1, 4096: 46 with 16 rows and eight waves, 54 with
//             four, 41 with 128 rows;  2 x 300, 4 over 4, 1500: 22, 23 and 30;
//             16 x 16, 32 over 4, 4096: 91, 79 and 58 (32 rows: never the fastest)
// Iterations (0.65 of their time where a CU holds one workgroup of two), starts,
// and the join's launch, parts and bytes (fitted with the rest: 8 TB/s, where a
// copy reaches 5.1); never less than reading the caches.  Against every tile in
// 1, 2, 4 .. 64 parts, 40 shapes drawn at random and eight single tokens with 600
// to 1200 units: 1.04 times the fastest in the geometric mean, within 5% of it in
// 38 and 20% in 44 of 48 (all eight of the latter within 3%).  The farthest: 38 x
// 1, 32 over 8 of width 128, 10541 keys: 106 for 74 in four parts; 54 x 40, 7
// over 1 of width 256, 116 keys: 24 for 17 with 128 rows; 7 x 1, 28 over 4 of
// width 128, 1528 keys: 12.6 for 9.7 with four waves in eight parts.  A
// batch of unequal histories gains nothing from more parts (64 sequences of 4096
// to 8192 keys, 32 heads over 8 of width 128: 85 in one part, 89 in two, 92 in
// three, each with its caches cold).
inline CacheAttnPlan plan_cache_attention(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len,
                                          bool split) {
  const CacheAttnShape* shapes = kCacheAttnShapes[D == 64 ? 0 : D == 128 ? 1 : 2];
  if (B * T * Hq > 1 << 22) split = false;                   // (the join, too, has fewer than 2^32 threads)
  const int64_t rows = T * (Hq / Hkv), blocks = plan_blocks(max_len);
  const double read = (double)B * Hkv * blocks * kCacheBlock * D * 1.125 / 5.3e6;   // the caches' bytes, once
  CacheAttnPlan best{};
  double best_cost = 1e300;
  for (int c = 0; c < kCacheShapes; ++c) {
    const CacheAttnShape& s = shapes[c];
    if (s.rows == 0) break;
    if (c > 0 && s.rows > shapes[c - 1].rows && rows <= shapes[c - 1].rows) break;   // a smaller tile holds them all
    const bool few = s.rows <= 32;
    const int64_t step = few ? s.waves : 1;                  // blocks of an iteration
    const int64_t tiles = (rows + s.rows - 1) / s.rows, units = B * Hkv * tiles;
    const int64_t slots = s.fit * kCacheCUs;
    int64_t most = split ? (blocks + step - 1) / step : 1;
    if (most > 64) most = 64;
    if (most > (1 << 20) / units) most = (1 << 20) / units;     // more rows than that fill the card by themselves
    if (most < 1) most = 1;
    for (int64_t parts = 1;; parts = parts * 2 < most ? parts * 2 : most) {
      const int64_t per = blocks < 1 ? 1 : (blocks + parts - 1) / parts;
      const int64_t iters = (per + step - 1) / step, rounds = (units * parts + slots - 1) / slots;
      const double work = rounds * iters * s.us * (s.fit > 1 && units * parts <= kCacheCUs ? 0.65 : 1.0);
      double cost = (work > read ? work : read) + s.start + (rounds - 1) * s.next;
      if (parts > 1) cost += 4.0 + 0.1 * parts + (double)parts * B * Hkv * rows * D * 8.0 / 8e6;
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
