// Which kernel, and how many parts of the key axis, cache_attention takes for
// a shape (host code).
#pragma once
#include <stdint.h>

namespace w4a4 {

struct CacheAttnPlan {
  int rows;      // query rows (token, head of the group) of a workgroup
  int tiles;     // row tiles of a sequence and KV head
  int parts;
};

constexpr int kFewWaves = 4;      // waves of a workgroup, each with key blocks of its own
constexpr int kCacheBlock = 64;   // keys of a block

inline CacheAttnPlan plan_cache_attention(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len,
                                          bool split) {
  const int64_t rows = T * (Hq / Hkv);
  CacheAttnPlan p;
  p.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : D == 256 ? 128 : 256;
  p.tiles = (int)((rows + p.rows - 1) / p.rows);
  const int64_t units = B * Hkv * p.tiles, blocks = (max_len + kCacheBlock - 1) / kCacheBlock;
  // Parts: up to three workgroups of the few-row kernel a CU with at least a
  // block a wave, or one of the many-row kernel.
  const bool few = p.rows <= 32;
  const int64_t most = few ? (blocks + kFewWaves - 1) / kFewWaves : (blocks + 1) / 2;
  int64_t parts = split ? (few ? 768 : 256) / units : 1;
  if (parts > most) parts = most;
  p.parts = (int)(parts < 1 ? 1 : parts);
  return p;
}

}  // namespace w4a4
