// Launchers of the operators around the 4-bit key/value cache behind the C
// ABI (host side).  Sizes, strides and pointers as checked by the entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/w4a4.h"

namespace w4a4 {

// kv_cache.hip
struct CacheIo {
  w4a4_kvcache c;
  int64_t M;
  const int32_t* slots;
  int f32;                     // else bf16
  void *k, *v;                 // read (append) or written (read)
  int64_t k_sm, k_sh, v_sm, v_sh;
};
hipError_t launch_cache_append(const CacheIo& a, hipStream_t st);
hipError_t launch_cache_read(const CacheIo& a, hipStream_t st);

// cache_attention.hip: workspace null or of cache_attention_workspace() bytes.
hipError_t launch_cache_attention(const w4a4_kvcache& c, const w4a4_cache_attn& a, void* workspace, hipStream_t st);
size_t cache_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len);

// rotary.hip
hipError_t launch_rotary_axes(const w4a4_rotary& r, hipStream_t st);

// gated_norm.hip
hipError_t launch_gated_norm(const w4a4_gated& g, hipStream_t st);

}  // namespace w4a4
