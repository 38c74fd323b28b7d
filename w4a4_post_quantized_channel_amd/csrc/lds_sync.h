// Waits and copies of the 16-bit operators' LDS pipelines.
#pragma once
#include "lds_dma.h"

namespace w4a4 {

// wait_vmcnt with every LDS read of this wave returned too: what a wave needs
// before a barrier after which others may overwrite what it has read.
template <int N>
__device__ __forceinline__ void wait_vmcnt_lds() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
}

// dma16_at without a scalar offset.
__device__ __forceinline__ void dma16_v(const v4u& rs, uint32_t lds, uint32_t off) {
  const uint32_t m = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(m), "v"(off), "s"(rs)
               : "memory", "m0");
}

}  // namespace w4a4
