// The activations of the 16-bit operators, in fp32.
#pragma once
#include "../../include/w4a4.h"
#include "device_common.h"

namespace w4a4 {

// z * sigmoid(u) with sigmoid(u) = 1 / (1 + exp(-u)); exp overflows to
// infinity for very negative u, which gives the right limit 0.
__device__ __forceinline__ float times_sigmoid(float z, float u) {
  return z * __builtin_amdgcn_rcpf(1.f + expf(-u));
}

// x Phi(x) is taken as x erfc(-x / sqrt 2) / 2, which keeps its relative
// accuracy where 1 + erf cancels; the tanh form 0.5 x (1 + tanh u) is
// x sigmoid(2 u).
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case W4A4_ACT_RELU: return z < 0.f ? 0.f : z;
    case W4A4_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);
    case W4A4_ACT_GELU_TANH: return times_sigmoid(z, 1.5957691216057308f * (z + 0.044715f * (z * z) * z));
    case W4A4_ACT_SILU: return times_sigmoid(z, z);
    default: return z;
  }
}

}  // namespace w4a4
