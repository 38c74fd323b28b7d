// The activations of the 16-bit operators, in fp32.
#pragma once
#include "../../include/w4a4.h"
#include "device_common.h"

namespace w4a4 {

// exp(x) to an ulp or two: the hardware's exp2 of x log2(e), with the part of
// the product that rounding lost (and of the constant) put back to first
// order.  Arguments past the normal range are clamped to its ends.
__device__ __forceinline__ float exp_f32(float x) {
  x = __builtin_amdgcn_fmed3f(x, -87.f, 88.f);
  const float t = x * 1.44269502f;
  const float r = __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, 1.44269502f, -t));
  const float y = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(y * r, 0.693147181f, y);
}

// z * sigmoid(u), sigmoid(u) = 1 / (1 + exp(-u)).  Past u = -87.3 the
// reciprocal would be subnormal, and the instruction gives zero, the limit.
__device__ __forceinline__ float times_sigmoid(float z, float u) {
  return z * __builtin_amdgcn_rcpf(1.f + exp_f32(-u));
}

// Activations by the code they need: none and ReLU; the sigmoid family; the
// error function.  KIND is a template parameter where the activation is
// unrolled many times.
enum { ACT_KIND_PLAIN = 0, ACT_KIND_SIGMOID = 1, ACT_KIND_ERF = 2 };
__host__ __device__ constexpr int act_kind(int act) {
  return act == W4A4_ACT_GELU ? ACT_KIND_ERF : act <= W4A4_ACT_RELU ? ACT_KIND_PLAIN : ACT_KIND_SIGMOID;
}

// x Phi(x) is taken as x erfc(-x / sqrt 2) / 2, which keeps its relative
// accuracy where 1 + erf cancels; the tanh form 0.5 x (1 + tanh u) is
// x sigmoid(2 u).
template <int KIND>
__device__ __forceinline__ float activate_kind(float z, int act) {
  if constexpr (KIND == ACT_KIND_PLAIN) return act == W4A4_ACT_RELU && z < 0.f ? 0.f : z;
  else if constexpr (KIND == ACT_KIND_ERF) return 0.5f * z * erfcf(z * -0.70710678118654752f);
  else {
    const float u = act == W4A4_ACT_GELU_TANH ? 1.5957691216057308f * __builtin_fmaf(0.044715f * z * z, z, z) : z;
    return times_sigmoid(z, u);
  }
}

__device__ __forceinline__ float activate(float z, int act) {
  const int kind = act_kind(act);
  if (kind == ACT_KIND_PLAIN) return activate_kind<ACT_KIND_PLAIN>(z, act);
  if (kind == ACT_KIND_ERF) return activate_kind<ACT_KIND_ERF>(z, act);
  return activate_kind<ACT_KIND_SIGMOID>(z, act);
}

}  // namespace w4a4
