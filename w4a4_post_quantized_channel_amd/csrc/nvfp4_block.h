// Exactly rounded NVFP4 quantization of 16 values, shared by the activation
// quantizer and the key/value cache.
#pragma once
#include "device_common.h"

namespace w4a4 {

constexpr float kTinyStep = 8.271806125530277e-25f;  // 2^-80

// RN(a / b) given r = RN(1 / b), for b >= 2^-80 and finite a.
__device__ __forceinline__ float div_rn(float a, float b, float r) {
  float q = a * r;
  float t = __builtin_fmaf(-b, q, a);
  q = __builtin_fmaf(t, r, q);
  t = __builtin_fmaf(-b, q, a);
  return __builtin_fmaf(t, r, q);
}

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

// Boundary screen for E2M1 quotients taken with one multiply,
// q0 = RN(v * RN(1/D)), which is within three representable steps of
// RN(v / D).  Every E2M1 rounding boundary (0.25, 0.75, 1.25, 1.75, 2.5,
// 3.5, 5) has at most three significant bits, so its low 16 bits are zero.
// If no q0 of a slot has its low 16 bits within 4 of a multiple of 2^16, no
// boundary lies between q0 and RN(v / D) and both give the same code;
// otherwise the slot is redone exactly.  Returns the minimum over the slot
// of ((bits(q0) + 4) mod 2^16).
__device__ __forceinline__ uint32_t near_boundary(const float (&q)[16]) {
  us2 mn = (us2){0xFFFF, 0xFFFF};
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const uint32_t p = __builtin_amdgcn_perm(__float_as_uint(q[i + 1]), __float_as_uint(q[i]), 0x05040100u);
    us2 t = __builtin_bit_cast(us2, p) + (us2){4, 4};
    mn = __builtin_elementwise_min(mn, t);
  }
  return (uint32_t)__builtin_elementwise_min(mn.x, mn.y);
}

constexpr float kBig = 1.2676506002282294e30f;     // 2^100
constexpr float kMinA = 8.077935669463161e-28f;    // 2^-90: dividends at or above keep residuals normal

// One NVFP4 block of 16 transformed values y = v * fl (fl a power of two,
// possibly negative): E4M3 block scale e and the 16 E2M1 codes packed in two
// dwords (low nibble first).  stab holds (S, RN(1/S)) per E4M3 code; live
// says whether the block exists (a screened slot past the end of a row must
// not take the exact path).
__device__ __forceinline__ uint32_t nvfp4_block16(const float (&v)[16], float fl, float g, float rg, bool g_fast,
                                                  const float2* stab, bool live, uint2& codes) {
  float mv = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) mv = fmaxf(mv, __builtin_fabsf(v[i]));
  const float m = mv * __builtin_fabsf(fl);                                             // max |y| of the block
  const float sb = m >= kMinA ? div_rn(m, 6.0f, 0.16666667163372040f) : m / 6.0f;      // RN(m / 6)
  const float sv = (g_fast && sb >= kMinA) ? div_rn(sb, g, rg) : sb / g;                // RN(sb / g)
  const uint32_t e = f32_to_e4m3_sat(sv);
  const float2 SR = stab[e];
  uint32_t w[2] = {0u, 0u};
  if (SR.x > 0.f) {
    const bool fast = SR.x >= kTinyStep && SR.x <= kBig;
    const float D = SR.x / fl, rD = SR.y * fl;   // exact power-of-two rescaling
    float q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = v[i] * rD;
    if (live && (!fast || near_boundary(q) <= 8u)) {
      if (fast) {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = div_rn(v[i], D, rD);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = (v[i] * fl) / SR.x;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t d = 0;
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[8 * h + 0], q[8 * h + 1], 1.0f, 0);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[8 * h + 2], q[8 * h + 3], 1.0f, 1);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[8 * h + 4], q[8 * h + 5], 1.0f, 2);
      d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, q[8 * h + 6], q[8 * h + 7], 1.0f, 3);
      // the converter writes -0 as 0x8; the packed format uses +0
      const uint32_t mag = d & 0x77777777u;
      const uint32_t nz = (mag + 0x77777777u) & 0x88888888u;
      w[h] = mag | (d & nz);
    }
  }
  codes = make_uint2(w[0], w[1]);
  return e;
}

}  // namespace w4a4
