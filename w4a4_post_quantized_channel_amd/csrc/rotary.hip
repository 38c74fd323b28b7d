// Rotary positions with several axes.
//
// Mathematics.  A pair (u, w) of a head is turned by pos * f.  The table holds
// f / (2 pi) as hi + lo, so the angle in turns is pos * hi + pos * lo; the
// rounding error of the first product is recovered by an fma, whole turns are
// dropped exactly, and what remains is below half a turn in 24 bits: the sine
// of position 10^6 is as good as that of position 1.
//
// A thread takes one pair of a token and applies it to every head.
#include "cache.h"
#include "device_common.h"

namespace w4a4 {

namespace {

__device__ __forceinline__ void sincos_of(float pos, float hi, float lo, float& c, float& s) {
  const float p = pos * hi;
  const float e = __builtin_fmaf(pos, hi, -p);              // exact
  const float turn = (p - __builtin_rintf(p)) + __builtin_fmaf(pos, lo, e);
  sincospif(2.f * turn, &s, &c);
}

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? ((const float*)p)[i] : bf16_bits_to_f32(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void store1(void* p, int64_t i, bool f32, float v) {
  if (f32) ((float*)p)[i] = v;
  else ((__bf16*)p)[i] = (__bf16)v;
}

__global__ void __launch_bounds__(256) rotary_kernel(w4a4_rotary a, int pairs, int items) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * items) return;
  const int64_t m = i / items;
  const int it = (int)(i % items);
  const bool f32 = a.dtype == W4A4_DT_F32;
  const int heads = (int)(a.Hq + a.Hk);
  if (it >= pairs) {                                          // a channel behind the pairs
    const int ch = 2 * pairs + it - pairs;
    for (int h = 0; h < heads; ++h) {
      const bool q = h < a.Hq;
      const int64_t x = q ? m * a.q_sm + h * a.q_sh : m * a.k_sm + (h - a.Hq) * a.k_sh;
      const int64_t y = q ? m * a.qo_sm + h * a.qo_sh : m * a.ko_sm + (h - a.Hq) * a.ko_sh;
      store1(q ? a.q_out : a.k_out, y + ch, f32, load1(q ? a.q : a.k, x + ch, f32));
    }
    return;
  }
  int axis = 0, end = a.sections[0];
  while (it >= end) end += a.sections[++axis];
  const int64_t pi = m * a.pos_sm + axis;
  const float pos = a.pos_dtype == W4A4_DT_I32 ? (float)((const int32_t*)a.pos)[pi] : ((const float*)a.pos)[pi];
  float c, s;
  sincos_of(pos, a.table[2 * it], a.table[2 * it + 1], c, s);
  const int c0 = a.pairs == W4A4_PAIRS_ADJACENT ? 2 * it : it;
  const int c1 = a.pairs == W4A4_PAIRS_ADJACENT ? 2 * it + 1 : it + pairs;
  for (int h = 0; h < heads; ++h) {
    const bool q = h < a.Hq;
    const int64_t x = q ? m * a.q_sm + h * a.q_sh : m * a.k_sm + (h - a.Hq) * a.k_sh;
    const int64_t y = q ? m * a.qo_sm + h * a.qo_sh : m * a.ko_sm + (h - a.Hq) * a.ko_sh;
    const void* src = q ? a.q : a.k;
    void* dst = q ? a.q_out : a.k_out;
    const float u = load1(src, x + c0, f32), w = load1(src, x + c1, f32);
    store1(dst, y + c0, f32, u * c - w * s);
    store1(dst, y + c1, f32, u * s + w * c);
  }
}

}  // namespace

hipError_t launch_rotary_axes(const w4a4_rotary& r, hipStream_t st) {
  const int pairs = r.sections[0] + r.sections[1] + r.sections[2] + r.sections[3];
  const int items = pairs + (int)r.D - 2 * pairs;
  rotary_kernel<<<(unsigned)((r.M * items + 255) / 256), 256, 0, st>>>(r, pairs, items);
  return hipGetLastError();
}

}  // namespace w4a4
