// Rotary positions with several axes.
//
// Mathematics.  A pair (u, w) of a head is turned by pos * f.  The table holds
// f / (2 pi) as hi + lo, so the angle in turns is pos * hi + pos * lo; the
// rounding error of the first product is recovered by an fma, whole turns are
// dropped exactly, and what remains is below half a turn in 24 bits: the sine
// of position 10^6 is as good as that of position 1.  An int32 position enters
// as fp32 and what that rounds off.
//
// A thread takes eight channels (16 bytes of bf16) of one token, or eight pairs
// where the halves of a head pair up, computes their sines once and applies them
// to its heads one after the other, four loads in flight.  Heads are cut into
// groups until there are enough workgroups; a pair's sines are then computed
// once a group.  Widths or pairs that are no multiples of eight: one pair a
// thread.
//
// Bound by memory: 12480 tokens of 16 + 16 heads of 128 in bf16 (204 MB) take 42
// us, 4.9 TB/s; a thread per pair took 96.  Heads of 72 with all 36 pairs in
// halves, which no eight pairs split, go by one pair a thread: 36 us, 3.2 TB/s,
// where adjacent pairs of the same width take 24.  Few tokens: 400 of 16 + 4 heads
// take 6 us, most of it the table entries and positions of a thread's eight pairs
// (four of adjacent ones), which are loaded under each pair's condition, one pair
// after the other.
#include "cache.h"
#include "device_common.h"
#include "divisor.h"

namespace w4a4 {

namespace {

typedef float v8f __attribute__((ext_vector_type(8)));

// A position: what fp32 holds of it, and the rest of an int32.
struct Pos {
  float x, rest;
};
__device__ __forceinline__ void sincos_of(const Pos& pos, float hi, float lo, float& c, float& s) {
  const float p = pos.x * hi;
  const float e = __builtin_fmaf(pos.x, hi, -p);            // exact
  const float turn = (p - __builtin_rintf(p)) + __builtin_fmaf(pos.rest, hi, __builtin_fmaf(pos.x, lo, e));
  sincospif(2.f * turn, &s, &c);
}

// 16 bytes at the alignment of their elements, which is all that global memory asks for.
typedef int v4i_of_bf16 __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 v8bf_of_bf16 __attribute__((ext_vector_type(8), aligned(2)));
typedef float v4f_of_f32 __attribute__((ext_vector_type(4), aligned(4)));

template <bool F32>
struct Row8;   // eight channels
template <>
struct Row8<false> {
  v4i d;
  __device__ __forceinline__ void load(const void* p, int64_t i) { d = *reinterpret_cast<const v4i_of_bf16*>((const uint16_t*)p + i); }
  __device__ __forceinline__ float get(int k) const {
    return __uint_as_float(k & 1 ? (uint32_t)d[k / 2] & 0xFFFF0000u : (uint32_t)d[k / 2] << 16);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
    const v8f a = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    *reinterpret_cast<v8bf_of_bf16*>((__bf16*)p + i) = __builtin_convertvector(a, v8bf);
  }
};
template <>
struct Row8<true> {
  v4f d[2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    d[0] = reinterpret_cast<const v4f_of_f32*>((const float*)p + i)[0];
    d[1] = reinterpret_cast<const v4f_of_f32*>((const float*)p + i)[1];
  }
  __device__ __forceinline__ float get(int k) const { return d[k / 4][k % 4]; }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
    reinterpret_cast<v4f_of_f32*>((float*)p + i)[0] = (v4f){v[0], v[1], v[2], v[3]};
    reinterpret_cast<v4f_of_f32*>((float*)p + i)[1] = (v4f){v[4], v[5], v[6], v[7]};
  }
};

struct RotaryArgs {
  w4a4_rotary a;
  int pairs, items;   // items of a token: vectors (or pairs and single channels)
  int heads;          // of a group
  Divisor by;         // items
};

__device__ __forceinline__ Pos position(const w4a4_rotary& a, int64_t m, int axis) {
  const int64_t i = m * a.pos_sm + axis;
  if (a.pos_dtype != W4A4_DT_I32) return {((const float*)a.pos)[i], 0.f};
  const int n = ((const int32_t*)a.pos)[i];
  const float x = fminf((float)n, 2147483520.f);             // (the largest fp32 number that is an int32)
  return {x, (float)(n - (int)x)};
}
// Token and item of element i.
__device__ __forceinline__ int64_t token_of(const RotaryArgs& p, int64_t i, bool small, int& it) {
  if (small) return div_by((int)i, p.by, it);
  const int64_t m = i / p.items;
  it = (int)(i - m * p.items);
  return m;
}
__device__ __forceinline__ int axis_of(const w4a4_rotary& a, int pair) {
  const int e0 = a.sections[0], e1 = e0 + a.sections[1], e2 = e1 + a.sections[2];
  return (pair >= e0) + (pair >= e1) + (pair >= e2);
}
// Element offsets of a token's head in its input and output.
__device__ __forceinline__ void offsets(const w4a4_rotary& a, int64_t m, int h, const void*& src, void*& dst, int64_t& x, int64_t& y) {
  const bool q = h < a.Hq;
  const int g = q ? h : h - (int)a.Hq;
  src = q ? a.q : a.k;
  dst = q ? a.q_out : a.k_out;
  x = m * (q ? a.q_sm : a.k_sm) + g * (q ? a.q_sh : a.k_sh);
  y = m * (q ? a.qo_sm : a.ko_sm) + g * (q ? a.qo_sh : a.ko_sh);
}

template <bool F32, bool HALVES>
__global__ void __launch_bounds__(256) rotary_vec_kernel(RotaryArgs p) {
  const w4a4_rotary& a = p.a;
  constexpr int AT = F32 ? 2 : 4;                              // heads loaded together
  const int64_t total = a.M * p.items;
  const int h0 = blockIdx.y * p.heads, h1 = min(h0 + p.heads, (int)(a.Hq + a.Hk));
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    int it;
    const int64_t m = token_of(p, i, total <= INT32_MAX, it);
    // channels c0 .. c0 + 7 and, for halves, their partners c1 .. c1 + 7
    const bool turned = HALVES ? it < p.pairs / 8 : true;
    const int c0 = HALVES && !turned ? 2 * p.pairs + (it - p.pairs / 8) * 8 : it * 8, c1 = c0 + p.pairs;
    constexpr int NP = HALVES ? 8 : 4;
    Row8<F32> u[AT], w[AT];
    auto fetch = [&](int h) {
#pragma unroll
      for (int k = 0; k < AT; ++k) {
        if (h + k >= h1) break;
        const void* src;
        void* dst;
        int64_t x, y;
        offsets(a, m, h + k, src, dst, x, y);
        u[k].load(src, x + c0);
        if (HALVES && turned) w[k].load(src, x + c1);
      }
    };
    fetch(h0);
    float c[NP], s[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int pair = HALVES ? c0 + k : c0 / 2 + k;
      c[k] = 1.f;
      s[k] = 0.f;
      if (turned && pair < p.pairs) {
        const float2 f = reinterpret_cast<const float2*>(a.table)[pair];
        sincos_of(position(a, m, axis_of(a, pair)), f.x, f.y, c[k], s[k]);
      }
    }
    for (int h = h0; h < h1; h += AT) {
      if (h > h0) fetch(h);
#pragma unroll
      for (int n = 0; n < AT; ++n) {
        if (h + n >= h1) break;
        const void* src;
        void* dst;
        int64_t x, y;
        offsets(a, m, h + n, src, dst, x, y);
        float v[8];
        if constexpr (HALVES) {
          if (!turned) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = u[n].get(k);
            Row8<F32>::store(dst, y + c0, v);
            continue;
          }
          float z[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[k] = u[n].get(k) * c[k] - w[n].get(k) * s[k];
            z[k] = u[n].get(k) * s[k] + w[n].get(k) * c[k];
          }
          Row8<F32>::store(dst, y + c0, v);
          Row8<F32>::store(dst, y + c1, z);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e = u[n].get(2 * k), f = u[n].get(2 * k + 1);
            const bool turn = c0 / 2 + k < p.pairs;           // else as it is, infinities too
            v[2 * k] = turn ? e * c[k] - f * s[k] : e;
            v[2 * k + 1] = turn ? e * s[k] + f * c[k] : f;
          }
          Row8<F32>::store(dst, y + c0, v);
        }
      }
    }
  }
}

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? ((const float*)p)[i] : bf16_bits_to_f32(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void store1(void* p, int64_t i, bool f32, float v) {
  if (f32) ((float*)p)[i] = v;
  else ((__bf16*)p)[i] = (__bf16)v;
}

__global__ void __launch_bounds__(256) rotary_kernel(RotaryArgs p) {
  const w4a4_rotary& a = p.a;
  const bool f32 = a.dtype == W4A4_DT_F32;
  const int64_t total = a.M * p.items;
  const int h0 = blockIdx.y * p.heads, h1 = min(h0 + p.heads, (int)(a.Hq + a.Hk));
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    int it;
    const int64_t m = token_of(p, i, total <= INT32_MAX, it);
    const bool turned = it < p.pairs;                          // else a channel behind the pairs
    float c = 1.f, s = 0.f;
    if (turned) sincos_of(position(a, m, axis_of(a, it)), a.table[2 * it], a.table[2 * it + 1], c, s);
    const int c0 = !turned ? p.pairs + it : a.pairs == W4A4_PAIRS_ADJACENT ? 2 * it : it;
    const int c1 = a.pairs == W4A4_PAIRS_ADJACENT ? 2 * it + 1 : it + p.pairs;
    for (int h = h0; h < h1; ++h) {
      const void* src;
      void* dst;
      int64_t x, y;
      offsets(a, m, h, src, dst, x, y);
      const float u = load1(src, x + c0, f32);
      if (turned) {
        const float w = load1(src, x + c1, f32);
        store1(dst, y + c0, f32, u * c - w * s);
        store1(dst, y + c1, f32, u * s + w * c);
      } else {
        store1(dst, y + c0, f32, u);
      }
    }
  }
}

}  // namespace

hipError_t launch_rotary_axes(const w4a4_rotary& r, hipStream_t st) {
  RotaryArgs p{};
  p.a = r;
  p.pairs = r.sections[0] + r.sections[1] + r.sections[2] + r.sections[3];
  const int D = (int)r.D, heads = (int)(r.Hq + r.Hk);
  const bool f32 = r.dtype == W4A4_DT_F32, halves = r.pairs == W4A4_PAIRS_HALVES;
  const bool vec = D % 8 == 0 && (!halves || p.pairs % 8 == 0);
  p.items = vec ? (halves ? D / 8 - p.pairs / 8 : D / 8) : D - p.pairs;
  p.by = divisor(p.items);
  int64_t blocks = (r.M * p.items + 255) / 256;
  // Groups of heads, down to four, until there are 1024 workgroups.
  int groups = 1;
  while (groups * 4 < heads && blocks * groups < 1024) groups *= 2;
  p.heads = (heads + groups - 1) / groups;
  if (blocks > 1 << 20) blocks = 1 << 20;                      // longer inputs are walked
  const dim3 grid((unsigned)blocks, (unsigned)((heads + p.heads - 1) / p.heads));
  if (!vec) rotary_kernel<<<grid, 256, 0, st>>>(p);
  else if (halves) f32 ? rotary_vec_kernel<true, true><<<grid, 256, 0, st>>>(p) : rotary_vec_kernel<false, true><<<grid, 256, 0, st>>>(p);
  else f32 ? rotary_vec_kernel<true, false><<<grid, 256, 0, st>>>(p) : rotary_vec_kernel<false, false><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace w4a4
