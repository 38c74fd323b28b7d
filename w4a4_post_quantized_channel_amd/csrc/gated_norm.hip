// The gated residual of a block fused with the norms on both sides of it.
//
// Mathematics.  x' = alpha x + gate u, with u = h or its rms norm; then the
// mean of x', its variance from differences to the mean (a large mean costs no
// accuracy), and y.  Sums go over a thread's values, the lanes of a wave and
// the waves, all in fp32.
//
// A row of up to 8192 channels stays in registers: each input is read once, each
// output written once.  Rows of up to 512 channels belong to one wave, four rows a
// workgroup; longer ones to a workgroup of one thread per eight channels (two or
// three times eight beyond 8192, which 128 registers do not hold: a multiple of
// eight keeps 12 of a thread's in scratch memory, 4096 rows of 16384 in bf16 take
// 116 us, 4.6 TB/s, and of 8192 57; another width 164, rows of 16383 take 311).
// Where the width is no multiple of eight, the channels behind the last eight are
// a thread's each: loads of single channels by one thread, one after the other,
// cost 777 rows of 1155 channels 4.4 us of 10.2.
// Rows that follow each other belong to the same workgroup, which keeps its
// channels' gate, scale and shift while they stay the same (read for every row
// they would be two thirds of what a compute unit loads at 5120 channels), and
// loads a row while it sums the one before.
//
// Bound by memory for many rows: 12480 of 5120 channels, fp32 stream, bf16 h and
// y (767 MB), take 155 us, 4.9 TB/s (a thread per channel took 985, a workgroup
// per row 237).  For few rows it is a launch and the chain of a row: loads, two
// or three sums, each with the weights that are loaded behind it, and the store,
// 4.1 us for 64 rows of 2048, 5.8 for the 777.
#include "cache.h"
#include "device_common.h"
#include "divisor.h"

namespace w4a4 {

namespace {

typedef float v8f __attribute__((ext_vector_type(8)));
// 16 bytes at the alignment of their elements, which is all that global memory asks for.
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4_of_f32 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u4_of_bf16 __attribute__((ext_vector_type(4), aligned(2)));

// Eight values of a row, or (TAIL, not all) the first one only, fp32 or bf16, as loaded.
struct Raw {
  uint32_t w[8];
  template <bool TAIL>
  __device__ __forceinline__ void load(const void* p, int64_t i, bool f32, bool all) {
    if (!TAIL || all) {
      if (f32) {
        const u4_of_f32* q = reinterpret_cast<const u4_of_f32*>((const float*)p + i);
        const u4_of_f32 a = q[0], b = q[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      } else {
        const u4_of_bf16 a = *reinterpret_cast<const u4_of_bf16*>((const uint16_t*)p + i);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      }
    } else {
      w[0] = f32 ? ((const uint32_t*)p)[i] : ((const uint16_t*)p)[i];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 0;
  }
  __device__ __forceinline__ void get(float (&v)[8], bool f32) const {
    if (f32) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    }
  }
};
template <bool TAIL>
__device__ __forceinline__ void load(float (&v)[8], const float* p, int64_t i, bool all) {
  if (!TAIL || all) {
    const u4_of_f32* q = reinterpret_cast<const u4_of_f32*>(p + i);
    const u4_of_f32 a = q[0], b = q[1];
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  } else {
    v[0] = p[i];
  }
}
template <bool TAIL>
__device__ __forceinline__ void store(void* p, int64_t i, bool f32, const float (&v)[8], bool all) {
  if (!TAIL || all) {
    const v8f a = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    if (f32) {
      u4_of_f32* q = reinterpret_cast<u4_of_f32*>((float*)p + i);
      q[0] = __builtin_bit_cast(u4, (v4f){v[0], v[1], v[2], v[3]});
      q[1] = __builtin_bit_cast(u4, (v4f){v[4], v[5], v[6], v[7]});
    } else {
      *reinterpret_cast<u4_of_bf16*>((__bf16*)p + i) = __builtin_bit_cast(u4, __builtin_convertvector(a, v8bf));
    }
  } else if (f32) {
    ((float*)p)[i] = v[0];
  } else {
    ((__bf16*)p)[i] = (__bf16)v[0];
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
// Sum over a wave, the same in every lane: inside rows of 16 by quad swaps and
// mirrors, then the rows' sums as scalars (exchanges through LDS take several
// times as long, and a short row waits for nothing else).
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);    // lane ^ 1
  v += dpp<0x4E>(v);    // lane ^ 2
  v += dpp<0x141>(v);   // the other quad of the half row
  v += dpp<0x140>(v);   // the other half row
  const int b = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

// Sum over the row's threads: of a wave, or of the workgroup through ``red``
// (a different one for every sum of a row, so one barrier each is enough).
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (WAVE) return v;
  const int nw = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < nw; ++w) s += red[w];
  return s;
}

// NI: items of a thread, eight channels each; TAIL: behind them C % 8 items of one.
template <int NI, bool WAVE, bool TAIL>
__global__ void __launch_bounds__(1024) gated_norm_kernel(w4a4_gated a, int rows, Divisor per) {
  __shared__ float red[WAVE ? 1 : 3][16];
  const int tpr = WAVE ? 64 : blockDim.x;                    // threads of a row
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int C = (int)a.C;
  const bool xf = a.x_dtype == W4A4_DT_F32, hf = a.h_dtype == W4A4_DT_F32, yf = a.y_dtype == W4A4_DT_F32;
  const float inv = 1.f / (float)C;
  // rows m0 .. m1 - 1
  const int64_t m0 = (WAVE ? 4 * (int64_t)blockIdx.x + (threadIdx.x >> 6) : blockIdx.x) * rows;
  const int64_t m1 = m0 + rows < a.M ? m0 + rows : a.M;
  const int full = C / 8;
  auto all = [&](int i) { return !TAIL || i * tpr + t < full; };
  auto at = [&](int i) { return all(i) ? (i * tpr + t) * 8 : 7 * full + i * tpr + t; };
  auto in = [&](int i) { return at(i) < C; };
  Raw nx[NI], nh[NI];                                        // a row as loaded
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!in(i)) continue;
      if (a.h) nh[i].template load<TAIL>(a.h, m * a.ldh + at(i), hf, all(i));
      nx[i].template load<TAIL>(a.x, m * a.ldx + at(i), xf, all(i));
    }
  };
#pragma unroll
  for (int i = 0; i < NI; ++i) nx[i].clear(), nh[i].clear();
  constexpr bool EARLY = NI == 1;                            // (registers for no more)
  if (EARLY && m0 < m1) fetch(m0);
  float g[NI][8], sc[NI][8], sh[NI][8];                      // of modulation row r
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) g[i][k] = 1.f, sc[i][k] = 0.f, sh[i][k] = 0.f;
  int64_t r = -1, rend = m0;                                 // and the first row behind it
  for (int64_t m = m0; m < m1; ++m) {
    if (m >= rend) {
      int rem;
      r = div_by((int)m, per, rem);
      rend = m - rem + per.d;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!in(i)) continue;
        if (a.gate) load<TAIL>(g[i], a.gate, r * a.gate_sr + at(i), all(i));
        if (a.y && a.scale) load<TAIL>(sc[i], a.scale, r * a.scale_sr + at(i), all(i));
        if (a.y && a.shift) load<TAIL>(sh[i], a.shift, r * a.shift_sr + at(i), all(i));
      }
    }
    if (!EARLY) fetch(m);
    float x[NI][8], u[NI][8];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      nx[i].get(x[i], xf);
      nh[i].get(u[i], hf);
    }
    if (EARLY && m + 1 < m1) fetch(m + 1);
    if (a.post_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += u[i][k] * u[i][k];
      const float post = 1.f / sqrtf(row_sum<WAVE>(ss, red[0]) * inv + a.eps);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!in(i)) continue;
        float w[8] = {};
        load<TAIL>(w, a.post_weight, at(i), all(i));
#pragma unroll
        for (int k = 0; k < 8; ++k) u[i][k] = u[i][k] * post * w[k];
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[i][k] = a.alpha * x[i][k] + u[i][k] * g[i][k];     // (zero past the end)
        s += x[i][k];
      }
      if (in(i) && a.x_out) store<TAIL>(a.x_out, m * a.ldxo + at(i), xf, x[i], all(i));
    }
    if (a.y) {
      const float mean = a.kind == W4A4_NORM_LAYER ? row_sum<WAVE>(s, red[WAVE ? 0 : 1]) * inv : 0.f;
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (in(i))
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[i][k] -= mean;
            if (k == 0 || all(i)) ss += x[i][k] * x[i][k];
          }
      const float rs = 1.f / sqrtf(row_sum<WAVE>(ss, red[WAVE ? 0 : 2]) * inv + a.eps);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!in(i)) continue;
        float w[8], bb[8], y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 1.f, bb[k] = 0.f;
        if (a.weight) load<TAIL>(w, a.weight, at(i), all(i));
        if (a.bias) load<TAIL>(bb, a.bias, at(i), all(i));
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = (x[i][k] * rs * w[k] + bb[k]) * (1.f + sc[i][k]) + sh[i][k];
        store<TAIL>(a.y, m * a.ldy + at(i), yf, y, all(i));
      }
    }
    // ``red`` is read by all before the next row's first sum writes it: rows with
    // one sum only, and the second of a pair of sums, are a barrier apart
    if constexpr (!WAVE) __syncthreads();
  }
}

}  // namespace

hipError_t launch_gated_norm(const w4a4_gated& g, hipStream_t st) {
  const int C = (int)g.C;
  // One row a workgroup (or wave) up to 2048 threads a CU, then runs of rows.
  // (Registers let 20 waves of a CU run at once, 16 where a wave has a row: 12480
  // rows of 5120 are 735 workgroups of ten waves, two of them a CU.)
  const int items = C / 8 + C % 8;
  const bool wave = items <= 64, tail = C % 8 != 0;
  const unsigned threads = wave ? 256 : items <= 1024 ? (unsigned)((items + 63) / 64 * 64) : 1024;
  const int64_t slots = 256 * (2048 / threads) * (wave ? 4 : 1);
  const int64_t rows = (g.M + slots - 1) / slots, units = (g.M + rows - 1) / rows;
  const unsigned grid = (unsigned)(wave ? (units + 3) / 4 : units);
  const Divisor per = divisor(g.M / g.R);
  auto launch = [&](auto kernel) { kernel<<<grid, threads, 0, st>>>(g, (int)rows, per); };
  if (wave) tail ? launch(gated_norm_kernel<1, true, true>) : launch(gated_norm_kernel<1, true, false>);
  else if (items <= 1024) tail ? launch(gated_norm_kernel<1, false, true>) : launch(gated_norm_kernel<1, false, false>);
  else tail ? launch(gated_norm_kernel<3, false, true>) : launch(gated_norm_kernel<2, false, false>);
  return hipGetLastError();
}

}  // namespace w4a4
