// The gated residual of a block fused with the norms on both sides of it.
//
// Mathematics.  x' = alpha x + gate u, with u = h or its rms norm; then the
// mean of x', its variance from differences to the mean (a large mean costs no
// accuracy), and y.  Sums go over a thread's values, the lanes of a wave and
// the waves, all in fp32.
//
// A row stays in registers: each input is read once, each output written once.
// Rows of up to 512 channels belong to one wave, four rows a workgroup; longer
// ones to a workgroup of one thread per eight channels (sixteen beyond 8192).
// Rows that follow each other belong to the same workgroup, which keeps its
// channels' gate, scale and shift while they stay the same (read for every row
// they would be two thirds of what a compute unit loads at 5120 channels), and
// loads a row while it sums the one before.  Where the width, a stride or an
// address does not allow 16-byte accesses a thread takes single channels, a
// workgroup apart.
#include "cache.h"
#include "device_common.h"
#include "divisor.h"

namespace w4a4 {

namespace {

typedef float v8f __attribute__((ext_vector_type(8)));

// VEC (8 or 1) values of a row, fp32 or bf16, as loaded.
template <int VEC>
struct Raw {
  uint32_t w[VEC];
  __device__ __forceinline__ void load(const void* p, int64_t i, bool f32) {
    if constexpr (VEC == 1) {
      w[0] = f32 ? ((const uint32_t*)p)[i] : (uint32_t)((const uint16_t*)p)[i] << 16;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>((const char*)p + i * (f32 ? 4 : 2));
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      if (f32) {
        const uint4 b = *reinterpret_cast<const uint4*>((const float*)p + i + 4);
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < VEC; ++k) w[k] = 0;
  }
  __device__ __forceinline__ void get(float (&v)[VEC], bool f32) const {
    if (VEC == 1 || f32) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = __uint_as_float(w[k]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    }
  }
};
template <int VEC>
__device__ __forceinline__ void load(float (&v)[VEC], const float* p, int64_t i) {
  Raw<VEC> r;
  r.load(p, i, true);
  r.get(v, true);
}
template <int VEC>
__device__ __forceinline__ void store(void* p, int64_t i, bool f32, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if (f32) ((float*)p)[i] = v[0];
    else ((__bf16*)p)[i] = (__bf16)v[0];
  } else if (f32) {
    *reinterpret_cast<v4f*>((float*)p + i) = (v4f){v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f*>((float*)p + i + 4) = (v4f){v[4], v[5], v[6], v[7]};
  } else {
    const v8f a = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    *reinterpret_cast<v8bf*>((__bf16*)p + i) = __builtin_convertvector(a, v8bf);
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

template <int VEC, int NI, bool WAVE>
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
  bool in[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) in[i] = (i * tpr + t) * VEC < C;
  Raw<VEC> nx[NI], nh[NI];                                   // the next row
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!in[i]) continue;
      if (a.h) nh[i].load(a.h, m * a.ldh + (i * tpr + t) * VEC, hf);
      nx[i].load(a.x, m * a.ldx + (i * tpr + t) * VEC, xf);
    }
  };
#pragma unroll
  for (int i = 0; i < NI; ++i) nx[i].clear(), nh[i].clear();
  if (m0 < m1) fetch(m0);
  float g[NI][VEC], sc[NI][VEC], sh[NI][VEC];                // of modulation row r
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) g[i][k] = 1.f, sc[i][k] = 0.f, sh[i][k] = 0.f;
  int64_t r = -1, rend = m0;                                 // and the first row behind it
  for (int64_t m = m0; m < m1; ++m) {
    if (m >= rend) {
      int rem;
      r = div_by((int)m, per, rem);
      rend = m - rem + per.d;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!in[i]) continue;
        const int c = (i * tpr + t) * VEC;
        if (a.gate) load<VEC>(g[i], a.gate, r * a.gate_sr + c);
        if (a.y && a.scale) load<VEC>(sc[i], a.scale, r * a.scale_sr + c);
        if (a.y && a.shift) load<VEC>(sh[i], a.shift, r * a.shift_sr + c);
      }
    }
    float x[NI][VEC], u[NI][VEC];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      nx[i].get(x[i], xf);
      nh[i].get(u[i], hf);
    }
    if (m + 1 < m1) fetch(m + 1);
    if (a.post_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss += u[i][k] * u[i][k];
      const float post = 1.f / sqrtf(row_sum<WAVE>(ss, red[0]) * inv + a.eps);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!in[i]) continue;
        float w[VEC];
        load<VEC>(w, a.post_weight, (i * tpr + t) * VEC);
#pragma unroll
        for (int k = 0; k < VEC; ++k) u[i][k] = u[i][k] * post * w[k];
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        x[i][k] = a.alpha * x[i][k] + u[i][k] * g[i][k];
        s += x[i][k];
      }
      if (in[i] && a.x_out) store<VEC>(a.x_out, m * a.ldxo + (i * tpr + t) * VEC, xf, x[i]);
    }
    if (a.y) {
      const float mean = a.kind == W4A4_NORM_LAYER ? row_sum<WAVE>(s, red[WAVE ? 0 : 1]) * inv : 0.f;
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (in[i])
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            x[i][k] -= mean;
            ss += x[i][k] * x[i][k];
          }
      const float rs = 1.f / sqrtf(row_sum<WAVE>(ss, red[WAVE ? 0 : 2]) * inv + a.eps);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!in[i]) continue;
        const int c = (i * tpr + t) * VEC;
        float w[VEC], bb[VEC], y[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = 1.f, bb[k] = 0.f;
        if (a.weight) load<VEC>(w, a.weight, c);
        if (a.bias) load<VEC>(bb, a.bias, c);
#pragma unroll
        for (int k = 0; k < VEC; ++k) y[k] = (x[i][k] * rs * w[k] + bb[k]) * (1.f + sc[i][k]) + sh[i][k];
        store<VEC>(a.y, m * a.ldy + c, yf, y);
      }
    }
    // ``red`` is read by all before the next row's first sum writes it: rows with
    // one sum only, and the second of a pair of sums, are a barrier apart
    if constexpr (!WAVE) __syncthreads();
  }
}

}  // namespace

hipError_t launch_gated_norm(const w4a4_gated& g, hipStream_t st) {
  // 16-byte accesses: eight channels of bf16, four of fp32 at a time
  auto fits = [&](const void* p, int64_t ld, bool f32) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % (f32 ? 4 : 8) == 0);
  };
  const bool vec = g.C % 8 == 0 && fits(g.x, g.ldx, g.x_dtype == W4A4_DT_F32) && fits(g.h, g.ldh, g.h_dtype == W4A4_DT_F32) &&
                   fits(g.x_out, g.ldxo, g.x_dtype == W4A4_DT_F32) && fits(g.y, g.ldy, g.y_dtype == W4A4_DT_F32) &&
                   fits(g.gate, g.gate_sr, true) && fits(g.scale, g.scale_sr, true) && fits(g.shift, g.shift_sr, true) &&
                   fits(g.post_weight, 0, true) && fits(g.weight, 0, true) && fits(g.bias, 0, true);
  const int C = (int)g.C;
  // One row a workgroup (or wave) until the card is full, then runs of rows.
  const bool wave = C <= (vec ? 512 : 256);
  const unsigned threads = wave ? 256 : vec ? (C <= 8192 ? (unsigned)((C / 8 + 63) / 64 * 64) : 1024)
                                      : C <= 4096 ? (unsigned)((C + 255) / 256 * 64) : 1024;
  const int64_t slots = 256 * (2048 / threads) * (wave ? 4 : 1);
  const int64_t rows = (g.M + slots - 1) / slots, units = (g.M + rows - 1) / rows;
  const unsigned grid = (unsigned)(wave ? (units + 3) / 4 : units);
  if (vec) {
    if (wave) gated_norm_kernel<8, 1, true><<<grid, threads, 0, st>>>(g, (int)rows, divisor(g.M / g.R));
    else if (C <= 8192) gated_norm_kernel<8, 1, false><<<grid, threads, 0, st>>>(g, (int)rows, divisor(g.M / g.R));
    else gated_norm_kernel<8, 2, false><<<grid, threads, 0, st>>>(g, (int)rows, divisor(g.M / g.R));
  } else {
    if (wave) gated_norm_kernel<1, 4, true><<<grid, threads, 0, st>>>(g, (int)rows, divisor(g.M / g.R));
    else if (C <= 4096) gated_norm_kernel<1, 4, false><<<grid, threads, 0, st>>>(g, (int)rows, divisor(g.M / g.R));
    else gated_norm_kernel<1, 16, false><<<grid, threads, 0, st>>>(g, (int)rows, divisor(g.M / g.R));
  }
  return hipGetLastError();
}

}  // namespace w4a4
