// The gated residual of a block fused with the norms on both sides of it.
//
// Mathematics.  x' = alpha x + gate u, with u = h or its rms norm; then the
// mean of x', its variance from differences to the mean (a large mean costs no
// accuracy), and y.  Sums go over a thread's values, the lanes of a wave and
// the waves, all in fp32.
//
// A row stays in registers: each input is read once, each output written once.
// Rows of up to 512 channels belong to one wave, four rows a workgroup; longer
// ones to a workgroup of one thread per eight channels (sixteen beyond 8192),
// so that every load of a row is in flight at once.  Where the width, a stride
// or an address does not allow 16-byte accesses a thread takes single channels,
// a workgroup apart.
#include "cache.h"
#include "device_common.h"

namespace w4a4 {

namespace {

typedef float v8f __attribute__((ext_vector_type(8)));

// VEC (8 or 1) values of row `p` from channel c on; rows of fp32 or bf16.
template <int VEC>
__device__ __forceinline__ void load(float (&v)[VEC], const void* p, int64_t i, bool f32) {
  if constexpr (VEC == 1) {
    v[0] = f32 ? ((const float*)p)[i] : bf16_bits_to_f32(((const uint16_t*)p)[i]);
  } else if (f32) {
    const v4f a = *reinterpret_cast<const v4f*>((const float*)p + i), b = *reinterpret_cast<const v4f*>((const float*)p + i + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = a[k], v[4 + k] = b[k];
  } else {
    const v4i a = *reinterpret_cast<const v4i*>((const uint16_t*)p + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float((uint32_t)a[k] << 16);
      v[2 * k + 1] = __uint_as_float((uint32_t)a[k] & 0xFFFF0000u);
    }
  }
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

// Sum over the row's threads: of a wave, or of the workgroup through ``red``
// (a different one for every sum, so one barrier each is enough).
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if constexpr (WAVE) return v;
  const int nw = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < nw; ++w) s += red[w];
  return s;
}

template <int VEC, int NI, bool WAVE>
__global__ void __launch_bounds__(1024) gated_norm_kernel(w4a4_gated a) {
  __shared__ float red[WAVE ? 1 : 3][16];
  const int tpr = WAVE ? 64 : blockDim.x;                    // threads of a row
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int C = (int)a.C;
  const float inv = 1.f / (float)C;
  const int64_t per = a.M / a.R;
  const int64_t step = WAVE ? 4 * (int64_t)gridDim.x : gridDim.x;
  for (int64_t m = WAVE ? 4 * (int64_t)blockIdx.x + (threadIdx.x >> 6) : blockIdx.x; m < a.M; m += step) {
    const int64_t r = a.R == 1 ? 0 : m / per;
    float x[NI][VEC], u[NI][VEC], g[NI][VEC], sc[NI][VEC], sh[NI][VEC];
    bool in[NI];
    // everything the row needs, before the first sum
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = (i * tpr + t) * VEC;
      in[i] = c < C;
#pragma unroll
      for (int k = 0; k < VEC; ++k) x[i][k] = 0.f, u[i][k] = 0.f, g[i][k] = 1.f, sc[i][k] = 0.f, sh[i][k] = 0.f;
      if (!in[i]) continue;
      if (a.h) load<VEC>(u[i], a.h, m * a.ldh + c, a.h_dtype == W4A4_DT_F32);
      load<VEC>(x[i], a.x, m * a.ldx + c, a.x_dtype == W4A4_DT_F32);
      if (a.gate) load<VEC>(g[i], a.gate, r * a.gate_sr + c, true);
      if (a.y && a.scale) load<VEC>(sc[i], a.scale, r * a.scale_sr + c, true);
      if (a.y && a.shift) load<VEC>(sh[i], a.shift, r * a.shift_sr + c, true);
    }
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
        load<VEC>(w, a.post_weight, (i * tpr + t) * VEC, true);
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
      if (in[i] && a.x_out) store<VEC>(a.x_out, m * a.ldxo + (i * tpr + t) * VEC, a.x_dtype == W4A4_DT_F32, x[i]);
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
        if (a.weight) load<VEC>(w, a.weight, c, true);
        if (a.bias) load<VEC>(bb, a.bias, c, true);
#pragma unroll
        for (int k = 0; k < VEC; ++k) y[k] = (x[i][k] * rs * w[k] + bb[k]) * (1.f + sc[i][k]) + sh[i][k];
        store<VEC>(a.y, m * a.ldy + c, a.y_dtype == W4A4_DT_F32, y);
      }
    }
    if constexpr (!WAVE) __syncthreads();   // ``red`` is read by all before the next row
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
  const int64_t most = 1 << 20;   // workgroups; more rows are walked
  const unsigned rows = (unsigned)(g.M < most ? g.M : most), quads = (unsigned)((g.M + 3) / 4 < most ? (g.M + 3) / 4 : most);
  const int C = (int)g.C;
  if (vec) {
    const unsigned threads = (unsigned)((C / 8 + 63) / 64 * 64);
    if (C <= 512) gated_norm_kernel<8, 1, true><<<quads, 256, 0, st>>>(g);
    else if (C <= 8192) gated_norm_kernel<8, 1, false><<<rows, threads, 0, st>>>(g);
    else gated_norm_kernel<8, 2, false><<<rows, 1024, 0, st>>>(g);
  } else {
    if (C <= 256) gated_norm_kernel<1, 4, true><<<quads, 256, 0, st>>>(g);
    else if (C <= 2048) gated_norm_kernel<1, 4, false><<<rows, (unsigned)((C + 255) / 256 * 64), 0, st>>>(g);
    else gated_norm_kernel<1, 16, false><<<rows, 1024, 0, st>>>(g);
  }
  return hipGetLastError();
}

}  // namespace w4a4
