// The gated residual of a block fused with the norms on both sides of it.
//
// A workgroup takes one row and keeps it in registers: x' = alpha x + gate u,
// its mean, then its variance from differences to the mean, each sum over the
// workgroup in fp32.
#include "cache.h"
#include "device_common.h"

namespace w4a4 {

namespace {

constexpr int kThreads = 256, kMost = 16384 / kThreads;

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? ((const float*)p)[i] : bf16_bits_to_f32(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void store1(void* p, int64_t i, bool f32, float v) {
  if (f32) ((float*)p)[i] = v;
  else ((__bf16*)p)[i] = (__bf16)v;
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += red[w];
  return s;
}

template <int NI>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(w4a4_gated a) {
  __shared__ float red[kThreads / 64];
  const int64_t m = blockIdx.x, r = m / (a.M / a.R);
  const int C = (int)a.C;
  const float inv = 1.f / (float)C;
  float x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) x[i] = 0.f;
  if (a.h) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * kThreads + threadIdx.x;
      if (c < C) x[i] = load1(a.h, m * a.ldh + c, a.h_dtype == W4A4_DT_F32);
      ss += x[i] * x[i];
    }
    float post = 1.f;
    if (a.post_weight) post = 1.f / sqrtf(block_sum(ss, red) * inv + a.eps);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * kThreads + threadIdx.x;
      if (c >= C) continue;
      if (a.post_weight) x[i] = x[i] * post * a.post_weight[c];
      if (a.gate) x[i] *= a.gate[r * a.gate_sr + c];
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = i * kThreads + threadIdx.x;
    if (c >= C) continue;
    x[i] = a.alpha * load1(a.x, m * a.ldx + c, a.x_dtype == W4A4_DT_F32) + x[i];
    s += x[i];
    if (a.x_out) store1(a.x_out, m * a.ldxo + c, a.x_dtype == W4A4_DT_F32, x[i]);
  }
  if (!a.y) return;
  const float mean = a.kind == W4A4_NORM_LAYER ? block_sum(s, red) * inv : 0.f;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (i * kThreads + threadIdx.x < C) ss += (x[i] - mean) * (x[i] - mean);
  const float rs = 1.f / sqrtf(block_sum(ss, red) * inv + a.eps);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = i * kThreads + threadIdx.x;
    if (c >= C) continue;
    float y = (x[i] - mean) * rs;
    if (a.weight) y *= a.weight[c];
    if (a.bias) y += a.bias[c];
    if (a.scale) y *= 1.f + a.scale[r * a.scale_sr + c];
    if (a.shift) y += a.shift[r * a.shift_sr + c];
    store1(a.y, m * a.ldy + c, a.y_dtype == W4A4_DT_F32, y);
  }
}

}  // namespace

hipError_t launch_gated_norm(const w4a4_gated& g, hipStream_t st) {
  const unsigned grid = (unsigned)g.M;
  if (g.C <= 8 * kThreads) gated_norm_kernel<8><<<grid, kThreads, 0, st>>>(g);
  else gated_norm_kernel<kMost><<<grid, kThreads, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace w4a4
