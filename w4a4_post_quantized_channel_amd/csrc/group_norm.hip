// Group normalisation with an activation on channels-last features.
//
// One workgroup per (sample, group): the mean, then the mean square
// difference to it, then the output, three passes over the group.
#include "activation.h"
#include "dense.h"
#include "device_common.h"

namespace w4a4 {

namespace {

__device__ __forceinline__ float norm_load(const void* p, int64_t i, int bf16) {
  return bf16 ? bf16_bits_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

__device__ float block_sum(float v, float* red) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += red[w];
  return s;
}

__global__ void __launch_bounds__(256) group_norm_kernel(NormArgs g) {
  __shared__ float red[4];
  const int64_t n = blockIdx.x / g.groups;
  const int cg = g.C / g.groups, c0 = (int)(blockIdx.x % g.groups) * cg;
  const int64_t cnt = g.S * cg;
  auto at = [&](int64_t i) { return n * g.x_sn + i / cg * g.x_ss + c0 + i % cg; };
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < cnt; i += 256) s += norm_load(g.x, at(i), g.bf16);
  const float mean = block_sum(s, red) / (float)cnt;
  s = 0.f;
  for (int64_t i = threadIdx.x; i < cnt; i += 256) {
    const float d = norm_load(g.x, at(i), g.bf16) - mean;
    s += d * d;
  }
  const float rstd = 1.f / sqrtf(block_sum(s, red) / (float)cnt + g.eps);
  for (int64_t i = threadIdx.x; i < cnt; i += 256) {
    const int c = c0 + (int)(i % cg);
    float v = (norm_load(g.x, at(i), g.bf16) - mean) * rstd;
    v = activate(v * (g.weight ? g.weight[c] : 1.f) + (g.bias ? g.bias[c] : 0.f), g.act);
    const int64_t o = n * g.y_sn + i / cg * g.y_ss + c;
    if (g.bf16) ((uint16_t*)g.y)[o] = (uint16_t)f32_to_bf16_bits(v);
    else ((float*)g.y)[o] = v;
  }
}

}  // namespace

size_t group_norm_workspace(int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_group_norm(const NormArgs& g, void*, hipStream_t st) {
  group_norm_kernel<<<dim3((unsigned)(g.N * g.groups)), 256, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace w4a4
