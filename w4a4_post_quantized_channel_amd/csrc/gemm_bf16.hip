// bf16 product with bias, activation and residual: y = act(x W^T + bias) + residual.
//
// One wave per 16 x 16 output tile, operands straight from global memory
// into v_mfma_f32_16x16x32_bf16; for SwiGLU the wave holds the gate's and the
// up projection's tile of the same columns.
#include "activation.h"
#include "dense.h"
#include "device_common.h"
#include "epilogue.h"

namespace w4a4 {

namespace {

__device__ __forceinline__ float bias_at(const DenseArgs& g, int n) {
  if (!g.bias) return 0.f;
  return g.bias_bf16 ? bf16_bits_to_f32(((const uint16_t*)g.bias)[n]) : ((const float*)g.bias)[n];
}

__global__ void __launch_bounds__(64) gemm_bf16_tile_kernel(DenseArgs g) {
  const int lane = threadIdx.x, lr = lane & 15, lk = (lane >> 4) * 8;
  const int m0 = blockIdx.y * 16, n0 = blockIdx.x * 16;
  const bool gated = g.act == W4A4_ACT_SWIGLU;
  v4f acc = {0, 0, 0, 0}, up = {0, 0, 0, 0};
  for (int k = 0; k < g.K; k += 32) {
    const v8bf a = load_bf16x8(g.x, g.ldx, m0 + lr, g.M, k + lk, g.K);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, load_bf16x8(g.w, g.ldw, n0 + lr, g.N, k + lk, g.K), acc, 0, 0, 0);
    if (gated)
      up = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          a, load_bf16x8(g.w + g.N * g.ldw, g.ldw, n0 + lr, g.N, k + lk, g.K), up, 0, 0, 0);
  }
  const int n = n0 + lr;
  if (n >= g.N) return;
  for (int r = 0; r < 4; ++r) {
    const int m = m0 + (lane >> 4) * 4 + r;
    if (m >= g.M) return;
    float z = acc[r] + bias_at(g, n);
    z = gated ? times_sigmoid(z, z) * (up[r] + bias_at(g, g.N + n)) : activate(z, g.act);
    if (g.residual)
      z += g.y_bf16 ? bf16_bits_to_f32(((const uint16_t*)g.residual)[m * g.ldr + n])
                    : ((const float*)g.residual)[m * g.ldr + n];
    if (g.y_bf16) ((uint16_t*)g.y)[m * g.ldy + n] = (uint16_t)f32_to_bf16_bits(z);
    else ((float*)g.y)[m * g.ldy + n] = z;
  }
}

}  // namespace

size_t gemm_bf16_workspace(int64_t, int64_t, int64_t, int) { return 0; }

hipError_t launch_gemm_bf16(const DenseArgs& g, void*, hipStream_t st) {
  gemm_bf16_tile_kernel<<<dim3((g.N + 15) / 16, (g.M + 15) / 16), 64, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace w4a4
