// Launchers of the 16-bit operators behind the C ABI (host side).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/w4a4.h"

namespace w4a4 {

// attention.hip: sizes and pointers as checked by the entry point; strides in
// elements.  workspace null or of prefix_attention_workspace() bytes.
hipError_t launch_prefix_attention(const w4a4_attn& a, void* workspace, hipStream_t st);
size_t prefix_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t P, int64_t S);

// gemm_bf16.hip
struct DenseArgs {
  const uint16_t* x;      // M x K
  const uint16_t* w;      // N (SwiGLU: 2 N) x K
  int64_t ldx, ldw;
  int M, N, K;            // N: output columns
  int act;                // W4A4_ACT_*
  const void* bias;       // [N or 2 N] or null
  int bias_bf16;
  const void* residual;   // M x N of the output's type, or null
  int64_t ldr;
  void* y;
  int y_bf16;
  int64_t ldy;
};
hipError_t launch_gemm_bf16(const DenseArgs& g, void* workspace, hipStream_t st);
size_t gemm_bf16_workspace(int64_t M, int64_t N, int64_t K, int act);

// group_norm.hip
struct NormArgs {
  const void* x;
  void* y;
  int bf16;
  int64_t N, S;
  int C, groups;
  int64_t x_sn, x_ss, y_sn, y_ss;
  const float* weight;    // or null
  const float* bias;      // or null
  float eps;
  int act;
};
hipError_t launch_group_norm(const NormArgs& g, void* workspace, hipStream_t st);
size_t group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups);

}  // namespace w4a4
