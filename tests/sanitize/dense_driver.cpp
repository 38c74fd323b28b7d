// Drives the 16-bit operators' argument checks under the host sanitizers:
// rejected calls launch nothing and set a message, accepted ones launch once.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "../../include/w4a4.h"
#include "../../w4a4_post_quantized_channel_amd/csrc/dense.h"

extern int g_launches;

namespace w4a4 {
hipError_t launch_prefix_attention(const w4a4_attn&, void*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
size_t prefix_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t P, int64_t) {
  return P > 4096 ? 1 << 20 : 0;
}
hipError_t launch_gemm_bf16(const DenseArgs&, void*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
size_t gemm_bf16_workspace(int64_t M, int64_t, int64_t K, int) { return M <= 64 && K >= 4096 ? 1 << 16 : 0; }
hipError_t launch_group_norm(const NormArgs&, void*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
size_t group_norm_workspace(int64_t, int64_t S, int64_t, int64_t) { return S > 1000 ? 4096 : 0; }
}  // namespace w4a4

namespace {
int failures = 0;

void expect(const char* what, int got, int want, int launches_before) {
  const bool launched = g_launches != launches_before;
  if (got != want || launched != (want == 0) || (want != 0 && std::strlen(w4a4_last_error()) == 0)) {
    std::printf("FAIL %s: status %d, want %d, launched %d\n", what, got, want, launched);
    ++failures;
  }
}

alignas(64) unsigned char mem[4096];

w4a4_attn attn() {
  w4a4_attn a{};
  a.B = 2; a.T = 3; a.Hq = 4; a.Hkv = 2; a.D = 64; a.P = 100; a.S = 10;
  a.scale = 0.125f;
  a.q = a.k_prefix = a.v_prefix = a.k_own = a.v_own = mem;
  a.out = mem + 2048;
  a.q_sb = a.o_sb = 768; a.q_st = a.o_st = 256; a.q_sh = a.o_sh = 64;
  a.kp_sp = a.vp_sp = 128; a.kp_sh = a.vp_sh = 64;
  a.ko_sb = a.vo_sb = 1280; a.ko_ss = a.vo_ss = 128; a.ko_sh = a.vo_sh = 64;
  return a;
}

#define ATTN(change, want)                                             \
  do {                                                                 \
    w4a4_attn a = attn();                                              \
    change;                                                            \
    const int before = g_launches;                                     \
    expect("attention: " #change, w4a4_prefix_attention(&a, nullptr, 0, nullptr), want, before); \
  } while (0)

int linear(int64_t M, int64_t N, int64_t K, const w4a4_epilogue* ep, int64_t ldx, int64_t ldw, int64_t ldy,
           int ydt = W4A4_DT_BF16, const void* x = mem, void* ws = nullptr, size_t wsb = 0) {
  return bf16_linear(x, ldx, mem, ldw, M, N, K, ep, mem + 2048, ydt, ldy, ws, wsb, nullptr);
}
#define LINEAR(want, ...)                                              \
  do {                                                                 \
    const int before = g_launches;                                     \
    expect("linear: " #__VA_ARGS__, linear(__VA_ARGS__), want, before);  \
  } while (0)

int norm(int64_t N, int64_t S, int64_t C, int64_t G, int64_t xss, float eps, int act, int dt = W4A4_DT_F32,
         void* ws = nullptr, size_t wsb = 0, const void* x = mem) {
  return w4a4_group_norm_act(x, dt, N, S, C, G, S * C, xss, nullptr, nullptr, eps, act, mem + 2048, S * C, C, ws, wsb,
                             nullptr);
}
#define NORM(want, ...)                                                \
  do {                                                                 \
    const int before = g_launches;                                     \
    expect("norm: " #__VA_ARGS__, norm(__VA_ARGS__), want, before);      \
  } while (0)
}  // namespace

int main() {
  ATTN(, 0);
  ATTN(a.D = 96, -2);
  ATTN(a.Hq = 5, -2);
  ATTN(a.B = -1, -1);
  ATTN(a.Hkv = 0, -1);
  ATTN(a.P = 1LL << 40, -2);
  ATTN(a.B = 1 << 20; a.T = 1 << 20, -2);
  ATTN(a.scale = INFINITY, -1);
  ATTN(a.causal = 2, -1);
  ATTN(a.q = nullptr, -1);
  ATTN(a.v_own = nullptr, -1);
  ATTN(a.k_prefix = mem + 8, -3);
  ATTN(a.q_st = 260, -3);
  ATTN(a.kp_sp = 1LL << 40, -2);
  ATTN(a.ko_sb = -8, -1);
  ATTN(a.vo_sb = 4, -3);
  ATTN(a.own_len = (const int32_t*)(mem + 2), -3);
  ATTN(a.P = 0; a.k_prefix = a.v_prefix = nullptr, 0);
  ATTN(a.S = 0; a.k_own = a.v_own = nullptr, 0);
  {
    const int before = g_launches;
    w4a4_attn a = attn();
    a.P = 8192;
    expect("attention: small workspace", w4a4_prefix_attention(&a, mem, 16, nullptr), -5, before);
    expect("attention: misaligned workspace", w4a4_prefix_attention(&a, mem + 4, 1 << 20, nullptr), -3, before);
    expect("attention: NULL", w4a4_prefix_attention(nullptr, nullptr, 0, nullptr), -1, before);
    a.B = 0;
    a.q = nullptr;
    if (w4a4_prefix_attention(&a, nullptr, 0, nullptr) != 0 || g_launches != before) ++failures;
  }

  w4a4_epilogue ep{W4A4_ACT_GELU, W4A4_DT_F32, mem, nullptr, 0};
  LINEAR(0, 4, 8, 64, nullptr, 64, 64, 8);
  LINEAR(0, 4, 8, 64, &ep, 64, 64, 8);
  LINEAR(-2, 4, 8, 60, nullptr, 64, 64, 8);
  LINEAR(-1, 4, 8, 0, nullptr, 64, 64, 8);
  LINEAR(-1, -4, 8, 64, nullptr, 64, 64, 8);
  LINEAR(-1, 4, 8, 64, nullptr, 56, 64, 8);
  LINEAR(-3, 4, 8, 64, nullptr, 68, 64, 8);
  LINEAR(-2, 4, 8, 64, nullptr, 1 << 23, 64, 8);
  LINEAR(-1, 4, 8, 64, nullptr, 64, 64, 7);
  LINEAR(-4, 4, 8, 64, nullptr, 64, 64, 8, W4A4_DT_I32);
  LINEAR(-1, 4, 8, 64, nullptr, 64, 64, 8, W4A4_DT_F32, nullptr);
  LINEAR(-3, 4, 8, 64, nullptr, 64, 64, 8, W4A4_DT_F32, mem + 8);
  LINEAR(-5, 4, 8, 8192, nullptr, 8192, 8192, 8, W4A4_DT_F32, mem, mem, 16);
  ep.act = 9;
  LINEAR(-4, 4, 8, 64, &ep, 64, 64, 8);
  ep = {W4A4_ACT_NONE, W4A4_DT_I32, mem, nullptr, 0};
  LINEAR(-4, 4, 8, 64, &ep, 64, 64, 8);
  ep = {W4A4_ACT_NONE, W4A4_DT_F32, mem + 2, nullptr, 0};
  LINEAR(-3, 4, 8, 64, &ep, 64, 64, 8);
  ep = {W4A4_ACT_NONE, W4A4_DT_F32, nullptr, mem, 4};
  LINEAR(-1, 4, 8, 64, &ep, 64, 64, 8);
  ep = {W4A4_ACT_NONE, W4A4_DT_F32, nullptr, mem + 2048, 16};
  LINEAR(-1, 4, 8, 64, &ep, 64, 64, 8);

  NORM(0, 2, 10, 32, 4, 32, 1e-5f, W4A4_ACT_SILU);
  NORM(-2, 2, 10, 32, 5, 32, 1e-5f, W4A4_ACT_SILU);
  NORM(-1, 2, 10, 32, 0, 32, 1e-5f, W4A4_ACT_SILU);
  NORM(-1, 2, 10, 32, 4, 31, 1e-5f, W4A4_ACT_SILU);
  NORM(-1, 2, 10, 32, 4, 32, -1.f, W4A4_ACT_SILU);
  NORM(-1, 2, 10, 32, 4, 32, NAN, W4A4_ACT_SILU);
  NORM(-4, 2, 10, 32, 4, 32, 1e-5f, W4A4_ACT_SWIGLU);
  NORM(-4, 2, 10, 32, 4, 32, 1e-5f, W4A4_ACT_NONE, W4A4_DT_I32);
  NORM(-2, 2, 10, 1 << 20, 4, 1 << 20, 1e-5f, W4A4_ACT_NONE);
  NORM(-1, 2, 10, 32, 4, 32, 1e-5f, W4A4_ACT_NONE, W4A4_DT_F32, nullptr, 0, nullptr);
  NORM(-3, 2, 10, 32, 4, 32, 1e-5f, W4A4_ACT_NONE, W4A4_DT_F32, nullptr, 0, mem + 2);
  NORM(-5, 2, 2000, 32, 4, 32, 1e-5f, W4A4_ACT_NONE, W4A4_DT_F32, mem, 16);

  // the workspace queries take anything
  if (w4a4_prefix_attention_workspace(-1, 1, 1, 1, 64, 1, 1) || w4a4_bf16_workspace_size(1, 1, 7, 0) ||
      w4a4_group_norm_workspace(1, 1, 7, 2) || !w4a4_prefix_attention_workspace(1, 1, 1, 1, 64, 8192, 1) ||
      !w4a4_bf16_workspace_size(1, 8, 8192, 0) || !w4a4_group_norm_workspace(1, 2000, 8, 2))
    ++failures;
  std::printf("ok: %d failures\n", failures);
  return failures != 0;
}
