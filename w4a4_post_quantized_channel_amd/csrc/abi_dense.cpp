// C ABI of the 16-bit operators: host-side argument checks and dispatch.
// Every check runs before any launch.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/w4a4.h"
#include "abi_util.h"
#include "dense.h"

using w4a4::aligned;
using w4a4::fail;
using w4a4::launch_status;
using w4a4::ok;

namespace {

int check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
  if (!ws) return ok();
  if (bytes < need) return fail(W4A4_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, bytes, need);
  if (!aligned(ws, 16)) return fail(W4A4_ERR_MISALIGNED, "%s: workspace not 16-byte aligned", fn);
  return ok();
}

// A stride the kernels address inside one tile with 32-bit offsets.
int check_stride(const char* fn, const char* what, int64_t s) {
  if (s < 0) return fail(W4A4_ERR_INVALID_ARG, "%s: negative %s stride", fn, what);
  if (s % 8 != 0) return fail(W4A4_ERR_MISALIGNED, "%s: %s stride %lld not a multiple of 8", fn, what, (long long)s);
  if (s > (1LL << 22)) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %s stride above 2^22 elements", fn, what);
  return ok();
}

int check_batch_stride(const char* fn, const char* what, int64_t s) {
  if (s < 0) return fail(W4A4_ERR_INVALID_ARG, "%s: negative %s batch stride", fn, what);
  if (s % 8 != 0) return fail(W4A4_ERR_MISALIGNED, "%s: %s batch stride not a multiple of 8", fn, what);
  return ok();
}

int check_pointer(const char* fn, const char* what, const void* p, size_t al) {
  if (!p) return fail(W4A4_ERR_INVALID_ARG, "%s: %s is NULL", fn, what);
  if (!aligned(p, al)) return fail(W4A4_ERR_MISALIGNED, "%s: %s not %zu-byte aligned", fn, what, al);
  return ok();
}

// Sizes of prefix_attention; also the workspace query's check.
int check_attn_sizes(const char* fn, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t P, int64_t S) {
  if (B < 0 || T < 0 || P < 0 || S < 0 || Hq <= 0 || Hkv <= 0)
    return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (D != 64 && D != 128 && D != 256)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: head width %lld is not 64, 128 or 256", fn, (long long)D);
  if (Hq % Hkv != 0)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %lld query heads over %lld KV heads", fn, (long long)Hq, (long long)Hkv);
  if (Hq > 65536 || P > (1LL << 30) || S > (1LL << 24) || T > (1LL << 24) || B > (1LL << 24) ||
      B * T > (1LL << 30) / Hq)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: sizes too large", fn);
  return ok();
}

}  // namespace

extern "C" {

int w4a4_prefix_attention(const w4a4_attn* desc, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "w4a4_prefix_attention";
  if (!desc) return fail(W4A4_ERR_INVALID_ARG, "%s: NULL descriptor", fn);
  w4a4_attn copy = *desc;
  w4a4_attn* a = &copy;
  // the stride of a dimension of one is not used and may be anything
  if (a->B == 1) a->q_sb = a->o_sb = a->ko_sb = a->vo_sb = 0;
  if (a->T == 1) a->q_st = a->o_st = 0;
  if (a->Hq == 1) a->q_sh = a->o_sh = 0;
  if (a->Hkv == 1) a->kp_sh = a->vp_sh = a->ko_sh = a->vo_sh = 0;
  if (a->P == 1) a->kp_sp = a->vp_sp = 0;
  if (a->S == 1) a->ko_ss = a->vo_ss = 0;
  int st = check_attn_sizes(fn, a->B, a->T, a->Hq, a->Hkv, a->D, a->P, a->S);
  if (st != W4A4_OK) return st;
  if (!std::isfinite(a->scale)) return fail(W4A4_ERR_INVALID_ARG, "%s: scale not finite", fn);
  if (a->causal != 0 && a->causal != 1) return fail(W4A4_ERR_INVALID_ARG, "%s: causal must be 0 or 1", fn);
  if (a->B == 0 || a->T == 0) return ok();
  struct Op {
    const char* what;
    const void* p;
    bool used;
    int64_t sb, ss, sh;
  } ops[] = {{"q", a->q, true, a->q_sb, a->q_st, a->q_sh},
             {"out", a->out, true, a->o_sb, a->o_st, a->o_sh},
             {"k_prefix", a->k_prefix, a->P > 0, 0, a->kp_sp, a->kp_sh},
             {"v_prefix", a->v_prefix, a->P > 0, 0, a->vp_sp, a->vp_sh},
             {"k_own", a->k_own, a->S > 0, a->ko_sb, a->ko_ss, a->ko_sh},
             {"v_own", a->v_own, a->S > 0, a->vo_sb, a->vo_ss, a->vo_sh}};
  for (const Op& o : ops) {
    if (!o.used) continue;
    if ((st = check_pointer(fn, o.what, o.p, 16)) != W4A4_OK) return st;
    if ((st = check_batch_stride(fn, o.what, o.sb)) != W4A4_OK) return st;
    if ((st = check_stride(fn, o.what, o.ss)) != W4A4_OK) return st;
    if ((st = check_stride(fn, o.what, o.sh)) != W4A4_OK) return st;
  }
  if (a->own_len && !aligned(a->own_len, 4)) return fail(W4A4_ERR_MISALIGNED, "%s: own_len misaligned", fn);
  const size_t need = w4a4::prefix_attention_workspace(a->B, a->T, a->Hq, a->Hkv, a->D, a->P, a->S);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != W4A4_OK) return st;
  return launch_status(w4a4::launch_prefix_attention(*a, need ? workspace : nullptr, (hipStream_t)stream), fn);
}

size_t w4a4_prefix_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t P, int64_t S) {
  if (check_attn_sizes("w4a4_prefix_attention_workspace", B, T, Hq, Hkv, D, P, S) != W4A4_OK || B == 0 || T == 0) return 0;
  return w4a4::prefix_attention_workspace(B, T, Hq, Hkv, D, P, S);
}

static int check_dense_sizes(const char* fn, int64_t M, int64_t N, int64_t K, int32_t act) {
  if (M < 0 || N < 0 || K <= 0) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (K % 8 != 0) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: K=%lld not a multiple of 8", fn, (long long)K);
  // (N is bounded by y's row stride)
  if (K > (1LL << 21) || M > (1LL << 30) || N > (1LL << 22) || (N > 0 && M > (1LL << 37) / N))
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: sizes too large", fn);
  if (act < W4A4_ACT_NONE || act > W4A4_ACT_SWIGLU)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: unknown activation %d", fn, act);
  return ok();
}

int bf16_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t M, int64_t N, int64_t K,
                const w4a4_epilogue* ep, void* y, int32_t y_dtype, int64_t ldy, void* workspace,
                size_t workspace_bytes, void* stream) {
  const char* fn = "bf16_linear";
  const w4a4_epilogue none = {W4A4_ACT_NONE, W4A4_DT_F32, nullptr, nullptr, 0};
  if (!ep) ep = &none;
  int st = check_dense_sizes(fn, M, N, K, ep->act);
  if (st != W4A4_OK) return st;
  if (y_dtype != W4A4_DT_F32 && y_dtype != W4A4_DT_BF16)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: y dtype %d not F32/BF16", fn, y_dtype);
  if (ep->bias && ep->bias_dtype != W4A4_DT_F32 && ep->bias_dtype != W4A4_DT_BF16)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: bias dtype %d not F32/BF16", fn, ep->bias_dtype);
  if (ldx < K || ldw < K || ldy < N || (ep->residual && ep->ldr < N))
    return fail(W4A4_ERR_INVALID_ARG, "%s: row stride below the row length", fn);
  if (ldx % 8 != 0 || ldw % 8 != 0) return fail(W4A4_ERR_MISALIGNED, "%s: ldx / ldw not a multiple of 8", fn);
  const int64_t top = 1LL << 22;
  if (ldx > top / 2 || ldw > top / 2 || ldy > top || (ep->residual && ep->ldr > top))
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: row stride too large", fn);
  if (M == 0 || N == 0) return ok();
  const size_t ysz = y_dtype == W4A4_DT_BF16 ? 2 : 4;
  if ((st = check_pointer(fn, "x", x, 16)) != W4A4_OK) return st;
  if ((st = check_pointer(fn, "w", w, 16)) != W4A4_OK) return st;
  if ((st = check_pointer(fn, "y", y, ysz)) != W4A4_OK) return st;
  if (ep->bias && !aligned(ep->bias, ep->bias_dtype == W4A4_DT_BF16 ? 2 : 4))
    return fail(W4A4_ERR_MISALIGNED, "%s: bias misaligned", fn);
  if (ep->residual && !aligned(ep->residual, ysz)) return fail(W4A4_ERR_MISALIGNED, "%s: residual misaligned", fn);
  if (ep->residual == y && ep->residual && ep->ldr != ldy)
    return fail(W4A4_ERR_INVALID_ARG, "%s: residual in place needs ldr == ldy", fn);
  const size_t need = w4a4::gemm_bf16_workspace(M, N, K, ep->act);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != W4A4_OK) return st;
  w4a4::DenseArgs g{};
  g.x = (const uint16_t*)x;
  g.w = (const uint16_t*)w;
  g.ldx = ldx;
  g.ldw = ldw;
  g.M = (int)M;
  g.N = (int)N;
  g.K = (int)K;
  g.act = ep->act;
  g.bias = ep->bias;
  g.bias_bf16 = ep->bias_dtype == W4A4_DT_BF16;
  g.residual = ep->residual;
  g.ldr = ep->ldr;
  g.y = y;
  g.y_bf16 = y_dtype == W4A4_DT_BF16;
  g.ldy = ldy;
  return launch_status(w4a4::launch_gemm_bf16(g, need ? workspace : nullptr, (hipStream_t)stream), fn);
}

size_t w4a4_bf16_workspace_size(int64_t M, int64_t N, int64_t K, int32_t act) {
  if (check_dense_sizes("w4a4_bf16_workspace_size", M, N, K, act) != W4A4_OK || M == 0 || N == 0) return 0;
  return w4a4::gemm_bf16_workspace(M, N, K, act);
}

static int check_norm_sizes(const char* fn, int64_t N, int64_t S, int64_t C, int64_t groups) {
  if (N < 0 || S < 0 || C <= 0 || groups <= 0) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (C % groups != 0)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %lld channels in %lld groups", fn, (long long)C, (long long)groups);
  if (C > 65536 || N > (1LL << 30) || S > (1LL << 30) || S > (1LL << 40) / C || N * groups > INT32_MAX)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: sizes too large", fn);
  return ok();
}

int w4a4_group_norm_act(const void* x, int32_t dtype, int64_t N, int64_t S, int64_t C, int64_t groups, int64_t x_sn,
                        int64_t x_ss, const float* weight, const float* bias, float eps, int32_t act, void* y,
                        int64_t y_sn, int64_t y_ss, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "w4a4_group_norm_act";
  int st = check_norm_sizes(fn, N, S, C, groups);
  if (st != W4A4_OK) return st;
  if (dtype != W4A4_DT_F32 && dtype != W4A4_DT_BF16)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: dtype %d not F32/BF16", fn, dtype);
  if (act < W4A4_ACT_NONE || act > W4A4_ACT_SILU)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: unknown activation %d", fn, act);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(W4A4_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (x_ss < C || y_ss < C || x_sn < 0 || y_sn < 0)
    return fail(W4A4_ERR_INVALID_ARG, "%s: position stride below C or negative sample stride", fn);
  if (x_ss > (1LL << 40) || y_ss > (1LL << 40)) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: position stride", fn);
  if (N == 0 || S == 0) return ok();
  const size_t sz = dtype == W4A4_DT_BF16 ? 2 : 4;
  if ((st = check_pointer(fn, "x", x, sz)) != W4A4_OK) return st;
  if ((st = check_pointer(fn, "y", y, sz)) != W4A4_OK) return st;
  if ((weight && !aligned(weight, 4)) || (bias && !aligned(bias, 4)))
    return fail(W4A4_ERR_MISALIGNED, "%s: weight / bias misaligned", fn);
  if (x == y && (x_ss != y_ss || x_sn != y_sn))
    return fail(W4A4_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  const size_t need = w4a4::group_norm_workspace(N, S, C, groups);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != W4A4_OK) return st;
  w4a4::NormArgs g{};
  g.x = x;
  g.y = y;
  g.bf16 = dtype == W4A4_DT_BF16;
  g.N = N;
  g.S = S;
  g.C = (int)C;
  g.groups = (int)groups;
  g.x_sn = x_sn;
  g.x_ss = x_ss;
  g.y_sn = y_sn;
  g.y_ss = y_ss;
  g.weight = weight;
  g.bias = bias;
  g.eps = eps;
  g.act = act;
  return launch_status(w4a4::launch_group_norm(g, need ? workspace : nullptr, (hipStream_t)stream), fn);
}

size_t w4a4_group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups) {
  if (check_norm_sizes("w4a4_group_norm_workspace", N, S, C, groups) != W4A4_OK || N == 0 || S == 0) return 0;
  return w4a4::group_norm_workspace(N, S, C, groups);
}

}  // extern "C"
