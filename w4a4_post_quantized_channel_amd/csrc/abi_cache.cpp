// C ABI of the operators around the 4-bit key/value cache: host-side argument
// checks and dispatch.  Every check runs before any launch.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/w4a4.h"
#include "abi_util.h"
#include "cache.h"
#include "cache_attention_plan.h"

using w4a4::aligned;
using w4a4::fail;
using w4a4::launch_status;
using w4a4::ok;

namespace {

int check_pointer(const char* fn, const char* what, const void* p, size_t al) {
  if (!p) return fail(W4A4_ERR_INVALID_ARG, "%s: %s is NULL", fn, what);
  if (!aligned(p, al)) return fail(W4A4_ERR_MISALIGNED, "%s: %s not %zu-byte aligned", fn, what, al);
  return ok();
}

// Strides are bounded so that (rows * stride) cannot pass 63 bits.
int check_stride(const char* fn, const char* what, int64_t s, int64_t multiple) {
  if (s < 0) return fail(W4A4_ERR_INVALID_ARG, "%s: negative %s stride", fn, what);
  if (s % multiple != 0)
    return fail(W4A4_ERR_MISALIGNED, "%s: %s stride %lld not a multiple of %lld", fn, what, (long long)s,
                (long long)multiple);
  if (s > (1LL << 30)) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %s stride above 2^30", fn, what);
  return ok();
}

// Rows of an output lie apart.
int check_apart(const char* fn, const char* what, int64_t s, int64_t row) {
  return s < row ? fail(W4A4_ERR_INVALID_ARG, "%s: %s stride below the row length", fn, what) : ok();
}

int check_float(const char* fn, const char* what, int32_t dtype) {
  if (dtype != W4A4_DT_F32 && dtype != W4A4_DT_BF16)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: %s dtype %d not F32/BF16", fn, what, dtype);
  return ok();
}

int check_head(const char* fn, int64_t Hkv, int64_t D) {
  if (Hkv <= 0) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (D != 64 && D != 128 && D != 256)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: head width %lld is not 64, 128 or 256", fn, (long long)D);
  if (Hkv > 65536) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: more than 65536 KV heads", fn);
  return ok();
}

int check_cache(const char* fn, const w4a4_kvcache* c) {
  if (!c) return fail(W4A4_ERR_INVALID_ARG, "%s: NULL cache", fn);
  int st = check_head(fn, c->Hkv, c->D);
  if (st != W4A4_OK) return st;
  if (c->n_pages <= 0) return fail(W4A4_ERR_INVALID_ARG, "%s: a cache has at least one page", fn);
  const int64_t p = c->page;
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: page of %lld tokens is not 16, 32, 64, 128 or 256", fn, (long long)p);
  if (c->n_pages > INT32_MAX / p) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: 2^31 tokens or more", fn);
  if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !std::isfinite(c->k_scale) || !std::isfinite(c->v_scale))
    return fail(W4A4_ERR_INVALID_ARG, "%s: the cache's scales must be positive and finite", fn);
  const struct {
    const char* what;
    const void* p;
    int64_t sp, row;
  } arrays[] = {{"k_codes", c->k_codes, c->k_codes_sp, c->D / 2},
                {"k_scales", c->k_scales, c->k_scales_sp, c->D / 16},
                {"v_codes", c->v_codes, c->v_codes_sp, c->D / 2},
                {"v_scales", c->v_scales, c->v_scales_sp, c->D / 16}};
  for (const auto& a : arrays) {
    if ((st = check_pointer(fn, a.what, a.p, 16)) != W4A4_OK) return st;
    if (a.sp < c->Hkv * p * a.row)
      return fail(W4A4_ERR_INVALID_ARG, "%s: %s page stride below a page's size", fn, a.what);
    if (a.sp % 16 != 0) return fail(W4A4_ERR_MISALIGNED, "%s: %s page stride not a multiple of 16", fn, a.what);
    if (a.sp > (1LL << 40) / c->n_pages)
      return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %s spans more than 2^40 bytes", fn, a.what);
  }
  return ok();
}

int check_io(const char* fn, const w4a4_kvcache* c, const void* k, int64_t k_sm, int64_t k_sh, const void* v,
             int64_t v_sm, int64_t v_sh, int32_t dtype, int64_t M, const int32_t* slots, bool written) {
  int st = check_cache(fn, c);
  if (st != W4A4_OK) return st;
  if ((st = check_float(fn, "k / v", dtype)) != W4A4_OK) return st;
  if (M < 0) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  // (the grid counts fewer than 2^32 threads, one per 16 channels of k and v)
  if (M > INT32_MAX || M > (1LL << 34) / (c->Hkv * c->D))
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: too many tokens", fn);
  if (M == 0) return ok();
  const struct {
    const char* what;
    const void* p;
    int64_t sm, sh;
  } rows[] = {{"k", k, k_sm, k_sh}, {"v", v, v_sm, v_sh}};
  for (const auto& r : rows) {
    if ((st = check_pointer(fn, r.what, r.p, 16)) != W4A4_OK) return st;
    if (M > 1 && (st = check_stride(fn, r.what, r.sm, 8)) != W4A4_OK) return st;
    if (c->Hkv > 1 && (st = check_stride(fn, r.what, r.sh, 8)) != W4A4_OK) return st;
    if (!written) continue;
    if (M > 1 && (st = check_apart(fn, r.what, r.sm, c->D)) != W4A4_OK) return st;
    if (c->Hkv > 1 && (st = check_apart(fn, r.what, r.sh, c->D)) != W4A4_OK) return st;
  }
  return check_pointer(fn, "slots", slots, 4);
}

w4a4::CacheIo cache_io(const w4a4_kvcache* c, const void* k, int64_t k_sm, int64_t k_sh, const void* v, int64_t v_sm,
                       int64_t v_sh, int32_t dtype, int64_t M, const int32_t* slots) {
  w4a4::CacheIo a{};
  a.c = *c;
  a.M = M;
  a.slots = slots;
  a.f32 = dtype == W4A4_DT_F32;
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  // the stride of a dimension of one is not used and may be anything
  a.k_sm = M > 1 ? k_sm : 0;
  a.v_sm = M > 1 ? v_sm : 0;
  a.k_sh = c->Hkv > 1 ? k_sh : 0;
  a.v_sh = c->Hkv > 1 ? v_sh : 0;
  return a;
}

// Sizes of w4a4_cache_attention; also the workspace query's check.
int check_attn_sizes(const char* fn, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len) {
  int st = check_head(fn, Hkv, D);
  if (st != W4A4_OK) return st;
  if (B < 0 || T < 0 || max_len < 0 || Hq <= 0) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (Hq % Hkv != 0)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %lld query heads over %lld KV heads", fn, (long long)Hq, (long long)Hkv);
  // (the grid counts fewer than 2^32 threads, 512 or fewer per 16 rows of a sequence and KV head)
  if (Hq > 65536 || max_len > (1LL << 30) || T > (1LL << 24) || B > (1LL << 24) || B * T > (1LL << 30) / Hq ||
      B * Hkv * ((T * (Hq / Hkv) + 15) / 16) > (1LL << 22))
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: sizes too large", fn);
  return ok();
}

}  // namespace

extern "C" {

int w4a4_cache_append(const w4a4_kvcache* c, const void* k, int64_t k_sm, int64_t k_sh, const void* v, int64_t v_sm,
                      int64_t v_sh, int32_t dtype, int64_t M, const int32_t* slots, void* stream) {
  const char* fn = "w4a4_cache_append";
  const int st = check_io(fn, c, k, k_sm, k_sh, v, v_sm, v_sh, dtype, M, slots, false);
  if (st != W4A4_OK || M == 0) return st;
  return launch_status(
      w4a4::launch_cache_append(cache_io(c, k, k_sm, k_sh, v, v_sm, v_sh, dtype, M, slots), (hipStream_t)stream), fn);
}

int w4a4_cache_read(const w4a4_kvcache* c, const int32_t* slots, int64_t M, void* k, int64_t k_sm, int64_t k_sh,
                    void* v, int64_t v_sm, int64_t v_sh, int32_t dtype, void* stream) {
  const char* fn = "w4a4_cache_read";
  const int st = check_io(fn, c, k, k_sm, k_sh, v, v_sm, v_sh, dtype, M, slots, true);
  if (st != W4A4_OK || M == 0) return st;
  return launch_status(
      w4a4::launch_cache_read(cache_io(c, k, k_sm, k_sh, v, v_sm, v_sh, dtype, M, slots), (hipStream_t)stream), fn);
}

int w4a4_cache_attention(const w4a4_kvcache* c, const w4a4_cache_attn* desc, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const char* fn = "w4a4_cache_attention";
  int st = check_cache(fn, c);
  if (st != W4A4_OK) return st;
  if (!desc) return fail(W4A4_ERR_INVALID_ARG, "%s: NULL descriptor", fn);
  w4a4_cache_attn copy = *desc;
  w4a4_cache_attn* a = &copy;
  // the stride of a dimension of one is not used and may be anything
  if (a->B == 1) a->q_sb = a->o_sb = a->table_sb = 0;
  if (a->T == 1) a->q_st = a->o_st = 0;
  if (a->Hq == 1) a->q_sh = a->o_sh = 0;
  if ((st = check_attn_sizes(fn, a->B, a->T, a->Hq, c->Hkv, c->D, a->max_len)) != W4A4_OK) return st;
  if (!std::isfinite(a->scale)) return fail(W4A4_ERR_INVALID_ARG, "%s: scale not finite", fn);
  if (a->causal != 0 && a->causal != 1) return fail(W4A4_ERR_INVALID_ARG, "%s: causal must be 0 or 1", fn);
  if (a->table_pages < 0) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (a->table_pages > (1LL << 30) / c->page)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: a table of more than 2^30 tokens", fn);
  if (a->B == 0 || a->T == 0) return ok();
  const struct {
    const char* what;
    const void* p;
    int64_t sb, st, sh;
  } rows[] = {{"q", a->q, a->q_sb, a->q_st, a->q_sh}, {"out", a->out, a->o_sb, a->o_st, a->o_sh}};
  for (const auto& r : rows) {
    if ((st = check_pointer(fn, r.what, r.p, 16)) != W4A4_OK) return st;
    if (r.sb < 0) return fail(W4A4_ERR_INVALID_ARG, "%s: negative %s batch stride", fn, r.what);
    if (r.sb % 8 != 0) return fail(W4A4_ERR_MISALIGNED, "%s: %s batch stride not a multiple of 8", fn, r.what);
    if (r.sb > (1LL << 38)) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %s batch stride above 2^38", fn, r.what);
    if ((st = check_stride(fn, r.what, r.st, 8)) != W4A4_OK) return st;
    if ((st = check_stride(fn, r.what, r.sh, 8)) != W4A4_OK) return st;
  }
  if ((a->B > 1 && (st = check_apart(fn, "out", a->o_sb, c->D)) != W4A4_OK) ||
      (a->T > 1 && (st = check_apart(fn, "out", a->o_st, c->D)) != W4A4_OK) ||
      (a->Hq > 1 && (st = check_apart(fn, "out", a->o_sh, c->D)) != W4A4_OK))
    return st;
  if (a->table_pages > 0 && (st = check_pointer(fn, "table", a->table, 4)) != W4A4_OK) return st;
  if (a->table_sb < 0 || (a->B > 1 && a->table_sb > (1LL << 38)))
    return fail(W4A4_ERR_INVALID_ARG, "%s: bad table stride", fn);
  if ((st = check_pointer(fn, "lens", a->lens, 4)) != W4A4_OK) return st;
  const size_t need = w4a4::cache_attention_workspace(a->B, a->T, a->Hq, c->Hkv, c->D, a->max_len);
  if (workspace) {
    if (workspace_bytes < need)
      return fail(W4A4_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace_bytes, need);
    if (!aligned(workspace, 16)) return fail(W4A4_ERR_MISALIGNED, "%s: workspace not 16-byte aligned", fn);
  }
  return launch_status(w4a4::launch_cache_attention(*c, *a, need ? workspace : nullptr, (hipStream_t)stream), fn);
}

size_t w4a4_cache_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len) {
  if (check_attn_sizes("w4a4_cache_attention_workspace", B, T, Hq, Hkv, D, max_len) != W4A4_OK || B == 0 || T == 0)
    return 0;
  // A shorter history can need more: its keys go into more parts.
  size_t most = 0;
  const int64_t blocks = w4a4::plan_blocks(max_len);
  for (int64_t n = 1; n <= blocks; n += w4a4::plan_step(n)) {
    const size_t need = w4a4::cache_attention_workspace(B, T, Hq, Hkv, D, n * w4a4::kCacheBlock);
    if (need > most) most = need;
  }
  return most;
}

int w4a4_rotary_axes(const w4a4_rotary* desc, void* stream) {
  const char* fn = "w4a4_rotary_axes";
  if (!desc) return fail(W4A4_ERR_INVALID_ARG, "%s: NULL descriptor", fn);
  w4a4_rotary r = *desc;
  if (r.M < 0 || r.Hq <= 0 || r.Hk < 0 || r.D <= 0) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (r.M > INT32_MAX || r.Hq > 65536 || r.Hk > 65536 || r.Hq + r.Hk > 65536 || r.D > 1024 || r.D % 2 != 0)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: sizes too large or an odd head width", fn);
  int st = check_float(fn, "q / k", r.dtype);
  if (st != W4A4_OK) return st;
  if (r.pos_dtype != W4A4_DT_I32 && r.pos_dtype != W4A4_DT_F32)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: positions' dtype %d not I32/F32", fn, r.pos_dtype);
  if (r.axes < 1 || r.axes > 4) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %d axes, 1 to 4 are taken", fn, r.axes);
  if (r.pairs != W4A4_PAIRS_ADJACENT && r.pairs != W4A4_PAIRS_HALVES)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: unknown pairing %d", fn, r.pairs);
  int64_t pairs = 0;
  for (int a = 0; a < 4; ++a) {
    if (r.sections[a] < 0 || (a >= r.axes && r.sections[a] != 0))
      return fail(W4A4_ERR_INVALID_ARG, "%s: bad section of axis %d", fn, a);
    pairs += r.sections[a];
  }
  if (pairs < 1 || 2 * pairs > r.D)
    return fail(W4A4_ERR_INVALID_ARG, "%s: sections of %lld pairs in a head of %lld", fn, (long long)pairs, (long long)r.D);
  if (r.M == 0) return ok();
  const size_t sz = r.dtype == W4A4_DT_BF16 ? 2 : 4;
  // the stride of a dimension of one is not used and may be anything
  if (r.M == 1) r.q_sm = r.qo_sm = r.k_sm = r.ko_sm = r.pos_sm = 0;
  if (r.Hq == 1) r.q_sh = r.qo_sh = 0;
  if (r.Hk <= 1) r.k_sh = r.ko_sh = 0;
  const struct {
    const char* what;
    const void* p;
    int64_t sm, sh, heads;
    bool written;
  } rows[] = {{"q", r.q, r.q_sm, r.q_sh, r.Hq, false},
              {"q_out", r.q_out, r.qo_sm, r.qo_sh, r.Hq, true},
              {"k", r.k, r.k_sm, r.k_sh, r.Hk, false},
              {"k_out", r.k_out, r.ko_sm, r.ko_sh, r.Hk, true}};
  for (const auto& t : rows) {
    if (t.heads == 0) continue;
    if ((st = check_pointer(fn, t.what, t.p, sz)) != W4A4_OK) return st;
    if ((st = check_stride(fn, t.what, t.sm, 1)) != W4A4_OK) return st;
    if ((st = check_stride(fn, t.what, t.sh, 1)) != W4A4_OK) return st;
    if (!t.written) continue;
    if (r.M > 1 && (st = check_apart(fn, t.what, t.sm, r.D)) != W4A4_OK) return st;
    if (t.heads > 1 && (st = check_apart(fn, t.what, t.sh, r.D)) != W4A4_OK) return st;
  }
  if ((r.q == r.q_out && (r.q_sm != r.qo_sm || r.q_sh != r.qo_sh)) ||
      (r.Hk > 0 && r.k == r.k_out && (r.k_sm != r.ko_sm || r.k_sh != r.ko_sh)))
    return fail(W4A4_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  if ((st = check_pointer(fn, "pos", r.pos, 4)) != W4A4_OK) return st;
  if ((st = check_stride(fn, "pos", r.pos_sm, 1)) != W4A4_OK) return st;
  if ((st = check_pointer(fn, "table", r.table, 8)) != W4A4_OK) return st;
  return launch_status(w4a4::launch_rotary_axes(r, (hipStream_t)stream), fn);
}

int w4a4_gated_norm(const w4a4_gated* desc, void* stream) {
  const char* fn = "w4a4_gated_norm";
  if (!desc) return fail(W4A4_ERR_INVALID_ARG, "%s: NULL descriptor", fn);
  w4a4_gated g = *desc;
  if (g.M < 0 || g.C <= 0 || g.R < (g.M > 0)) return fail(W4A4_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (g.C > 16384 || g.M > INT32_MAX) return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: sizes too large", fn);
  if (g.R > 0 && g.M % g.R != 0)
    return fail(W4A4_ERR_UNSUPPORTED_SHAPE, "%s: %lld rows over %lld rows of modulations", fn, (long long)g.M,
                (long long)g.R);
  int st = check_float(fn, "x", g.x_dtype);
  if (st != W4A4_OK) return st;
  if (g.h && (st = check_float(fn, "h", g.h_dtype)) != W4A4_OK) return st;
  if (g.y && (st = check_float(fn, "y", g.y_dtype)) != W4A4_OK) return st;
  if (g.kind != W4A4_NORM_LAYER && g.kind != W4A4_NORM_RMS)
    return fail(W4A4_ERR_UNSUPPORTED_FORMAT, "%s: unknown norm %d", fn, g.kind);
  if (!(g.eps >= 0.f) || !std::isfinite(g.eps)) return fail(W4A4_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (!std::isfinite(g.alpha)) return fail(W4A4_ERR_INVALID_ARG, "%s: alpha not finite", fn);
  if (g.M == 0) return ok();
  if (!g.x_out && !g.y) return fail(W4A4_ERR_INVALID_ARG, "%s: neither x_out nor y is wanted", fn);
  if (!g.h && (g.gate || g.post_weight))
    return fail(W4A4_ERR_INVALID_ARG, "%s: gate and post_weight belong to h, which is NULL", fn);
  const struct {
    const char* what;
    const void* p;
    int64_t ld, rows;
    size_t size;
    bool used;
  } mats[] = {{"x", g.x, g.ldx, g.M, g.x_dtype == W4A4_DT_BF16 ? 2u : 4u, true},
              {"h", g.h, g.ldh, g.M, g.h_dtype == W4A4_DT_BF16 ? 2u : 4u, g.h != nullptr},
              {"x_out", g.x_out, g.ldxo, g.M, g.x_dtype == W4A4_DT_BF16 ? 2u : 4u, g.x_out != nullptr},
              {"y", g.y, g.ldy, g.M, g.y_dtype == W4A4_DT_BF16 ? 2u : 4u, g.y != nullptr},
              {"gate", g.gate, g.gate_sr, g.R, 4, g.gate != nullptr},
              {"scale", g.scale, g.scale_sr, g.R, 4, g.scale != nullptr},
              {"shift", g.shift, g.shift_sr, g.R, 4, g.shift != nullptr},
              {"post_weight", g.post_weight, 0, 1, 4, g.post_weight != nullptr},
              {"weight", g.weight, 0, 1, 4, g.weight != nullptr},
              {"bias", g.bias, 0, 1, 4, g.bias != nullptr}};
  for (const auto& m : mats) {
    if (!m.used) continue;
    if ((st = check_pointer(fn, m.what, m.p, m.size)) != W4A4_OK) return st;
    if (m.rows == 1) continue;   // the stride of a dimension of one is not used and may be anything
    if ((st = check_stride(fn, m.what, m.ld, 1)) != W4A4_OK) return st;
  }
  if (g.M > 1 && ((g.x_out && g.ldxo < g.C) || (g.y && g.ldy < g.C)))
    return fail(W4A4_ERR_INVALID_ARG, "%s: an output's row stride below C", fn);
  if (g.M > 1 && g.x_out == g.x && g.ldx != g.ldxo)
    return fail(W4A4_ERR_INVALID_ARG, "%s: in place needs equal strides", fn);
  if (g.M == 1) g.ldx = g.ldh = g.ldxo = g.ldy = 0;
  if (g.R == 1) g.gate_sr = g.scale_sr = g.shift_sr = 0;
  return launch_status(w4a4::launch_gated_norm(g, (hipStream_t)stream), fn);
}

}  // extern "C"
