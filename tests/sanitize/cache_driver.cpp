// Drives the argument checks of the operators around the 4-bit cache under the
// host sanitizers: rejected calls launch nothing and set a message, accepted
// ones launch once.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "../../include/w4a4.h"
#include "../../w4a4_post_quantized_channel_amd/csrc/cache.h"

extern int g_launches;

namespace w4a4 {
hipError_t launch_cache_append(const CacheIo&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_cache_read(const CacheIo&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_cache_attention(const w4a4_kvcache&, const w4a4_cache_attn&, void*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
size_t cache_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t max_len) {
  return max_len > 4096 ? 1 << 20 : 0;
}
hipError_t launch_rotary_axes(const w4a4_rotary&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_gated_norm(const w4a4_gated&, hipStream_t) { ++g_launches; return hipSuccess; }
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
int32_t* ints() { return reinterpret_cast<int32_t*>(mem); }

w4a4_kvcache cache() {
  w4a4_kvcache c{};
  c.n_pages = 8; c.page = 16; c.Hkv = 2; c.D = 64;
  c.k_scale = c.v_scale = 0.25f;
  c.k_codes = c.v_codes = c.k_scales = c.v_scales = mem;
  c.k_codes_sp = c.v_codes_sp = 1024;
  c.k_scales_sp = c.v_scales_sp = 128;
  return c;
}

w4a4_cache_attn attn() {
  w4a4_cache_attn a{};
  a.B = 2; a.T = 3; a.Hq = 4; a.max_len = 100;
  a.scale = 0.125f;
  a.q = mem; a.out = mem + 2048;
  a.q_sb = a.o_sb = 768; a.q_st = a.o_st = 256; a.q_sh = a.o_sh = 64;
  a.table = ints(); a.table_sb = 7; a.table_pages = 7; a.lens = ints();
  return a;
}

w4a4_rotary rotary() {
  w4a4_rotary r{};
  r.M = 5; r.Hq = 4; r.Hk = 2; r.D = 64;
  r.dtype = W4A4_DT_BF16; r.pos_dtype = W4A4_DT_I32; r.axes = 3;
  r.sections[0] = 12; r.sections[1] = r.sections[2] = 10;
  r.pos = mem; r.pos_sm = 3; r.table = (const float*)mem;
  r.q = r.k = mem; r.q_out = r.k_out = mem + 1024;
  r.q_sm = r.qo_sm = 256; r.k_sm = r.ko_sm = 128;
  r.q_sh = r.qo_sh = r.k_sh = r.ko_sh = 64;
  return r;
}

w4a4_gated gated() {
  w4a4_gated g{};
  g.M = 6; g.C = 40; g.R = 2; g.alpha = 1.f; g.eps = 1e-6f;
  g.x_dtype = W4A4_DT_F32; g.h_dtype = g.y_dtype = W4A4_DT_BF16;
  g.x = mem; g.h = mem + 1024; g.x_out = mem; g.y = mem + 2048;
  g.ldx = g.ldh = g.ldxo = g.ldy = 40;
  g.gate = g.scale = g.shift = (const float*)mem;
  g.gate_sr = g.scale_sr = g.shift_sr = 120;
  g.post_weight = g.weight = g.bias = (const float*)mem;
  return g;
}

#define ATTN(change, want)                                             \
  do {                                                                 \
    w4a4_kvcache c = cache();                                          \
    w4a4_cache_attn a = attn();                                        \
    change;                                                            \
    const int before = g_launches;                                     \
    expect("attention: " #change, w4a4_cache_attention(&c, &a, nullptr, 0, nullptr), want, before); \
  } while (0)

struct Io {
  const void* k = mem;
  const void* v = mem;
  int64_t k_sm = 128, k_sh = 64, v_sm = 128, v_sh = 64, M = 9;
  int32_t dtype = W4A4_DT_BF16;
  const int32_t* slots = ints();
};
#define IO(change, append, read)                                       \
  do {                                                                 \
    w4a4_kvcache c = cache();                                          \
    Io i;                                                              \
    change;                                                            \
    int before = g_launches;                                           \
    expect("append: " #change, w4a4_cache_append(&c, i.k, i.k_sm, i.k_sh, i.v, i.v_sm, i.v_sh, i.dtype, i.M, i.slots, nullptr), append, before); \
    before = g_launches;                                               \
    expect("read: " #change, w4a4_cache_read(&c, i.slots, i.M, (void*)i.k, i.k_sm, i.k_sh, (void*)i.v, i.v_sm, i.v_sh, i.dtype, nullptr), read, before); \
  } while (0)

#define ROTARY(change, want)                                           \
  do {                                                                 \
    w4a4_rotary r = rotary();                                          \
    change;                                                            \
    const int before = g_launches;                                     \
    expect("rotary: " #change, w4a4_rotary_axes(&r, nullptr), want, before); \
  } while (0)

#define GATED(change, want)                                            \
  do {                                                                 \
    w4a4_gated g = gated();                                            \
    change;                                                            \
    const int before = g_launches;                                     \
    expect("gated: " #change, w4a4_gated_norm(&g, nullptr), want, before); \
  } while (0)
}  // namespace

int main() {
  // the cache itself
  IO(, 0, 0);
  IO(c.D = 96, -2, -2);
  IO(c.Hkv = 0, -1, -1);
  IO(c.Hkv = 1 << 20, -2, -2);
  IO(c.n_pages = 0, -1, -1);
  IO(c.page = 24, -2, -2);
  IO(c.page = 8, -2, -2);
  IO(c.page = 512, -2, -2);
  IO(c.n_pages = 1LL << 28, -2, -2);
  IO(c.k_scale = 0.f, -1, -1);
  IO(c.v_scale = -1.f, -1, -1);
  IO(c.v_scale = NAN, -1, -1);
  IO(c.k_scale = INFINITY, -1, -1);
  IO(c.k_codes = nullptr, -1, -1);
  IO(c.v_scales = mem + 8, -3, -3);
  IO(c.v_codes_sp = 1008, -1, -1);
  IO(c.k_scales_sp = 112, -1, -1);
  IO(c.k_scales_sp = 136, -3, -3);
  IO(c.k_codes_sp = 1LL << 42, -2, -2);
  // rows
  IO(i.k = nullptr, -1, -1);
  IO(i.v = mem + 8, -3, -3);
  IO(i.k_sm = 132, -3, -3);
  IO(i.v_sh = -8, -1, -1);
  IO(i.v_sm = 1LL << 31, -2, -2);
  IO(i.k_sm = 0, 0, -1);           // one row for all tokens may be read, not written
  IO(i.v_sh = 32, 0, -1);
  IO(i.M = -1, -1, -1);
  IO(i.M = 1LL << 31, -2, -2);
  IO(i.dtype = W4A4_DT_I32, -4, -4);
  IO(i.slots = nullptr, -1, -1);
  IO(i.slots = (const int32_t*)(mem + 2), -3, -3);
  IO(i.M = 1; i.k_sm = -3; i.v_sm = 5, 0, 0);
  IO(c.Hkv = 1; i.k_sh = -3; i.v_sh = 5, 0, 0);
  {
    const int before = g_launches;
    w4a4_kvcache c = cache();
    if (w4a4_cache_append(&c, nullptr, 0, 0, nullptr, 0, 0, W4A4_DT_BF16, 0, nullptr, nullptr) != 0 ||
        w4a4_cache_read(&c, nullptr, 0, nullptr, 0, 0, nullptr, 0, 0, W4A4_DT_F32, nullptr) != 0 || g_launches != before)
      ++failures;
    expect("append: NULL", w4a4_cache_append(nullptr, mem, 0, 0, mem, 0, 0, W4A4_DT_BF16, 1, ints(), nullptr), -1, before);
  }

  ATTN(, 0);
  ATTN(c.D = 32, -2);
  ATTN(c.k_codes = nullptr, -1);
  ATTN(a.Hq = 5, -2);
  ATTN(a.Hq = 0, -1);
  ATTN(a.B = -1, -1);
  ATTN(a.max_len = -1, -1);
  ATTN(a.max_len = 1LL << 31, -2);
  ATTN(a.B = 1 << 20; a.T = 1 << 20, -2);
  ATTN(a.scale = NAN, -1);
  ATTN(a.causal = 2, -1);
  ATTN(a.q = nullptr, -1);
  ATTN(a.out = mem + 8, -3);
  ATTN(a.q_st = 260, -3);
  ATTN(a.q_sh = -64, -1);
  ATTN(a.q_sb = 1LL << 40, -2);
  ATTN(a.o_st = 0, -1);
  ATTN(a.o_sh = 32, -1);
  ATTN(a.table = nullptr, -1);
  ATTN(a.table = (const int32_t*)(mem + 2), -3);
  ATTN(a.table_sb = -1, -1);
  ATTN(a.table_pages = -1, -1);
  ATTN(a.table_pages = 1LL << 40, -2);
  ATTN(a.lens = nullptr, -1);
  ATTN(a.table_pages = 0; a.table = nullptr, 0);
  ATTN(a.max_len = 0, 0);
  ATTN(a.B = 1; a.q_sb = a.o_sb = a.table_sb = -1, 0);
  ATTN(a.T = 1; a.q_st = a.o_st = -1, 0);
  {
    const int before = g_launches;
    w4a4_kvcache c = cache();
    w4a4_cache_attn a = attn();
    a.max_len = 8192;
    expect("attention: small workspace", w4a4_cache_attention(&c, &a, mem, 16, nullptr), -5, before);
    expect("attention: misaligned workspace", w4a4_cache_attention(&c, &a, mem + 4, 1 << 20, nullptr), -3, before);
    expect("attention: NULL", w4a4_cache_attention(&c, nullptr, nullptr, 0, nullptr), -1, before);
    expect("attention: NULL cache", w4a4_cache_attention(nullptr, &a, nullptr, 0, nullptr), -1, before);
    a.B = 0;
    a.q = nullptr;
    if (w4a4_cache_attention(&c, &a, nullptr, 0, nullptr) != 0 || g_launches != before) ++failures;
    if (w4a4_cache_attention_workspace(-1, 1, 1, 1, 64, 1) || w4a4_cache_attention_workspace(1, 1, 1, 0, 64, 8192) ||
        w4a4_cache_attention_workspace(1, 1, 1, 1, 63, 8192) || !w4a4_cache_attention_workspace(1, 1, 1, 1, 64, 8192))
      ++failures;
  }

  ROTARY(, 0);
  ROTARY(r.Hk = 0; r.k = nullptr; r.k_out = nullptr, 0);
  ROTARY(r.q_out = (void*)r.q; r.k_out = (void*)r.k, 0);
  ROTARY(r.q_out = (void*)r.q; r.qo_sm = 512, -1);
  ROTARY(r.M = -1, -1);
  ROTARY(r.Hq = 0, -1);
  ROTARY(r.Hk = -1, -1);
  ROTARY(r.D = 63, -2);
  ROTARY(r.D = 2048, -2);
  ROTARY(r.M = 1LL << 32, -2);
  ROTARY(r.Hq = 65536; r.Hk = 1, -2);
  ROTARY(r.dtype = W4A4_DT_I32, -4);
  ROTARY(r.pos_dtype = W4A4_DT_BF16, -4);
  ROTARY(r.pairs = 2, -4);
  ROTARY(r.axes = 0, -2);
  ROTARY(r.axes = 5, -2);
  ROTARY(r.axes = 2, -1);
  ROTARY(r.sections[1] = -1, -1);
  ROTARY(r.sections[0] = 13, -1);
  ROTARY(r.sections[0] = r.sections[1] = r.sections[2] = 0, -1);
  ROTARY(r.q = nullptr, -1);
  ROTARY(r.k_out = nullptr, -1);
  ROTARY(r.q = mem + 1, -3);
  ROTARY(r.pos = nullptr, -1);
  ROTARY(r.table = nullptr, -1);
  ROTARY(r.table = (const float*)(mem + 4), -3);
  ROTARY(r.q_sm = -1, -1);
  ROTARY(r.qo_sm = 0, -1);
  ROTARY(r.ko_sh = 63, -1);
  ROTARY(r.k_sh = 1LL << 31, -2);
  ROTARY(r.M = 1; r.q_sm = r.qo_sm = r.k_sm = r.ko_sm = r.pos_sm = -1, 0);
  {
    const int before = g_launches;
    w4a4_rotary r = rotary();
    r.M = 0;
    r.q = nullptr;
    if (w4a4_rotary_axes(&r, nullptr) != 0 || g_launches != before) ++failures;
    expect("rotary: NULL", w4a4_rotary_axes(nullptr, nullptr), -1, before);
  }

  GATED(, 0);
  GATED(g.h = nullptr, -1);
  GATED(g.h = nullptr; g.gate = nullptr; g.post_weight = nullptr, 0);
  GATED(g.x_out = nullptr, 0);
  GATED(g.y = nullptr, 0);
  GATED(g.y = nullptr; g.x_out = nullptr, -1);
  GATED(g.R = 0, -1);
  GATED(g.R = 4, -2);
  GATED(g.C = 0, -1);
  GATED(g.C = 16385, -2);
  GATED(g.M = -1, -1);
  GATED(g.M = 1LL << 32, -2);
  GATED(g.eps = -1.f, -1);
  GATED(g.eps = NAN, -1);
  GATED(g.alpha = INFINITY, -1);
  GATED(g.kind = 2, -4);
  GATED(g.x_dtype = W4A4_DT_I32, -4);
  GATED(g.h_dtype = 9, -4);
  GATED(g.y_dtype = 9, -4);
  GATED(g.x = nullptr, -1);
  GATED(g.x = mem + 2, -3);
  GATED(g.y = mem + 1, -3);
  GATED(g.gate = (const float*)(mem + 2), -3);
  GATED(g.ldh = -1, -1);
  GATED(g.ldh = 0, 0);             // one row of h for all
  GATED(g.ldy = 39, -1);
  GATED(g.ldxo = 80, -1);          // in place with another stride
  GATED(g.scale_sr = 1LL << 31, -2);
  GATED(g.M = 1; g.R = 1; g.ldx = g.ldh = g.ldxo = g.ldy = g.gate_sr = -1, 0);
  {
    const int before = g_launches;
    w4a4_gated g = gated();
    g.M = 0;
    g.x = nullptr;
    if (w4a4_gated_norm(&g, nullptr) != 0 || g_launches != before) ++failures;
    g.R = 0;
    if (w4a4_gated_norm(&g, nullptr) != 0 || g_launches != before) ++failures;
    expect("gated: NULL", w4a4_gated_norm(nullptr, nullptr), -1, before);
  }
  std::printf("ok: %d failures\n", failures);
  return failures != 0;
}
