// Attention over the 4-bit key/value cache.
//
// A wave takes one query head of one token: 64 keys at a time, one a lane,
// their scores, the running maximum and sum of the softmax, then the values
// channel by channel.
#include "cache.h"
#include "device_common.h"

namespace w4a4 {

namespace {

__device__ __forceinline__ float e2m1(uint32_t c) {
  const uint32_t n = c & 7u;
  const float mag = n < 2 ? 0.5f * n : __uint_as_float(((n >> 1) + 126u) << 23 | (n & 1u) << 22);
  return c & 8u ? -mag : mag;
}

template <int D>
__global__ void __launch_bounds__(64) attn_row_kernel(w4a4_kvcache c, w4a4_cache_attn a) {
  __shared__ float q[D], ps[64];
  __shared__ int pages[64];
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int h = (int)(row % a.Hq), t = (int)(row / a.Hq % a.T), b = (int)(row / a.Hq / a.T);
  const int hk = h / (int)(a.Hq / c.Hkv), page = (int)c.page;
  for (int d = lane; d < D; d += 64)
    q[d] = bf16_bits_to_f32(((const uint16_t*)a.q)[b * a.q_sb + t * a.q_st + h * a.q_sh + d]) * a.scale * c.k_scale;
  int64_t len = a.lens[b];
  len = len < a.max_len ? len : a.max_len;
  len = len < a.table_pages * page ? len : a.table_pages * page;
  if (a.causal) len = len - a.T + t + 1;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[D / 64] = {};
  for (int64_t j0 = 0; j0 < len; j0 += 64) {
    const int64_t j = j0 + lane;
    int pg = -1;
    if (j < len) pg = a.table[b * a.table_sb + j / page];
    if (pg < 0 || pg >= c.n_pages) pg = -1;
    float s = -INFINITY;
    if (pg >= 0) {
      const int64_t r = (int64_t)hk * page + j % page;
      const uint8_t* cd = (const uint8_t*)c.k_codes + pg * c.k_codes_sp + r * (D / 2);
      const uint8_t* sc = (const uint8_t*)c.k_scales + pg * c.k_scales_sp + r * (D / 16);
      s = 0.f;
      for (int k = 0; k < D / 16; ++k) {
        float x = 0.f;
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = cd[k * 8 + i];
          x += e2m1(w) * q[k * 16 + 2 * i] + e2m1(w >> 4) * q[k * 16 + 2 * i + 1];
        }
        s += x * e4m3_to_f32(sc[k] & 0x7Fu);
      }
    }
    float mx = s;
    for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
    const float p = pg >= 0 ? expf(s - ms) : 0.f, f = expf(m - ms);
    m = mn;
    l = l * f + p;
    ps[lane] = p;
    pages[lane] = pg;
    __syncthreads();
    for (int e = 0; e < D / 64; ++e) {
      const int d = e * 64 + lane;
      float acc = 0.f;
      for (int k = 0; k < 64; ++k) {
        if (pages[k] < 0) continue;
        const int64_t r = (int64_t)hk * page + (j0 + k) % page;
        const uint32_t w = ((const uint8_t*)c.v_codes)[pages[k] * c.v_codes_sp + r * (D / 2) + d / 2];
        const uint32_t sc = ((const uint8_t*)c.v_scales)[pages[k] * c.v_scales_sp + r * (D / 16) + d / 16];
        acc += ps[k] * (e2m1(d & 1 ? w >> 4 : w) * e4m3_to_f32(sc & 0x7Fu));
      }
      o[e] = o[e] * f + acc;
    }
    __syncthreads();
  }
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  const float inv = l == 0.f ? 0.f : c.v_scale / l;
  for (int e = 0; e < D / 64; ++e)
    ((__bf16*)a.out)[b * a.o_sb + t * a.o_st + h * a.o_sh + e * 64 + lane] = (__bf16)(o[e] * inv);
}

}  // namespace

size_t cache_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len) {
  (void)B, (void)T, (void)Hq, (void)Hkv, (void)D, (void)max_len;
  return 0;
}

hipError_t launch_cache_attention(const w4a4_kvcache& c, const w4a4_cache_attn& a, void* workspace, hipStream_t st) {
  (void)workspace;
  const unsigned grid = (unsigned)(a.B * a.T * a.Hq);
  if (c.D == 64) attn_row_kernel<64><<<grid, 64, 0, st>>>(c, a);
  else if (c.D == 128) attn_row_kernel<128><<<grid, 64, 0, st>>>(c, a);
  else attn_row_kernel<256><<<grid, 64, 0, st>>>(c, a);
  return hipGetLastError();
}

}  // namespace w4a4
