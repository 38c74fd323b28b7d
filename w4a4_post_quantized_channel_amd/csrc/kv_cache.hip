// Writing keys and values to the NVFP4 cache, and reading them back.
//
// Mathematics.  16 channels of a row share one scale: e = E4M3(amax / 6 / g),
// codes E2M1(x / (e g)), every quotient the correctly rounded one
// (nvfp4_block16, the activation quantizer's own); a value read is code * e *
// g.  Products code * e have at most six significant bits, so with g a power
// of two they are exact in bf16.
//
// A thread takes one block of 16 channels.
#include "cache.h"
#include "device_common.h"
#include "nvfp4_block.h"

namespace w4a4 {

namespace {

// Block of 16 channels `i` of the call: token, head, k or v, block of the row.
struct Place {
  int64_t m;
  int h, blk;
  bool v;
  int64_t page;   // -1: the slot is outside the cache
  int tok;
};

__device__ __forceinline__ Place place(const CacheIo& a, int64_t i) {
  const int nb = (int)a.c.D / 16, H = (int)a.c.Hkv;
  Place p;
  p.blk = (int)(i % nb);
  i /= nb;
  p.h = (int)(i % H);
  i /= H;
  p.v = i & 1;
  p.m = i >> 1;
  const int slot = a.slots[p.m], page = (int)a.c.page;
  p.page = slot >= 0 && slot < (int)(a.c.n_pages * page) ? slot / page : -1;
  p.tok = slot % page;
  return p;
}

__device__ __forceinline__ int64_t row_of(const CacheIo& a, const Place& p) {   // within a page
  return p.h * a.c.page + p.tok;
}

template <bool F32>
__global__ void __launch_bounds__(256) cache_append_kernel(CacheIo a) {
  __shared__ float2 steps[2][128];   // (e g, 1 / (e g)) of every scale code
  {
    const int t = threadIdx.x, e = t & 127;
    const float S = e < 0x7F ? e4m3_to_f32((uint32_t)e) * (t < 128 ? a.c.k_scale : a.c.v_scale) : 0.f;
    steps[t >> 7][e] = make_float2(S, S > 0.f ? 1.0f / S : 0.f);
  }
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * 2 * a.c.Hkv * (a.c.D / 16)) return;
  const Place p = place(a, i);
  if (p.page < 0) return;
  const int64_t off = (p.v ? p.m * a.v_sm + p.h * a.v_sh : p.m * a.k_sm + p.h * a.k_sh) + p.blk * 16;
  const void* src = p.v ? a.v : a.k;
  float x[16];
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const v4f w = reinterpret_cast<const v4f*>((const float*)src + off)[j];
#pragma unroll
      for (int n = 0; n < 4; ++n) x[4 * j + n] = w[n];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const v4i w = reinterpret_cast<const v4i*>((const uint16_t*)src + off)[j];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        x[8 * j + 2 * n] = __uint_as_float((uint32_t)w[n] << 16);
        x[8 * j + 2 * n + 1] = __uint_as_float((uint32_t)w[n] & 0xFFFF0000u);
      }
    }
  }
  const float g = p.v ? a.c.v_scale : a.c.k_scale;
  uint2 codes;
  const uint32_t e = nvfp4_block16(x, 1.f, g, 1.f / g, g >= kTinyStep && g <= kBig, steps[p.v], true, codes);
  const int64_t row = row_of(a, p);
  uint8_t* cd = (uint8_t*)(p.v ? a.c.v_codes : a.c.k_codes) + p.page * (p.v ? a.c.v_codes_sp : a.c.k_codes_sp);
  uint8_t* sc = (uint8_t*)(p.v ? a.c.v_scales : a.c.k_scales) + p.page * (p.v ? a.c.v_scales_sp : a.c.k_scales_sp);
  *reinterpret_cast<uint2*>(cd + row * (a.c.D / 2) + p.blk * 8) = codes;
  sc[row * (a.c.D / 16) + p.blk] = (uint8_t)e;
}

template <bool F32>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheIo a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * 2 * a.c.Hkv * (a.c.D / 16)) return;
  const Place p = place(a, i);
  uint2 codes = make_uint2(0, 0);
  float s = 0.f;
  if (p.page >= 0) {
    const int64_t row = row_of(a, p);
    const uint8_t* cd = (const uint8_t*)(p.v ? a.c.v_codes : a.c.k_codes) + p.page * (p.v ? a.c.v_codes_sp : a.c.k_codes_sp);
    const uint8_t* sc = (const uint8_t*)(p.v ? a.c.v_scales : a.c.k_scales) + p.page * (p.v ? a.c.v_scales_sp : a.c.k_scales_sp);
    codes = *reinterpret_cast<const uint2*>(cd + row * (a.c.D / 2) + p.blk * 8);
    s = e4m3_to_f32(sc[row * (a.c.D / 16) + p.blk] & 0x7Fu);
  }
  const float g = p.v ? a.c.v_scale : a.c.k_scale;
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t c = ((j < 8 ? codes.x : codes.y) >> (4 * (j & 7))) & 15u;
    const uint32_t n = c & 7u;
    const float mag = n < 2 ? 0.5f * n : __uint_as_float(((n >> 1) + 126u) << 23 | (n & 1u) << 22);
    x[j] = (c & 8u ? -mag : mag) * s * g;   // the first product is exact
  }
  const int64_t off = (p.v ? p.m * a.v_sm + p.h * a.v_sh : p.m * a.k_sm + p.h * a.k_sh) + p.blk * 16;
  void* dst = p.v ? a.v : a.k;
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      reinterpret_cast<v4f*>((float*)dst + off)[j] = (v4f){x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v4i w;
#pragma unroll
      for (int n = 0; n < 4; ++n)
        w[n] = (int)(f32_to_bf16_bits(x[8 * j + 2 * n]) | f32_to_bf16_bits(x[8 * j + 2 * n + 1]) << 16);
      reinterpret_cast<v4i*>((uint16_t*)dst + off)[j] = w;
    }
  }
}

unsigned grid_of(const CacheIo& a) {
  const int64_t n = a.M * 2 * a.c.Hkv * (a.c.D / 16);
  return (unsigned)((n + 255) / 256);
}

}  // namespace

hipError_t launch_cache_append(const CacheIo& a, hipStream_t st) {
  if (a.f32) cache_append_kernel<true><<<grid_of(a), 256, 0, st>>>(a);
  else cache_append_kernel<false><<<grid_of(a), 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheIo& a, hipStream_t st) {
  if (a.f32) cache_read_kernel<true><<<grid_of(a), 256, 0, st>>>(a);
  else cache_read_kernel<false><<<grid_of(a), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace w4a4
