// Writing keys and values to the NVFP4 cache, and reading them back.
//
// Mathematics.  16 channels of a row share one scale: e = E4M3(amax / 6 / g),
// codes E2M1(x / (e g)), every quotient the correctly rounded one
// (nvfp4_block16, the activation quantizer's own); a value read is code * e *
// g.  Products code * e have at most six significant bits, so with g a power
// of two they are exact in bf16.
//
// A thread takes one block of 16 channels; a workgroup a run of tokens of one
// head, so that tokens which follow each other in a page are written, and read,
// in whole lines, while a token's head is D * 2 bytes side by side on the other
// end.
//
// Bound by memory: 12480 tokens of 16 heads of 128, bf16 (102 MB and 29 MB of
// cache), append in 23.4 us (5.6 TB/s, part of it from the last-level cache) and
// read in 28.1 (4.7); a workgroup per token, all its heads, took 72 in all.  One
// token of each of 64 sequences is a launch, the slot, the row and the
// quotients: 3.5 us each.
#include "cache.h"
#include "device_common.h"
#include "divisor.h"
#include "nvfp4_block.h"

namespace w4a4 {

namespace {

struct Args {
  CacheIo io;
  int lnb, lp;        // log2 of the blocks of a row and of the tokens of a page
  int run;            // tokens of a workgroup
  Divisor heads;      // 2 Hkv: keys, then values
};

// Block of 16 channels of the call: token, head, k or v, block of the row.
struct Place {
  bool live, v;
  int64_t m;
  int h, blk;
  int64_t page;       // -1: the slot is outside the cache
  int tok;
};

__device__ __forceinline__ Place place(const Args& p) {
  const CacheIo& a = p.io;
  Place q;
  int hv;
  const int first = div_by((int)blockIdx.x, p.heads, hv);
  q.v = hv >= (int)a.c.Hkv;
  q.h = q.v ? hv - (int)a.c.Hkv : hv;
  q.blk = threadIdx.x & ((1 << p.lnb) - 1);
  q.m = (int64_t)first * p.run + (threadIdx.x >> p.lnb);
  q.live = q.m < a.M;
  q.page = -1;
  q.tok = 0;
  if (!q.live) return q;
  const int slot = a.slots[q.m];
  if (slot >= 0 && slot < (int)(a.c.n_pages << p.lp)) q.page = slot >> p.lp;
  q.tok = slot & ((1 << p.lp) - 1);
  return q;
}

template <bool F32>
__global__ void __launch_bounds__(256) cache_append_kernel(Args p) {
  const CacheIo& a = p.io;
  __shared__ float2 steps[128];      // (e g, 1 / (e g)) of every scale code
  const Place q = place(p);
  const float g = q.v ? a.c.v_scale : a.c.k_scale;
  const int64_t off = (q.v ? q.m * a.v_sm + q.h * a.v_sh : q.m * a.k_sm + q.h * a.k_sh) + q.blk * 16;
  const void* src = q.v ? a.v : a.k;
  float x[16];
  // the row first, then the table; a row that is skipped reads nothing
  if (q.page < 0) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = 0.f;
  } else if constexpr (F32) {
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
  if (threadIdx.x < 128) {
    const int e = threadIdx.x;
    const float S = e < 0x7F ? e4m3_to_f32((uint32_t)e) * g : 0.f;
    steps[e] = make_float2(S, S > 0.f ? 1.0f / S : 0.f);
  }
  __syncthreads();
  if (q.page < 0) return;
  uint2 codes;
  const uint32_t e = nvfp4_block16(x, 1.f, g, 1.f / g, g >= kTinyStep && g <= kBig, steps, true, codes);
  const int64_t row = ((int64_t)q.h << p.lp) + q.tok;
  uint8_t* cd = (uint8_t*)(q.v ? a.c.v_codes : a.c.k_codes) + q.page * (q.v ? a.c.v_codes_sp : a.c.k_codes_sp);
  uint8_t* sc = (uint8_t*)(q.v ? a.c.v_scales : a.c.k_scales) + q.page * (q.v ? a.c.v_scales_sp : a.c.k_scales_sp);
  *reinterpret_cast<uint2*>(cd + row * (a.c.D / 2) + q.blk * 8) = codes;
  sc[row * (a.c.D / 16) + q.blk] = (uint8_t)e;
}

template <bool F32>
__global__ void __launch_bounds__(256) cache_read_kernel(Args p) {
  const CacheIo& a = p.io;
  const Place q = place(p);
  if (!q.live) return;
  uint2 codes = make_uint2(0, 0);
  float s = 0.f;
  if (q.page >= 0) {
    const int64_t row = ((int64_t)q.h << p.lp) + q.tok;
    const uint8_t* cd = (const uint8_t*)(q.v ? a.c.v_codes : a.c.k_codes) + q.page * (q.v ? a.c.v_codes_sp : a.c.k_codes_sp);
    const uint8_t* sc = (const uint8_t*)(q.v ? a.c.v_scales : a.c.k_scales) + q.page * (q.v ? a.c.v_scales_sp : a.c.k_scales_sp);
    codes = *reinterpret_cast<const uint2*>(cd + row * (a.c.D / 2) + q.blk * 8);
    s = e4m3_to_f32(sc[row * (a.c.D / 16) + q.blk] & 0x7Fu);
  }
  const float g = q.v ? a.c.v_scale : a.c.k_scale;
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t c = ((j < 8 ? codes.x : codes.y) >> (4 * (j & 7))) & 15u;
    const uint32_t n = c & 7u;
    const float mag = n < 2 ? 0.5f * n : __uint_as_float(((n >> 1) + 126u) << 23 | (n & 1u) << 22);
    x[j] = (c & 8u ? -mag : mag) * s * g;   // the first product is exact
  }
  const int64_t off = (q.v ? q.m * a.v_sm + q.h * a.v_sh : q.m * a.k_sm + q.h * a.k_sh) + q.blk * 16;
  void* dst = q.v ? a.v : a.k;
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

Args args_of(const CacheIo& io, unsigned& grid) {
  Args p{};
  p.io = io;
  p.lnb = io.c.D == 64 ? 2 : io.c.D == 128 ? 3 : 4;
  p.lp = io.c.page == 16 ? 4 : io.c.page == 32 ? 5 : io.c.page == 64 ? 6 : io.c.page == 128 ? 7 : 8;
  p.run = 256 >> p.lnb;
  p.heads = divisor(2 * io.c.Hkv);
  grid = (unsigned)((io.M + p.run - 1) / p.run * 2 * io.c.Hkv);
  return p;
}

}  // namespace

hipError_t launch_cache_append(const CacheIo& a, hipStream_t st) {
  unsigned grid;
  const Args p = args_of(a, grid);
  if (a.f32) cache_append_kernel<true><<<grid, 256, 0, st>>>(p);
  else cache_append_kernel<false><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheIo& a, hipStream_t st) {
  unsigned grid;
  const Args p = args_of(a, grid);
  if (a.f32) cache_read_kernel<true><<<grid, 256, 0, st>>>(p);
  else cache_read_kernel<false><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace w4a4
