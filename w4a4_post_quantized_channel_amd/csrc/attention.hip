// Attention of a batch over one shared prefix and each sequence's own keys.
//
// One wave per query row: 64 keys at a time, a lane per key for the scores
// and a lane per D / 64 columns for the values, with the running maximum m
// and sum l of the softmax (acc and l are rescaled by exp(m_old - m_new)
// whenever m grows).
#include "dense.h"
#include "device_common.h"

namespace w4a4 {

namespace {

template <int D>
__global__ void __launch_bounds__(64) attn_row_kernel(w4a4_attn a) {
  __shared__ float qs[D], ps[64];
  const int lane = threadIdx.x;
  const int64_t id = blockIdx.x;
  const int h = (int)(id % a.Hq), t = (int)(id / a.Hq % a.T);
  const int64_t b = id / (a.Hq * a.T);
  const int hk = h / (int)(a.Hq / a.Hkv);
  const float c2 = a.scale * 1.4426950408889634f;   // exp(scale s) = exp2(c2 s)
  const uint16_t* q = (const uint16_t*)a.q + b * a.q_sb + t * a.q_st + h * a.q_sh;
  for (int d = lane; d < D; d += 64) qs[d] = bf16_bits_to_f32(q[d]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc[D / 64] = {};
  auto block = [&](const uint16_t* k, int64_t ks, const uint16_t* v, int64_t vs, int64_t j0, int64_t end,
                   const uint8_t* keep) {
    const int64_t j = j0 + lane;
    float s = -INFINITY;
    if (j < end && (!keep || keep[j])) {
      float dot = 0.f;
      for (int d = 0; d < D; d += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(k + j * ks + d);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += qs[d + e] * bf16_bits_to_f32((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
      }
      s = dot * c2;
    }
    float mx = s;
    for (int o = 32; o; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    const float mn = fmaxf(m, mx);
    const float ms = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ms), p = exp2f(s - ms);
    m = mn;
    l = l * f + p;
    ps[lane] = p;
    __syncthreads();
    for (int e = 0; e < D / 64; ++e) acc[e] *= f;
    for (int jj = 0; jj < 64 && j0 + jj < end; ++jj) {
      if (keep && !keep[j0 + jj]) continue;
      for (int e = 0; e < D / 64; ++e) acc[e] += ps[jj] * bf16_bits_to_f32(v[(j0 + jj) * vs + lane + 64 * e]);
    }
    __syncthreads();
  };
  for (int64_t j0 = 0; j0 < a.P; j0 += 64)
    block((const uint16_t*)a.k_prefix + hk * a.kp_sh, a.kp_sp, (const uint16_t*)a.v_prefix + hk * a.vp_sh, a.vp_sp, j0,
          a.P, a.prefix_keep);
  int64_t end = a.own_len ? min((int64_t)max(a.own_len[b], 0), a.S) : a.S;
  if (a.causal) end = max(min(end, end - a.T + 1 + t), (int64_t)0);
  for (int64_t j0 = 0; j0 < end; j0 += 64)
    block((const uint16_t*)a.k_own + b * a.ko_sb + hk * a.ko_sh, a.ko_ss,
          (const uint16_t*)a.v_own + b * a.vo_sb + hk * a.vo_sh, a.vo_ss, j0, end, nullptr);
  for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o);
  uint16_t* out = (uint16_t*)a.out + b * a.o_sb + t * a.o_st + h * a.o_sh;
  for (int e = 0; e < D / 64; ++e)
    out[lane + 64 * e] = (uint16_t)f32_to_bf16_bits(l > 0.f ? acc[e] / l : l == 0.f ? 0.f : NAN);
}

}  // namespace

size_t prefix_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_prefix_attention(const w4a4_attn& a, void*, hipStream_t st) {
  const dim3 grid((unsigned)(a.B * a.T * a.Hq));
  if (a.D == 64) attn_row_kernel<64><<<grid, 64, 0, st>>>(a);
  else if (a.D == 128) attn_row_kernel<128><<<grid, 64, 0, st>>>(a);
  else attn_row_kernel<256><<<grid, 64, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace w4a4
