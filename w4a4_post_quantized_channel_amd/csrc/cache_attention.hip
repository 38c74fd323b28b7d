// Attention over the 4-bit key/value cache.
//
// Mathematics.  The rows of a sequence and KV head are its queries (row = t G
// + g, G query heads per KV head).  Keys come in blocks of 64; a row keeps its
// running maximum m (in units of exp2), its sum l and its output o in fp32:
//   p = 2^b exp2(c s - m),  l += sum p,  o += p V,   c = scale log2 e * k_scale.
// m only moves when a score exceeds it by more than kLazy: until then p is at
// most 2^(b + kLazy), which costs no accuracy (p and l scale alike), and o and l
// need no rescaling.  b (kFewUp, kManyUp) puts p into the upper part of fp16's
// range, so that what a long history's small probabilities lose below 2^-14 is
// 2^-25 against a sum of at least 2^b.
//
// Types.  A cached value code * e (E2M1 times E4M3, at most six significant
// bits, 2^-10 to 2880) is exact in fp16, so both products run on fp16 matrix
// instructions with nothing lost on the cache's side; the static scales k_scale
// and v_scale enter c and the last division.  A query row is multiplied by the
// power of two that puts its largest channel at 2^13: bf16's eight bits then
// fit fp16 for every channel down to 2^-27 of the largest.  Probabilities are
// rounded to fp16 (off by 2^-11 of them, an eighth of the output's own rounding:
// in fp32 or as two fp16 numbers the second product would take twice as long).
//
// A wave works alone on every NW-th block of its workgroup's part, for
// 16 MT rows at once:
//  - S^T = K Q^T with v_mfma_f32_16x16x32_f16.  The order of channels inside a
//    product is free, so lane (key r, group g) takes the D / 4 channels from
//    g D / 4: they lie side by side, and a key's codes go from global memory
//    straight into the operand (convert, times scale), never through LDS.
//  - O^T = V^T P^T takes keys as the inner index.  A lane holds of its query
//    the scores of keys 16 t + 4 g + i, and P^T takes them in that order, so P
//    never moves between lanes.  V's codes go through LDS as they are, and the
//    4-bit transposing read (16 rows x 16 channels per 16 lanes) hands each
//    lane 16 keys of one channel in the same order; their scales lie in LDS as
//    fp16, one row of 64 keys per 16 channels.
// The waves' (m, l, o) are joined through LDS, the parts through the workspace
// by a second kernel.
//
// What bounds it.  One token each of 64 sequences, 32 heads over 8 of 128, 4096
// to 8192 keys: the caches' 463 MB at 5.5 TB/s, 84 us (a device copy reaches
// 5.1).  There each key is read by one workgroup only, past the caches (at widths
// 128 and 256): 92 us against 102 with ordinary loads (7% slower where the
// history fits the 256 MB cache and is read again at once), and in one part: 85
// against 89 in two and 92 in three.  Parts follow max_len: where one sequence of
// a batch is far longer than the rest, its workgroups walk it alone.  A chunk of
// 8 x 50 queries, 16 heads over 4, 2090 keys (21 us): turns
// of 7000 cycles in which two waves a SIMD convert codes (1150 cycles a block and
// wave), multiply (1024) and take exponentials (600), one after the other for
// each wave; 64 rows a wave convert half as often but leave one wave a SIMD: 34.
// Blocks of absent pages take the time of others.  2 x 13 queries, 8 heads over
// one of 256, 5131 keys (14.4 us and 2.8 of join): one
// turn a wave; seven row tiles read the same keys through the L2s, 4 MB each.
// One workgroup's call (1 query, 317 keys) takes 5.5 to 6 us: arguments, lens and
// table, keys and the join wait for each other (the table waiting for lens: 0.3
// more; a second barrier in the join: 0.3 more).
#include "cache.h"
#include "cache_attention_plan.h"
#include "device_common.h"
#include "divisor.h"

namespace w4a4 {

namespace {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i lds_v2i;

constexpr float kLazy = 8.f, kFewUp = 7.f;   // p < 2^15
// Where |m| reaches this its last place, an eighth and more, is no small part of
// what p may grow by (from 2^24 on p passed fp16, or all of a row's were lost).
// Such a row's scores are summed from minus a base on, the score that m stands
// for.  The kernel for many rows always starts its sums there (no time at width
// 128, 2% at 64); the one for few takes its keys once more, with bases, where a
// row turns out to need one: in its loop they cost 2 to 7%.
constexpr float kFar = 1048576.f;
constexpr int BN = kCacheBlock;

struct Args {
  w4a4_kvcache c;
  w4a4_cache_attn a;
  int rows;              // T G rows of a sequence and KV head
  int lp;                // log2 of the page
  Divisor g, tiles, heads, parts;
  float c2, cpost;       // > 0: |scale| log2 e k_scale = c2 * cpost
  float qmul;            // 1, -1 (scale < 0) or 0 (scale of zero: c2 is 1)
  float v, vpost;        // v_scale = v * vpost: v over a sum of weights is no subnormal number
  float* po;             // parts > 1: [part][b][head][row][D], else null
  float* pml;            // [part][b][head][row][2]
};

// N bytes of a lane's codes or scales, in 32-bit words.
template <int BYTES>
struct Words {
  static constexpr int N = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t w[N];
};
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
// ONCE: no other workgroup reads them, and they leave the caches first (16 bytes
// or more; width 64 takes 8 and reads them in the ordinary way).
template <int BYTES, bool ONCE = false>
__device__ __forceinline__ Words<BYTES> load_words(const uint8_t* p) {
  Words<BYTES> r;
  if constexpr (BYTES == 1) r.w[0] = *p;
  else if constexpr (BYTES == 2) r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  else if constexpr (BYTES == 4) r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const u4* a = reinterpret_cast<const u4*>(p) + i;
      const u4 v = ONCE ? __builtin_nontemporal_load(a) : *a;
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

// E4M3 magnitude times 2^-8 as fp16: the seven bits are an fp16 number's upper
// ones with another bias (subnormals included; 0x7F reads as 480).
__device__ __forceinline__ uint32_t scale_bits(uint32_t byte) { return (byte & 0x7Fu) << 7; }
__device__ __forceinline__ v2h both(uint32_t bits) { return __builtin_bit_cast(v2h, bits | bits << 16); }

// Eight codes times 2^8 times their scales (as scale_bits gives them, in pairs).
__device__ __forceinline__ v8h decode8(uint32_t w, v2h s0, v2h s1, v2h s2, v2h s3) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.f, 0) * s0;
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.f, 1) * s1;
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.f, 2) * s2;
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.f, 3) * s3;
  return (v8h){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Maximum and sum over the four lane groups that hold a query.
__device__ __forceinline__ float group_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float group_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2bf));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2h));
}

// Four outputs as bf16.
__device__ __forceinline__ uint2 pack_out(const Args& p, v4f x) {
  x *= p.vpost;
  return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

// The factor 2^(13 - floor(log2 amax)) of a query row, and its inverse.  Rows
// of infinities keep theirs (factor 2^-114: Inf stays Inf), zeros stay zero.
__device__ __forceinline__ float row_factor(float amax, float& inverse) {
  int e = (int)(__float_as_uint(amax) >> 23);
  e = e < 14 ? 14 : e > 254 ? 254 : e;
  inverse = __uint_as_float((uint32_t)(e - 13) << 23);
  return __uint_as_float((uint32_t)(267 - e) << 23);
}

// What turns a row's scores into units of exp2.  Never zero (-inf, which is
// excluded, times it stays -inf) and never infinite (zero times it stays zero).
__device__ __forceinline__ float score_factor(const Args& p, float inverse) {
  return fminf(fmaxf(p.c2 * inverse * p.cpost, 1.17549435e-38f), 3.40282347e38f);
}

// The next m of a row that moves to its scores' maximum ``most``, and what its
// scores, taken relative to minus ``from``, change by.  Beside a base m is what
// that was rounded by, or, where this is far as well, left out.
__device__ __forceinline__ float rebase(bool moves, float most, float factor, float& m, float from) {
  if (!moves) return 0.f;
  const float top = most - from, full = top * factor;
  if (__builtin_fabsf(full) < kFar) {
    m = full;
    return -from;
  }
  const float step = -top - from, rest = (most + step) * factor;
  const bool far = __builtin_fabsf(rest) >= kFar;
  m = far ? 0.f : rest;
  return far ? -most : step;
}
// At the end: m as other sums of the row know it, rounded, and the factor that
// what was taken relative to the exact one gets for that (a last place of 60 and
// more is left as it is: scores that differ by less than it differ by their own
// rounding).
__device__ __forceinline__ float to_m(float from, float factor, float& m) {
  if (from == 0.f) return 1.f;
  const float rest = m;
  m = __builtin_fmaf(-from, factor, rest);
  return __builtin_amdgcn_exp2f(fminf(fmaxf(__builtin_fmaf(-from, factor, -m) + rest, -30.f), 30.f));
}

template <int D_, int MT_, int NW_, bool ONCE_>
struct Few {
  static constexpr int D = D_, MT = MT_, NW = NW_, R = 16 * MT;
  static constexpr bool ONCE = ONCE_;           // one row tile: every key is read by one workgroup
  static constexpr int KS = D / 32;             // steps of the first product
  static constexpr int DT = D / 16;             // channel tiles, scales of a row
  static constexpr int CB = D / 8;              // bytes of codes a lane takes of a key
  static constexpr int VCH = D / 16;            // 8-byte chunks of a value row
  static constexpr int VCODES = BN * D / 2, VSCALES = DT * BN * 2;
  static constexpr int WAVE = VCODES + VSCALES;
  static constexpr int PITCH = D + 4;           // floats of a row in the join
  static constexpr int JOIN = NW * R * (PITCH + 2) * 4;
  static constexpr int LDS = NW * WAVE > JOIN ? NW * WAVE : JOIN;
};

// Keys a query row sees: those below its limit.
struct Limit {
  int len, reach, back;      // keys of the sequence; keys there can be; T if causal
  __device__ __forceinline__ Limit(const Args& p, int b) {
    len = max(p.a.lens[b], 0);
    reach = (int)min(p.a.max_len, p.a.table_pages << p.lp);
    back = p.a.causal ? (int)p.a.T : 0;
  }
  __device__ __forceinline__ int operator()(int t) const { return min(back ? len - back + t + 1 : len, reach); }
};

template <typename C>
__global__ void __launch_bounds__(64 * C::NW, 2) attn_few_kernel(Args p) {
  constexpr int D = C::D, MT = C::MT, NW = C::NW, R = C::R, KS = C::KS, DT = C::DT;
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // workgroup -> (sequence, head, part, tile): the tiles that read the same
  // keys follow each other on an XCD
  const int nwg = gridDim.x, wid = blockIdx.x;
  const int u = nwg % 8 == 0 ? (wid % 8) * (nwg / 8) + wid / 8 : wid;
  int tile, part, hk;
  const int b = div_by(div_by(div_by(u, p.tiles, tile), p.parts, part), p.heads, hk);
  const w4a4_kvcache& c = p.c;
  const w4a4_cache_attn& a = p.a;
  const int G = (int)p.g.d, page = 1 << p.lp;

  // Table entries of a block's four groups of 16 keys, one a lane group, whether
  // held or not (without a table any integer).  Neither this load nor those of a
  // block is ever left out, so that waits can count the younger ones: past the
  // end all lanes read the first bytes of page 0 (one request instead of one a
  // line).
  const int entries = (int)a.table_pages;
  const int32_t* table = entries > 0 ? a.table + b * a.table_sb : a.lens;
  auto load_pages = [&](int blk) { return table[max(min((blk * BN + 16 * lg) >> p.lp, entries - 1), 0)]; };
  int pg = 0, pg1 = 0;
  if (part == 0) pg = load_pages(wave), pg1 = load_pages(wave + NW);   // while lens is on its way

  const int r0 = tile * R, nrows = min(R, p.rows - r0);
  int rem;
  const Limit limit(p, b);
  const int first = limit(div_by(r0, p.g, rem));            // the tile's lowest limit
  const int last = limit(div_by(r0 + nrows - 1, p.g, rem));   // and highest
  const int nblk = (max(last, 0) + BN - 1) / BN;
  const int per = (nblk + (int)p.parts.d - 1) / (int)p.parts.d;
  const int lo = min(part * per, nblk), hi = min(lo + per, nblk);
  if (part != 0) pg = load_pages(lo + wave), pg1 = load_pages(lo + wave + NW);

  Words<C::CB> kw[4], vw[4];        // a block's codes and scales: K by tiles of 16 keys
  Words<C::CB / 8> ksw[4];
  Words<DT> vsw;
  uint32_t bad = 0;                 // groups whose page is absent
  const uint8_t* kc = (const uint8_t*)c.k_codes + (int64_t)hk * page * (D / 2);
  const uint8_t* ks = (const uint8_t*)c.k_scales + (int64_t)hk * page * DT;
  const uint8_t* vc = (const uint8_t*)c.v_codes + (int64_t)hk * page * (D / 2);
  const uint8_t* vs = (const uint8_t*)c.v_scales + (int64_t)hk * page * DT;
  const uint32_t kco = lr * (D / 2) + lg * C::CB, kso = lr * DT + lg * (DT / 4), vco = lane * C::CB;
  // an entry of a block; -1: the page is absent, or past the end (page 0 is read then, its keys are excluded)
  const int end = min(last, hi * BN);
  auto held = [&](int blk, int pg) { return blk * BN + 16 * lg < end && (uint32_t)pg < (uint32_t)c.n_pages ? pg : -1; };
  auto load_k = [&](int blk, int pg) {
    const uint64_t x = __ballot(pg < 0);
    bad = (uint32_t)(x & 1) | (uint32_t)(x >> 15 & 2) | (uint32_t)(x >> 30 & 4) | (uint32_t)(x >> 45 & 8);
    pg = max(pg, 0);
    const bool in = blk < hi;
    const uint32_t ko = in ? kco : 0, so = in ? kso : 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t pt = __builtin_amdgcn_readlane(pg, 16 * t);
      const int tok = (blk * BN + 16 * t) & (page - 1);
      kw[t] = load_words<C::CB, C::ONCE>(kc + (pt * c.k_codes_sp + tok * (D / 2)) + ko);
      ksw[t] = load_words<C::CB / 8>(ks + (pt * c.k_scales_sp + tok * DT) + so);
    }
  };
  auto load_v = [&](int blk, int pg) {
    pg = max(pg, 0);
    const bool in = blk < hi;
    const uint32_t vo = in ? vco : 0, so = in ? (((blk * BN + 16 * lg) & (page - 1)) + lr) * DT : 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t pt = __builtin_amdgcn_readlane(pg, 16 * t);
      vw[t] = load_words<C::CB, C::ONCE>(vc + (pt * c.v_codes_sp + ((blk * BN + 16 * t) & (page - 1)) * (D / 2)) + vo);
    }
    vsw = load_words<DT>(vs + (pg * c.v_scales_sp) + so);
  };

  pg = held(lo + wave, pg);
  // loads stay in this order, so that a wait for the older ones leaves the younger in flight
  auto in_order = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  in_order();
  load_v(lo + wave, pg);
  in_order();
  load_k(lo + wave, pg);
  in_order();

  // queries, limits
  v8h qf[MT][KS];
  float cr[MT], m[MT], l[MT];
  int lim[MT];
#pragma unroll
  for (int x = 0; x < MT; ++x) {
    const int row = r0 + min(x * 16 + lr, nrows - 1);    // rows past the end repeat the last
    int g;
    const int t = div_by(row, p.g, g);
    lim[x] = limit(t);
    const uint16_t* q = (const uint16_t*)a.q + b * a.q_sb + t * a.q_st + (int64_t)(hk * G + g) * a.q_sh + lg * (D / 4);
    float f[KS][8], amax = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint4 v = *reinterpret_cast<const uint4*>(q + 8 * s);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[s][2 * i] = __uint_as_float(w[i] << 16);
        f[s][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        amax = fmaxf(amax, fmaxf(__builtin_fabsf(f[s][2 * i]), __builtin_fabsf(f[s][2 * i + 1])));
      }
    }
    float inv;
    const float fac = row_factor(group_max(amax), inv) * p.qmul;
    cr[x] = score_factor(p, inv);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) qf[x][s][i] = (_Float16)(f[s][i] * fac);
    m[x] = -INFINITY;
    l[x] = 0.f;                                          // this lane group's keys only
  }
  v4f o[MT][DT];
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int d = 0; d < DT; ++d) o[x][d] = (v4f){0.f, 0.f, 0.f, 0.f};

  // This wave's LDS.  Row r of codes at r D / 2, its 8-byte chunks swizzled so
  // that the 64 rows of a transposing read spread over the banks.
  uint8_t* vl = smem + wave * C::WAVE;
  uint8_t* sl = vl + C::VCODES;
  auto chunk = [](int row) { return (row >> (D == 64 ? 3 : D == 128 ? 2 : 1)) & (C::VCH - 1); };
  // the row whose codes this lane hands to the transposing read: key 16 t + 4 lg + i
  const int trow = 16 * (lr >> 2) + 4 * lg + (lr & 3);
  const uint32_t tbase = (uint32_t)(trow * (D / 2)), tswz = chunk(trow);

  bool far = false;                                      // some m was too large to go without a base
  float from[MT];                                        // with bases: minus them, what sums of scores start from
  // The next block's values are loaded when this one's are in LDS, its keys when
  // this one's are multiplied: into the registers that those leave.
  auto walk = [&](auto based_) {
    constexpr bool based = based_();
    for (int blk = lo + wave; blk < hi; blk += NW) {
      const int j0 = blk * BN;
      const uint32_t absent = bad;
      pg = held(blk + NW, pg1);
      pg1 = load_pages(blk + 2 * NW);

      // V into LDS: piece t holds keys 16 t .. 16 t + 15, CB bytes a lane
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 16 * t + lane / (D / 2 / C::CB), ch = lane % (D / 2 / C::CB) * (C::CB / 8), z = chunk(row);
#pragma unroll
        for (int i = 0; i < C::CB / 8; ++i)
          *reinterpret_cast<uint2*>(vl + row * (D / 2) + ((ch + i) ^ z) * 8) =
              make_uint2(vw[t].w[2 * i], vw[t].w[2 * i + 1]);
      }
      // scales of key 16 lg + lr, in the order of the second product: t = lg, (g, i) from lr
      {
        const int at = (lr >> 2) * 16 + lg * 4 + (lr & 3);
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<uint16_t*>(sl + (d * BN + at) * 2) = (uint16_t)scale_bits(vsw.w[d / 4] >> (8 * (d & 3)));
      }

      in_order();
      load_v(blk + NW, pg);
      in_order();

      v4f s[MT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          const float z = based ? from[x] : 0.f;
          s[x][t] = (v4f){z, z, z, z};
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const v2h sc = both(scale_bits(ksw[t].w[0] >> (8 * (k / 2))));
          const v8h kf = decode8(kw[t].w[k], sc, sc, sc, sc);
#pragma unroll
          for (int x = 0; x < MT; ++x) s[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[x][k], s[x][t], 0, 0, 0);
        }
      }
      in_order();
      load_k(blk + NW, pg);
      in_order();
      if (absent || j0 + BN > first) {
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          const int vis = lim[x] - j0 - 4 * lg;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[x][t][i] = 16 * t + i < vis && !(absent >> t & 1) ? s[x][t][i] : -INFINITY;
        }
      }
      v8h pf[MT][2];
#pragma unroll
      for (int x = 0; x < MT; ++x) {
        float tm = s[x][0][0];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) tm = fmaxf(tm, s[x][t][i]);
        const float most = group_max(tm);
        tm = most * cr[x];
        if (__any(tm > m[x] + kLazy)) {
          const float mn = tm > m[x] + kLazy ? tm : m[x];   // only the rows that need it move
          const float f = __builtin_amdgcn_exp2f(m[x] - (mn == -INFINITY ? 0.f : mn));
          l[x] *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[x][d] *= f;
          if constexpr (based) {
            const float step = rebase(tm > m[x] + kLazy, most, cr[x], m[x], from[x]);
#pragma unroll
            for (int t = 0; t < 4; ++t) s[x][t] += step;
            from[x] += step;
          } else {
            far |= __any(__builtin_fabsf(mn) >= kFar && mn != -INFINITY);
            m[x] = mn;
          }
        }
        const float nm = m[x] == -INFINITY ? 0.f : kFewUp - m[x];
        uint32_t w[8];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][t][i], cr[x], nm));
            const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][t][i + 1], cr[x], nm));
            l0 += e0;
            l1 += e1;
            w[2 * t + i / 2] = pack_f16(e0, e1);   // the second product takes p with 11 significant bits; l keeps 24
          }
        l[x] += l0 + l1;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          pf[x][h] = __builtin_bit_cast(v8h, (v4i){(int)w[4 * h], (int)w[4 * h + 1], (int)w[4 * h + 2], (int)w[4 * h + 3]});
      }
      // A wave's LDS accesses keep their order; the compiler has to keep it too.
      asm volatile("" ::: "memory");
      v2i vcd[DT];
      uint4 vsc[DT][2];
      auto read_v = [&](int d) {
        vcd[d] = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_v2i*)(vl + tbase + ((d ^ tswz) * 8)));
        const uint4* sp = reinterpret_cast<const uint4*>(sl + (d * BN + lg * 16) * 2);
        vsc[d][0] = sp[0], vsc[d][1] = sp[1];
      };
      read_v(0);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        if (d + 1 < DT) read_v(d + 1);
        __builtin_amdgcn_sched_barrier(0);   // else, short of registers, reads wait right before their products
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 q4 = vsc[d][h];
          const v8h vf = decode8((uint32_t)vcd[d][h], __builtin_bit_cast(v2h, q4.x), __builtin_bit_cast(v2h, q4.y),
                                 __builtin_bit_cast(v2h, q4.z), __builtin_bit_cast(v2h, q4.w));
#pragma unroll
          for (int x = 0; x < MT; ++x) o[x][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[x][h], o[x][d], 0, 0, 0);
        }
      }
      asm volatile("" ::: "memory");
    }
  };
  struct Without { constexpr bool operator()() const { return false; } };
  struct With { constexpr bool operator()() const { return true; } };
  walk(Without());
  if (__builtin_expect(far, 0)) {                        // once more, from the start
    pg = held(lo + wave, load_pages(lo + wave));
    pg1 = load_pages(lo + wave + NW);
    load_v(lo + wave, pg);
    load_k(lo + wave, pg);
#pragma unroll
    for (int x = 0; x < MT; ++x) {
      m[x] = -INFINITY;
      l[x] = from[x] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[x][d] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    walk(With());
#pragma unroll
    for (int x = 0; x < MT; ++x) {
      const float f = to_m(from[x], cr[x], m[x]);
      l[x] *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[x][d] *= f;
    }
  }

  // Join the waves: each leaves its (m, l) and its o in LDS, and all threads sum
  // them, scaled to the common maximum.
  float* red = reinterpret_cast<float*>(smem);
  float* ml = red + NW * R * C::PITCH;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < MT; ++x) {
    l[x] = group_sum(l[x]);
    if (lg == 0) {
      ml[(wave * R + x * 16 + lr) * 2] = m[x];
      ml[(wave * R + x * 16 + lr) * 2 + 1] = l[x];
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<v4f*>(&red[(wave * R + x * 16 + lr) * C::PITCH + 16 * d + 4 * lg]) = o[x][d];
  }
  __syncthreads();
  for (int e = tid; e < nrows * (D / 4); e += 64 * NW) {
    const int rr = e / (D / 4), d = e % (D / 4) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) M = fmaxf(M, ml[(k * R + rr) * 2]);
    const float ms = M == -INFINITY ? 0.f : M;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float f = __builtin_amdgcn_exp2f(ml[(k * R + rr) * 2] - ms);
      L += ml[(k * R + rr) * 2 + 1] * f;
      acc += *reinterpret_cast<const v4f*>(&red[(k * R + rr) * C::PITCH + d]) * f;
    }
    const int row = r0 + rr;
    if (p.po) {
      const int64_t x = (((int64_t)part * a.B + b) * c.Hkv + hk) * p.rows + row;
      *reinterpret_cast<v4f*>(p.po + x * D + d) = acc;
      if (d == 0) *reinterpret_cast<v2f*>(p.pml + x * 2) = (v2f){M, L};
    } else {
      const float inv = L == 0.f ? 0.f : p.v / L;
      int g;
      const int t = div_by(row, p.g, g);
      uint16_t* out = (uint16_t*)a.out + b * a.o_sb + t * a.o_st + (int64_t)(hk * G + g) * a.o_sh + d;
      *reinterpret_cast<uint2*>(out) = pack_out(p, acc * inv);
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup of W waves (eight; four at D = 256) of 32 rows each
// shares every block of keys, converted to fp16 once and kept in LDS.
//
// Products.  S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_32x32x16_f16: a lane
// has one query (lane % 32) and of 32 keys the scores of keys 8 (i / 4) +
// 4 (lane / 32) + i % 4.  The second product takes its 16 keys per step in that
// order, V^T comes from LDS through the transposing read (4 keys x 16 channels
// per 16 lanes), and P never moves between lanes.
//
// A wave overlaps its own work as far as it can.  Keys go by halves of a
// block: phase 1 of half u multiplies half u + 1 by the queries while it turns
// the scores of half u into probabilities; phase 2 multiplies those by V while
// it converts codes of a later block.  A barrier stands between phase 1 and
// phase 2 of a block's first half: between two of them V of block i and K of
// block i + 1 are read, and V of block i + 1 and K of block i + 2 written to the
// other buffers.
//
// Maximum.  Probabilities are taken with the m at hand.  Only where a lane's
// sum of half a block passes kMost (or there is no m yet) the maximum is looked
// for and the probabilities are taken again; p is at most kMost, l at least
// 2^kManyUp then.
//
// What bounds it.  A frame of 2 x 1560 queries, 16 heads of 128, 12480 keys: 319
// GFLOP in 352 to 358 us, 0.9 PFLOP/s (a large library product: 1.4).  Of the
// 352, products alone take 202, fragment reads add 27, softmax 75, conversions
// 24, loads 16; matrix and vector units are each busy half the time, and 224 of
// 256 CUs have a tile.  64 rows a wave and 4 waves: 393 to 403; two blocks a
// barrier: 364.  One wave a SIMD (D = 256) where the queries and sums of 32 rows
// take the registers of two.
// ---------------------------------------------------------------------------
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v4i lds_v4i;

constexpr float kMost = 32768.f, kManyUp = 5.f;

template <int D_, int W_>
struct Many {
  static constexpr int D = D_, W = W_;
  static constexpr int R = W * 32;
  static constexpr int RB = 2 * D, MAT = BN * RB;       // bytes of a row, of a block of K or V
  static constexpr int KC = D / 16, DB = D / 32;        // steps, channel blocks
  static constexpr int MATS = 8 / W;                    // W = 8: waves 0-3 convert K, 4-7 V; W = 4: each both
  static constexpr int CB = D / 8;                      // bytes of codes a thread converts of one of them
  static constexpr int STRIDE = 2 / MATS;               // conversions of a chunk: every second or fourth step
  static constexpr int AHEAD = 4;                       // steps a fragment is read ahead
  static constexpr int LDS = 4 * MAT;                   // two blocks of K, two of V
  static_assert(KC % AHEAD == 0, "a phase's last fragments and the next one's first take the same registers");
};

// 16-byte chunk swizzles of an LDS row.  K: the rows of a chunk column, read 32
// at a time, spread over the banks.  V: so do 4 rows of 4 adjacent chunks, which
// the transposing read takes, and (the lower bits) the rows written together.
template <int D>
__device__ __forceinline__ int swz_k(int row) {
  return D == 64 ? (row >> 1) & 7 : row & 15;
}
template <int D>
__device__ __forceinline__ int swz_v(int row) {
  return D == 64 ? ((row >> 1) & 1) << 2 | ((row >> 2) & 1) : (row & 3) << 2 | ((row >> 2) & 3);
}
// The row of its group of 16 that a thread converts of V, so that 16 lanes
// write all banks (four lanes a row; of K the rows in order do that).
template <int D>
__device__ __forceinline__ int write_row_v(int i) {
  return D == 64 ? (i & 9) | (i & 2) << 1 | (i & 4) >> 1 : (i & 3) << 2 | i >> 2;
}
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <typename C>
__global__ void __launch_bounds__(64 * C::W, C::W / 4) attn_many_kernel(Args p) {
  constexpr int D = C::D, R = C::R, MATS = C::MATS, KC = C::KC, DB = C::DB, AHEAD = C::AHEAD;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];   // K of even and odd blocks, V of them
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const int nwg = gridDim.x, wid = blockIdx.x;
  const int u = nwg % 8 == 0 ? (wid % 8) * (nwg / 8) + wid / 8 : wid;
  int tile, part, hk;
  const int b = div_by(div_by(div_by(u, p.tiles, tile), p.parts, part), p.heads, hk);
  const w4a4_kvcache& c = p.c;
  const w4a4_cache_attn& a = p.a;
  const int G = (int)p.g.d, page = 1 << p.lp;

  const int r0 = tile * R, nrows = min(R, p.rows - r0);
  int rem;
  const Limit limit(p, b);
  const int last = limit(div_by(r0 + nrows - 1, p.g, rem));
  const int first = limit(div_by(r0 + min(wave * 32, nrows - 1), p.g, rem));   // of this wave
  const int nblk = (max(last, 0) + BN - 1) / BN;
  const int per = (nblk + (int)p.parts.d - 1) / (int)p.parts.d;
  const int lo = min(part * per, nblk), n = min(lo + per, nblk) - lo;
  // (without keys there may be no table: any integer then)
  const int32_t* table = n > 0 ? a.table + b * a.table_sb : a.lens;

  // pages of the four groups of 16 keys from key `j` of this part on, one a lane group
  auto load_pages = [&](int j) {
    j += 16 * (lane >> 4);
    const int key = lo * BN + j;
    const bool in = j < n * BN && key < last;
    const int pg = table[in ? key >> p.lp : 0];   // no branch: the waits of later loads count this one
    return in ? pg : -1;
  };
  auto absent = [&](int pg) -> uint32_t {
    const uint64_t x = __ballot(pg < 0 || pg >= c.n_pages);
    return (uint32_t)(x & 1) | (uint32_t)(x >> 15 & 2) | (uint32_t)(x >> 30 & 4) | (uint32_t)(x >> 45 & 8);
  };
  // This thread converts a row of each block of K, or V, or both: row `in` of
  // the group of 16, chunks of eight channels chunk(0), chunk(1), ...
  const int grp = wave & 3, cq = lane & 3;
  auto chunk = [&](int x) { return D == 256 ? (x >> 2) * 16 + cq * 4 + (x & 3) : cq * (D / 32) + x; };
  constexpr int PIECES = D == 256 ? 2 : 1, PB = C::CB / PIECES;   // adjacent chunks: PB bytes of codes
  struct Raw {
    Words<PB> codes[PIECES];
    Words<PB / 8> scales[PIECES];
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  struct Mat {
    const uint8_t *codes, *scales;   // the head's, page 0
    int64_t codes_sp, scales_sp;
    uint32_t coff, soff, at;         // this lane's bytes in a group of 16 rows; its row in LDS, buffer 0
    int z;                           // the row's swizzle
  } mat[MATS];
#pragma unroll
  for (int x = 0; x < MATS; ++x) {
    const bool v = MATS == 2 ? x == 1 : wave >= 4;
    const int in = v ? write_row_v<D>(lane >> 2) : lane >> 2;
    mat[x].codes = (const uint8_t*)(v ? c.v_codes : c.k_codes) + (int64_t)hk * page * (D / 2);
    mat[x].scales = (const uint8_t*)(v ? c.v_scales : c.k_scales) + (int64_t)hk * page * (D / 16);
    mat[x].codes_sp = v ? c.v_codes_sp : c.k_codes_sp;
    mat[x].scales_sp = v ? c.v_scales_sp : c.k_scales_sp;
    mat[x].coff = in * (D / 2) + cq * PB;
    mat[x].soff = in * (D / 16) + cq * (PB / 8);
    mat[x].at = lds0 + (v ? 2 * C::MAT : 0) + (16 * grp + in) * C::RB;
    mat[x].z = v ? swz_v<D>(in) : swz_k<D>(in);
  }
  const uint32_t n_pages = (uint32_t)c.n_pages;
  auto load_raw = [&](const Mat& t, int j, int pgs) {     // keys from j (of the part) on, on pages pgs
    uint32_t pg = (uint32_t)__builtin_amdgcn_readlane(pgs, 16 * grp);
    pg = pg < n_pages ? pg : 0;                           // any page: its keys are excluded
    const uint32_t tok = (uint32_t)((lo * BN + j + 16 * grp) & (page - 1));
    const uint8_t* cp = t.codes + (pg * t.codes_sp + tok * (D / 2));
    const uint8_t* sp = t.scales + (pg * t.scales_sp + tok * (D / 16));
    Raw r;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      r.codes[i] = load_words<PB>(cp + t.coff + i * 64);
      r.scales[i] = load_words<PB / 8>(sp + t.soff + i * 8);
    }
    return r;
  };
  auto store = [&](const Mat& t, const Raw& r, int x, uint32_t buf) {   // the thread's chunk x, converted
    constexpr int N = PB / 4;
    const v2h sc = both(scale_bits(r.scales[x / N].w[0] >> (8 * (x % N / 2))));
    *(lds_v4i*)(t.at + buf + ((chunk(x) ^ t.z) << 4)) =
        __builtin_bit_cast(v4i, decode8(r.codes[x / N].w[x % N], sc, sc, sc, sc));
  };

  int pg[4];                                              // of the next blocks
#pragma unroll
  for (int x = 0; x < 4; ++x) pg[x] = load_pages(x * BN);
  // The blocks that are converted before the first product: of K one more than
  // of V (a wave that converts V alone converts that one in the loop).
  const bool only_v = MATS == 1 && wave >= 4;
  Raw raw[MATS], early[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) early[x] = load_raw(mat[0], x * BN, pg[x]);

  // queries: row tile r0, wave, set, lane
  v8h qf[KC];
  float cr, m = -INFINITY, l = 0.f;                       // l: this half's keys only
  int lim;
  {
    const int row = r0 + min(wave * 32 + lr, nrows - 1);   // rows past the end repeat the last
    int g;
    const int t = div_by(row, p.g, g);
    lim = limit(t);
    const uint16_t* q = (const uint16_t*)a.q + b * a.q_sb + t * a.q_st + (int64_t)(hk * G + g) * a.q_sh + h * 8;
    uint4 v[KC];
    float amax = 0.f;
#pragma unroll
    for (int s = 0; s < KC; ++s) v[s] = *reinterpret_cast<const uint4*>(q + 16 * s);
#pragma unroll
    for (int s = 0; s < KC; ++s) {
      const uint32_t w[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        amax = fmaxf(amax, fmaxf(__uint_as_float(w[i] << 16 & 0x7FFFFFFFu), __uint_as_float(w[i] & 0x7FFF0000u)));
    }
    float inv;
    const float fac = row_factor(half_max(amax), inv) * p.qmul;
    cr = score_factor(p, inv);
#pragma unroll
    for (int s = 0; s < KC; ++s) {
      const uint32_t w[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
      v4i f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = (int)pack_f16(__uint_as_float(w[i] << 16) * fac, __uint_as_float(w[i] & 0xFFFF0000u) * fac);
      qf[s] = __builtin_bit_cast(v8h, f);
      // with one wave a SIMD it stays in accumulation registers, from where the products take it
      if constexpr (C::W == 4) asm volatile("" : "+a"(qf[s]));
    }
  }
  v16f o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

  // addresses of the fragment reads in the buffers that are read next
  const uint32_t ka = lds0 + lr * C::RB + ((h ^ swz_k<D>(lr)) << 4);
  const int vr = 4 * h + ((lane & 15) >> 2);
  const int vch = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  uint32_t kad[KC], vad[2][DB];                           // V: rows vr and vr + 8 (the swizzle repeats every 16)
#pragma unroll
  for (int k = 0; k < KC; ++k) kad[k] = ka ^ (k << 5);    // the swizzle is an exclusive or of the chunk
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      vad[e][d] = lds0 + 2 * C::MAT + (vr + 8 * e) * C::RB + (((4 * d + vch) ^ swz_v<D>(vr + 8 * e)) << 4) + (lane & 1) * 8;
  v4i frag[AHEAD];
  // fragment t of K: 32 keys of half `half`, channels 16 t
  auto fetch_k = [&](int t, int half) { frag[t % AHEAD] = *(lds_v4i*)(kad[t] + half * 32 * C::RB); };
  // fragment t of V: keys 16 (t / DB) of half `half`, channels 32 (t % DB)
  auto fetch_v = [&](int t, int half) {
    const int off = (half * 32 + t / DB * 16) * C::RB;
    const v4s v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(vad[0][t % DB] + off));
    const v4s v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(vad[1][t % DB] + off));
    frag[t % AHEAD] = __builtin_bit_cast(v4i, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  typedef v16f Scores;     // of 32 keys
  uint32_t pk[8];
  float lb;
  const v2h one = {(_Float16)1.f, (_Float16)1.f};
  auto prob = [&](const Scores& s, int w, float nm) {   // probabilities 2 w and 2 w + 1
    const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * w], cr, nm));
    const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * w + 1], cr, nm));
    pk[w] = pack_f16(e0, e1);   // the second product takes p with 11 significant bits, and so does the sum
    lb = __builtin_amdgcn_fdot2(__builtin_bit_cast(v2h, pk[w]), one, lb, false);
  };
  // scores of keys from j0 (of the part) on that a row does not see; bad: absent groups of 16
  auto exclude = [&](Scores& s, int j0, uint32_t bad) {
    j0 += lo * BN;
    if ((bad & 3) == 0 && j0 + 32 <= first) return;
    const int vis = lim - j0 - 4 * h;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      s[e] = 8 * (e >> 2) + (e & 3) < vis && !(bad >> (e >> 3) & 1) ? s[e] : -INFINITY;
  };
  auto sync = [&]() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // minus the row's base: what sums of scores start from
  v16f from = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  asm volatile("" : "+v"(from));                          // (registers of its own, not copies of one for every sum)
  auto qk = [&](Scores& s, int t, const v8h& f) {
    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, qf[t], t == 0 ? from : s, 0, 0, 0);
  };

  // Phase 1: scores `s` to probabilities, products of K's half `half` to `next`.
  auto phase1 = [&](Scores& s, Scores& next, auto half_, auto then_, auto&& extra) {
    constexpr int half = half_(), then = then_();    // then: the half of V whose fragments come next, or -1
    const float nm = m == -INFINITY ? 0.f : kManyUp - m;
    lb = 0.f;
#pragma unroll
    for (int t = 0; t < KC; ++t) {
      const v8h f = __builtin_bit_cast(v8h, frag[t % AHEAD]);
      qk(next, t, f);
#pragma unroll
      for (int w = t * 8 / KC; w < (t + 1) * 8 / KC; ++w) prob(s, w, nm);
      extra(t);
      if (t + AHEAD < KC) fetch_k(t + AHEAD, half);
      else if constexpr (then >= 0) fetch_v(t + AHEAD - KC, then);
    }
    if (__any(!(lb <= kMost) || m == -INFINITY)) {
      float tm = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) tm = fmaxf(tm, s[e]);
      const float most = half_max(tm);
      tm = most * cr;
      // only the rows that need it move: no row's result depends on its neighbours
      const bool moves = (half_max(lb) > kMost || m == -INFINITY) && tm > m;
      const float f = __builtin_amdgcn_exp2f(m - (moves ? tm : m == -INFINITY ? 0.f : m));
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= f;
      const float step = rebase(moves, most, cr, m, from[0]);
      if (__any(step != 0.f)) {
        s += step;
        next += step;
        from += step;
        asm volatile("" : "+v"(from));
      }
      lb = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) prob(s, w, m == -INFINITY ? 0.f : kManyUp - m);
    }
    l += lb;
  };
  // Phase 2: the probabilities by V's half `half`; convert(t) is called in every step.
  auto phase2 = [&](auto half_, auto then_, auto&& convert) {
    constexpr int half = half_(), then = then_();    // then: the half of K whose fragments come next
#pragma unroll
    for (int t = 0; t < KC; ++t) {
      convert(t);
      const v8h f = __builtin_bit_cast(v8h, frag[t % AHEAD]);
      const uint32_t* w = &pk[t / DB * 4];
      const v4i pv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
      o[t % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, __builtin_bit_cast(v8h, pv), o[t % DB], 0, 0, 0);
      if (t + AHEAD < KC) fetch_v(t + AHEAD, half);
      else fetch_k(t + AHEAD - KC, then);
    }
  };
  struct None { constexpr int operator()() const { return -1; } };
  struct First { constexpr int operator()() const { return 0; } };
  struct Second { constexpr int operator()() const { return 1; } };
  auto flip = [&](int k, int v) {
#pragma unroll
    for (int i = 0; i < KC; ++i) kad[i] += k;
#pragma unroll
    for (int d = 0; d < DB; ++d) vad[0][d] += v, vad[1][d] += v;
  };

  Scores s0, s1;               // of the first and second half of a block
  if (n > 0) {
    uint32_t bad = absent(pg[0]), next_bad = 0;
    int next_pg = -1;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (y == 1 && only_v) continue;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) store(mat[0], early[y], x, y * C::MAT);
    }
    if constexpr (MATS == 2) {
      raw[1] = load_raw(mat[1], 0, pg[0]);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) store(mat[1], raw[1], x, 0);
    }
    sync();
#pragma unroll
    for (int t = 0; t < KC; ++t) {
      fetch_k(t, 0);
      qk(s0, t, __builtin_bit_cast(v8h, frag[t % AHEAD]));
    }
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) fetch_k(t, 1);
    // What an iteration converts first: in the order in which it loads them, so
    // that a wait for the older one leaves the younger in flight.
    raw[0] = load_raw(mat[0], (only_v ? 1 : 2) * BN, only_v ? pg[1] : pg[2]);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MATS == 2) raw[1] = load_raw(mat[1], BN, pg[1]);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    for (int i = 0; i < n; ++i) {
      const uint32_t bufk = (i & 1) * C::MAT, bufv = C::MAT - bufk;   // of blocks i + 2 and i + 1
      const uint32_t buf0 = only_v ? bufv : bufk;
      exclude(s0, i * BN, bad);
      phase1(s0, s1, Second(), None(), [&](int t) {
        if (t == 1) next_bad = absent(pg[1]);
      });
      flip(i & 1 ? -C::MAT : C::MAT, 0);
      sync();
#pragma unroll
      for (int t = 0; t < AHEAD; ++t) fetch_v(t, 0);
      phase2(First(), First(), [&](int t) {
        if (t % (2 * C::STRIDE) == 0) store(mat[0], raw[0], t / (2 * C::STRIDE), buf0);
        if (MATS == 2 && t == KC - 1) raw[0] = load_raw(mat[0], (i + 3) * BN, pg[3]);
      });
      exclude(s1, i * BN + 32, bad >> 2);
      phase1(s1, s0, First(), Second(), [&](int t) {
        if (t == 1) next_pg = load_pages((i + 4) * BN);
      });
      phase2(Second(), Second(), [&](int t) {
        if constexpr (MATS == 2) {
          if (t % 2 == 0) store(mat[1], raw[1], t / 2, bufv);
          if (t == KC - 1) raw[1] = load_raw(mat[1], (i + 2) * BN, pg[2]);
        } else {
          if (t % 4 == 0) store(mat[0], raw[0], D / 64 + t / 4, buf0);
          if (t == KC - 1) raw[0] = load_raw(mat[0], (i + (only_v ? 2 : 3)) * BN, only_v ? pg[2] : pg[3]);
        }
      });
      flip(0, i & 1 ? -C::MAT : C::MAT);
      bad = next_bad;
#pragma unroll
      for (int x = 0; x < 3; ++x) pg[x] = pg[x + 1];
      pg[3] = next_pg;
    }
  }

  l = half_sum(l);
  const int rl = wave * 32 + lr, row = r0 + rl;
  if (rl >= nrows) return;
  if (p.po) {
    const float f = to_m(from[0], cr, m);
    const int64_t at = (((int64_t)part * a.B + b) * c.Hkv + hk) * p.rows + row;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<v4f*>(p.po + at * D + 32 * d + 8 * i + 4 * h) =
            (v4f){o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]} * f;
    if (h == 0) *reinterpret_cast<v2f*>(p.pml + at * 2) = (v2f){m, l * f};
  } else {
    const float inv = l == 0.f ? 0.f : p.v / l;
    int g;
    const int t = div_by(row, p.g, g);
    uint16_t* out = (uint16_t*)a.out + b * a.o_sb + t * a.o_st + (int64_t)(hk * G + g) * a.o_sh;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint2*>(out + 32 * d + 8 * i + 4 * h) =
            pack_out(p, (v4f){o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]} * inv);
  }
}

// Joins the parts of a row: kJoin groups of D / 4 lanes a row take every kJoin-th
// part, four in flight, 16 bytes of each a lane, and meet in LDS.  A launch and
// two dependent loads: 2.8 us for 16 parts of 208 rows of 256 (one group a row:
// 4.8).
constexpr int kJoin = 4;
template <int D>
__global__ void __launch_bounds__(256) cache_join_kernel(Args p) {
  const w4a4_cache_attn& a = p.a;
  constexpr int LPR = D / 4, GROUPS = 256 / LPR, ROWS = GROUPS / kJoin;
  __shared__ v4f accs[GROUPS][LPR];
  __shared__ v2f mls[GROUPS];
  const int group = threadIdx.x / LPR, x = threadIdx.x % LPR, first = group % kJoin;
  const int64_t gr = (int64_t)blockIdx.x * ROWS + group / kJoin;
  const int64_t all = a.B * p.c.Hkv * p.rows, at = min(gr, all - 1);
  const int parts = (int)p.parts.d;
  float M = -INFINITY, L = 0.f;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = first; k0 < parts; k0 += 4 * kJoin) {
    v2f ml[4];
    v4f o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = min(k0 + i * kJoin, parts - 1);
      ml[i] = *reinterpret_cast<const v2f*>(p.pml + (k * all + at) * 2);
      o[i] = *reinterpret_cast<const v4f*>(p.po + (k * all + at) * D + 4 * x);
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k0 + i * kJoin >= parts) ml[i][0] = -INFINITY;      // (one that another group takes)
      mn = fmaxf(mn, ml[i][0]);
    }
    const float ms = mn == -INFINITY ? 0.f : mn, f = __builtin_amdgcn_exp2f(M - ms);
    M = mn;
    L *= f;
    acc *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k0 + i * kJoin >= parts) break;
      const float e = __builtin_amdgcn_exp2f(ml[i][0] - ms);
      L += ml[i][1] * e;
      acc += o[i] * e;
    }
  }
  accs[group][x] = acc;
  if (x == 0) mls[group] = (v2f){M, L};
  __syncthreads();
  if (first != 0 || gr >= all) return;
#pragma unroll
  for (int i = 1; i < kJoin; ++i) M = fmaxf(M, mls[group + i][0]);
  const float ms = M == -INFINITY ? 0.f : M;
  L = 0.f;
  acc = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kJoin; ++i) {
    const float e = __builtin_amdgcn_exp2f(mls[group + i][0] - ms);
    L += mls[group + i][1] * e;
    acc += accs[group + i][x] * e;
  }
  const float inv = L == 0.f ? 0.f : p.v / L;
  const int row = (int)(gr % p.rows), bh = (int)(gr / p.rows);
  int hk, g;
  const int b = div_by(bh, p.heads, hk), t = div_by(row, p.g, g);
  uint16_t* out = (uint16_t*)a.out + b * a.o_sb + t * a.o_st + (int64_t)(hk * (int)p.g.d + g) * a.o_sh + 4 * x;
  *reinterpret_cast<uint2*>(out) = pack_out(p, acc * inv);
}

template <int D, int MT, int NW>
void launch_few(const Args& p, hipStream_t st) {
  const unsigned grid = (unsigned)(p.a.B * p.c.Hkv * p.tiles.d * p.parts.d);
  if (D > 64 && p.tiles.d == 1) attn_few_kernel<Few<D, MT, NW, D != 64>><<<grid, 64 * NW, 0, st>>>(p);
  else attn_few_kernel<Few<D, MT, NW, false>><<<grid, 64 * NW, 0, st>>>(p);
}

template <typename C>
void launch_many(const Args& p, hipStream_t st) {
  attn_many_kernel<C><<<(unsigned)(p.a.B * p.c.Hkv * p.tiles.d * p.parts.d), 64 * C::W, 0, st>>>(p);
}

}  // namespace

size_t cache_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len) {
  const CacheAttnPlan pl = plan_cache_attention(B, T, Hq, Hkv, D, max_len, true);
  return pl.parts > 1 ? (size_t)pl.parts * B * T * Hq * (D + 2) * 4 : 0;
}

hipError_t launch_cache_attention(const w4a4_kvcache& c, const w4a4_cache_attn& a, void* workspace, hipStream_t st) {
  const CacheAttnPlan pl = plan_cache_attention(a.B, a.T, a.Hq, c.Hkv, c.D, a.max_len, workspace != nullptr);
  Args p{};
  p.c = c;
  p.a = a;
  const int64_t g = a.Hq / c.Hkv;
  p.rows = (int)(a.T * g);
  p.lp = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : c.page == 128 ? 7 : 8;
  p.g = divisor(g);
  p.tiles = divisor(pl.tiles);
  p.heads = divisor(c.Hkv);
  p.parts = divisor(pl.parts);
  const double c2 = (double)a.scale * c.k_scale * 1.4426950408889634;
  p.qmul = c2 > 0 ? 1.f : c2 < 0 ? -1.f : 0.f;
  // as a product, which meets the queries' factors where fp32 alone has no bits left for it, or no number
  const double mag = c2 == 0 ? 1.0 : c2 < 0 ? -c2 : c2;
  p.cpost = mag < 0x1p-64 ? 0x1p-64f : mag > 0x1p64 ? 0x1p64f : 1.f;
  p.c2 = (float)(mag / p.cpost);
  const bool tiny = c.v_scale < 0x1p-63f;                    // (weights, 2^15 at most, of 2^30 keys sum to 2^45)
  p.v = tiny ? c.v_scale * 0x1p96f : c.v_scale;
  p.vpost = tiny ? 0x1p-96f : 1.f;
  if (pl.parts > 1) {
    p.po = (float*)workspace;
    p.pml = p.po + (size_t)pl.parts * a.B * a.T * a.Hq * c.D;
  }
  const bool four = pl.waves == 4;
  if (c.D == 64) {
    if (pl.rows == 16) four ? launch_few<64, 1, 4>(p, st) : launch_few<64, 1, 8>(p, st);
    else if (pl.rows == 32) launch_few<64, 2, 8>(p, st);
    else launch_many<Many<64, 8>>(p, st);
  } else if (c.D == 128) {
    if (pl.rows == 16) four ? launch_few<128, 1, 4>(p, st) : launch_few<128, 1, 8>(p, st);
    else if (pl.rows == 32) launch_few<128, 2, 8>(p, st);
    else launch_many<Many<128, 8>>(p, st);
  } else {
    if (pl.rows == 16) four ? launch_few<256, 1, 4>(p, st) : launch_few<256, 1, 8>(p, st);
    else launch_many<Many<256, 4>>(p, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.parts == 1) return e;
  const int64_t all = a.B * c.Hkv * (int64_t)p.rows;
  const int per = 256 / ((int)c.D / 4) / kJoin;
  const unsigned grid = (unsigned)((all + per - 1) / per);
  if (c.D == 64) cache_join_kernel<64><<<grid, 256, 0, st>>>(p);
  else if (c.D == 128) cache_join_kernel<128><<<grid, 256, 0, st>>>(p);
  else cache_join_kernel<256><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace w4a4
