// Attention of a batch over one shared prefix and each sequence's own keys.
//
// Mathematics.  For a KV head, the rows of the product are all queries of the
// batch that read it (row = (b T + t) G + g, G query heads per KV head), so
// the prefix is an ordinary key / value matrix for rows of different
// sequences and is read once per row tile, not once per sequence.  Keys come
// in blocks; a row keeps its running maximum m (in units of exp2), its sum l
// and its output o, all in fp32:
//   p = exp2(c s - m),  l += sum p,  o += p V,   c = scale log2 e.
// m only moves when a score exceeds it by more than kLazy: until then p is at
// most 2^kLazy, which costs no accuracy (p and l scale alike), and o and l
// need no rescaling.
//
// Products.  S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_32x32x16_bf16: the
// accumulator layout gives a lane one query (lane % 32) and 16 keys, so the
// softmax needs one exchange between the wave's halves per block and m, l
// and the rescaling are per lane.  The 16 scores a lane holds of 32 keys are
// keys 8 (i / 4) + 4 (lane / 32) + i % 4; the second product takes its 16
// keys per step in that same order, with V^T read from LDS through the
// transposing read (4 keys x 16 columns per 16 lanes), so P never moves
// between lanes.
//
// Work split.  A workgroup holds WQ x WK waves: WQ groups of 32 rows, and WK
// key groups that take every WK-th block and are joined through LDS at the
// end.  Blocks are copied global -> LDS (16 bytes a lane, XOR-swizzled on the
// way so that the fragment reads are free of bank conflicts) into NBUF
// buffers per key group.  The block list of a row tile, prefix blocks then
// the own blocks of its sequences, is cut into `parts` for shapes with few
// rows; partial (m, l, o) go to the workspace and a second kernel joins them.
#include "dense.h"
#include "device_common.h"
#include "lds_dma.h"

namespace w4a4 {

namespace {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef const __attribute__((address_space(3))) v4i lds_v4i;

constexpr float kLazy = 8.f;
constexpr int kNoBad = 1 << 30;

struct AttnArgs {
  w4a4_attn a;
  int rows;         // B T G rows of a KV head
  int rpt;          // rows of a tile
  int tg, g;        // T G, G
  int tiles, parts;
  int np, ns;       // prefix blocks; own blocks of a sequence
  float c2;         // |scale| log2 e
  uint32_t qflip;   // sign bits flipped in q when scale < 0
  float* po;        // parts > 1: [part][head][row][D], else null
  float* pml;       // [part][head][row][2]
};

template <int D_, int WQ_, int WK_, int BN_, int NBUF_>
struct ACfg {
  static constexpr int D = D_, WQ = WQ_, WK = WK_, BN = BN_, NBUF = NBUF_;
  static constexpr int NW = WQ * WK;
  static constexpr int RB = 2 * D;                  // bytes of a key or value row
  static constexpr int MAT = BN * RB;               // bytes of a block of one of them
  static constexpr int STAGE = 2 * MAT;
  static constexpr int NI = MAT / 1024 / WQ;        // copy instructions per wave and matrix
  static constexpr int RPI = 1024 / RB;             // rows per copy instruction
  static constexpr int KC = D / 16, DB = D / 32, SB = BN / 32;
  static constexpr int PITCH = D + 4;               // floats of a row in the joining of key groups
  static constexpr int PIPE = WK * NBUF * STAGE;
  static constexpr int JOIN = WK > 1 ? NW * 32 * (PITCH + 2) * 4 : 0;
  static constexpr int LDS = PIPE > JOIN ? PIPE : JOIN;
  static_assert(MAT % (1024 * WQ) == 0 && BN % 32 == 0, "whole copies");
  static_assert(LDS <= 156 * 1024, "LDS");
};

// 16-byte chunk swizzles of an LDS row (see the header of this file): K rows
// are read 16 at a time in the same chunk column, V rows 4 at a time over 4
// adjacent chunks.
template <int D>
__device__ __forceinline__ int swz_k(int row) {
  return D == 64 ? (row >> 1) & 7 : row & 15;
}
template <int D>
__device__ __forceinline__ int swz_v(int row) {
  return D == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2;
}

__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){a, b}, v2bf));
}

template <int BN>
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n >= 64 ? ~0ull : (1ull << n) - 1;
}

// A block of the list: prefix keys (b < 0) or own keys of sequence b.
struct Slot {
  int b, j0, valid;   // valid: keys of the block inside the prefix or the sequence's length
};

template <typename C>
__global__ void __launch_bounds__(64 * C::NW) __attribute__((amdgpu_waves_per_eu((C::NW + 3) / 4, (C::NW + 3) / 4)))
attn_tile_kernel(AttnArgs p) {
  constexpr int D = C::D, BN = C::BN, WQ = C::WQ, WK = C::WK;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  __shared__ int sbad[WK][2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave % WQ, wk = wave / WQ;
  const int h = lane >> 5, lr = lane & 31;

  // Workgroup -> (head, part, tile), tiles fastest, in contiguous runs per
  // XCD: the tiles that read the same keys share an L2.
  const int nwg = gridDim.x, wid = blockIdx.x;
  const int u = nwg % 8 == 0 ? (wid % 8) * (nwg / 8) + wid / 8 : wid;
  const int tile = u % p.tiles, part = u / p.tiles % p.parts, hk = u / p.tiles / p.parts;
  const w4a4_attn& a = p.a;

  const int r0 = tile * p.rpt, nrows = min(p.rpt, p.rows - r0);
  const int b0 = r0 / p.tg, nseq = (r0 + nrows - 1) / p.tg - b0 + 1;
  const int64_t total = p.np + (int64_t)nseq * p.ns;
  const int lo = (int)(total * part / p.parts), hi = (int)(total * (part + 1) / p.parts);
  const int iters = (hi - lo + WK - 1) / WK;

  // this lane's row: query, sequence, and how many of its own keys it sees
  const int rl = wq * 32 + lr, row = r0 + rl;
  const bool live = rl < nrows;
  const int rb = live ? row / p.tg : -1, rt = live ? (row % p.tg) / p.g : 0, rg = live ? row % p.g : 0;
  auto own_length = [&](int b) {
    return a.own_len ? max(0, min(a.own_len[b], (int)a.S)) : (int)a.S;
  };
  int rlim = live ? own_length(rb) : 0;
  if (a.causal) rlim = max(0, min(rlim, rlim - (int)a.T + 1 + rt));
  const int wb0 = (r0 + wq * 32) / p.tg, wb1 = (min(r0 + wq * 32 + 32, r0 + nrows) - 1) / p.tg;   // this wave's sequences
  const bool wave_live = wq * 32 < nrows;
  // own value rows are seen by some rows of a wave and not by others
  const bool mixed = a.causal || nseq > 1;

  v8bf qf[C::KC];
  {
    const uint16_t* q = (const uint16_t*)a.q + rb * a.q_sb + rt * a.q_st + (int64_t)(hk * p.g + rg) * a.q_sh + h * 8;
#pragma unroll
    for (int c = 0; c < C::KC; ++c) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live) v = *reinterpret_cast<const uint4*>(q + c * 16);
      v.x ^= p.qflip; v.y ^= p.qflip; v.z ^= p.qflip; v.w ^= p.qflip;
      qf[c] = __builtin_bit_cast(v8bf, v);
    }
  }

  auto slot_at = [&](int it) {
    Slot s{-1, 0, 0};
    const int i = lo + it * WK + wk;
    if (i >= hi) return s;
    if (i < p.np) {
      s.j0 = i * BN;
      s.valid = min(BN, (int)a.P - s.j0);
    } else {
      const int o = i - p.np;
      s.b = b0 + o / p.ns;
      s.j0 = o % p.ns * BN;
      s.valid = max(0, min(BN, own_length(s.b) - s.j0));
    }
    return s;
  };

  // Copies.  Instruction n of a matrix covers rows n RPI + [0, RPI), lane l
  // chunk l % (D / 8) of row l / (D / 8); excluded rows (past the end, or not
  // kept) take an out-of-range offset and arrive as zeros, so whatever
  // lies there never enters a product.
  const uint32_t lds0 = lds_addr(smem);
  const int cr = lane / (D / 8), cc = lane % (D / 8);
  auto copy = [&](const Slot& s, uint64_t mask, uint32_t dst, const void* base, int64_t stride, bool is_k) {
    const v4u rs = rsrc_words((const uint16_t*)base + s.j0 * stride, 0x7FFFFFFFu);
    const uint32_t st2 = (uint32_t)stride * 2;
    const uint32_t voff = cr * st2;
    const bool full = mask == low_bits<BN>(BN);
#pragma unroll
    for (int k = 0; k < C::NI; ++k) {
      const int n = k * WQ + wq, rw = n * C::RPI;
      const int chunk = cc ^ (is_k ? swz_k<D>(rw + cr) : swz_v<D>(rw + cr));
      uint32_t off = voff + chunk * 16;
      if (!full) off = (mask >> (rw + cr)) & 1 ? off : kOOB;
      dma16_at(rs, dst + n * 1024, off, rw * st2);
    }
  };
  auto issue = [&](const Slot& s, uint64_t mask, int buf) {
    if (mask == 0) return;
    const uint32_t dst = lds0 + (wk * C::NBUF + buf) * C::STAGE;
    if (s.b < 0) {
      copy(s, mask, dst, (const uint16_t*)a.k_prefix + hk * a.kp_sh, a.kp_sp, true);
      copy(s, mask, dst + C::MAT, (const uint16_t*)a.v_prefix + hk * a.vp_sh, a.vp_sp, false);
    } else {
      copy(s, mask, dst, (const uint16_t*)a.k_own + s.b * a.ko_sb + hk * a.ko_sh, a.ko_ss, true);
      copy(s, mask, dst + C::MAT, (const uint16_t*)a.v_own + s.b * a.vo_sb + hk * a.vo_sh, a.vo_ss, false);
    }
  };
  // keep bytes of a block, one per lane, loaded an iteration before they are balloted
  auto load_keep = [&](const Slot& s) -> uint32_t {
    if (!a.prefix_keep || s.b >= 0 || lane >= s.valid) return 1;
    return a.prefix_keep[s.j0 + lane];
  };
  auto slot_mask = [&](const Slot& s, uint32_t keep) -> uint64_t {
    const uint64_t in = low_bits<BN>(s.valid);
    return a.prefix_keep && s.b < 0 ? in & __ballot(keep != 0) : in;
  };
  auto group_sync = [&]() {
    asm volatile("" ::: "memory");
    if constexpr (WQ > 1) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  v16f o[C::DB];
#pragma unroll
  for (int d = 0; d < C::DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;   // l: this half's keys only
  bool poisoned = false;

  // LDS addresses of the fragment reads, relative to a stage
  const uint32_t ka = lr * C::RB + ((h ^ swz_k<D>(lr)) << 4);
  const int vr = 4 * h + ((lane & 15) >> 2);
  const uint32_t va = C::MAT + vr * C::RB + (((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swz_v<D>(vr)) << 4) + (lane & 1) * 8;

  if (tid < WK) sbad[tid][0] = sbad[tid][1] = kNoBad;
  __syncthreads();

  Slot cur, nxt = slot_at(0);
  uint64_t cmask, nmask = slot_mask(nxt, load_keep(nxt));
  if (iters > 0) issue(nxt, nmask, 0);
  Slot after = slot_at(1);
  uint32_t keep = load_keep(after);

  for (int it = 0; it < iters; ++it) {
    wait_vmcnt<0>();
    group_sync();   // the block has landed and the other buffer is no longer read
    cur = nxt;
    cmask = nmask;
    nxt = after;
    nmask = slot_mask(nxt, keep);
    if constexpr (C::NBUF > 1) {
      if (it + 1 < iters) issue(nxt, nmask, (it + 1) & 1);
      after = slot_at(it + 2);
      keep = load_keep(after);
    }
    const uint32_t stage = lds0 + (wk * C::NBUF + (C::NBUF > 1 ? (it & 1) : 0)) * C::STAGE;

    // Own values that some rows of the tile must not see: a chunk with a NaN
    // or Inf is zeroed and the rows that do see its key are marked.
    if (mixed && lo + it * WK + WK > p.np) {
      if (cur.b >= 0 && cmask != 0) {
#pragma unroll
        for (int k = 0; k < C::NI; ++k) {
          const int n = k * WQ + wq;
          auto* ptr = (__attribute__((address_space(3))) v4i*)(stage + C::MAT + n * 1024 + lane * 16);
          const v4i v = *ptr;
          uint32_t bad = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= (((uint32_t)v[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
          if (bad) {
            *ptr = (v4i){0, 0, 0, 0};
            atomicMin(&sbad[wk][it & 1], n * C::RPI + cr);
          }
        }
      }
      if (wq == 0 && lane == 0) sbad[wk][(it + 1) & 1] = kNoBad;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      group_sync();
      if (cur.b >= 0 && rb == cur.b && cur.j0 + sbad[wk][it & 1] < rlim) poisoned = true;
    }

    const bool mine = cmask != 0 && wave_live && (cur.b < 0 || (cur.b >= wb0 && cur.b <= wb1));
    if (mine) {
      v16f s[C::SB];
#pragma unroll
      for (int b = 0; b < C::SB; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
        for (int c = 0; c < C::KC; ++c) {
          const v4i kf = *(lds_v4i*)(stage + (ka ^ (c << 5)) + b * 32 * C::RB);
          s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, kf), qf[c], s[b], 0, 0, 0);
        }
      }
      if (cur.b >= 0) {
        const int vis = (rb == cur.b ? rlim - cur.j0 : 0) - 4 * h;
#pragma unroll
        for (int b = 0; b < C::SB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = 32 * b + 8 * (i >> 2) + (i & 3) < vis ? s[b][i] : -INFINITY;
      } else if (cmask != low_bits<BN>(BN)) {
#pragma unroll
        for (int b = 0; b < C::SB; ++b) {
          const uint32_t w = (uint32_t)(cmask >> (32 * b)) >> (4 * h);
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = (w >> (8 * (i >> 2) + (i & 3))) & 1 ? s[b][i] : -INFINITY;
        }
      }
      float tm = s[0][0];
#pragma unroll
      for (int b = 0; b < C::SB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) tm = fmaxf(tm, s[b][i]);
      tm = half_max(tm) * p.c2;
      if (__any(tm > m + kLazy)) {
        const float mn = fmaxf(m, tm);
        const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < C::DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] *= f;
      }
      const float nm = m == -INFINITY ? 0.f : -m;
      uint32_t pk[C::SB][8];
      float l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int b = 0; b < C::SB; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], p.c2, nm));
          const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i + 1], p.c2, nm));
          l0 += e0;
          l1 += e1;
          pk[b][i >> 1] = pack_bf16(e0, e1);   // the second product takes p with 8 significant bits; l keeps 24
        }
      l += l0 + l1;
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk) {
        const uint32_t* w = &pk[kk >> 1][(kk & 1) * 4];
        const v4i pv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
#pragma unroll
        for (int d = 0; d < C::DB; ++d) {
          const uint32_t ad = stage + (va ^ (d << 6)) + kk * 16 * C::RB;
          const v4s v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)ad);
          const v4s v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(ad + 8 * C::RB));
          const auto vv = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, vv), __builtin_bit_cast(v8bf, pv), o[d],
                                                         0, 0, 0);
        }
      }
    }
    if constexpr (C::NBUF == 1) {
      group_sync();
      if (it + 1 < iters) issue(nxt, nmask, 0);
      after = slot_at(it + 2);
      keep = load_keep(after);
    }
  }
  wait_vmcnt<0>();   // no copy may land in memory that is used differently below

  l = half_sum(l);
  if (poisoned) l = NAN;

  if constexpr (WK > 1) {
    // Join the key groups: every wave leaves its (m, l) and its o scaled to
    // the common maximum in LDS; group 0's rows are summed by all waves.
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
    float* ml = red + C::NW * 32 * C::PITCH;
    if (h == 0) {
      ml[(wave * 32 + lr) * 2] = m;
      ml[(wave * 32 + lr) * 2 + 1] = l;
    }
    __syncthreads();
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < WK; ++k) mx = fmaxf(mx, ml[((k * WQ + wq) * 32 + lr) * 2]);
    const float f = __builtin_amdgcn_exp2f(m - (mx == -INFINITY ? 0.f : mx));
#pragma unroll
    for (int d = 0; d < C::DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<v4f*>(&red[(wave * 32 + lr) * C::PITCH + 32 * d + 8 * i + 4 * h]) =
            (v4f){o[d][4 * i] * f, o[d][4 * i + 1] * f, o[d][4 * i + 2] * f, o[d][4 * i + 3] * f};
    __syncthreads();
    for (int e = tid; e < WQ * 32 * (D / 4); e += 64 * C::NW) {
      const int rr = e / (D / 4), d = e % (D / 4) * 4;
      if (rr >= nrows) continue;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < WK; ++k) M = fmaxf(M, ml[(k * WQ * 32 + rr) * 2]);
      v4f acc = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const int x = k * WQ * 32 + rr;
        L += ml[x * 2 + 1] * __builtin_amdgcn_exp2f(ml[x * 2] - (M == -INFINITY ? 0.f : M));
        acc += *reinterpret_cast<const v4f*>(&red[x * C::PITCH + d]);
      }
      const int gr = r0 + rr;
      if (p.parts > 1) {
        const int64_t x = ((int64_t)part * a.Hkv + hk) * p.rows + gr;
        *reinterpret_cast<v4f*>(p.po + x * D + d) = acc;
        if (d == 0) *reinterpret_cast<v2f*>(p.pml + x * 2) = (v2f){M, L};
      } else {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        uint16_t* out = (uint16_t*)a.out + gr / p.tg * a.o_sb + gr % p.tg / p.g * a.o_st +
                        (int64_t)(hk * p.g + gr % p.g) * a.o_sh + d;
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
      }
    }
  } else {
    if (!live) return;
    if (p.parts > 1) {
      const int64_t x = ((int64_t)part * a.Hkv + hk) * p.rows + row;
#pragma unroll
      for (int d = 0; d < C::DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<v4f*>(p.po + x * D + 32 * d + 8 * i + 4 * h) =
              (v4f){o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
      if (h == 0) *reinterpret_cast<v2f*>(p.pml + x * 2) = (v2f){m, l};
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint16_t* out = (uint16_t*)a.out + rb * a.o_sb + rt * a.o_st + (int64_t)(hk * p.g + rg) * a.o_sh;
#pragma unroll
      for (int d = 0; d < C::DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint2*>(out + 32 * d + 8 * i + 4 * h) =
              make_uint2(pack_bf16(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                         pack_bf16(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv));
    }
  }
}

// Joins the parts of a row: D / 4 lanes a row, 16 bytes of each part a lane.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs p) {
  const w4a4_attn& a = p.a;
  constexpr int LPR = D / 4;
  const int64_t gr = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const int d = threadIdx.x % LPR * 4;
  const int64_t all = (int64_t)a.Hkv * p.rows;
  if (gr >= all) return;
  float M = -INFINITY, L = 0.f;
  for (int k = 0; k < p.parts; ++k) M = fmaxf(M, p.pml[(k * all + gr) * 2]);
  const float ms = M == -INFINITY ? 0.f : M;
  v4f acc = {0, 0, 0, 0};
  for (int k = 0; k < p.parts; ++k) {
    const v2f ml = *reinterpret_cast<const v2f*>(p.pml + (k * all + gr) * 2);
    const float f = __builtin_amdgcn_exp2f(ml[0] - ms);
    L += ml[1] * f;
    acc += *reinterpret_cast<const v4f*>(p.po + (k * all + gr) * D + d) * f;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int hk = (int)(gr / p.rows), row = (int)(gr % p.rows);
  uint16_t* out = (uint16_t*)a.out + row / p.tg * a.o_sb + row % p.tg / p.g * a.o_st + (int64_t)(hk * p.g + row % p.g) * a.o_sh + d;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
}

struct AttnPlan {
  int cfg;     // index of the (WQ, WK) pair
  int rpt, tiles, parts, np, ns;
};

struct Shape {
  int wq, wk, bn;
};
// (WQ, WK, BN) per head width; the kernels below are instantiated from it.
constexpr Shape kShapes[3][4] = {{{1, 4, 64}, {2, 4, 64}, {4, 2, 64}, {8, 1, 64}},     // D = 64
                                 {{1, 4, 32}, {2, 4, 32}, {4, 2, 64}, {8, 1, 64}},     // D = 128
                                 {{1, 4, 32}, {2, 2, 32}, {4, 1, 32}, {4, 1, 32}}};    // D = 256
constexpr int kCUs = 256;

AttnPlan plan_attention(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t P, int64_t S, bool split) {
  const Shape* sh = kShapes[D == 64 ? 0 : D == 128 ? 1 : 2];
  const int64_t tg = T * (Hq / Hkv), rows = B * tg;
  AttnPlan best{};
  double best_cost = 1e300;
  for (int c = 0; c < 4; ++c) {
    if (D == 256 && c == 3) break;
    const int64_t R = 32 * sh[c].wq;
    const int64_t rpt = tg <= R ? R / tg * tg : R;
    const int64_t tiles = (rows + rpt - 1) / rpt;
    const int64_t np = (P + sh[c].bn - 1) / sh[c].bn, ns = (S + sh[c].bn - 1) / sh[c].bn;
    const int64_t nseq = tg <= R ? rpt / tg : (R + tg - 1) / tg + (R % tg != 0);
    const int64_t total = np + (nseq < B ? nseq : B) * ns;
    const int64_t units = Hkv * tiles;
    // parts: one round of the card's CUs, with at least one block per key group
    int64_t parts = 1;
    if (split && units < kCUs) parts = kCUs / units;
    const int64_t cap = (total + sh[c].wk - 1) / sh[c].wk;
    if (parts > cap) parts = cap < 1 ? 1 : cap;
    const int64_t per = (total + parts * sh[c].wk - 1) / (parts * sh[c].wk);    // iterations of a workgroup
    const int64_t rounds = (units * parts + kCUs - 1) / kCUs;
    // microseconds: an iteration, and the join's launch and traffic
    const double iter = (sh[c].bn / 64.0) * (D / 128.0) * (sh[c].wq * sh[c].wk > 4 ? 1.5 : 1.0);
    double cost = rounds * (per * iter + 2.0);
    if (parts > 1) cost += 3.0 + parts * Hkv * rows * (double)D * 8.0 / 4e6;
    if (cost < best_cost) {
      best_cost = cost;
      best = {c, (int)rpt, (int)tiles, (int)parts, (int)np, (int)ns};
    }
  }
  return best;
}

template <typename C>
void launch_tiles(const AttnArgs& p, hipStream_t st) {
  attn_tile_kernel<C><<<(unsigned)(p.a.Hkv * p.tiles * p.parts), 64 * C::NW, 0, st>>>(p);
}

}  // namespace

size_t prefix_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t P, int64_t S) {
  const AttnPlan pl = plan_attention(B, T, Hq, Hkv, D, P, S, true);
  return pl.parts > 1 ? (size_t)pl.parts * B * T * Hq * (D + 2) * 4 : 0;
}

hipError_t launch_prefix_attention(const w4a4_attn& a, void* workspace, hipStream_t st) {
  const AttnPlan pl = plan_attention(a.B, a.T, a.Hq, a.Hkv, a.D, a.P, a.S, workspace != nullptr);
  AttnArgs p{};
  p.a = a;
  p.g = (int)(a.Hq / a.Hkv);
  p.tg = (int)a.T * p.g;
  p.rows = (int)(a.B * p.tg);
  p.rpt = pl.rpt;
  p.tiles = pl.tiles;
  p.parts = pl.parts;
  p.np = pl.np;
  p.ns = pl.ns;
  // A scale of zero weighs all keys alike; the tiny positive factor keeps
  // -inf (excluded) times the scale at -inf.
  const float c2 = (a.scale < 0 ? -a.scale : a.scale) * 1.4426950408889634f;
  p.c2 = c2 < 1e-30f ? 1e-30f : c2;
  p.qflip = a.scale < 0 ? 0x80008000u : 0;
  if (pl.parts > 1) {
    p.po = (float*)workspace;
    p.pml = p.po + (size_t)pl.parts * a.Hkv * p.rows * a.D;
  }
  if (a.D == 64) {
    if (pl.cfg == 0) launch_tiles<ACfg<64, 1, 4, 64, 2>>(p, st);
    else if (pl.cfg == 1) launch_tiles<ACfg<64, 2, 4, 64, 2>>(p, st);
    else if (pl.cfg == 2) launch_tiles<ACfg<64, 4, 2, 64, 2>>(p, st);
    else launch_tiles<ACfg<64, 8, 1, 64, 2>>(p, st);
  } else if (a.D == 128) {
    if (pl.cfg == 0) launch_tiles<ACfg<128, 1, 4, 32, 2>>(p, st);
    else if (pl.cfg == 1) launch_tiles<ACfg<128, 2, 4, 32, 2>>(p, st);
    else if (pl.cfg == 2) launch_tiles<ACfg<128, 4, 2, 64, 2>>(p, st);
    else launch_tiles<ACfg<128, 8, 1, 64, 2>>(p, st);
  } else {
    if (pl.cfg == 0) launch_tiles<ACfg<256, 1, 4, 32, 1>>(p, st);
    else if (pl.cfg == 1) launch_tiles<ACfg<256, 2, 2, 32, 2>>(p, st);
    else launch_tiles<ACfg<256, 4, 1, 32, 2>>(p, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.parts == 1) return e;
  const int64_t all = a.Hkv * (int64_t)p.rows;
  const int per = 256 / ((int)a.D / 4);
  const unsigned grid = (unsigned)((all + per - 1) / per);
  if (a.D == 64) attn_join_kernel<64><<<grid, 256, 0, st>>>(p);
  else if (a.D == 128) attn_join_kernel<128><<<grid, 256, 0, st>>>(p);
  else attn_join_kernel<256><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace w4a4
