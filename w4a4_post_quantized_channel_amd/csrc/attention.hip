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
// end.  A block's K and V go global -> LDS XOR-swizzled, so that the fragment
// reads are free of bank conflicts (none counted), into NBUF buffers per key
// group.  The block list of a row tile, prefix blocks then the own blocks of
// its sequences, is cut into `parts` for shapes with few rows; partial
// (m, l, o) go to the workspace and a second kernel joins them.
//
// Probabilities enter the second product as bf16: its rate is 16 times that of
// the 32-bit product, and a second bf16 product for what rounding lost would
// cost half as much time again.  Against 64 bits the output is off by 0.0022
// (relative, rms) where its own rounding to bf16 alone gives 0.0017.
//
// What bounds it (one MI355X).  Many rows (16 x 64 queries, 32 heads over 8,
// width 128, 16384 + 192 keys, 277 GFLOP): 270-284 us, 0.98-1.03 PFLOP/s, 55%
// of the matrix cycles at the 1.7 GHz the card holds there; a phase takes
// about 1750 cycles where its 32 products need 1024, the rest being the
// softmax's vector work, the issue of copies and the barriers.  Few rows: one
// block in flight a key group, whose load is waited out.  A decoding batch (64
// x 1 over 8192 + 256 keys) takes 35 us for 12 such iterations, of which the
// load path of a CU (43 bytes a cycle, all waves loading) is 9 to 11; a third
// of its blocks are own keys, seen by 4 of a tile's 64 rows.
#include "attention_plan.h"
#include "dense.h"
#include "device_common.h"
#include "lds_sync.h"

namespace w4a4 {

namespace {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef const __attribute__((address_space(3))) v4i lds_v4i;

constexpr float kLazy = 8.f;
constexpr int kNoBad = 1 << 30;

// Division by a number fixed for a launch: m = floor(2^32 / d) + 1 gives the
// quotient or one more (2^32 - 1 for d = 1: or one less).
struct Divisor {
  uint32_t d, m;
};
inline Divisor divisor(int64_t d) {
  return {(uint32_t)d, d == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / (uint64_t)d + 1)};
}
__device__ __forceinline__ int div_by(int x, const Divisor& v, int& rem) {
  int q = (int)__umulhi((uint32_t)x, v.m), r = x - q * (int)v.d;
  if (r < 0) --q, r += (int)v.d;
  if (r >= (int)v.d) ++q, r -= (int)v.d;
  rem = r;
  return q;
}

struct AttnArgs {
  w4a4_attn a;
  int rows;         // B T G rows of a KV head
  int rpt;          // rows of a tile
  Divisor tg, g;    // T G, G
  Divisor tiles, heads;
  int parts;
  int np;           // prefix blocks
  Divisor ns;       // own blocks of a sequence (1 if none)
  int own;          // 0: no own keys
  int per;          // blocks of a part
  float c2;         // |scale| log2 e
  uint32_t qflip;   // sign bits flipped in q when scale < 0
  float* po;        // parts > 1: [part][head][row][D], else null
  float* pml;       // [part][head][row][2]
};

template <int D_, int WQ_, int WK_, int BN_, int NBUF_>
struct ACfg {
  static constexpr int D = D_, WQ = WQ_, WK = WK_, BN = BN_, NBUF = NBUF_;
  static constexpr int NW = WQ * WK;
  static constexpr bool PINGPONG = WQ == 8 && NBUF == 4;
  static constexpr int RB = 2 * D;                  // bytes of a key or value row
  static constexpr int MAT = BN * RB;               // bytes of a block of one of them
  static constexpr int STAGE = 2 * MAT;
  static constexpr int NI = MAT / 1024 / WQ;        // copy instructions per wave and matrix
  static constexpr int RPI = 1024 / RB;             // rows per copy instruction
  static constexpr int AHEAD = D == 256 ? 3 : WQ == 1 ? 4 : 6;    // MFMA steps an operand is read ahead
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
  __shared__ int sbad[WK][3], slen[32 * C::WQ];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave % WQ, wk = wave / WQ;
  const int h = lane >> 5, lr = lane & 31;

  // Workgroup -> (part, tile, head), heads fastest, in contiguous runs per
  // XCD.  An XCD thus reads the same few key rows for all heads: where the
  // heads of a key lie side by side, one head alone is 2 D bytes in every
  // 2 D Hkv and would use few of the L2's channels.
  const int nwg = gridDim.x, wid = blockIdx.x;
  const int u = nwg % 8 == 0 ? (wid % 8) * (nwg / 8) + wid / 8 : wid;
  int tile, hk;
  const int part = div_by(div_by(u, p.heads, hk), p.tiles, tile);
  const w4a4_attn& a = p.a;

  const int r0 = tile * p.rpt, nrows = min(p.rpt, p.rows - r0);
  int rem;
  const int b0 = div_by(r0, p.tg, rem), nseq = div_by(r0 + nrows - 1, p.tg, rem) - b0 + 1;
  const int64_t total = p.np + (p.own ? (int64_t)nseq * (int)p.ns.d : 0);
  const int lo = (int)min((int64_t)part * p.per, total), hi = (int)min((int64_t)lo + p.per, total);

  // A block on its way from global memory to LDS, 16 bytes a lane and piece:
  // piece k of a matrix covers rows n RPI + [0, RPI), n = k WQ + wq, lane l
  // chunk l % (D / 8) of row l / (D / 8).  Excluded rows (past the end, or not
  // kept) take an out-of-range offset and arrive as zeros, so whatever lies
  // there never enters a product.
  const uint32_t lds0 = lds_addr(smem);
  const int cr = lane / (D / 8), cc = lane % (D / 8);
  v4i piece[2 * C::NI];
  auto load_matrix = [&](const Slot& s, uint64_t mask, const uint16_t* base, int64_t stride, bool is_k) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(base + s.j0 * stride, 0x7FFFFFFFu);
    const uint32_t st2 = (uint32_t)stride * 2, voff = cr * st2;
    const bool full = mask == low_bits<BN>(BN);
#pragma unroll
    for (int k = 0; k < C::NI; ++k) {
      const int rw = (k * WQ + wq) * C::RPI;
      uint32_t off = voff + rw * st2 + (cc ^ (is_k ? swz_k<D>(rw + cr) : swz_v<D>(rw + cr))) * 16;
      if (!full) off = (mask >> (rw + cr)) & 1 ? off : kOOB;
      piece[is_k ? k : C::NI + k] = __builtin_bit_cast(v4i, buf_load16(rs, off));
    }
  };
  auto load_block = [&](const Slot& s, uint64_t mask) {
    if (mask == 0) return;
    if (s.b < 0) {
      load_matrix(s, mask, (const uint16_t*)a.k_prefix + hk * a.kp_sh, a.kp_sp, true);
      load_matrix(s, mask, (const uint16_t*)a.v_prefix + hk * a.vp_sh, a.vp_sp, false);
    } else {
      load_matrix(s, mask, (const uint16_t*)a.k_own + s.b * a.ko_sb + hk * a.ko_sh, a.ko_ss, true);
      load_matrix(s, mask, (const uint16_t*)a.v_own + s.b * a.vo_sb + hk * a.vo_sh, a.vo_ss, false);
    }
  };
  auto store_block = [&](int buf) {
    const uint32_t dst = lds0 + (wk * C::NBUF + buf) * C::STAGE + lane * 16;
#pragma unroll
    for (int k = 0; k < 2 * C::NI; ++k)
      *(__attribute__((address_space(3))) v4i*)(dst + (k >= C::NI ? C::MAT : 0) + ((k % C::NI) * WQ + wq) * 1024) = piece[k];
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
  auto prefix_slot = [&](int i) {
    const int j0 = i * BN;
    return Slot{-1, j0, min(BN, (int)a.P - j0)};
  };
  auto group_sync = [&]() {
    asm volatile("" ::: "memory");
    if constexpr (WQ > 1) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // The first prefix blocks are under way before anything else is loaded.
  const int pend = min(hi, p.np);
  Slot nxt{-1, 0, 0};
  uint64_t nmask = 0;
  const bool early = !C::PINGPONG && lo + wk < pend;
  if (early) {
    nxt = prefix_slot(lo + wk);
    nmask = slot_mask(nxt, load_keep(nxt));
    load_block(nxt, nmask);
  }

  // lengths of the tile's sequences
  for (int i = tid; i < nseq; i += 64 * C::NW) slen[i] = a.own_len ? max(0, min(a.own_len[b0 + i], (int)a.S)) : (int)a.S;
  if (tid < WK) sbad[tid][0] = sbad[tid][1] = sbad[tid][2] = kNoBad;

  // this lane's row: query, sequence
  const int rl = wq * 32 + lr, row = r0 + rl;
  const bool live = rl < nrows;
  int rt, rg, rb = div_by(live ? row : r0, p.tg, rem);
  rt = div_by(rem, p.g, rg);
  const bool wave_live = wq * 32 < nrows;
  const int wb0 = div_by(r0 + (wave_live ? wq * 32 : 0), p.tg, rem);   // this wave's sequences
  const int wb1 = div_by(min(r0 + wq * 32 + 32, r0 + nrows) - 1, p.tg, rem);
  // own value rows are seen by some rows of a wave and not by others
  const bool mixed = a.causal || nseq > 1;

  v8bf qf[C::KC];
  {
    const uint16_t* q = (const uint16_t*)a.q + rb * a.q_sb + rt * a.q_st + (int64_t)(hk * (int)p.g.d + rg) * a.q_sh + h * 8;
#pragma unroll
    for (int c = 0; c < C::KC; ++c) {
      uint4 v = *reinterpret_cast<const uint4*>(q + c * 16);   // rows past the end repeat the tile's first
      v.x ^= p.qflip; v.y ^= p.qflip; v.z ^= p.qflip; v.w ^= p.qflip;
      qf[c] = __builtin_bit_cast(v8bf, v);
    }
  }

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
  const uint32_t va = vr * C::RB + (((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swz_v<D>(vr)) << 4) + (lane & 1) * 8;

  // Scores of a block -> probabilities (bf16, in the order the second product
  // takes them), with m, l and, when m moves, o brought up to date.
  uint32_t pk[C::SB][8];
  auto softmax = [&](v16f (&s)[C::SB]) {
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
  };
  auto exclude = [&](v16f (&s)[C::SB], uint64_t mask) {
#pragma unroll
    for (int b = 0; b < C::SB; ++b) {
      const uint32_t w = (uint32_t)(mask >> (32 * b)) >> (4 * h);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = (w >> (8 * (i >> 2) + (i & 3))) & 1 ? s[b][i] : -INFINITY;
    }
  };
  // LDS addresses of this lane's fragment reads in buffer 0; buffers, row
  // blocks and key steps are constant offsets from them
  uint32_t kad[C::KC], vad[C::DB];
#pragma unroll
  for (int c = 0; c < C::KC; ++c) kad[c] = lds0 + wk * C::NBUF * C::STAGE + (ka ^ (c << 5));
#pragma unroll
  for (int d = 0; d < C::DB; ++d) vad[d] = lds0 + wk * C::NBUF * C::STAGE + C::MAT + (va ^ (d << 6));
  // The products of a block as a list of steps, one MFMA each, with the LDS
  // reads kAhead steps in front of their MFMA (left to itself the compiler
  // reads each operand right before its use and waits out the latency every
  // time).  Both products have as many steps.  Together they start with
  // kAhead steps of P V, whose operands can be read before the barrier in
  // front, and then alternate.
  constexpr int kSteps = C::KC * C::SB;
  static_assert(kSteps == BN / 16 * C::DB, "products of equal length");
  constexpr int kAhead = C::AHEAD;
  static_assert(kAhead <= kSteps, "steps");
  v4i frag[kAhead];
  enum { QK = 1, PV = 2, BOTH = 3 };
  auto step_is_k = [](int what, int t) {
    return what == QK || (what == BOTH && (t >= 2 * kSteps - kAhead || (t >= kAhead && (t - kAhead) % 2 == 0)));
  };
  auto step_index = [](int what, int t) {
    if (what != BOTH || t < kAhead) return t;
    if (t >= 2 * kSteps - kAhead) return t - kSteps;
    return (t - kAhead) / 2 + ((t - kAhead) % 2 == 0 ? 0 : kAhead);
  };
  auto fetch = [&](int what, int t, int koff, int voff) {
    const int x = step_index(what, t);
    if (step_is_k(what, t)) {
      frag[t % kAhead] = *(lds_v4i*)(kad[x / C::SB] + koff + x % C::SB * 32 * C::RB);
    } else {
      const uint32_t ad = vad[x % C::DB] + voff + x / C::DB * 16 * C::RB;
      const v4s v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)ad);
      const v4s v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(ad + 8 * C::RB));
      frag[t % kAhead] = __builtin_bit_cast(v4i, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  auto fetch_first = [&](int what, int koff, int voff) {
#pragma unroll
    for (int t = 0; t < kAhead; ++t) fetch(what, t, koff, voff);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto products = [&](v16f (&s)[C::SB], auto what_, int koff, int voff) {
    constexpr int what = what_();
    constexpr int n = what == BOTH ? 2 * kSteps : kSteps;
#pragma unroll
    for (int t = 0; t < n; ++t) {
      const int x = step_index(what, t);
      const v8bf op = __builtin_bit_cast(v8bf, frag[t % kAhead]);
      if (step_is_k(what, t)) {
        s[x % C::SB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(op, qf[x / C::SB], s[x % C::SB], 0, 0, 0);
      } else {
        const uint32_t* w = &pk[x / C::DB >> 1][(x / C::DB & 1) * 4];
        const v4i pv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
        o[x % C::DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(op, __builtin_bit_cast(v8bf, pv), o[x % C::DB], 0, 0, 0);
      }
      if (t + kAhead < n) fetch(what, t + kAhead, koff, voff);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  struct Qk { constexpr int operator()() const { return QK; } };
  struct Pv { constexpr int operator()() const { return PV; } };
  struct Both { constexpr int operator()() const { return BOTH; } };
  auto clear = [&](v16f (&s)[C::SB]) {
#pragma unroll
    for (int b = 0; b < C::SB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
  };

  // Prefix blocks with eight waves of rows: waves 0-3 and 4-7 (one of each on
  // every SIMD) run half an iteration apart, so that one multiplies while the
  // other does its softmax.  Phase 2 i: waves 0-3 take the products M(i)
  // (block i - 1 times V, block i times K), waves 4-7 softmax S(i - 1); phase
  // 2 i + 1: the other way round.  A barrier ends every phase.  Stage i (K and
  // V of block i) is read in phases 2 i to 2 i + 3.  S(i) copies stage i + 2
  // into the buffer of stage i - 2 (a copy takes about 100 cycles to issue,
  // too long between the products of M); each wave waits for its copies of
  // stage i + 1 in phase 2 i + 1, between M(i) and S(i).
  int glo = lo;
  if constexpr (C::PINGPONG) {
    const int n = pend - lo;
    glo = max(lo, p.np);
    if (n > 0) {
      const bool second = wave >= 4;
      auto block_at = [&](int i) {
        Slot b = prefix_slot(lo + i);
        if (i >= n) b.valid = 0;
        return b;
      };
      // stages are copied in order: the bases step by a block, the lanes'
      // offsets stay
      uint64_t kbase = (uint64_t)((const uint16_t*)a.k_prefix + hk * a.kp_sh + (int64_t)lo * BN * a.kp_sp);
      uint64_t vbase = (uint64_t)((const uint16_t*)a.v_prefix + hk * a.vp_sh + (int64_t)lo * BN * a.vp_sp);
      uint32_t off[2 * C::NI];
#pragma unroll
      for (int k = 0; k < C::NI; ++k) {
        const int row = (k * WQ + wq) * C::RPI + cr;
        off[k] = (uint32_t)(row * a.kp_sp * 2) + (cc ^ swz_k<D>(row)) * 16;
        off[C::NI + k] = (uint32_t)(row * a.vp_sp * 2) + (cc ^ swz_v<D>(row)) * 16;
      }
      auto copy_one = [&](int i, int k, uint64_t mask) {   // copy k of 2 NI of stage i
        const bool isv = k >= C::NI;
        const int n_ = (isv ? k - C::NI : k) * WQ + wq;
        const uint64_t b = isv ? vbase : kbase;
        const v4u rs = {(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, 0x7FFFFFFFu, 0x00020000u};
        const uint32_t dst = lds0 + (i & 3) * C::STAGE + (isv ? C::MAT : 0) + n_ * 1024;
        if (mask == low_bits<BN>(BN)) dma16_v(rs, dst, off[k]);
        else dma16_v(rs, dst, (mask >> (n_ * C::RPI + cr)) & 1 ? off[k] : kOOB);
      };
      auto next_stage = [&]() {
        kbase += BN * a.kp_sp * 2;
        vbase += BN * a.vp_sp * 2;
      };
      uint64_t m0, m1, m2 = 0;   // masks of blocks i, i + 1, i + 2
      uint32_t keep;             // keep bytes of block i + 2
      {
        const Slot s0 = block_at(0), s1 = block_at(1);
        const uint32_t k0 = load_keep(s0), k1 = load_keep(s1);
        keep = load_keep(block_at(2));
        m0 = slot_mask(s0, k0);
        m1 = slot_mask(s1, k1);
#pragma unroll
        for (int k = 0; k < 2 * C::NI; ++k) copy_one(0, k, m0);
        next_stage();
        if (n > 1)
#pragma unroll
          for (int k = 0; k < 2 * C::NI; ++k) copy_one(1, k, m1);
        next_stage();
      }
      // M(0) has no block before it: its V, in the buffer of stage -1, and P are zero
#pragma unroll
      for (int k = 0; k < C::NI; ++k)
        *(__attribute__((address_space(3))) v4i*)(lds0 + 3 * C::STAGE + C::MAT + (k * WQ + wq) * 1024 + lane * 16) =
            (v4i){0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < C::SB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) pk[b][i] = 0;
#pragma unroll
      for (int d = 0; d < C::DB; ++d) vad[d] += 3 * C::STAGE;
      auto phase = [&]() {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      };
      v16f s[C::SB];
      wait_vmcnt<0>();
      phase();
      if (second) phase();
      fetch_first(BOTH, 0, 0);
      for (int i = 0; i < n; ++i) {
        __builtin_amdgcn_s_setprio(1);
        clear(s);
        products(s, Both(), 0, 0);
        __builtin_amdgcn_s_setprio(0);
        const int kstep = (i & 3) == 3 ? -3 * C::STAGE : C::STAGE, vstep = (i & 3) == 0 ? -3 * C::STAGE : C::STAGE;
#pragma unroll
        for (int c = 0; c < C::KC; ++c) kad[c] += kstep;
#pragma unroll
        for (int d = 0; d < C::DB; ++d) vad[d] += vstep;
        if (second) wait_vmcnt<0>();   // stage i + 1
        phase();
        if (!second) wait_vmcnt<0>();
        asm volatile("" ::: "memory");
        if (i + 2 < n) {
          m2 = slot_mask(block_at(i + 2), keep);
#pragma unroll
          for (int k = 0; k < 2 * C::NI; ++k) copy_one(i + 2, k, m2);
          next_stage();
          keep = load_keep(block_at(i + 3));
        }
        fetch_first(PV, 0, 0);   // the first operands of M(i + 1)
        if (m0 != low_bits<BN>(BN)) exclude(s, m0);
        softmax(s);
        m0 = m1;
        m1 = m2;
        phase();
      }
      products(s, Pv(), 0, 0);
      if (!second) phase();
#pragma unroll
      for (int c = 0; c < C::KC; ++c) kad[c] -= (n & 3) * C::STAGE;
#pragma unroll
      for (int d = 0; d < C::DB; ++d) vad[d] -= ((n - 1) & 3) * C::STAGE;
      __syncthreads();
    }
  }

  // Everything else, block by block: own keys, and prefix keys with fewer waves.
  __syncthreads();   // lengths and flags are set
  int rlim = live ? slen[rb - b0] : 0;   // own keys this row sees
  if (a.causal) rlim = max(0, min(rlim, rlim - (int)a.T + 1 + rt));
  const int iters = (hi - glo + WK - 1) / WK;
  auto slot_at = [&](int it) {
    Slot s{-1, 0, 0};
    const int i = glo + it * WK + wk;
    if (i >= hi) return s;
    if (i < p.np) return prefix_slot(i);
    int blk;
    const int sq = div_by(i - p.np, p.ns, blk);
    s.b = b0 + sq;
    s.j0 = blk * BN;
    s.valid = max(0, min(BN, __builtin_amdgcn_readfirstlane(slen[sq]) - s.j0));
    return s;
  };
  if (!early && iters > 0) {
    nxt = slot_at(0);
    nmask = slot_mask(nxt, load_keep(nxt));
    load_block(nxt, nmask);
  }
  Slot after = slot_at(1);
  uint32_t keep = load_keep(after);

  // Iteration `it` stores its block from registers to LDS, loads the next one
  // into them, and multiplies.  With one wave per key group the wave's own
  // order of LDS accesses is all the synchronisation there is, and one buffer
  // is enough.
  //
  // Own values that some rows of the tile must not see: a piece with a NaN or
  // Inf is stored as zeros, and the rows that do see its key are marked.  The
  // lowest such key of iteration `it` is in sbad[][it % 3]; the next
  // iteration's is cleared a barrier before it is written.
  for (int it = 0, third = 0; it < iters; ++it, third = third == 2 ? 0 : third + 1) {
    const Slot cur = nxt;
    const uint64_t cmask = nmask;
    const int buf = C::NBUF > 1 ? (it & 1) : 0;
    if (mixed && cur.b >= 0 && cmask != 0) {
#pragma unroll
      for (int k = C::NI; k < 2 * C::NI; ++k) {
        uint32_t bad = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= (((uint32_t)piece[k][e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
        if (bad) {
          piece[k] = (v4i){0, 0, 0, 0};
          atomicMin(&sbad[wk][third], ((k - C::NI) * WQ + wq) * C::RPI + cr);
        }
      }
    }
    if (cmask != 0) store_block(buf);
    if (wq == 0 && lane == 0) sbad[wk][third == 2 ? 0 : third + 1] = kNoBad;
    nxt = after;
    nmask = it + 1 < iters ? slot_mask(nxt, keep) : 0;
    load_block(nxt, nmask);
    after = slot_at(it + 2);
    keep = load_keep(after);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    group_sync();   // stored by all, and the other buffer is no longer read
    const int boff = buf * C::STAGE;
    if (mixed && cur.b >= 0 && live && rb == cur.b && cur.j0 + sbad[wk][third] < rlim) poisoned = true;

    const bool mine = cmask != 0 && wave_live && (cur.b < 0 || (cur.b >= wb0 && cur.b <= wb1));
    if (mine) {
      v16f s[C::SB];
      clear(s);
      fetch_first(QK, boff, 0);
      products(s, Qk(), boff, 0);
      if (cur.b >= 0) {
        const int vis = (rb == cur.b ? rlim - cur.j0 : 0) - 4 * h;
#pragma unroll
        for (int b = 0; b < C::SB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = 32 * b + 8 * (i >> 2) + (i & 3) < vis ? s[b][i] : -INFINITY;
      } else if (cmask != low_bits<BN>(BN)) {
        exclude(s, cmask);
      }
      softmax(s);
      fetch_first(PV, 0, boff);
      products(s, Pv(), 0, boff);
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
        int og, ob = div_by(gr, p.tg, rem), ot = div_by(rem, p.g, og);
        uint16_t* out = (uint16_t*)a.out + ob * a.o_sb + ot * a.o_st + (int64_t)(hk * (int)p.g.d + og) * a.o_sh + d;
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
      uint16_t* out = (uint16_t*)a.out + rb * a.o_sb + rt * a.o_st + (int64_t)(hk * (int)p.g.d + rg) * a.o_sh;
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
#pragma unroll 4
  for (int k = 0; k < p.parts; ++k) M = fmaxf(M, p.pml[(k * all + gr) * 2]);
  const float ms = M == -INFINITY ? 0.f : M;
  v4f acc = {0, 0, 0, 0};
#pragma unroll 4
  for (int k = 0; k < p.parts; ++k) {
    const v2f ml = *reinterpret_cast<const v2f*>(p.pml + (k * all + gr) * 2);
    const float f = __builtin_amdgcn_exp2f(ml[0] - ms);
    L += ml[1] * f;
    acc += *reinterpret_cast<const v4f*>(p.po + (k * all + gr) * D + d) * f;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int hk = (int)gr / p.rows, row = (int)gr % p.rows;
  int rem, g, b = div_by(row, p.tg, rem), t = div_by(rem, p.g, g);
  uint16_t* out = (uint16_t*)a.out + b * a.o_sb + t * a.o_st + (int64_t)(hk * (int)p.g.d + g) * a.o_sh + d;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
}

template <typename C>
void launch_tiles(const AttnArgs& p, hipStream_t st) {
  attn_tile_kernel<C><<<(unsigned)(p.a.Hkv * p.tiles.d * p.parts), 64 * C::NW, 0, st>>>(p);
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
  const int64_t g = a.Hq / a.Hkv;
  p.g = divisor(g);
  p.tg = divisor(a.T * g);
  p.rows = (int)(a.B * a.T * g);
  p.rpt = pl.rpt;
  p.tiles = divisor(pl.tiles);
  p.parts = pl.parts;
  p.heads = divisor(a.Hkv);
  p.np = pl.np;
  p.ns = divisor(pl.ns > 0 ? pl.ns : 1);
  p.own = pl.ns > 0;
  p.per = pl.per;
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
    if (pl.cfg == 0) launch_tiles<ACfg<64, 1, 8, 64, 1>>(p, st);
    else if (pl.cfg == 1) launch_tiles<ACfg<64, 2, 4, 64, 2>>(p, st);
    else if (pl.cfg == 2) launch_tiles<ACfg<64, 4, 2, 64, 2>>(p, st);
    else launch_tiles<ACfg<64, 8, 1, 64, 4>>(p, st);
  } else if (a.D == 128) {
    if (pl.cfg == 0) launch_tiles<ACfg<128, 1, 8, 32, 1>>(p, st);
    else if (pl.cfg == 1) launch_tiles<ACfg<128, 2, 4, 32, 2>>(p, st);
    else if (pl.cfg == 2) launch_tiles<ACfg<128, 4, 2, 64, 2>>(p, st);
    else launch_tiles<ACfg<128, 8, 1, 64, 4>>(p, st);
  } else {
    if (pl.cfg == 0) launch_tiles<ACfg<256, 2, 2, 32, 2>>(p, st);
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
