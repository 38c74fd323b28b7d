// bf16 product with bias, activation and residual:
//   y = act(x W^T + bias) + residual.
//
// Tiles of BM x BN outputs, K in stages of 64 (a 128-byte line per row).
// Stages are copied global -> LDS with 16-byte copies (XOR-swizzled 16-byte
// slots, see swz128) into NBUF buffers, NBUF - 1 stages ahead, and multiplied
// with v_mfma_f32_16x16x32_bf16.  W is the first operand and x the second,
// so that a lane's four accumulators are four adjacent columns of one output
// row.  The epilogue passes 16 rows at a time through LDS as fp32, so that
// bias, activation and residual work on whole row segments and every store
// is 16 bytes of a row.
//
// SwiGLU: 16-row fragments of a W tile alternate between the gate's rows and
// the up projection's, so one wave holds both factors of its outputs.
//
// Few output tiles: K is split over workgroups; fp32 partial sums go to the
// workspace and a second kernel adds them in order and runs the epilogue.
//
// What bounds it (one MI355X).  4096 x 5120 x 5120 with bias and GELU: 256
// tiles of 256 x 320 are one round of the card, 162-180 us (1.2-1.3 PFLOP/s)
// against 153 us of matrix time at the rate a large library product reaches.
// A direct copy takes about 100 cycles to issue; with its 9 copies a stage up
// front the loop ran 200 us, one to a step 192; the epilogue that read bias
// and residual per chunk cost 36 us of that, the present one under 10.
// 64 x 2048 x 8192: 14 us, of which the second launch and the partial sums
// take 5 and the weights' 33.5 MB 6.6 at the copy rate.
#include "activation.h"
#include "dense.h"
#include "device_common.h"
#include "gemm_bf16_plan.h"
#include "lds_sync.h"

namespace w4a4 {

namespace {

// Slot swizzle of a 128-byte LDS row: the 16 rows of a fragment read land on
// distinct banks in each of the read's four cycles.
__device__ __forceinline__ int swz128(int row) {
  return ((row >> 1) & 1) ^ (row & 4) ^ (((row >> 3) & 1) * 6);
}

// Eight adjacent columns of an output row, from column n.  Bias and residual
// are read ahead of the sums they are added to.
struct Bias8 {
  float b[8], up[8];   // up: SwiGLU's second factor
};
template <bool GATED>
__device__ __forceinline__ Bias8 load_bias8(const DenseArgs& g, int n) {
  Bias8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = min(n + e, g.N - 1);   // past the end: read but not used
    r.b[e] = r.up[e] = 0.f;
    if (!g.bias) continue;
    if (g.bias_bf16) {
      r.b[e] = bf16_bits_to_f32(((const uint16_t*)g.bias)[i]);
      if (GATED) r.up[e] = bf16_bits_to_f32(((const uint16_t*)g.bias)[g.N + i]);
    } else {
      r.b[e] = ((const float*)g.bias)[i];
      if (GATED) r.up[e] = ((const float*)g.bias)[g.N + i];
    }
  }
  return r;
}

// Residual of a chunk as its bits (bf16: four words, fp32: eight).
// vec: 16-byte accesses to y and the residual are aligned.
struct Res8 {
  uint32_t w[8];
};
__device__ __forceinline__ Res8 load_res8(const DenseArgs& g, int m, int n, bool vec) {
  Res8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r.w[e] = 0;
  if (!g.residual || m >= g.M || n >= g.N) return r;
  const int64_t at = m * g.ldr + n;
  if (n + 8 <= g.N && vec) {
    const uint4* p = reinterpret_cast<const uint4*>((const char*)g.residual + at * (g.y_bf16 ? 2 : 4));
    const uint4 a = p[0];
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    if (!g.y_bf16) {
      const uint4 b = p[1];
      r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < g.N) {
        if (g.y_bf16) r.w[e >> 1] |= (uint32_t)((const uint16_t*)g.residual)[at + e] << (16 * (e & 1));
        else r.w[e] = ((const uint32_t*)g.residual)[at + e];
      }
  }
  return r;
}

// act(z + bias) + residual (SwiGLU: silu(z + bias) (u + bias) + residual),
// one rounding, store.
template <int KIND, bool GATED>
__device__ __forceinline__ void finish8(const DenseArgs& g, float (&z)[8], const float (&u)[8], const Bias8& b,
                                        const Res8& res, int m, int n, bool vec) {
  if (m >= g.M || n >= g.N) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v = z[e] + b.b[e];
    if constexpr (GATED) v = times_sigmoid(v, v) * (u[e] + b.up[e]);
    else v = activate_kind<KIND>(v, g.act);
    const float r = !g.y_bf16 ? __uint_as_float(res.w[e])
                              : __uint_as_float(e & 1 ? res.w[e >> 1] & 0xFFFF0000u : res.w[e >> 1] << 16);
    z[e] = v + r;
  }
  const bool whole = n + 8 <= g.N && vec;
  const int64_t yo = m * g.ldy + n;
  // non-temporal: the output is not read again here
  if (g.y_bf16) {
    uint16_t* y = (uint16_t*)g.y + yo;
    v4i w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      typedef float v2f __attribute__((ext_vector_type(2)));
      w[e] = __builtin_bit_cast(int, __builtin_convertvector((v2f){z[2 * e], z[2 * e + 1]}, v2bf));
    }
    if (whole) {
      __builtin_nontemporal_store(w, reinterpret_cast<v4i*>(y));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < g.N) y[e] = (uint16_t)((uint32_t)w[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* y = (float*)g.y + yo;
    if (whole) {
      __builtin_nontemporal_store((v4f){z[0], z[1], z[2], z[3]}, reinterpret_cast<v4f*>(y));
      __builtin_nontemporal_store((v4f){z[4], z[5], z[6], z[7]}, reinterpret_cast<v4f*>(y) + 1);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < g.N) y[e] = z[e];
    }
  }
}

__host__ __device__ inline bool vec_ok(const DenseArgs& g) {
  const uintptr_t esz = g.y_bf16 ? 2 : 4;
  uintptr_t bits = (uintptr_t)g.y | (uintptr_t)g.ldy * esz;
  if (g.residual) bits |= (uintptr_t)g.residual | (uintptr_t)g.ldr * esz;
  return bits % 16 == 0;
}

struct GemmPlanArgs {
  DenseArgs g;
  int tiles_m, tiles_n, splits;
  int stages;        // K stages in all
  float* part;       // splits > 1: [split][m][W row], row length pn
  int pn;
};

template <int TI_, int TJ_, int WR_, int WC_, int NBUF_>
struct GCfg {
  static constexpr int TI = TI_, TJ = TJ_, WR = WR_, WC = WC_, NBUF = NBUF_;
  static constexpr int NW = WR * WC;
  static constexpr int BM = WR * TI * 16, BN = WC * TJ * 16;   // BN: rows of W
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int NA = BM / 8, NB = BN / 8;               // copy instructions of a stage
  static constexpr int PA = (NA + NW - 1) / NW, PB = (NB + NW - 1) / NW, DPS = PA + PB;
  static constexpr int PITCH = TJ * 16 + 4;                    // floats of an epilogue row
  static constexpr int PIPE = NBUF * STAGE + 1024;             // + the target of padding copies
  static constexpr int EPI = NW * 16 * PITCH * 4;
  static constexpr int LDS = PIPE > EPI ? PIPE : EPI;
  static_assert(LDS <= 160 * 1024 && DPS * (NBUF - 2) <= 63, "limits");
};

template <typename C, int KIND, bool GATED>
__global__ void __launch_bounds__(64 * C::NW) __attribute__((amdgpu_waves_per_eu((C::NW + 3) / 4, 8)))
gemm_bf16_kernel(GemmPlanArgs p) {
  constexpr int TI = C::TI, TJ = C::TJ, NW = C::NW;
  static_assert(!GATED || TJ % 2 == 0, "gate and up fragments in pairs");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  const DenseArgs& g = p.g;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WC * TI * 16, wn = wave % C::WC * TJ * 16;

  // Workgroup -> tile: contiguous runs per XCD, groups of four row tiles
  // walked column by column, K splits outermost.
  const int nwg = gridDim.x, wid = blockIdx.x;
  int t = nwg % 8 == 0 ? (wid % 8) * (nwg / 8) + wid / 8 : wid;
  const int per = p.tiles_m * p.tiles_n, split = t / per;
  t %= per;
  constexpr int GM = 4;
  const int grp = t / (GM * p.tiles_n), gm0 = grp * GM, gh = min(GM, p.tiles_m - gm0);
  const int tm = gm0 + t % (GM * p.tiles_n) % gh, tn = t % (GM * p.tiles_n) / gh;
  const int m0 = tm * C::BM, n0 = tn * (GATED ? C::BN / 2 : C::BN);
  const int s0 = (int)((int64_t)p.stages * split / p.splits), s1 = (int)((int64_t)p.stages * (split + 1) / p.splits);

  // Copies: instruction n of an operand covers 8 rows; lane l chunk slot
  // l % 8 of row l / 8.  Rows past the end and columns past K take an
  // out-of-range offset and arrive as zeros.
  const uint32_t lds0 = lds_addr(smem);
  const v4u rsA = rsrc_words(g.x + (int64_t)m0 * g.ldx, 0x7FFFFFFFu);
  const v4u rsB = rsrc_words(g.w + (int64_t)n0 * g.ldw, 0x7FFFFFFFu);
  const v4u rsU = GATED ? rsrc_words(g.w + ((int64_t)g.N + n0) * g.ldw, 0x7FFFFFFFu) : rsB;
  const int crow = lane >> 3, cslot = lane & 7;
  uint32_t offA[C::PA], offB[C::PB];
  // NW is even: the row's bits that the swizzle takes are the same in every instruction of a wave
  const int col = (cslot ^ swz128((wave & 1) * 8 + crow)) * 16;
#pragma unroll
  for (int k = 0; k < C::PA; ++k) {
    const int n = k * NW + wave, row = n * 8 + crow;
    offA[k] = n < C::NA && m0 + row < g.M ? (uint32_t)(row * g.ldx * 2) + col : kOOB;
  }
#pragma unroll
  for (int k = 0; k < C::PB; ++k) {
    const int n = k * NW + wave, row = n * 8 + crow;
    const int nl = GATED ? (row >> 5) * 16 + (row & 15) : row;   // output column within the tile
    offB[k] = n < C::NB && n0 + nl < g.N ? (uint32_t)(nl * g.ldw * 2) + col : kOOB;
  }
  const int kbytes = g.K * 2;
  // copy k of DPS of stage s
  auto copy_one = [&](int s, int k) {
    const bool isa = k < C::PA;
    const int n = (isa ? k : k - C::PA) * NW + wave;
    const uint32_t base = lds0 + (uint32_t)((s - s0) % C::NBUF) * C::STAGE;
    const uint32_t pad = lds0 + C::NBUF * C::STAGE;
    const int left = s < s1 ? kbytes - s * 128 : 0;   // bytes of this stage's rows
    const uint32_t k0 = left > 0 ? s * 128u : 0;
    const bool real = isa ? (C::NA % NW == 0 || n < C::NA) : (C::NB % NW == 0 || n < C::NB);
    dma16_at(isa ? rsA : (GATED && (n & 2)) ? rsU : rsB, real ? base + (isa ? 0 : C::A_BYTES) + n * 1024 : pad,
             col < left ? (isa ? offA[k < C::PA ? k : 0] : offB[k >= C::PA ? k - C::PA : 0]) : kOOB, k0);
  };

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  int aoff[2], boff[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    aoff[k] = (wm + lr) * 128 + (((4 * k + lq) ^ swz128(lr)) << 4);
    boff[k] = C::A_BYTES + (wn + lr) * 128 + (((4 * k + lq) ^ swz128(lr)) << 4);
  }

  // A stage is 2 TI steps of TJ products: step t multiplies fragment t % TI of
  // x with all of W's fragments of K half t / TI.  x fragments are read two
  // steps ahead, W's second half during the first, and the next stage's
  // copies, which take about 100 cycles each to issue, go one to a step.
  // The order is pinned: left to itself the compiler reads operands right
  // before their use.
#pragma unroll
  for (int b = 0; b < C::NBUF - 1; ++b)
#pragma unroll
    for (int k = 0; k < C::DPS; ++k) copy_one(s0 + b, k);
  constexpr int RING = 3, STEPS = 2 * TI, CPS = (C::DPS + STEPS - 1) / STEPS, BPS = (TJ + TI - 1) / TI;
  for (int s = s0; s < s1; ++s) {
    wait_vmcnt_lds<C::DPS * (C::NBUF - 2)>();   // stage s has landed (later ones may be in flight), s - 1 is read
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();           // for every wave
    asm volatile("" ::: "memory");
    const uint8_t* base = smem + (s - s0) % C::NBUF * C::STAGE;
    v8bf a[RING], b[2][TJ];
    auto read_a = [&](int t) {
      a[t % RING] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(base + aoff[t / TI] + t % TI * 2048));
    };
    auto read_b = [&](int k, int j) {
      b[k][j] = __builtin_bit_cast(v8bf, *reinterpret_cast<const uint4*>(base + boff[k] + j * 2048));
    };
    read_a(0);
#pragma unroll
    for (int j = 0; j < TJ; ++j) read_b(0, j);
    read_a(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      if (t + 2 < STEPS) read_a(t + 2);
      if (t < TI)
#pragma unroll
        for (int j = t * BPS; j < (t + 1) * BPS && j < TJ; ++j) read_b(1, j);
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        acc[t % TI][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[t / TI][j], a[t % RING], acc[t % TI][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = t * CPS; k < (t + 1) * CPS && k < C::DPS; ++k) copy_one(s + C::NBUF - 1, k);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  wait_vmcnt<0>();
  __syncthreads();   // no copy in flight, no stage being read: LDS is free for the epilogue

  if (p.splits > 1) {
    // partial sums: a lane's four values are adjacent W rows
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int m = m0 + wm + i * 16 + lr;
      float* row = p.part + ((int64_t)split * g.M + m) * p.pn + tn * C::BN + wn + lq * 4;
      if (m < g.M)
#pragma unroll
        for (int j = 0; j < TJ; ++j) *reinterpret_cast<v4f*>(row + j * 16) = acc[i][j];
    }
    return;
  }
  // Epilogue: 16 rows at a time through this wave's slice of LDS.  A lane
  // keeps its 8 columns, so that bias is read once; OC lanes share a row.
  const bool vec = vec_ok(g);
  float* buf = reinterpret_cast<float*>(smem) + wave * 16 * C::PITCH;
  constexpr int OC = (GATED ? TJ / 2 : TJ) * 2;      // 8-column chunks of a row
  constexpr int RPP = 64 / OC, PASSES = (16 + RPP - 1) / RPP;
  const int ch = lane % OC, prow = lane / OC;
  const int n = n0 + (GATED ? wn / 2 : wn) + ch * 8;
  const float* src = buf + (GATED ? (ch >> 1) * 32 + (ch & 1) * 8 : ch * 8);
  const Bias8 bias = load_bias8<GATED>(g, n);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int mb = m0 + wm + i * 16;
    Res8 res[PASSES];
#pragma unroll
    for (int q = 0; q < PASSES; ++q) res[q] = load_res8(g, prow < RPP && prow + q * RPP < 16 ? mb + prow + q * RPP : g.M, n, vec);
#pragma unroll
    for (int j = 0; j < TJ; ++j) *reinterpret_cast<v4f*>(buf + lr * C::PITCH + j * 16 + lq * 4) = acc[i][j];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
      const int row = prow + q * RPP;
      if (prow < RPP && row < 16) {
        float z[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const v4f v = *reinterpret_cast<const v4f*>(src + row * C::PITCH + e);
          const v4f w = GATED ? *reinterpret_cast<const v4f*>(src + row * C::PITCH + 16 + e) : v4f{0, 0, 0, 0};
#pragma unroll
          for (int x = 0; x < 4; ++x) z[e + x] = v[x], u[e + x] = w[x];
        }
        finish8<KIND, GATED>(g, z, u, bias, res[q], mb + row, n, vec);
      }
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_sched_barrier(0);   // one row block's registers at a time
  }
}

// At most 16 rows (decoding): one launch, no LDS on the way.  A workgroup
// takes 16 output columns and its eight waves a share of K each, operands
// straight from global memory (16 bytes a lane, kRowsAhead steps of 32 K in
// flight); the waves' sums are added in order through LDS.
constexpr int kRowsAhead = 8;

template <int KIND, bool GATED>
__global__ void __launch_bounds__(64 * kRowsWaves) gemm_bf16_rows_kernel(DenseArgs g) {
  constexpr int F = GATED ? 2 : 1, PITCH = 20;
  __shared__ __attribute__((aligned(16))) float red[F][kRowsWaves][16][PITCH];
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;
  const int steps = (g.K + 31) / 32, per = (steps + kRowsWaves - 1) / kRowsWaves;
  const int s1 = min(steps, (wave + 1) * per);
  const bool row_on = lr < g.M, col_on = n0 + lr < g.N;
  const uint16_t* x = g.x + (int64_t)(row_on ? lr : 0) * g.ldx + lq * 8;
  const uint16_t* w = g.w + (int64_t)(col_on ? n0 + lr : 0) * g.ldw + lq * 8;
  const uint16_t* up = w + (int64_t)g.N * g.ldw;
  const v4i zero = {0, 0, 0, 0};
  auto chunk = [&](const uint16_t* p, int s, bool on) {
    on = on && s < s1 && s * 32 + lq * 8 < g.K;
    return on ? *reinterpret_cast<const v4i*>(p + (int64_t)s * 32) : zero;
  };
  v4f acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = v4f{0, 0, 0, 0};
  for (int s = wave * per; s < s1; s += kRowsAhead) {
    v4i a[kRowsAhead], b[F][kRowsAhead];
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) {
      a[k] = chunk(x, s + k, row_on);
      b[0][k] = chunk(w, s + k, col_on);
      if constexpr (GATED) b[F - 1][k] = chunk(up, s + k, col_on);
    }
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k)
#pragma unroll
      for (int f = 0; f < F; ++f)
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, b[f][k]), __builtin_bit_cast(v8bf, a[k]),
                                                         acc[f], 0, 0, 0);
  }
#pragma unroll
  for (int f = 0; f < F; ++f) *reinterpret_cast<v4f*>(&red[f][wave][lr][lq * 4]) = acc[f];
  __syncthreads();
  const int m = threadIdx.x >> 1, c = (threadIdx.x & 1) * 8;
  if (m >= g.M) return;
  const bool vec = vec_ok(g);
  const Bias8 bias = load_bias8<GATED>(g, n0 + c);
  const Res8 res = load_res8(g, m, n0 + c, vec);
  float z[8], u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    z[e] = u[e] = 0.f;
#pragma unroll
    for (int k = 0; k < kRowsWaves; ++k) {
      z[e] += red[0][k][m][c + e];
      if constexpr (GATED) u[e] += red[F - 1][k][m][c + e];
    }
  }
  finish8<KIND, GATED>(g, z, u, bias, res, m, n0 + c, vec);
}

// Adds the K splits in order and runs the epilogue: 8 columns a thread.
template <int KIND, bool GATED>
__global__ void __launch_bounds__(64) gemm_bf16_join_kernel(GemmPlanArgs p) {
  const DenseArgs& g = p.g;
  const int chunks = (g.N + 7) / 8;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (id >= (int64_t)g.M * chunks) return;
  const int m = (int)(id / chunks), n = (int)(id % chunks) * 8;
  // column n of the partial rows: SwiGLU rows hold 16 gate then 16 up values
  const int col = GATED ? (n >> 4) * 32 + (n & 15) : n;
  const float* src = p.part + (int64_t)m * p.pn + col;
  const int64_t step = (int64_t)g.M * p.pn;
  v4f z0 = {0, 0, 0, 0}, z1 = z0, u0 = z0, u1 = z0;
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s, src += step) {
    z0 += *reinterpret_cast<const v4f*>(src);
    z1 += *reinterpret_cast<const v4f*>(src + 4);
    if constexpr (GATED) {
      u0 += *reinterpret_cast<const v4f*>(src + 16);
      u1 += *reinterpret_cast<const v4f*>(src + 20);
    }
  }
  float z[8], u[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) z[e] = z0[e], z[e + 4] = z1[e], u[e] = u0[e], u[e + 4] = u1[e];
  finish8<KIND, GATED>(g, z, u, load_bias8<GATED>(g, n), load_res8(g, m, n, vec_ok(g)), m, n, vec_ok(g));
}

// kTiles
using T256x320 = GCfg<8, 5, 2, 4, 2>;   // not for SwiGLU (odd fragment count)
using T256x256 = GCfg<8, 4, 2, 4, 2>;
using T128x256 = GCfg<4, 4, 2, 4, 3>;
using T128x128 = GCfg<4, 2, 2, 4, 4>;
using T64x128 = GCfg<2, 2, 2, 4, 5>;
using T32x128 = GCfg<2, 2, 1, 4, 6>;
template <typename C>
constexpr bool is_tile(int i) {
  return kTiles[i].bm == C::BM && kTiles[i].bn == C::BN && kTiles[i].threads == 64 * C::NW && (!kTiles[i].gated || C::TJ % 2 == 0);
}
static_assert(is_tile<T256x320>(0) && is_tile<T256x256>(1) && is_tile<T128x256>(2) && is_tile<T128x128>(3) &&
              is_tile<T64x128>(4) && is_tile<T32x128>(5), "kTiles");

template <typename C, bool GATED>
void launch_kind(const GemmPlanArgs& p, hipStream_t st) {
  const unsigned grid = (unsigned)(p.tiles_m * p.tiles_n * p.splits);
  const int kind = act_kind(p.g.act);
  if (GATED || (kind == ACT_KIND_SIGMOID && p.splits == 1))
    gemm_bf16_kernel<C, ACT_KIND_SIGMOID, GATED><<<grid, 64 * C::NW, 0, st>>>(p);
  else if constexpr (!GATED) {
    if (kind == ACT_KIND_ERF && p.splits == 1) gemm_bf16_kernel<C, ACT_KIND_ERF, false><<<grid, 64 * C::NW, 0, st>>>(p);
    else gemm_bf16_kernel<C, ACT_KIND_PLAIN, false><<<grid, 64 * C::NW, 0, st>>>(p);   // a split stores plain sums
  }
}

template <typename C>
void launch_tile(const GemmPlanArgs& p, hipStream_t st) {
  if (p.g.act != W4A4_ACT_SWIGLU) launch_kind<C, false>(p, st);
  else if constexpr (C::TJ % 2 == 0) launch_kind<C, true>(p, st);
}

}  // namespace

size_t gemm_bf16_workspace(int64_t M, int64_t N, int64_t K, int act) {
  const GemmPlan pl = plan_gemm(M, N, K, act, true);
  return !pl.rows && pl.splits > 1 ? (size_t)pl.splits * M * pl.pn * 4 : 0;
}

hipError_t launch_gemm_bf16(const DenseArgs& g, void* workspace, hipStream_t st) {
  // a workspace that no split needs is null here: the plan is the same then
  const GemmPlan pl = plan_gemm(g.M, g.N, g.K, g.act, workspace != nullptr);
  if (pl.rows) {
    const unsigned grid = (unsigned)((g.N + 15) / 16);
    const int kind = act_kind(g.act), threads = 64 * kRowsWaves;
    if (g.act == W4A4_ACT_SWIGLU) gemm_bf16_rows_kernel<ACT_KIND_SIGMOID, true><<<grid, threads, 0, st>>>(g);
    else if (kind == ACT_KIND_SIGMOID) gemm_bf16_rows_kernel<ACT_KIND_SIGMOID, false><<<grid, threads, 0, st>>>(g);
    else if (kind == ACT_KIND_ERF) gemm_bf16_rows_kernel<ACT_KIND_ERF, false><<<grid, threads, 0, st>>>(g);
    else gemm_bf16_rows_kernel<ACT_KIND_PLAIN, false><<<grid, threads, 0, st>>>(g);
    return hipGetLastError();
  }
  GemmPlanArgs p{g, pl.tiles_m, pl.tiles_n, pl.splits, (g.K + 63) / 64, (float*)workspace, pl.pn};
  switch (pl.tile) {
    case 0: launch_tile<T256x320>(p, st); break;
    case 1: launch_tile<T256x256>(p, st); break;
    case 2: launch_tile<T128x256>(p, st); break;
    case 3: launch_tile<T128x128>(p, st); break;
    case 4: launch_tile<T64x128>(p, st); break;
    default: launch_tile<T32x128>(p, st); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.splits == 1) return e;
  const int64_t items = (int64_t)g.M * ((g.N + 7) / 8);
  const unsigned grid = (unsigned)((items + 63) / 64);
  const int kind = act_kind(g.act);
  if (g.act == W4A4_ACT_SWIGLU) gemm_bf16_join_kernel<ACT_KIND_SIGMOID, true><<<grid, 64, 0, st>>>(p);
  else if (kind == ACT_KIND_SIGMOID) gemm_bf16_join_kernel<ACT_KIND_SIGMOID, false><<<grid, 64, 0, st>>>(p);
  else if (kind == ACT_KIND_ERF) gemm_bf16_join_kernel<ACT_KIND_ERF, false><<<grid, 64, 0, st>>>(p);
  else gemm_bf16_join_kernel<ACT_KIND_PLAIN, false><<<grid, 64, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace w4a4
