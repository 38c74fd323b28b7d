// Group normalisation with an activation on channels-last features.
//
// Memory bound: the features are read once for the statistics and once for
// the output; the second read comes from the 256 MB last-level cache where
// the features fit it.  1597440 x 96 bf16 (306 MB): 50 us for the moments, 6
// to join them, 109-119 for the output, against 120 us for one read and one
// write at the rate of a device copy (5.1 TB/s).  Small inputs (1560 x 384:
// 13.7 us) are two launches of dependent memory latencies.
//
// Statistics.  A thread keeps V adjacent channels and walks down the
// positions of its slab, so loads are whole lines and a lane's groups are
// fixed.  It sums d and d^2 of differences d = x - x0 to the channel's first
// value in the slab (exact to an ulp, so a large mean costs no accuracy), in
// runs of kRun positions joined in fp64 (channel_moments).  Sums become (count, mean, M2) and are joined by
//   mean = mean_a + (mean_b - mean_a) n_b / n,
//   M2 = M2_a + M2_b + (mean_b - mean_a)^2 n_a n_b / n,
// over the threads of a channel, over the channels of a group, and over the
// slabs of a sample, always in the same order: no atomics, the same bits
// every time.
//
// With a workspace the positions of a sample are cut into slabs that fill the
// card; one kernel takes the moments of each (slab, group), one writes the
// output.  The output kernel joins the slabs itself when they are few;
// otherwise a third kernel does.  Without a workspace, when a sample is small
// or a group too wide, one workgroup does a run of groups of a sample by
// itself.
#include "activation.h"
#include "dense.h"
#include "device_common.h"

namespace w4a4 {

namespace {

constexpr int kThreads = 256, kCUs = 256;
constexpr int kRun = 64;           // positions a thread sums in fp32 before it joins
constexpr int kMaxSlabs = 2048;
constexpr int kJoinInline = 64;    // slabs the output kernel joins by itself
constexpr int64_t kSlabElems = 8192;

struct Moments {
  float n, mean, m2;
};

__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  const float w = n > 0.f ? b.n * __builtin_amdgcn_rcpf(n) : 0.f;
  const float d = b.mean - a.mean;
  return {n, a.mean + d * w, a.m2 + b.m2 + d * d * (a.n * w)};
}

// Joins over the L = 2^k <= 64 adjacent lanes that share a result.
__device__ __forceinline__ Moments join_lanes(Moments m, int L) {
  for (int o = 1; o < L; o <<= 1) {
    const Moments x = {__shfl_xor(m.n, o), __shfl_xor(m.mean, o), __shfl_xor(m.m2, o)};
    m = (threadIdx.x & o) ? join(x, m) : join(m, x);
  }
  return m;
}

// Moments first, first + step, ... of `slabs`, `stride` apart; eight loads in flight.
__device__ __forceinline__ Moments join_slabs(const Moments* ws, int slabs, int stride, int first, int step) {
  Moments m = {0.f, 0.f, 0.f};
  for (int i = first; i < slabs; i += 8 * step) {
    Moments x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = ws[(int64_t)min(i + k * step, slabs - 1) * stride];
      if (i + k * step >= slabs) x[k].n = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (x[k].n > 0.f) m = join(m, x[k]);
  }
  return m;
}

// Lanes for each of `items` results of a workgroup.
__device__ __forceinline__ int lanes_per(int items) {
  int L = 1;
  while (L < 64 && items * L * 2 <= kThreads) L *= 2;
  return L;
}

__device__ __forceinline__ float2 mean_rstd(const Moments& m, float eps) {
  return make_float2(m.mean, 1.f / sqrtf(m.m2 / m.n + eps));
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// Output that nothing here reads again: a non-temporal store leaves the
// features in the caches.
template <typename T, int V>
__device__ __forceinline__ void store_once(const Vec<T, V>& r, T* to) {
  if constexpr (sizeof(r) == 16) __builtin_nontemporal_store(__builtin_bit_cast(v4i, r), reinterpret_cast<v4i*>(to));
  else *reinterpret_cast<Vec<T, V>*>(to) = r;
}

__device__ __forceinline__ float to_f32(uint16_t b) { return bf16_bits_to_f32(b); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ void from_f32(uint16_t& o, float f) { o = __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ void from_f32(float& o, float f) { o = f; }

// SiLU on the way to bf16 takes the hardware exp2 (a few parts in 10^6,
// against 2^-8 of the output).
template <typename T, int KIND>
__device__ __forceinline__ float activate_for(float z, int act) {
  if constexpr (sizeof(T) == 2 && KIND == ACT_KIND_SIGMOID) {
    if (act == W4A4_ACT_SILU) return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
  }
  return activate_kind<KIND>(z, act);
}

// How a sample is cut.  A workgroup covers `gpb` whole groups, `cols` threads
// across their channels and kThreads / cols positions deep.
struct Split {
  int gpb, cols, blocks;
  int slabs;
  int64_t len;     // positions of a slab
};

// Moments of the channels [c, c + V) of each thread over positions [s0, s1),
// joined over the threads of a channel into mom[0 .. cols * V).
//
// LONG: a walk may have more than kRun positions and is summed in runs, fp32
// inside a run, the runs joined in fp64, and the next run's differences taken
// to the mean so far.  One fp32 sum over 10^5 positions is off by up to a few
// parts in 10^3 where its terms are alike (each is rounded the same way), and
// a first value far from the rest would cost accuracy all along the walk.
// (Inside one run it costs at most 64 u of its own square per position, 1e-4
// of the variance it makes itself; unequal terms average far below that.)
// Without LONG the kernels save its registers (0.1-0.2 us of 8-14).
template <typename T, int V, bool LONG>
__device__ __forceinline__ void channel_moments(const NormArgs& g, const T* x, int64_t s0, int64_t s1, int c, int cend,
                                                int cols, Moments* mom) {
  const int rows = kThreads / cols, col = threadIdx.x % cols, depth = threadIdx.x / cols;
  float sh[V], s[V], q[V];
  double mean[V], m2[V];   // of the runs before, `done` positions
  int64_t done = 0;
  int cnt = 0;             // positions in s and q
#pragma unroll
  for (int e = 0; e < V; ++e) sh[e] = s[e] = q[e] = 0.f;
  auto fold = [&]() {
    const double nb = cnt, inv = 1.0 / nb, w = nb / (double)(done + cnt);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const double ms = s[e] * inv, mb = sh[e] + ms, m2b = fmax(q[e] - s[e] * ms, 0.0);
      const double d = done > 0 ? mb - mean[e] : 0.0;
      m2[e] = done > 0 ? m2[e] + m2b + d * d * (done * w) : m2b;
      mean[e] = done > 0 ? mean[e] + d * w : mb;
      sh[e] = (float)mean[e];
      s[e] = q[e] = 0.f;
    }
    done += cnt;
  };
  if (c < cend && depth < rows && s0 + depth < s1) {
    const T* p = x + (s0 + depth) * g.x_ss + c;
    const int64_t step = (int64_t)rows * g.x_ss;
    const Vec<T, V> f = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
    for (int e = 0; e < V; ++e) sh[e] = to_f32(f.v[e]);
    auto add = [&](const Vec<T, V>& u) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = to_f32(u.v[e]) - sh[e];
        s[e] += d;
        q[e] = __builtin_fmaf(d, d, q[e]);
      }
    };
    auto walk = [&](int k) {
      for (; k >= 4; k -= 4, p += 4 * step) {   // four loads in flight
        Vec<T, V> u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const Vec<T, V>*>(p + i * step);
#pragma unroll
        for (int i = 0; i < 4; ++i) add(u[i]);
      }
      for (; k > 0; --k, p += step) add(*reinterpret_cast<const Vec<T, V>*>(p));
    };
    if constexpr (LONG) {
      for (int64_t left = (s1 - s0 - depth + rows - 1) / rows; left > 0;) {
        cnt = (int)min(left, (int64_t)kRun);
        walk(cnt);
        fold();
        left -= cnt;
      }
    } else {
      cnt = (int)((uint32_t)(s1 - s0 - depth + rows - 1) / (uint32_t)rows);
      walk(cnt);
    }
  }
  const int width = cols * V;
  if (LONG && depth < rows && done > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) mom[depth * width + col * V + e] = {(float)done, (float)mean[e], (float)m2[e]};
  } else if (depth < rows) {
    const float n = (float)cnt, inv = cnt > 0 ? 1.f / n : 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float ms = s[e] * inv;
      mom[depth * width + col * V + e] = {n, sh[e] + ms, fmaxf(q[e] - s[e] * ms, 0.f)};
    }
  }
  __syncthreads();
  const int L = lanes_per(width);
  for (int ch = threadIdx.x / L; ch < width; ch += kThreads / L) {
    Moments m = {0.f, 0.f, 0.f};
    for (int r = threadIdx.x % L; r < rows; r += L) m = join(m, mom[r * width + ch]);
    m = join_lanes(m, L);
    if (threadIdx.x % L == 0) mom[ch] = m;   // the column's other rows have been read by this wave
  }
  __syncthreads();
}

// The output of a thread's channels over positions [s0, s1): kBatch rows are
// loaded while the kBatch before them are worked on; the first ones when the
// object is made, ahead of the statistics.
template <typename T, int V, int KIND>
struct Applier {
  static constexpr int kBatch = 8;
  const T* p;
  T* o;
  int64_t xs, ys;
  int left;
  Vec<T, V> u[kBatch];
  float w[V], b[V];

  __device__ __forceinline__ Applier(const NormArgs& g, int64_t n, int64_t s0, int64_t s1, int c, int cols, bool on) {
    const int rows = kThreads / cols, depth = threadIdx.x / cols;
    // a slab's positions fit 32 bits (the entry point refuses more)
    left = on && depth < rows && s0 + depth < s1 ? (int)((uint32_t)(s1 - s0 - depth + rows - 1) / (uint32_t)rows) : 0;
    xs = (int64_t)rows * g.x_ss;
    ys = (int64_t)rows * g.y_ss;
    p = (const T*)g.x + n * g.x_sn + (s0 + depth) * g.x_ss + c;
    o = (T*)g.y + n * g.y_sn + (s0 + depth) * g.y_ss + c;
    load(u);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[e] = g.weight && on ? g.weight[c + e] : 1.f;
      b[e] = g.bias && on ? g.bias[c + e] : 0.f;
    }
  }
  __device__ __forceinline__ void load(Vec<T, V> (&to)[kBatch]) {   // the kBatch rows at p
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < left) to[i] = *reinterpret_cast<const Vec<T, V>*>(p + i * xs);
  }
  __device__ __forceinline__ void run(const NormArgs& g, const float (&mu)[V], const float (&rs)[V]) {
    if (left <= 0) return;
    float k[V];
#pragma unroll
    for (int e = 0; e < V; ++e) k[e] = rs[e] * w[e];
    while (true) {
      Vec<T, V> next[kBatch];
      const int had = left;
      left -= kBatch;
      p += kBatch * xs;
      load(next);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i < had) {
          Vec<T, V> r;
#pragma unroll
          for (int e = 0; e < V; ++e)
            from_f32(r.v[e], activate_for<T, KIND>(__builtin_fmaf(to_f32(u[i].v[e]) - mu[e], k[e], b[e]), g.act));
          store_once<T, V>(r, o + i * ys);
        }
      o += kBatch * ys;
      if (left <= 0) return;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) u[i] = next[i];
    }
  }
};

// Moments of (sample, slab, group).
template <typename T, int V, bool LONG>
__global__ void __launch_bounds__(kThreads) norm_moments_kernel(NormArgs g, Split sp, Moments* ws) {
  __shared__ Moments mom[kThreads * V];
  const int cg = g.C / g.groups;
  const int g0 = blockIdx.y * sp.gpb, ng = min(sp.gpb, g.groups - g0);
  const int64_t n = blockIdx.z;
  const int64_t s0 = blockIdx.x * sp.len, s1 = min(g.S, s0 + sp.len);
  channel_moments<T, V, LONG>(g, (const T*)g.x + n * g.x_sn, s0, s1, g0 * cg + (threadIdx.x % sp.cols) * V, (g0 + ng) * cg,
                        sp.cols, mom);
  const int L = lanes_per(ng);
  for (int i = threadIdx.x / L; i < ng; i += kThreads / L) {
    Moments m = {0.f, 0.f, 0.f};
    for (int c = threadIdx.x % L; c < cg; c += L) m = join(m, mom[i * cg + c]);
    m = join_lanes(m, L);
    if (threadIdx.x % L == 0) ws[(n * sp.slabs + blockIdx.x) * g.groups + g0 + i] = m;
  }
}

// (mean, 1 / deviation) of a (sample, group) from its slabs.
__global__ void __launch_bounds__(kThreads) norm_join_kernel(NormArgs g, int slabs, const Moments* ws, float2* stat) {
  __shared__ Moments part[kThreads / 64];
  const int64_t n = blockIdx.x / g.groups;
  const int grp = blockIdx.x % g.groups;
  Moments m = join_lanes(join_slabs(ws + n * slabs * g.groups + grp, slabs, g.groups, threadIdx.x, kThreads), 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 64; ++w) m = join(m, part[w]);
  stat[blockIdx.x] = mean_rstd(m, g.eps);
}

// The output of a slab; stat null: the slabs' moments are joined here.
template <typename T, int V, int KIND>
__global__ void __launch_bounds__(kThreads) norm_apply_kernel(NormArgs g, Split sp, const Moments* ws, const float2* stat) {
  __shared__ float2 st[kThreads * V];
  const int cg = g.C / g.groups;
  const int g0 = blockIdx.y * sp.gpb, ng = min(sp.gpb, g.groups - g0);
  const int64_t n = blockIdx.z;
  const int cl = (threadIdx.x % sp.cols) * V;   // channel within the block
  // slabs last to first: what the moments kernel read last is still cached
  const int64_t s0 = (sp.slabs - 1 - (int)blockIdx.x) * sp.len, s1 = min(g.S, s0 + sp.len);
  Applier<T, V, KIND> out(g, n, s0, s1, g0 * cg + cl, sp.cols, cl < ng * cg);
  if (stat) {
    for (int i = threadIdx.x; i < ng; i += kThreads) st[i] = stat[n * g.groups + g0 + i];
  } else {
    const int L = lanes_per(ng);
    for (int i = threadIdx.x / L; i < ng; i += kThreads / L) {
      Moments m = join_slabs(ws + n * sp.slabs * g.groups + g0 + i, sp.slabs, g.groups, threadIdx.x % L, L);
      m = join_lanes(m, L);
      if (threadIdx.x % L == 0) st[i] = mean_rstd(m, g.eps);
    }
  }
  __syncthreads();
  if (cl >= ng * cg) return;
  float mu[V], rs[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float2 v = st[(cl + e) / cg];
    mu[e] = v.x;
    rs[e] = v.y;
  }
  out.run(g, mu, rs);
}

// A run of whole groups of one sample, statistics and output.  A group wider
// than the workgroup (ng == 1 then) is taken in chunks of its channels.
template <typename T, int V, int KIND, bool LONG>
__global__ void __launch_bounds__(kThreads) norm_whole_kernel(NormArgs g, int gpb, int cols) {
  __shared__ Moments mom[kThreads * V];
  __shared__ float2 st[kThreads * V];
  const int cg = g.C / g.groups;
  const int64_t n = blockIdx.y;
  const int g0 = blockIdx.x * gpb, ng = min(gpb, g.groups - g0);
  const int c0 = g0 * cg, cend = c0 + ng * cg, width = cols * V;
  const T* x = (const T*)g.x + n * g.x_sn;
  const int L = lanes_per(ng);
  Moments tot = {0.f, 0.f, 0.f};
  for (int cc = c0; cc < cend; cc += width) {
    channel_moments<T, V, LONG>(g, x, 0, g.S, cc + (threadIdx.x % cols) * V, cend, cols, mom);
    for (int i = threadIdx.x / L; i < ng; i += kThreads / L) {
      Moments m = ng == 1 ? tot : Moments{0.f, 0.f, 0.f};
      const int cnt = ng == 1 ? min(width, cend - cc) : cg;
      for (int c = threadIdx.x % L; c < cnt; c += L) m = join(m, mom[i * cg + c]);
      tot = m;
      if (cc + width >= cend) {
        m = join_lanes(m, L);
        if (threadIdx.x % L == 0) st[i] = mean_rstd(m, g.eps);
      }
    }
    __syncthreads();
  }
  for (int cc = c0; cc < cend; cc += width) {
    const int c = cc + (threadIdx.x % cols) * V;
    if (c >= cend) break;
    float mu[V], rs[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 v = st[(c + e - c0) / cg];
      mu[e] = v.x;
      rs[e] = v.y;
    }
    Applier<T, V, KIND>(g, n, 0, g.S, c, cols, true).run(g, mu, rs);
  }
}

// Slabs of a sample: about eight workgroups a CU over all samples, at least
// kSlabElems elements each.
int slabs_for(int64_t N, int64_t S, int64_t C, int64_t groups) {
  const int64_t elems = S * C;
  // Groups that fill a workgroup by themselves are cut when there are too few
  // of them for the card and they are long.  us, cut / whole, bf16: 1 x 64 x
  // 512 11.8 / 14.1, 2 x 4096 x 512 14.9 / 478, 128 x 64 x 1024 20.8 / 22.5,
  // but 1 x 32 x 512 11.9 / 10.4 and 250 x 64 x 1024 34.6 / 25.0.
  if (C / groups > kThreads && (N * groups > kCUs / 2 || elems < 4 * kSlabElems)) return 1;
  int64_t want = kMaxSlabs / N;
  if (want > elems / kSlabElems) want = elems / kSlabElems;
  if (want > S) want = S;
  // a third launch and more slabs than that gain less than they cost
  if (want > kJoinInline && want < 4 * kJoinInline) want = kJoinInline;
  return want < 2 ? 1 : (int)want;
}

// Whether a thread of `cols` across the channels meets more than kRun of S positions.
bool walk_is_long(int64_t S, int cols) { return S > (int64_t)kRun * (kThreads / cols); }

size_t stat_bytes(int64_t N, int64_t groups) { return (size_t)(N * groups * 8 + 255) / 256 * 256; }

template <typename T, int V, int KIND>
hipError_t run_kind(const NormArgs& g, void* workspace, hipStream_t st) {
  const int cg = g.C / g.groups;
  const int slabs = slabs_for(g.N, g.S, g.C, g.groups);
  // whole groups a workgroup can cover; vectors may straddle groups only
  // where the workgroup covers all of them
  int gpb = cg >= kThreads * V ? 1 : kThreads * V / cg;
  if (gpb > g.groups) gpb = g.groups;
  // A group of more channels than a workgroup covers (2048 in bf16, 1024 in
  // fp32, fewer where alignment narrows V) is not cut.
  if (!workspace || slabs == 1 || cg > kThreads * V) {
    // small: few channels a workgroup, so that more of them share the sample
    if (cg % V == 0)
      while (gpb > 1 && gpb * cg > 16 * V) gpb = (gpb + 1) / 2;
    const int w = (gpb * cg + V - 1) / V, cols = w < kThreads ? w : kThreads;
    // a grid's second dimension ends at 65535, and a layer norm has a sample per token
    NormArgs part = g;
    for (int64_t left = g.N; left > 0; left -= part.N) {
      part.N = left < 65535 ? left : 65535;
      const dim3 grid((g.groups + gpb - 1) / gpb, (unsigned)part.N);
      if (walk_is_long(g.S, cols)) norm_whole_kernel<T, V, KIND, true><<<grid, kThreads, 0, st>>>(part, gpb, cols);
      else norm_whole_kernel<T, V, KIND, false><<<grid, kThreads, 0, st>>>(part, gpb, cols);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      part.x = (const T*)part.x + part.N * g.x_sn;
      part.y = (T*)part.y + part.N * g.y_sn;
    }
    return hipSuccess;
  }
  Split sp;
  sp.gpb = gpb;
  sp.cols = (gpb * cg + V - 1) / V;
  sp.blocks = (g.groups + gpb - 1) / gpb;
  sp.len = (g.S + slabs - 1) / slabs;
  sp.slabs = (int)((g.S + sp.len - 1) / sp.len);
  float2* stat = (float2*)workspace;
  Moments* mom = (Moments*)((char*)workspace + stat_bytes(g.N, g.groups));
  const dim3 grid(sp.slabs, sp.blocks, (unsigned)g.N);
  if (walk_is_long(sp.len, sp.cols)) norm_moments_kernel<T, V, true><<<grid, kThreads, 0, st>>>(g, sp, mom);
  else norm_moments_kernel<T, V, false><<<grid, kThreads, 0, st>>>(g, sp, mom);
  const bool inline_join = sp.slabs <= kJoinInline;
  if (!inline_join) norm_join_kernel<<<(unsigned)(g.N * g.groups), kThreads, 0, st>>>(g, sp.slabs, mom, stat);
  norm_apply_kernel<T, V, KIND><<<grid, kThreads, 0, st>>>(g, sp, mom, inline_join ? nullptr : stat);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t run(const NormArgs& g, void* workspace, hipStream_t st) {
  switch (act_kind(g.act)) {
    case ACT_KIND_PLAIN: return run_kind<T, V, ACT_KIND_PLAIN>(g, workspace, st);
    case ACT_KIND_ERF: return run_kind<T, V, ACT_KIND_ERF>(g, workspace, st);
    default: return run_kind<T, V, ACT_KIND_SIGMOID>(g, workspace, st);
  }
}

}  // namespace

size_t group_norm_workspace(int64_t N, int64_t S, int64_t C, int64_t groups) {
  const int slabs = slabs_for(N, S, C, groups);
  return slabs == 1 ? 0 : stat_bytes(N, groups) + (size_t)N * slabs * groups * sizeof(Moments);
}

hipError_t launch_group_norm(const NormArgs& g, void* workspace, hipStream_t st) {
  // Widest vector that the channel count, the strides and the pointers allow.
  const int esz = g.bf16 ? 2 : 4;
  auto fits = [&](int V) {
    const int64_t b = V * esz;
    if (g.C % V || g.x_ss % V || g.y_ss % V || (g.N > 1 && (g.x_sn % V || g.y_sn % V))) return false;
    if ((uintptr_t)g.x % b || (uintptr_t)g.y % b) return false;
    return (g.C / g.groups) % V == 0 || g.C <= kThreads * V;   // straddling vectors: all groups in one workgroup
  };
  if (g.bf16) {
    if (fits(8)) return run<uint16_t, 8>(g, workspace, st);
    if (fits(4)) return run<uint16_t, 4>(g, workspace, st);
    if (fits(2)) return run<uint16_t, 2>(g, workspace, st);
    return run<uint16_t, 1>(g, workspace, st);
  }
  if (fits(4)) return run<float, 4>(g, workspace, st);
  if (fits(2)) return run<float, 2>(g, workspace, st);
  return run<float, 1>(g, workspace, st);
}

}  // namespace w4a4
