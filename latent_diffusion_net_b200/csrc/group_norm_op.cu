// Group norm with an activation on channels-last tensors, and its gradients.
//
// Per image and group, over rows x (C/G) values: xh = (x - mean) * rstd,
// z = gamma * xh + beta, y = act(z). With dz = dy * act'(z) and u = gamma * dz:
//   dbeta = sum dz, dgamma = sum dz * xh (over images and rows),
//   dx = rstd * (u - mean(u) - xh * mean(u * xh)).
//
// Bound by memory: forward reads x and writes y, backward reads x and dy and
// writes dx. Groups are independent, so an image's channels are cut into slices of
// whole groups, and a thread block cluster takes one slice of one image:
//   gn_cluster_fwd / _bwd_kernel  where the slice (of x, or of x and dy) fits into the
//       shared memory of up to eight CTAs: read once, summed, the sums joined
//       through distributed shared memory, normalised from shared memory
//   otherwise two kernels: the first sums over a share of an image's rows per CTA,
//       the second joins the shares and walks the same rows from their end, where L2 may
//       still hold what the first one read last
// Sums are joined in a fixed order, so results repeat bit for bit.
// Measured (BF16, SiLU): 768 x 768 x 128 forward 92 us, 302 MB of x and y at 3.3 TB/s (x is
// read twice; the second kernel takes 58 us for 302 MB with cold caches: a CTA loads eight rows
// a thread, waits and stores, and has nothing under way meanwhile); 4 x 9216 rows x 320 forward
// 24 us (one wave of 128 CTAs: all load, join, then store), gradients 31 us; 144 rows x 1280
// forward 8.2 us, which is launch, cluster barriers and two latencies.
//
// A thread owns one 16-byte vector of channels for all its rows (channel terms
// stay in registers, a warp reads whole sectors whatever C/G is). Statistics are FP32
// pairs (mean, sum of squared deviations from it) at every level: a thread's rows
// about their own mean, the threads of a channel, the channels of a group, the shares.
// Every term of the squares is positive and part of the result, so neither a mean far
// from zero nor an outlier, wherever it stands, costs precision (squares about the
// first value of a group lost 2^-24 (distance / deviation)^2 a value: with an outlier in
// that place y was off by up to 1e-3).
#include <string.h>

#include <algorithm>
#include <numeric>

#include "op_common.cuh"
#include "profile.h"

namespace sdo {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxChannels = 8192;  // per-channel sums of a CTA: 64 KB of shared memory
constexpr int kSms = 148;
constexpr int kMaxChunks = 160;  // shares of one image: kSms up to a multiple of 32
constexpr int kMaxCluster = 8;
constexpr size_t kClusterSmem = 220 * 1024;

struct GnArgs {
  const void *x, *gamma, *beta, *dy;
  void* out;  // y or dx
  float* stats;
  float *dgamma, *dbeta;
  float *pg, *pc;  // shares: per group [batch][G][chunks][2], per channel [batch][chunks][2][C]
  int64_t rows, chunk_rows, ldx, ldy;
  int32_t batch, C, G, cpg, act, chunks;
  int32_t slices, width;  // cluster kernels: slices of an image, channels of one
  float eps;
  int* err;  // cleared by the first kernel of a call (none of them waits)
};

struct Plan {
  bool cluster[2];  // forward, backward
  int ctas[2], width[2];
  int64_t cta_rows[2];
  int chunks[2];
  int64_t chunk_rows[2];
  size_t pg_floats, pc_floats;
};

// Shared memory of a cluster kernel: `tensors` vectors per thread and row pass, the
// row threads' sums, per-channel sums, per-group results (two buffers).
size_t cluster_smem(int width, int groups, int vec, int64_t cta_rows, int tensors) {
  const int cols = width / vec, rows_t = kThreads / cols;
  const int64_t iters = (cta_rows + rows_t - 1) / rows_t;
  if (iters > 64) return SIZE_MAX;
  return (size_t)iters * kThreads * 16 * tensors + (size_t)2 * vec * kThreads * 4 + (size_t)2 * width * 4 +
         (size_t)4 * groups * 4;
}

Plan make_plan(const sd_group_norm_cfg& c) {
  Plan p;
  memset(&p, 0, sizeof(p));
  const int vec = c.dtype == SD_DTYPE_F32 ? 4 : 8, size = 16 / vec;
  const int cpg = c.channels / c.groups;
  const bool wide = c.channels % vec == 0 && c.ld_x % vec == 0 && c.ld_y % vec == 0;
  const int unit = std::lcm(cpg, vec);  // narrowest slice of whole groups and whole vectors
  for (int back = 0; back < 2 && wide && c.channels % unit == 0; ++back) {
    const int n = c.channels / unit;
    double best = 0;  // in passes, see below
    for (int k = 1; k <= n; ++k) {
      if (n % k) continue;
      const int width = unit * k, cols = width / vec;
      // slices of 64 bytes and more: narrower ones waste parts of sectors
      if (cols > kThreads || (width * size < 64 && k < n)) continue;
      const int rows_t = kThreads / cols;
      for (int ctas = 1; ctas <= kMaxCluster; ctas *= 2) {
        const int64_t rows = (c.rows + ctas - 1) / ctas;
        if (ctas > 1 && rows < rows_t) break;
        if (cluster_smem(width, width / cpg, vec, rows, 1 + back) > kClusterSmem) continue;
        // Measured: a wave of clusters takes about 7 us and 0.5 us (0.75 us for gradients)
        // for each pass of its threads over their rows, more where a row of the slice
        // is few sectors, so that the parts outside it count (80 bytes: a third). One CTA
        // fits on an SM, and of larger clusters fewer fit on the GPU.
        const int64_t total = (int64_t)c.batch * (n / k) * ctas, room = ctas <= 2 ? 148 : ctas == 4 ? 132 : 120;
        const double part = 1 + 24.0 / (width * size);
        const double cost = (double)((total + room - 1) / room) * ((rows + rows_t - 1) / rows_t * part + 12);
        if (!p.cluster[back] || cost < best) {
          best = cost;
          p.cluster[back] = true;
          p.ctas[back] = ctas;
          p.width[back] = width;
          p.cta_rows[back] = rows;
        }
      }
    }
    // The two kernels, measured: 14 us and 0.5 us per MB of x, gradients 10.5 us and
    // 0.93 us per MB. (16 x 256 rows x 1280: 14 us in clusters, 21 in two kernels; 2 x 16384 x
    // 320: 35 and 25.)
    if (p.cluster[back]) {
      const double mb = 1e-6 * c.batch * c.rows * c.channels * size;
      if (best * (back ? 0.7 : 0.5) > (back ? 10.5 + 0.93 * mb : 14 + 0.5 * mb)) p.cluster[back] = false;
    }
  }
  for (int back = 0; back < 2; ++back) {
    // one wave of CTAs, four rows or more for each thread. Two CTAs per SM have too few
    // registers for the loads under way (9216 x 320 x 4 forward: 31 us, one CTA 26), and a
    // second wave pays the joins again (gradients: 41 us, 31 in one).
    const int cols = std::max(1, std::min(kThreads, c.channels / (wide ? vec : 1)));
    const int64_t least = 4 * (int64_t)(kThreads / cols);
    int64_t n = kSms / c.batch;
    n = std::max<int64_t>(std::min<int64_t>(n, (c.rows + least - 1) / least), 1);
    p.chunk_rows[back] = (c.rows + n - 1) / n;
    p.chunks[back] = (int)((c.rows + p.chunk_rows[back] - 1) / p.chunk_rows[back]);
    if (!p.cluster[back])
      p.pg_floats = std::max(p.pg_floats, (size_t)c.batch * p.chunks[back] * c.groups * 2);
  }
  p.pc_floats = (size_t)c.batch * (p.cluster[1] ? 1 : p.chunks[1]) * c.channels * 2;
  return p;
}

// V channels at p (16-byte aligned when V > 1).
template <typename T, int V>
struct Raw {
  uint4 v;
};
template <typename T>
struct Raw<T, 1> {
  T v;
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  Raw<T, V> r;
  if constexpr (V == 1)
    r.v = *p;
  else
    r.v = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void to_float(const Raw<T, V>& r, float (&f)[V]) {
  if constexpr (V == 1)
    f[0] = Elem<T>::to_f(r.v);
  else
    unpack_vec<T, V>(r.v, f);
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&f)[V]) {
  if constexpr (V == 1)
    *p = Elem<T>::from_f(f[0]);
  else
    __stcs(reinterpret_cast<uint4*>(p), pack_vec<T, V>(f));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Pairwise arithmetic on V channels (packed FP32 for even V).
template <int V>
__device__ __forceinline__ void v_add(const float (&x)[V], const float (&y)[V], float (&o)[V]) {
  if constexpr (V % 2) {
    o[0] = x[0] + y[0];
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2) add2(x[j], x[j + 1], y[j], y[j + 1], o[j], o[j + 1]);
  }
}
template <int V>
__device__ __forceinline__ void v_mul(const float (&x)[V], const float (&y)[V], float (&o)[V]) {
  if constexpr (V % 2) {
    o[0] = x[0] * y[0];
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2) mul2(x[j], x[j + 1], y[j], y[j + 1], o[j], o[j + 1]);
  }
}
template <int V>
__device__ __forceinline__ void v_fma(const float (&x)[V], const float (&y)[V], const float (&z)[V], float (&o)[V]) {
  if constexpr (V % 2) {
    o[0] = fmaf(x[0], y[0], z[0]);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2) fma2v(x[j], x[j + 1], y[j], y[j + 1], z[j], z[j + 1], o[j], o[j + 1]);
  }
}

// Per-channel terms of the V channels a thread owns: z = (x + nm) * sc + be, where
// nm = -mean and sc = rstd * gamma.
template <int V>
struct Cols {
  float nm[V], sc[V], be[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_affine(const GnArgs& a, int c, Cols<V>& t) {
  const T *gamma = static_cast<const T*>(a.gamma), *beta = static_cast<const T*>(a.beta);
#pragma unroll
  for (int j = 0; j < V; ++j) t.sc[j] = 1.f, t.be[j] = 0.f;
  if (gamma) to_float<T, V>(load_raw<T, V>(gamma + c), t.sc);
  if (beta) to_float<T, V>(load_raw<T, V>(beta + c), t.be);
}
// The first group of a thread's V channels and, where groups are narrower than the
// vector, each channel's own: one division per thread.
struct Groups {
  int g, left, cpg;  // group of the next channel, channels of it left
  __device__ __forceinline__ Groups(int c, int per) : g(c / per), left(per - c % per), cpg(per) {}
  __device__ __forceinline__ int next() {
    const int r = g;
    if (--left == 0) {
      ++g;
      left = cpg;
    }
    return r;
  }
};
// Takes mean and rstd pairs of the channels' groups into
// the terms; rs receives rstd.
template <int V>
__device__ __forceinline__ void add_stats(const float* st, int c, int cpg, Cols<V>& t, float (&rs)[V]) {
  Groups gr(c, cpg);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int g = gr.next();
    t.nm[j] = -st[2 * g];
    rs[j] = st[2 * g + 1];
    t.sc[j] *= rs[j];
  }
}
template <int V>
__device__ __forceinline__ void normalise(const Cols<V>& t, float (&f)[V], int act) {
  v_add<V>(f, t.nm, f);
  v_fma<V>(f, t.sc, t.be, f);
  act_vec<V>(f, act);
}
// f = x -> x - mean, d = dy -> dz
template <int V>
__device__ __forceinline__ void grad_terms(const Cols<V>& t, float (&f)[V], float (&d)[V], int act) {
  v_add<V>(f, t.nm, f);
  if (act != SD_ACT_NONE) {
    float z[V], a[V];
    v_fma<V>(f, t.sc, t.be, z);
    act_grad_vec<V>(z, d, a, act);
  }
}
// dx = rstd (gamma dz - m1 - xh m2) = sc dz + b2 (x - mean) + b1
template <int V>
struct GradCols {
  float b1[V], b2[V];
};
template <int V>
__device__ __forceinline__ void grad_cols(const float* mu, int c, int cpg, const float (&rs)[V],
                                          GradCols<V>& o) {
  Groups gr(c, cpg);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int g = gr.next();
    o.b1[j] = -rs[j] * mu[2 * g];
    o.b2[j] = -rs[j] * rs[j] * mu[2 * g + 1];
  }
}
template <int V>
__device__ __forceinline__ void grad_out(const Cols<V>& t, const GradCols<V>& k, float (&f)[V], const float (&d)[V]) {
  v_fma<V>(f, k.b2, k.b1, f);
  v_fma<V>(d, t.sc, f, f);
}

// Adds the per-thread sums s0, s1 of V channels over the CTA's row threads, in
// row-thread order, into ch[c] and ch[C + c].
template <int V>
__device__ __forceinline__ void reduce_rows(float* red, float* ch, int C, int c_first, int tx, int ty, int cols_t,
                                            int rows_t, bool active, const float (&s0)[V], const float (&s1)[V]) {
  __syncthreads();
  if (active) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      red[(ty * 2 * V + j) * cols_t + tx] = s0[j];
      red[(ty * 2 * V + V + j) * cols_t + tx] = s1[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * V * cols_t; i += kThreads) {
    const int j = i / cols_t, t = i % cols_t;
    float a = 0.f;
#pragma unroll 8
    for (int y = 0; y < rows_t; ++y) a += red[(y * 2 * V + j) * cols_t + t];
    ch[(j >= V ? C : 0) + c_first + t * V + (j >= V ? j - V : j)] = a;
  }
}

// Joins the row threads' pairs (mean, squares about it) of V channels into the channels'
// pairs ch[c] and ch[C + c]: squares = sum of squares_t + n_t (mean_t - mean)^2. As many lanes
// share a channel as the CTA has (one lane each: 4 x 9216 x 320 forward 31 us instead of 29).
template <int V>
__device__ __forceinline__ void reduce_moments(float* red, float* ch, int C, int c_first, int tx, int ty, int cols_t,
                                               int rows_t, bool active, int64_t rows, const float (&mean)[V],
                                               const float (&sq)[V]) {
  __syncthreads();
  if (active) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      red[(ty * 2 * V + j) * cols_t + tx] = mean[j];
      red[(ty * 2 * V + V + j) * cols_t + tx] = sq[j];
    }
  }
  __syncthreads();
  const int64_t full = rows / rows_t;
  const int more = (int)(rows - full * rows_t);  // the first threads take a row more
  const float n0 = (float)full, n1 = (float)(full + 1), inv = rows > 0 ? 1.f / (float)rows : 0.f;
  int lanes = 1;
  while (lanes < 32 && 2 * lanes * V * cols_t <= kThreads) lanes *= 2;
  const int total = V * cols_t * lanes, sub = threadIdx.x & (lanes - 1);
  for (int i = threadIdx.x; i - (int)(threadIdx.x & 31) < total; i += kThreads) {  // whole warps
    const int at = min(i, total - 1) / lanes, j = at / cols_t, t = at % cols_t;
    const float *m = red + j * cols_t + t, *q = m + V * cols_t;
    const int step = 2 * V * cols_t;
    const float base = m[0];
    float d = 0.f, s = 0.f;
#pragma unroll 4
    for (int y = sub; y < rows_t; y += lanes) d = fmaf(y < more ? n1 : n0, m[y * step] - base, d);
    for (int o = lanes >> 1; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    d *= inv;
#pragma unroll 4
    for (int y = sub; y < rows_t; y += lanes) {
      const float e = (m[y * step] - base) - d;
      s += fmaf((y < more ? n1 : n0) * e, e, q[y * step]);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (sub == 0 && i < total) {
      const int c = c_first + t * V + j;
      ch[c] = base + d;
      ch[C + c] = s;
    }
  }
}
// A warp joins the pairs of a group's channels (`rows` values each).
__device__ __forceinline__ float2 join_channels(const float* ch, int C, int cpg, int64_t rows) {
  const int lane = threadIdx.x & 31;
  const float base = ch[0];
  float d = 0.f, s = 0.f;
  for (int i = lane; i < cpg; i += 32) d += ch[i] - base;
  d = warp_sum(d) / (float)cpg;
  for (int i = lane; i < cpg; i += 32) {
    const float e = (ch[i] - base) - d;
    s += fmaf((float)rows * e, e, ch[C + i]);
  }
  return make_float2(base + d, warp_sum(s));
}

// ------------------------------------------------------------------ one slice per cluster
// All of a thread's rows are asked for ahead (16 forward, 8 of both tensors backward)
// straight into shared memory: with four in registers 4 x 9216 x 320 took 30 us, so 22.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// p[i] of CTA `rank` of the cluster
__device__ __forceinline__ float peer_float(const float* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// 16 bytes from global to shared memory, without a register; a thread reads back only what
// it asked for itself, so its own wait suffices.
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows that a thread takes of first, first + step, ... below end (a CTA's share: below 2^31).
__device__ __forceinline__ int thread_rows(int64_t first, int64_t end, int step) {
  return first < end ? ((int)(end - first) + step - 1) / step : 0;
}

struct Slice {
  int64_t n, r0, r1;
  int c0, tx, ty, cols, rows_t;
  bool active;
};
__device__ __forceinline__ Slice my_slice(const GnArgs& a, int vec, uint32_t rank, uint32_t ctas) {
  Slice s;
  const int64_t cl = blockIdx.x / ctas;
  s.n = cl / a.slices;
  s.c0 = (int)(cl % a.slices) * a.width;
  s.r0 = min(a.rows, rank * a.chunk_rows);
  s.r1 = min(a.rows, s.r0 + a.chunk_rows);
  s.cols = a.width / vec;
  s.rows_t = kThreads / s.cols;
  s.tx = threadIdx.x % s.cols;
  s.ty = threadIdx.x / s.cols;
  s.active = s.ty < s.rows_t;
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gn_cluster_fwd_kernel(const __grid_constant__ GnArgs a) {
  constexpr int V = kVec<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const Slice s = my_slice(a, V, rank, ctas);
  const int iters = (int)((a.chunk_rows + s.rows_t - 1) / s.rows_t), groups = a.width / a.cpg;
  uint4* tile = reinterpret_cast<uint4*>(smem);                       // [iters][threads]
  float* red = reinterpret_cast<float*>(tile + (size_t)iters * kThreads);
  float* ch = red + 2 * V * kThreads;                                 // [2][width]
  float* part = ch + 2 * a.width;                                     // [groups][2] mean, squared deviations
  float* res = part + 2 * groups;                                     // [groups][2] mean, rstd
  const int c = s.c0 + s.tx * V;
  Cols<V> t;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const T* x = static_cast<const T*>(a.x) + s.n * a.rows * a.ldx;
  float mean[V], sq[V];
#pragma unroll
  for (int j = 0; j < V; ++j) mean[j] = sq[j] = 0.f;
  if (s.active) {
    constexpr int kAhead = 16;
    const int n = thread_rows(s.r0 + s.ty, s.r1, s.rows_t);
    const int64_t step = s.rows_t * a.ldx;
    const T* p = x + (s.r0 + s.ty) * a.ldx + c;
    uint4* own = tile + threadIdx.x;
    for (int i = 0; i < kAhead; ++i, p += step) {
      if (i < n) copy_async(own + i * kThreads, p);
      copy_commit();
    }
    load_affine<T, V>(a, c, t);
    // the mean about the first row, then the squares about the mean from shared memory
    float nk[V], f[V];
    for (int i = 0; i < n; ++i, p += step) {
      copy_wait<kAhead - 1>();
      unpack_vec<T, V>(own[i * kThreads], f);
      if (i + kAhead < n) copy_async(own + (i + kAhead) * kThreads, p);
      copy_commit();
      if (i == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) nk[j] = -f[j];
      }
      v_add<V>(f, nk, f);
      v_add<V>(mean, f, mean);
    }
    if (n > 0) {
      const float inv = -1.f / (float)n;
#pragma unroll
      for (int j = 0; j < V; ++j) nk[j] = fmaf(mean[j], inv, nk[j]);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        unpack_vec<T, V>(own[i * kThreads], f);
        v_add<V>(f, nk, f);
        v_fma<V>(f, f, sq, sq);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) mean[j] = -nk[j];
    }
  }
  reduce_moments<V>(red, ch, a.width, 0, s.tx, s.ty, s.cols, s.rows_t, s.active, s.r1 - s.r0, mean, sq);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < groups; g += kThreads / 32) {
    const float2 v = join_channels(ch + g * a.cpg, a.width, a.cpg, s.r1 - s.r0);
    if (lane == 0) {
      part[2 * g] = v.x;
      part[2 * g + 1] = v.y;
    }
  }
  cluster_sync();
  for (int g = threadIdx.x; g < groups; g += kThreads) {
    float m = 0.f, q = 0.f;
    float pm[kMaxCluster], w[kMaxCluster];
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      pm[i] = w[i] = 0.f;
      if (i < (int)ctas) {
        const int64_t lo = min(a.rows, i * a.chunk_rows), hi = min(a.rows, lo + a.chunk_rows);
        w[i] = (float)(hi - lo) / (float)a.rows;
        pm[i] = peer_float(part + 2 * g, i);
        q += peer_float(part + 2 * g + 1, i);
        m += w[i] * pm[i];
      }
    }
    q /= (float)a.rows * a.cpg;
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) q += w[i] * (pm[i] - m) * (pm[i] - m);
    const float rstd = 1.f / sqrtf(q + a.eps);
    res[2 * g] = m;
    res[2 * g + 1] = rstd;
    if (a.stats && rank == 0) {
      float* o = a.stats + (s.n * a.G + s.c0 / a.cpg + g) * 2;
      o[0] = m;
      o[1] = rstd;
    }
  }
  __syncthreads();
  if (s.active) {
    float rs[V];
    add_stats<V>(res, s.tx * V, a.cpg, t, rs);
    T* y = static_cast<T*>(a.out) + s.n * a.rows * a.ldy + c;
    int it = 0;
#pragma unroll 2
    for (int64_t r = s.r0 + s.ty; r < s.r1; r += s.rows_t, ++it) {
      float f[V];
      unpack_vec<T, V>(tile[it * kThreads + threadIdx.x], f);
      normalise<V>(t, f, a.act);
      *reinterpret_cast<uint4*>(y + r * a.ldy) = pack_vec<T, V>(f);
    }
  }
  cluster_sync();  // a CTA's sums stay readable until all have read them
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gn_cluster_bwd_kernel(const __grid_constant__ GnArgs a) {
  constexpr int V = kVec<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const Slice s = my_slice(a, V, rank, ctas);
  const int iters = (int)((a.chunk_rows + s.rows_t - 1) / s.rows_t), groups = a.width / a.cpg;
  uint4* tx_ = reinterpret_cast<uint4*>(smem);           // [iters][threads] x
  uint4* td = tx_ + (size_t)iters * kThreads;            // dy
  float* red = reinterpret_cast<float*>(td + (size_t)iters * kThreads);
  float* ch = red + 2 * V * kThreads;                    // [2][width] sum dz, sum dz * xh of this CTA
  float* part = ch + 2 * a.width;                        // [groups][2] the same weighted by gamma
  float* res = part + 2 * groups;                        // [groups][2] mean(u), mean(u * xh)
  const int c = s.c0 + s.tx * V;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const T* x = static_cast<const T*>(a.x) + s.n * a.rows * a.ldx + c;
  const T* dy = static_cast<const T*>(a.dy) + s.n * a.rows * a.ldy + c;
  const T* gamma = static_cast<const T*>(a.gamma);
  Cols<V> t;
  float s0[V], s1[V], rs[V];
#pragma unroll
  for (int j = 0; j < V; ++j) s0[j] = s1[j] = rs[j] = 0.f;
  if (s.active) {
    constexpr int kAhead = 8;
    const int n = thread_rows(s.r0 + s.ty, s.r1, s.rows_t);
    const int64_t step_x = s.rows_t * a.ldx, step_y = s.rows_t * a.ldy;
    const T *px = x + (s.r0 + s.ty) * a.ldx, *pd = dy + (s.r0 + s.ty) * a.ldy;
    uint4 *own_x = tx_ + threadIdx.x, *own_d = td + threadIdx.x;
    auto ask = [&](int i) {
      if (i < n) {
        copy_async(own_x + i * kThreads, px);
        copy_async(own_d + i * kThreads, pd);
      }
      copy_commit();
      px += step_x;
      pd += step_y;
    };
    for (int i = 0; i < kAhead; ++i) ask(i);
    load_affine<T, V>(a, c, t);
    add_stats<V>(a.stats + s.n * a.G * 2, c, a.cpg, t, rs);
    for (int i = 0; i < n; ++i) {
      copy_wait<kAhead - 1>();
      float f[V], d[V];
      unpack_vec<T, V>(own_x[i * kThreads], f);
      unpack_vec<T, V>(own_d[i * kThreads], d);
      ask(i + kAhead);
      grad_terms<V>(t, f, d, a.act);
      v_add<V>(s0, d, s0);
      v_fma<V>(d, f, s1, s1);
    }
  }
  v_mul<V>(s1, rs, s1);  // sum dz (x - mean) -> sum dz * xh
  reduce_rows<V>(red, ch, a.width, 0, s.tx, s.ty, s.cols, s.rows_t, s.active, s0, s1);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < groups; g += kThreads / 32) {
    float sum = 0.f, q = 0.f;
    for (int i = lane; i < a.cpg; i += 32) {
      const int cc = g * a.cpg + i;
      const float w = gamma ? Elem<T>::to_f(gamma[s.c0 + cc]) : 1.f;
      sum += w * ch[cc];
      q += w * ch[a.width + cc];
    }
    sum = warp_sum(sum);
    q = warp_sum(q);
    if (lane == 0) {
      part[2 * g] = sum;
      part[2 * g + 1] = q;
    }
  }
  cluster_sync();
  const float inv = 1.f / ((float)a.rows * a.cpg);
  for (int i = threadIdx.x; i < 2 * groups; i += kThreads) {
    float v = 0.f;
    for (uint32_t k = 0; k < ctas; ++k) v += peer_float(part + i, k);
    res[i] = v * inv;
  }
  if (a.dgamma || a.dbeta) {
    // the image's channel sums, a share of the channels per CTA; of several images they
    // are joined by a kernel of their own
    for (int i = rank * kThreads + threadIdx.x; i < 2 * a.width; i += ctas * kThreads) {
      float v = 0.f;
      for (uint32_t k = 0; k < ctas; ++k) v += peer_float(ch + i, k);
      const bool second = i >= a.width;
      const int cc = s.c0 + (second ? i - a.width : i);
      if (a.batch > 1)
        a.pc[(s.n * 2 + second) * a.C + cc] = v;
      else if (float* o = second ? a.dgamma : a.dbeta)
        o[cc] = v;
    }
  }
  __syncthreads();
  if (s.active) {
    GradCols<V> k;
    grad_cols<V>(res, s.tx * V, a.cpg, rs, k);
    T* dx = static_cast<T*>(a.out) + s.n * a.rows * a.ldx + c;
    int it = 0;
#pragma unroll 2
    for (int64_t r = s.r0 + s.ty; r < s.r1; r += s.rows_t, ++it) {
      float f[V], d[V];
      unpack_vec<T, V>(tx_[it * kThreads + threadIdx.x], f);
      unpack_vec<T, V>(td[it * kThreads + threadIdx.x], d);
      grad_terms<V>(t, f, d, a.act);
      grad_out<V>(t, k, f, d);
      *reinterpret_cast<uint4*>(dx + r * a.ldx) = pack_vec<T, V>(f);
    }
  }
  cluster_sync();  // a CTA's sums stay readable until all have read them
}

// dgamma and dbeta from per-channel parts [parts][2][C], 32 channels per CTA.
__device__ __forceinline__ void join_params(const GnArgs& a, int64_t parts, int block) {
  __shared__ float part[2][kThreads];
  const int c = block * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float s = 0.f, q = 0.f;
  if (c < a.C) {
#pragma unroll 4
    for (int64_t p = slice; p < parts; p += kThreads / 32) {
      s += a.pc[p * 2 * a.C + c];
      q += a.pc[p * 2 * a.C + a.C + c];
    }
  }
  part[0][threadIdx.x] = s;
  part[1][threadIdx.x] = q;
  __syncthreads();
  if (slice == 0 && c < a.C) {
    for (int i = 1; i < kThreads / 32; ++i) {
      s += part[0][i * 32 + threadIdx.x];
      q += part[1][i * 32 + threadIdx.x];
    }
    if (a.dbeta) a.dbeta[c] = s;
    if (a.dgamma) a.dgamma[c] = q;
  }
}
__global__ void __launch_bounds__(kThreads) gn_param_join_kernel(const __grid_constant__ GnArgs a) {
  pdl_wait();
  pdl_trigger();
  join_params(a, a.batch, blockIdx.x);
}

// ------------------------------------------------------------------ two kernels

// Shares of the forward statistics: (mean, sum of squared deviations) per group.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_stats_share_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ float ch[];  // [2][C]
  __shared__ float red[2 * V * kThreads];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const int64_t n = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x % a.chunks;
  const int64_t r0 = chunk * a.chunk_rows, r1 = min(a.rows, r0 + a.chunk_rows);
  const T* x = static_cast<const T*>(a.x) + n * a.rows * a.ldx;
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    const bool active = ty < rows_t;
    const int c = (c0 + tx) * V;
    float mean[V], sq[V];
#pragma unroll
    for (int j = 0; j < V; ++j) mean[j] = sq[j] = 0.f;
    if (active) {
      // eight rows at a time: their mean (about the thread's first row), the squares about
      // it, and the pair joined to that of the rows before
      constexpr int U = 8;
      const T* p = x + (r0 + ty) * a.ldx + c;
      const int64_t step = rows_t * a.ldx;
      const int n = thread_rows(r0 + ty, r1, rows_t);
      float nk[V];
      if (n > 0) {
        to_float<T, V>(load_raw<T, V>(p), nk);
#pragma unroll
        for (int j = 0; j < V; ++j) nk[j] = -nk[j];
      }
      for (int left = n; left > 0; left -= U, p += U * step) {
        Raw<T, V> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < left) raw[u] = load_raw<T, V>(p + u * step);
        float f[V], d[V], kb[V];
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u >= left) break;
          to_float<T, V>(raw[u], f);
          v_add<V>(f, nk, f);
          v_add<V>(d, f, d);
        }
        const float before = (float)(n - left), cnt = (float)min(left, U), inv = 1.f / cnt;
        const float w = cnt / (before + cnt), wn = before * w;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          kb[j] = fmaf(-inv, d[j], nk[j]);
          d[j] = fmaf(inv, d[j], -mean[j]);  // this mean less the one before
          mean[j] = fmaf(w, d[j], mean[j]);
          sq[j] = fmaf(wn * d[j], d[j], sq[j]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u >= left) break;
          to_float<T, V>(raw[u], f);
          v_add<V>(f, kb, f);
          v_fma<V>(f, f, sq, sq);
        }
      }
      if (n > 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) mean[j] -= nk[j];
      }
    }
    reduce_moments<V>(red, ch, a.C, c0 * V, tx, ty, cols_t, rows_t, active, r1 - r0, mean, sq);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < a.G; g += kThreads / 32) {
    const float2 v = join_channels(ch + g * a.cpg, a.C, a.cpg, r1 - r0);
    if (lane == 0) {
      float* o = a.pg + ((n * a.G + g) * a.chunks + chunk) * 2;
      o[0] = v.x;
      o[1] = v.y;
    }
  }
}

// y = act(z) from the joined shares; each CTA joins its image's shares itself.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_apply_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ float gs[];  // [G][2] mean, rstd
  pdl_wait();
  pdl_trigger();
  const int64_t n = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x % a.chunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float2* pg = reinterpret_cast<const float2*>(a.pg) + n * a.chunks * a.G;
  for (int g = warp; g < a.G; g += kThreads / 32) {
    float2 s[kMaxChunks / 32];
    float cnt[kMaxChunks / 32];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxChunks / 32; ++i) {
      const int p = i * 32 + lane;
      s[i] = p < a.chunks ? pg[(int64_t)g * a.chunks + p] : make_float2(0.f, 0.f);
      cnt[i] = p < a.chunks ? (float)(min(a.rows, (p + 1) * a.chunk_rows) - p * a.chunk_rows) / (float)a.rows : 0.f;
      m += cnt[i] * s[i].x;
    }
    m = warp_sum(m);
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxChunks / 32; ++i) {
      const float d = s[i].x - m;
      q += s[i].y / ((float)a.rows * a.cpg) + cnt[i] * d * d;
    }
    q = warp_sum(q);
    if (lane == 0) {
      const float rstd = 1.f / sqrtf(q + a.eps);
      gs[2 * g] = m;
      gs[2 * g + 1] = rstd;
      if (a.stats && chunk == 0) {
        a.stats[(n * a.G + g) * 2] = m;
        a.stats[(n * a.G + g) * 2 + 1] = rstd;
      }
    }
  }
  __syncthreads();
  const int64_t r0 = chunk * a.chunk_rows, r1 = min(a.rows, r0 + a.chunk_rows);
  const T* x = static_cast<const T*>(a.x) + n * a.rows * a.ldx;
  T* y = static_cast<T*>(a.out) + n * a.rows * a.ldy;
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    if (ty >= rows_t) continue;
    const int c = (c0 + tx) * V;
    Cols<V> t;
    float rs[V];
    load_affine<T, V>(a, c, t);
    add_stats<V>(gs, c, a.cpg, t, rs);
    // several rows are read before the first is written: y may be x, so the compiler
    // would not move a read across a write
    constexpr int U = 8;
    const int64_t last = r1 - 1 - ty, step_x = rows_t * a.ldx, step_y = rows_t * a.ldy;
    const T* p = x + last * a.ldx + c;
    T* o = y + last * a.ldy + c;
    for (int left = thread_rows(r0 + ty, r1, rows_t); left > 0; left -= U, p -= U * step_x, o -= U * step_y) {
      Raw<T, V> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < left) raw[u] = load_raw<T, V>(p - u * step_x);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= left) break;
        float f[V];
        to_float<T, V>(raw[u], f);
        normalise<V>(t, f, a.act);
        store_v<T, V>(o - u * step_y, f);
      }
    }
  }
}

// Shares of the backward sums: per channel (sum dz, sum dz*xh), per group the
// same weighted by gamma.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_grad_share_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ float ch[];  // [2][C]
  __shared__ float red[2 * V * kThreads];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const int64_t n = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x % a.chunks;
  const int64_t r0 = chunk * a.chunk_rows, r1 = min(a.rows, r0 + a.chunk_rows);
  const T* x = static_cast<const T*>(a.x) + n * a.rows * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + n * a.rows * a.ldy;
  const T* gamma = static_cast<const T*>(a.gamma);
  const float* stats = a.stats + n * a.G * 2;
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    const bool active = ty < rows_t;
    const int c = (c0 + tx) * V;
    float s0[V], s1[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s0[j] = s1[j] = 0.f;
    if (active) {
      Cols<V> t;
      float rs[V];
      load_affine<T, V>(a, c, t);
      add_stats<V>(stats, c, a.cpg, t, rs);
      constexpr int U = 4;
      const int64_t step_x = rows_t * a.ldx, step_y = rows_t * a.ldy;
      const T *px = x + (r0 + ty) * a.ldx + c, *pd = dy + (r0 + ty) * a.ldy + c;
      for (int left = thread_rows(r0 + ty, r1, rows_t); left > 0; left -= U, px += U * step_x, pd += U * step_y) {
        Raw<T, V> rx[U], rd[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < left) {
            rx[u] = load_raw<T, V>(px + u * step_x);
            rd[u] = load_raw<T, V>(pd + u * step_y);
          }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u >= left) break;
          float f[V], d[V];
          to_float<T, V>(rx[u], f);
          to_float<T, V>(rd[u], d);
          grad_terms<V>(t, f, d, a.act);
          v_add<V>(s0, d, s0);
          v_fma<V>(d, f, s1, s1);
        }
      }
      v_mul<V>(s1, rs, s1);  // sum dz (x - mean) -> sum dz * xh
    }
    reduce_rows<V>(red, ch, a.C, c0 * V, tx, ty, cols_t, rows_t, active, s0, s1);
  }
  __syncthreads();
  if (a.dgamma || a.dbeta) {
    float* o = a.pc + (int64_t)blockIdx.x * 2 * a.C;
    for (int i = threadIdx.x; i < 2 * a.C; i += kThreads) o[i] = ch[i];
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < a.G; g += kThreads / 32) {
    float s = 0.f, q = 0.f;
    for (int i = lane; i < a.cpg; i += 32) {
      const int c = g * a.cpg + i;
      const float w = gamma ? Elem<T>::to_f(gamma[c]) : 1.f;
      s += w * ch[c];
      q += w * ch[a.C + c];
    }
    s = warp_sum(s);
    q = warp_sum(q);
    if (lane == 0) {
      float* o = a.pg + ((n * a.G + g) * a.chunks + chunk) * 2;
      o[0] = s;
      o[1] = q;
    }
  }
}

// dx from the joined shares; the CTAs behind those of dx join dgamma and dbeta,
// 32 channels each.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_grad_apply_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ float gs[];  // [G][2] mean(u), mean(u * xh)
  pdl_wait();
  pdl_trigger();
  const int64_t shares = (int64_t)a.batch * a.chunks;
  if (blockIdx.x >= shares) {
    join_params(a, shares, (int)(blockIdx.x - shares));
    return;
  }
  const int64_t n = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x % a.chunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float2* pg = reinterpret_cast<const float2*>(a.pg) + n * a.chunks * a.G;
  const float inv = 1.f / ((float)a.rows * a.cpg);
  for (int g = warp; g < a.G; g += kThreads / 32) {
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxChunks / 32; ++i) {
      const int p = i * 32 + lane;
      const float2 v = p < a.chunks ? pg[(int64_t)g * a.chunks + p] : make_float2(0.f, 0.f);
      s += v.x;
      q += v.y;
    }
    s = warp_sum(s);
    q = warp_sum(q);
    if (lane == 0) {
      gs[2 * g] = s * inv;
      gs[2 * g + 1] = q * inv;
    }
  }
  __syncthreads();
  const int64_t r0 = chunk * a.chunk_rows, r1 = min(a.rows, r0 + a.chunk_rows);
  const T* x = static_cast<const T*>(a.x) + n * a.rows * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + n * a.rows * a.ldy;
  T* dx = static_cast<T*>(a.out) + n * a.rows * a.ldx;
  const float* stats = a.stats + n * a.G * 2;
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    if (ty >= rows_t) continue;
    const int c = (c0 + tx) * V;
    Cols<V> t;
    float rs[V];
    GradCols<V> k;
    load_affine<T, V>(a, c, t);
    add_stats<V>(stats, c, a.cpg, t, rs);
    grad_cols<V>(gs, c, a.cpg, rs, k);
    constexpr int U = 2;  // reads before writes, as above
    const int64_t last = r1 - 1 - ty, step_x = rows_t * a.ldx, step_y = rows_t * a.ldy;
    const T *px = x + last * a.ldx + c, *pd = dy + last * a.ldy + c;
    T* o = dx + last * a.ldx + c;
    for (int left = thread_rows(r0 + ty, r1, rows_t); left > 0;
         left -= U, px -= U * step_x, pd -= U * step_y, o -= U * step_x) {
      Raw<T, V> rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < left) {
          rx[u] = load_raw<T, V>(px - u * step_x);
          rd[u] = load_raw<T, V>(pd - u * step_y);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= left) break;
        float f[V], d[V];
        to_float<T, V>(rx[u], f);
        to_float<T, V>(rd[u], d);
        grad_terms<V>(t, f, d, a.act);
        grad_out<V>(t, k, f, d);
        store_v<T, V>(o - u * step_x, f);
      }
    }
  }
}

// ------------------------------------------------------------------ host side

sd_status check(const sd_group_norm_cfg* c) {
  if (!c) return SD_ERR_NULL_ARG;
  if (c->batch < 0 || c->rows < 0 || c->channels <= 0 || c->groups <= 0 || c->channels % c->groups) return SD_ERR_BAD_SHAPE;
  if ((c->ld_x && c->ld_x < c->channels) || (c->ld_y && c->ld_y < c->channels)) return SD_ERR_BAD_SHAPE;
  if (!(c->eps > 0.f)) return SD_ERR_BAD_SHAPE;
  if (c->channels > kMaxChannels || c->dtype < SD_DTYPE_BF16 || c->dtype > SD_DTYPE_F32 || c->act < SD_ACT_NONE ||
      c->act > SD_ACT_GELU)
    return SD_ERR_UNSUPPORTED;
  // element counts within 63 bits, CTA counts within a grid's x extent
  const int64_t ld = c->ld_x > c->ld_y ? c->ld_x : c->ld_y;
  if (c->rows > (int64_t)1 << 36 || ld > (int64_t)1 << 24 || c->batch > 1 << 18) return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

cudaError_t launch_cluster(void (*kernel)(GnArgs), unsigned grid, unsigned ctas, size_t smem, cudaStream_t st,
                           const GnArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T>
sd_status run_cluster(const sd_group_norm_cfg& c, GnArgs& a, const Plan& p, int back, const Device& dev,
                      cudaStream_t st) {
  a.width = p.width[back];
  a.slices = c.channels / a.width;
  a.chunk_rows = p.cta_rows[back];
  const size_t smem = cluster_smem(a.width, a.width / a.cpg, kVec<T>, a.chunk_rows, 1 + back);
  const unsigned ctas = (unsigned)p.ctas[back], grid = (unsigned)(c.batch * a.slices) * ctas;
  const double bytes = (double)c.batch * c.rows * c.channels * sizeof(T) * (2 + back);
  if (!back) {
    OP_TRY((allow_smem<gn_cluster_fwd_kernel<T>>(kClusterSmem, dev.index)));
    sdp::Scope sc("gn_cluster_fwd", sdp::F_GN_APPLY, 0, bytes, st);
    return launched(launch_cluster(gn_cluster_fwd_kernel<T>, grid, ctas, smem, st, a));
  }
  OP_TRY((allow_smem<gn_cluster_bwd_kernel<T>>(kClusterSmem, dev.index)));
  const bool more = c.batch > 1 && (a.dgamma || a.dbeta);
  sdp::Scope sc("gn_cluster_bwd", sdp::F_GN_APPLY, 0, bytes, st, more ? 2 : 1);
  OP_TRY(launched(launch_cluster(gn_cluster_bwd_kernel<T>, grid, ctas, smem, st, a)));
  if (!more) return SD_OK;
  return launched(launch_pdl(gn_param_join_kernel, dim3((c.channels + 31) / 32), dim3(kThreads), 0, st, a));
}

template <typename T, int V>
sd_status run_pair(const sd_group_norm_cfg& c, GnArgs& a, const Plan& p, int back, const Device& dev, cudaStream_t st) {
  const size_t sums = (size_t)2 * c.channels * sizeof(float), gsum = (size_t)2 * c.groups * sizeof(float);
  const unsigned ctas = (unsigned)(c.batch * (int64_t)p.chunks[back]);
  const double e = sizeof(T), n = (double)c.batch * c.rows * c.channels;
  if (!back) {
    OP_TRY((allow_smem<gn_stats_share_kernel<T, V>>(2 * kMaxChannels * sizeof(float), dev.index)));
    OP_TRY((allow_smem<gn_apply_kernel<T, V>>(2 * kMaxChannels * sizeof(float), dev.index)));
    {
      sdp::Scope sc("gn_stats_share", sdp::F_GN_STATS, 0, n * e, st);
      OP_TRY(launched(launch_pdl(gn_stats_share_kernel<T, V>, dim3(ctas), dim3(kThreads), sums, st, a)));
    }
    sdp::Scope sc("gn_apply_act", sdp::F_GN_APPLY, 0, 2 * n * e, st);
    return launched(launch_pdl(gn_apply_kernel<T, V>, dim3(ctas), dim3(kThreads), gsum, st, a));
  }
  OP_TRY((allow_smem<gn_grad_share_kernel<T, V>>(2 * kMaxChannels * sizeof(float), dev.index)));
  OP_TRY((allow_smem<gn_grad_apply_kernel<T, V>>(2 * kMaxChannels * sizeof(float), dev.index)));
  {
    sdp::Scope sc("gn_grad_share", sdp::F_GN_STATS, 0, 2 * n * e, st);
    OP_TRY(launched(launch_pdl(gn_grad_share_kernel<T, V>, dim3(ctas), dim3(kThreads), sums, st, a)));
  }
  const unsigned more = a.dgamma || a.dbeta ? (c.channels + 31) / 32 : 0;
  sdp::Scope sc("gn_grad_apply", sdp::F_GN_APPLY, 0, 3 * n * e, st);
  return launched(launch_pdl(gn_grad_apply_kernel<T, V>, dim3(ctas + more), dim3(kThreads), gsum, st, a));
}

template <typename T>
sd_status run_type(const sd_group_norm_cfg& c, GnArgs& a, const Plan& p, int back, const Device& dev, cudaStream_t st) {
  if (p.cluster[back]) return run_cluster<T>(c, a, p, back, dev, st);
  // 16-byte accesses when every row of every tensor starts on a 16-byte boundary
  const int v = kVec<T>;
  if (c.channels % v == 0 && a.ldx % v == 0 && a.ldy % v == 0) return run_pair<T, kVec<T>>(c, a, p, back, dev, st);
  return run_pair<T, 1>(c, a, p, back, dev, st);
}

sd_status dispatch(const sd_group_norm_cfg& c, GnArgs& a, const Plan& p, int back, cudaStream_t st) {
  Device dev;
  OP_TRY(current_device(&dev));
  if (c.dtype == SD_DTYPE_BF16) return run_type<__nv_bfloat16>(c, a, p, back, dev, st);
  if (c.dtype == SD_DTYPE_F16) return run_type<__half>(c, a, p, back, dev, st);
  return run_type<float>(c, a, p, back, dev, st);
}

void fill(const sd_group_norm_cfg& c, const Plan& p, int back, void* ws, GnArgs* a) {
  memset(a, 0, sizeof(*a));
  a->batch = c.batch;
  a->rows = c.rows;
  a->C = c.channels;
  a->G = c.groups;
  a->cpg = c.channels / c.groups;
  a->act = c.act;
  a->eps = c.eps;
  a->ldx = c.ld_x ? c.ld_x : c.channels;
  a->ldy = c.ld_y ? c.ld_y : c.channels;
  a->chunks = p.chunks[back];
  a->chunk_rows = p.chunk_rows[back];
  a->err = static_cast<int*>(ws);
  uint8_t* w = static_cast<uint8_t*>(ws) + kOpHeader;
  a->pg = reinterpret_cast<float*>(w);
  a->pc = reinterpret_cast<float*>(w + up256(p.pg_floats * sizeof(float)));
}

size_t space(const Plan& p) {
  return kOpHeader + up256(p.pg_floats * sizeof(float)) + up256(p.pc_floats * sizeof(float));
}

}  // namespace
}  // namespace sdo

using namespace sdo;

extern "C" {

size_t sd_group_norm_workspace_size(const sd_group_norm_cfg* cfg) {
  if (check(cfg) != SD_OK) return 0;
  if (cfg->batch == 0 || cfg->rows == 0) return kOpHeader;
  return space(make_plan(*cfg));
}

sd_status sd_group_norm_fwd(const sd_group_norm_cfg* cfg, const void* x, const void* gamma, const void* beta, void* y,
                            float* stats, void* workspace, size_t ws_bytes, sd_stream_t stream) {
  OP_TRY(check(cfg));
  if (cfg->batch == 0 || cfg->rows == 0) return SD_OK;
  if (!x || !y) return SD_ERR_NULL_ARG;
  if (misaligned(x) || misaligned(gamma) || misaligned(beta) || misaligned(y) || misaligned(stats))
    return SD_ERR_MISALIGNED;
  const Plan p = make_plan(*cfg);
  OP_TRY(check_workspace(space(p), workspace, ws_bytes));
  GnArgs a;
  fill(*cfg, p, 0, workspace, &a);
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.stats = stats;
  return dispatch(*cfg, a, p, 0, (cudaStream_t)stream);
}

sd_status sd_group_norm_bwd(const sd_group_norm_cfg* cfg, const void* x, const void* gamma, const void* beta,
                            const float* stats, const void* dy, void* dx, float* dgamma, float* dbeta, void* workspace,
                            size_t ws_bytes, sd_stream_t stream) {
  OP_TRY(check(cfg));
  if (misaligned(x) || misaligned(gamma) || misaligned(beta) || misaligned(stats) || misaligned(dy) ||
      misaligned(dx) || misaligned(dgamma) || misaligned(dbeta))
    return SD_ERR_MISALIGNED;
  if (cfg->batch == 0 || cfg->rows == 0) {
    Device dev;
    OP_TRY(current_device(&dev));
    const size_t n = (size_t)cfg->channels * sizeof(float);
    if (dgamma) OP_TRY(launched(cudaMemsetAsync(dgamma, 0, n, (cudaStream_t)stream)));
    if (dbeta) OP_TRY(launched(cudaMemsetAsync(dbeta, 0, n, (cudaStream_t)stream)));
    return SD_OK;
  }
  if (!x || !stats || !dy || !dx) return SD_ERR_NULL_ARG;
  const Plan p = make_plan(*cfg);
  OP_TRY(check_workspace(space(p), workspace, ws_bytes));
  GnArgs a;
  fill(*cfg, p, 1, workspace, &a);
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = const_cast<float*>(stats);
  a.dy = dy;
  a.out = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  return dispatch(*cfg, a, p, 1, (cudaStream_t)stream);
}

}  // extern "C"
