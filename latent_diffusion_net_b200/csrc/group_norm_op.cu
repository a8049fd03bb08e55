// Group norm with an activation on channels-last tensors, and its gradients.
//
// Per image and group, over rows x (C/G) values: xh = (x - mean) * rstd,
// z = gamma * xh + beta, y = act(z). With dz = dy * act'(z) and u = gamma * dz:
//   dbeta = sum dz, dgamma = sum dz * xh (over images and rows),
//   dx = rstd * (u - mean(u) - xh * mean(u * xh)).
//
// Bound by memory: forward reads x and writes y, backward reads x and dy and
// writes dx. Both run as two kernels: the first sums over a share of an
// image's rows per CTA, the second combines the shares in a fixed order (so
// results repeat bit for bit) and walks the same rows from their end, so that it
// finds the rows that the first one read last still in L2.
//
// A thread owns one 16-byte vector of channels for all its rows (channel terms
// stay in registers, a warp reads whole sectors whatever C/G is); sums are FP32
// per channel, relative to the first value of the share's group, and shares
// are joined from (mean, sum of squared deviations), so a mean far from zero
// costs no precision.
#include <string.h>

#include "op_common.cuh"
#include "profile.h"

namespace sdo {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxChannels = 8192;  // per-channel sums of a CTA: 64 KB of shared memory
constexpr int kMaxChunks = 256;     // shares of one image
constexpr int kTargetCtas = 592;    // four CTAs for each of 148 SMs

struct GnArgs {
  const void *x, *gamma, *beta, *dy;
  void* out;  // y or dx
  float* stats;
  float *dgamma, *dbeta;
  float *pg, *pc;  // shares: per group [batch][chunks][G][2], per channel [batch][chunks][2][C]
  int64_t rows, chunk_rows, ldx, ldy;
  int32_t batch, C, G, cpg, act, chunks;
  float eps;
  int* err;  // cleared by the first kernel of a call (none of them waits)
};

struct Plan {
  int chunks;
  int64_t chunk_rows;
  size_t pg_floats, pc_floats;
};

Plan make_plan(const sd_group_norm_cfg& c) {
  Plan p;
  // enough CTAs to fill the GPU, at least 16 rows in each
  int64_t n = (kTargetCtas + c.batch - 1) / c.batch;
  if (n > kMaxChunks) n = kMaxChunks;
  if (n > (c.rows + 15) / 16) n = (c.rows + 15) / 16;
  if (n < 1) n = 1;
  p.chunk_rows = (c.rows + n - 1) / n;
  p.chunks = (int)((c.rows + p.chunk_rows - 1) / p.chunk_rows);
  p.pg_floats = (size_t)c.batch * p.chunks * c.groups * 2;
  p.pc_floats = (size_t)c.batch * p.chunks * c.channels * 2;
  return p;
}

template <typename T, int V>
struct Row {
  uint4 raw;
  float f[V];
};

// V channels at p (16-byte aligned when V > 1).
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = Elem<T>::to_f(*p);
  } else {
    unpack_vec<T, V>(*reinterpret_cast<const uint4*>(p), f);
  }
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
    for (int y = 0; y < rows_t; ++y) a += red[(y * 2 * V + j) * cols_t + t];
    ch[(j >= V ? C : 0) + c_first + t * V + (j >= V ? j - V : j)] = a;
  }
}

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
  const T* first = x + r0 * a.ldx;
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    const bool active = ty < rows_t;
    const int c = (c0 + tx) * V;
    float k[V], s0[V], s1[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      k[j] = Elem<T>::to_f(first[(c + j) / a.cpg * a.cpg]);
      s0[j] = s1[j] = 0.f;
    }
    if (active) {
      const T* p = x + c;
#pragma unroll 4
      for (int64_t r = r0 + ty; r < r1; r += rows_t) {
        float f[V];
        load_v<T, V>(p + r * a.ldx, f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = f[j] - k[j];
          s0[j] += d;
          s1[j] = fmaf(d, d, s1[j]);
        }
      }
    }
    reduce_rows<V>(red, ch, a.C, c0 * V, tx, ty, cols_t, rows_t, active, s0, s1);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float cnt = (float)(r1 - r0) * a.cpg, inv = 1.f / cnt;
  for (int g = warp; g < a.G; g += kThreads / 32) {
    float s = 0.f, q = 0.f;
    for (int i = lane; i < a.cpg; i += 32) {
      s += ch[g * a.cpg + i];
      q += ch[a.C + g * a.cpg + i];
    }
    s = warp_sum(s);
    q = warp_sum(q);
    if (lane == 0) {
      const float d = s * inv;
      float* o = a.pg + ((int64_t)blockIdx.x * a.G + g) * 2;
      o[0] = Elem<T>::to_f(first[g * a.cpg]) + d;
      o[1] = fmaxf(q - s * d, 0.f);
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
      s[i] = p < a.chunks ? pg[(int64_t)p * a.G + g] : make_float2(0.f, 0.f);
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
  const T *gamma = static_cast<const T*>(a.gamma), *beta = static_cast<const T*>(a.beta);
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    if (ty >= rows_t) continue;
    const int c = (c0 + tx) * V;
    float m[V], sc[V], sh[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = (c + j) / a.cpg;
      m[j] = gs[2 * g];
      sc[j] = gs[2 * g + 1] * (gamma ? Elem<T>::to_f(gamma[c + j]) : 1.f);
      sh[j] = beta ? Elem<T>::to_f(beta[c + j]) : 0.f;
    }
#pragma unroll 4
    for (int64_t r = r1 - 1 - ty; r >= r0; r -= rows_t) {
      float f[V];
      load_v<T, V>(x + r * a.ldx + c, f);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = act_f(fmaf(f[j] - m[j], sc[j], sh[j]), a.act);
      store_v<T, V>(y + r * a.ldy + c, f);
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
  const T *gamma = static_cast<const T*>(a.gamma), *beta = static_cast<const T*>(a.beta);
  const float* stats = a.stats + n * a.G * 2;
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    const bool active = ty < rows_t;
    const int c = (c0 + tx) * V;
    float m[V], rs[V], ga[V], be[V], s0[V], s1[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = (c + j) / a.cpg;
      m[j] = stats[2 * g];
      rs[j] = stats[2 * g + 1];
      ga[j] = gamma ? Elem<T>::to_f(gamma[c + j]) : 1.f;
      be[j] = beta ? Elem<T>::to_f(beta[c + j]) : 0.f;
      s0[j] = s1[j] = 0.f;
    }
    if (active) {
#pragma unroll 2
      for (int64_t r = r0 + ty; r < r1; r += rows_t) {
        float f[V], d[V];
        load_v<T, V>(x + r * a.ldx + c, f);
        load_v<T, V>(dy + r * a.ldy + c, d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (f[j] - m[j]) * rs[j];
          float act, slope;
          act_grad_f(fmaf(xh, ga[j], be[j]), a.act, act, slope);
          const float dz = d[j] * slope;
          s0[j] += dz;
          s1[j] = fmaf(dz, xh, s1[j]);
        }
      }
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
      float* o = a.pg + ((int64_t)blockIdx.x * a.G + g) * 2;
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
    __shared__ float part[2][kThreads];
    const int c = (int)(blockIdx.x - shares) * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    float s = 0.f, q = 0.f;
    if (c < a.C) {
#pragma unroll 4
      for (int64_t p = slice; p < shares; p += kThreads / 32) {
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
      const float2 v = p < a.chunks ? pg[(int64_t)p * a.G + g] : make_float2(0.f, 0.f);
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
  const T *gamma = static_cast<const T*>(a.gamma), *beta = static_cast<const T*>(a.beta);
  const float* stats = a.stats + n * a.G * 2;
  const int cols = a.C / V;
  for (int c0 = 0; c0 < cols; c0 += kThreads) {
    const int cols_t = min(kThreads, cols - c0), rows_t = kThreads / cols_t;
    const int tx = threadIdx.x % cols_t, ty = threadIdx.x / cols_t;
    if (ty >= rows_t) continue;
    const int c = (c0 + tx) * V;
    float m[V], rs[V], ga[V], be[V], m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = (c + j) / a.cpg;
      m[j] = stats[2 * g];
      rs[j] = stats[2 * g + 1];
      ga[j] = gamma ? Elem<T>::to_f(gamma[c + j]) : 1.f;
      be[j] = beta ? Elem<T>::to_f(beta[c + j]) : 0.f;
      m1[j] = gs[2 * g];
      m2[j] = gs[2 * g + 1];
    }
#pragma unroll 2
    for (int64_t r = r1 - 1 - ty; r >= r0; r -= rows_t) {
      float f[V], d[V];
      load_v<T, V>(x + r * a.ldx + c, f);
      load_v<T, V>(dy + r * a.ldy + c, d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (f[j] - m[j]) * rs[j];
        float act, slope;
        act_grad_f(fmaf(xh, ga[j], be[j]), a.act, act, slope);
        f[j] = rs[j] * (d[j] * slope * ga[j] - m1[j] - xh * m2[j]);
      }
      store_v<T, V>(dx + r * a.ldx + c, f);
    }
  }
}

sd_status check(const sd_group_norm_cfg* c) {
  if (!c) return SD_ERR_NULL_ARG;
  if (c->batch < 0 || c->rows < 0 || c->channels <= 0 || c->groups <= 0 || c->channels % c->groups) return SD_ERR_BAD_SHAPE;
  if ((c->ld_x && c->ld_x < c->channels) || (c->ld_y && c->ld_y < c->channels)) return SD_ERR_BAD_SHAPE;
  if (!(c->eps > 0.f)) return SD_ERR_BAD_SHAPE;
  if (c->channels > kMaxChannels || c->dtype < SD_DTYPE_BF16 || c->dtype > SD_DTYPE_F32 || c->act < SD_ACT_NONE ||
      c->act > SD_ACT_GELU)
    return SD_ERR_UNSUPPORTED;
  // element counts within 48 bits, CTA counts within a grid's x extent
  const int64_t ld = c->ld_x > c->ld_y ? c->ld_x : c->ld_y;
  if (c->rows > (int64_t)1 << 40 || ld > (int64_t)1 << 24 || c->batch > 1 << 22) return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

template <typename T, int V>
sd_status run(const sd_group_norm_cfg& c, GnArgs& a, const Plan& p, bool grad, const Device& dev, cudaStream_t st) {
  const size_t sums = (size_t)2 * c.channels * sizeof(float), gsum = (size_t)2 * c.groups * sizeof(float);
  const unsigned ctas = (unsigned)(c.batch * (int64_t)p.chunks);
  const double e = sizeof(T), n = (double)c.batch * c.rows * c.channels;
  if (!grad) {
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
sd_status run_type(const sd_group_norm_cfg& c, GnArgs& a, const Plan& p, bool grad, const Device& dev,
                   cudaStream_t st) {
  // 16-byte accesses when every row of every tensor starts on a 16-byte boundary
  const int v = kVec<T>;
  if (c.channels % v == 0 && a.ldx % v == 0 && a.ldy % v == 0) return run<T, kVec<T>>(c, a, p, grad, dev, st);
  return run<T, 1>(c, a, p, grad, dev, st);
}

sd_status dispatch(const sd_group_norm_cfg& c, GnArgs& a, const Plan& p, bool grad, cudaStream_t st) {
  Device dev;
  OP_TRY(current_device(&dev));
  if (c.dtype == SD_DTYPE_BF16) return run_type<__nv_bfloat16>(c, a, p, grad, dev, st);
  if (c.dtype == SD_DTYPE_F16) return run_type<__half>(c, a, p, grad, dev, st);
  return run_type<float>(c, a, p, grad, dev, st);
}

void fill(const sd_group_norm_cfg& c, const Plan& p, void* ws, GnArgs* a) {
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
  a->chunks = p.chunks;
  a->chunk_rows = p.chunk_rows;
  a->err = static_cast<int*>(ws);
  uint8_t* w = static_cast<uint8_t*>(ws) + kOpHeader;
  a->pg = reinterpret_cast<float*>(w);
  a->pc = reinterpret_cast<float*>(w + up256(p.pg_floats * sizeof(float)));
}

}  // namespace
}  // namespace sdo

using namespace sdo;

extern "C" {

size_t sd_group_norm_workspace_size(const sd_group_norm_cfg* cfg) {
  if (check(cfg) != SD_OK) return 0;
  if (cfg->batch == 0 || cfg->rows == 0) return kOpHeader;
  const Plan p = make_plan(*cfg);
  return kOpHeader + up256(p.pg_floats * sizeof(float)) + up256(p.pc_floats * sizeof(float));
}

sd_status sd_group_norm_fwd(const sd_group_norm_cfg* cfg, const void* x, const void* gamma, const void* beta, void* y,
                            float* stats, void* workspace, size_t ws_bytes, sd_stream_t stream) {
  OP_TRY(check(cfg));
  if (cfg->batch == 0 || cfg->rows == 0) return SD_OK;
  if (!x || !y) return SD_ERR_NULL_ARG;
  if (misaligned(x) || misaligned(gamma) || misaligned(beta) || misaligned(y) || misaligned(stats))
    return SD_ERR_MISALIGNED;
  OP_TRY(check_workspace(sd_group_norm_workspace_size(cfg), workspace, ws_bytes));
  const Plan p = make_plan(*cfg);
  GnArgs a;
  fill(*cfg, p, workspace, &a);
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.stats = stats;
  return dispatch(*cfg, a, p, false, (cudaStream_t)stream);
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
  OP_TRY(check_workspace(sd_group_norm_workspace_size(cfg), workspace, ws_bytes));
  const Plan p = make_plan(*cfg);
  GnArgs a;
  fill(*cfg, p, workspace, &a);
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = const_cast<float*>(stats);
  a.dy = dy;
  a.out = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  return dispatch(*cfg, a, p, true, (cudaStream_t)stream);
}

}  // extern "C"
