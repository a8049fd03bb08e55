// Gradients of the attention operator. With P = exp(s - lse) recomputed tile by tile,
//   delta_i = sum_d dO_id O_id,  dP = dO V^T,  dS = P (dP - delta) (1 - tanh^2),
//   dV = P^T dO,  dK = scale dS^T Q (both summed over the heads that share a key head),
//   dQ = scale dS K.
//
// Bound by the tensor cores (10 D operations a pair in five products). Two kernels
// recompute S and dP each, so that every gradient is accumulated by one CTA in a
// fixed order: no atomics, results repeat bit for bit.
//   attn_dq_kernel   128 queries of one head walk their key tiles. delta from the saved
//                    o carries o's rounding, which is no longer small beside dP - delta
//                    where a row sees few keys; since the exact dS of a row sums to
//                    zero, the row sum e of the computed P (dP - delta) is delta's
//                    error, and dQ = scale (dS K - e P K) with P K as a third
//                    accumulator is exact to FP32. The corrected delta is left for
//   attn_dkv_kernel  a CTA owns 128 keys of one key head and walks the (head, query
//                    tile) pairs that may see them: S^T = K Q^T and dP^T = V dO^T
//                    have the keys as rows, so P^T and dS^T go from registers to
//                    TMEM as A operands of dV += P^T dO and dK += dS^T Q, and no
//                    transposed copy of anything is made
// Long walks are cut into parts, as in the forward kernel; FP32 parts are joined in order.
//
// 608 threads, one CTA per SM: warps 0-15 turn scores into P and dS (four warps per
// TMEM lane quarter, 32 of the columns each: with eight warps of 64 columns a tile took
// 1.2 to 1.4 times as long), warp 16 loads by TMA, one thread of warp 17 issues the
// products around S and P, one of warp 18 those around dP and dS: beside sixteen busy
// warps a thread issues one product in 80 to 100 cycles, so that one thread for all
// five was what the others waited for. S of the next tile runs beside dS of this one. P and dS
// are rounded to the inputs' type (the tensor core takes no other); everything else is
// FP32. FP16 has too few exponents for them, so for FP16 inputs both carry factors that
// are powers of two and taken out of the results again:
//   P   2^15 (P <= 1, and FP16 ends at 2^16): probabilities, times the cap's slope in dq,
//       keep their full precision down to 2^-29
//   dS  is bounded by what dO and V hold, not by k_len: |dS| <= 2 |dO_i| max |v_j|. The
//       factor brings that bound to 2^14 .. 2^15, whatever a loss scale made of dO: in
//       dQ one for each row i, in dK one for each CTA (largest |dO_i|, largest |v_j| of
//       its keys). attn_delta_kernel leaves the norms; rows that see nothing and keys
//       behind the last one take no part. The cap's slope is no part of the bound: where it
//       is below 2^-12 for all keys of a row, dS has fewer bits than FP16's eleven
//
// Measured (BF16): a step of 128 x 128 pairs takes 2.0 us an SM at head_dim 64, 2.6 at 128,
// 3.6 with capped scores; 2 x 4096 tokens causal, 10 heads of 64 293 us (FP16, with its
// factors, 4 % more); 9216 tokens, 5 heads 643 us (423 TFLOP/s of the formula's five products;
// the two kernels compute eight).
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "attention_op.cuh"
#include "profile.h"

namespace sdo {
namespace {

constexpr int kThreads = 608;
constexpr int kComputeWarps = 16;
constexpr int kSms = 148;
constexpr int kMaxSplits = 32;

struct GradArgs {
  AttnArgs f;
  int32_t qpad;         // query rows of lse2 and delta: a multiple of 128
  int32_t qblocks;      // 128-query tiles
  float* nlse;          // [B][H][qpad] -lse in log2 units; -inf where a row sees nothing or does not exist
  float* ndelta;        // [B][H][qpad] -delta
  const float* lse;
  const void* d_o;
  float out_scale, v_scale;  // factors of dQ and dK, of dV
  float shift;               // of P, as a power of two
  // FP16: norms of the rows of dO [B][H][qpad] (0 where a row sees nothing), the largest of
  // each 32 [B][H][qblocks][4], and the largest norm of a row of v in each key tile [B][KV][ktiles]
  float *do_norm, *do_max, *v_max;
  const void* v;
  int64_t vs[3];
  int64_t row_ctas;          // attn_delta_kernel: CTAs of rows, before those of key tiles
  int64_t s0[3], s1[3];      // output strides: dQ, or dK and dV
  void *out0, *out1;
  float* part;               // FP32 parts [2][slots][128][D]
  float* part_e;             // attn_dq_kernel: their row sums e [slots][128]
  int64_t slots;
};

struct __align__(64) GradMaps {
  CUtensorMap q, k, v, d_o;
};

// FP16: the largest norm of the rows of v in one key tile, rows behind the last key left
// out; 16 lanes a row.
__device__ __forceinline__ void tile_norm(const GradArgs& g, int64_t w) {
  __shared__ uint32_t top;
  const AttnArgs& a = g.f;
  const int kt = (int)(w % a.ktiles), kv = (int)(w / a.ktiles % a.KV), b = (int)(w / a.ktiles / a.KV);
  if (threadIdx.x == 0) top = 0;
  __syncthreads();
  const int d = (threadIdx.x & 15) * 8, end = min(keys_of(a, b), (kt + 1) * kTile);
  float m = 0.f;
  bool odd = false;  // NaN, which a maximum would pass over
#pragma unroll 4
  for (int k = 0; k < kTile; k += 16) {
    const int j = kt * kTile + k + (int)(threadIdx.x >> 4);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (j < end && d < a.D)
      x = *reinterpret_cast<const uint4*>(static_cast<const __half*>(g.v) + b * g.vs[0] + j * g.vs[1] + kv * g.vs[2] + d);
    float u[8], s = 0.f;
    unpack_vec<__half, 8>(x, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(u[e], u[e], s);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    odd = odd || s != s;
    m = fmaxf(m, s);
  }
  m = odd ? INFINITY : sqrtf(m);
  // numbers that are not negative compare like their bits
  const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
  if ((threadIdx.x & 31) == 0) atomicMax(&top, most);
  __syncthreads();
  if (threadIdx.x == 0) g.v_max[w] = __uint_as_float(top);
}
// FP16: the power of two that brings 2 `bound` below 2^15 (and to 2^14 at least); 1 where the
// bound is 0 or no number.
__device__ __forceinline__ float ds_factor(float bound) {
  const int e = (int)(__float_as_uint(bound) >> 23) - 127;  // bound in 2^e .. 2^(e + 1)
  return e > -100 && e < 100 ? __uint_as_float((uint32_t)(127 + 13 - e) << 23) : 1.f;
}

// -lse in log2 units and -delta for rows up to qpad: 2^shift lanes share a row, eight
// head dimensions each, and take four rows so that eight loads are under way.
template <typename T>
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ GradArgs g, int shift) {
  pdl_wait();
  pdl_trigger();
  const AttnArgs& a = g.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  if constexpr (Elem<T>::kF16) {
    if (blockIdx.x >= g.row_ctas) {
      tile_norm(g, blockIdx.x - g.row_ctas);
      return;
    }
  }
  const int sub = threadIdx.x & ((1 << shift) - 1), groups = 256 >> shift;
  const int64_t rows = (int64_t)a.B * a.H * g.qpad, r0 = blockIdx.x * (int64_t)groups * 4 + (threadIdx.x >> shift);
  uint4 x[4], y[4];
  float lse[4];
  int64_t to[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = r0 + k * groups;
    // rows in the order of (token, head), in which o lies when it is contiguous; 64-bit
    // divisions, of which each row needs three, would take longer than the reads
    int h, i, b;
    if (rows <= UINT32_MAX) {
      const uint32_t t = (uint32_t)r / (uint32_t)a.H;
      h = (int)((uint32_t)r - t * (uint32_t)a.H);
      b = (int)(t / (uint32_t)g.qpad);
      i = (int)(t - (uint32_t)b * (uint32_t)g.qpad);
    } else {
      h = (int)(r % a.H);
      i = (int)(r / a.H % g.qpad);
      b = (int)(r / a.H / g.qpad);
    }
    to[k] = ((int64_t)b * a.H + h) * g.qpad + i;
    x[k] = y[k] = make_uint4(0u, 0u, 0u, 0u);
    lse[k] = -INFINITY;
    if (r < rows && i < a.Nq) {
      if (sub * 8 < a.D) {
        const int64_t at = b * a.os[0] + i * a.os[1] + h * a.os[2] + sub * 8;
        x[k] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.o) + at);
        y[k] = *reinterpret_cast<const uint4*>(static_cast<const T*>(g.d_o) + at);
      }
      if (sub == 0) lse[k] = g.lse[((int64_t)b * a.H + h) * a.Nq + i];
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = r0 + k * groups;
    float u[8], v[8], s = 0.f, n = 0.f;
    unpack_vec<T, 8>(x[k], u);
    unpack_vec<T, 8>(y[k], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(u[e], v[e], s);
    for (int o = 1 << shift >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (Elem<T>::kF16) {
#pragma unroll
      for (int e = 0; e < 8; ++e) n = fmaf(v[e], v[e], n);
      for (int o = 1 << shift >> 1; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (sub == 0 && r < rows) g.do_norm[to[k]] = lse[k] == -INFINITY ? 0.f : n == n ? sqrtf(n) : INFINITY;
    }
    if (sub == 0 && r < rows) {
      g.nlse[to[k]] = lse[k] == -INFINITY ? -INFINITY : fmaf(-lse[k], kLog2e, g.shift);
      g.ndelta[to[k]] = -s;
    }
  }
}

// What becomes of one 16-column chunk of scores: p, p times the cap's slope (pf), and as FP16
// pairs where asked for the slope times kSlopeScale, or the rest p - pf (REST). The scores'
// columns lie `c` columns from the diagonal's column p0.
// SHAPED: cap or bias; MASKED: columns outside [from, to) and of other documents are hidden.
constexpr float kSlopeScale = 32768.f;  // slopes down to 2^-29 keep FP16's full precision
struct ScoreTerms {
  float slope, p0;
  int from, to, doc;
  const int32_t* sdoc;  // the columns' documents, or null
};
template <bool SHAPED, bool MASKED, bool REST = false>
__device__ __forceinline__ void probabilities(const AttnArgs& a, const ScoreTerms& s, const uint32_t (&r)[16], int c,
                                              const float (&nl)[16], float* p, float* pf, uint32_t* side = nullptr) {
  bool small = false;
  if constexpr (SHAPED) {
    if (a.cap_out != 0.f) {
      // neither padded keys (columns from `to` on, or a row that starts behind its columns) nor
      // queries that see nothing take part in choosing the form
      float top = 0.f;
#pragma unroll
      for (int u = 0; u < 16; u += 2) {
        float x0 = fabsf(__uint_as_float(r[u])), x1 = fabsf(__uint_as_float(r[u + 1]));
        if constexpr (MASKED) {
          if (c + u >= s.to || nl[u] == -INFINITY) x0 = 0.f;
          if (c + u + 1 >= s.to || nl[u + 1] == -INFINITY) x1 = 0.f;
        }
        top = max3f(top, x0, x1);
      }
      if (MASKED && s.from >= kTile) top = 0.f;
      small = __all_sync(0xffffffffu, top * a.cap_in <= kTanhSmall);
    }
  }
  auto two = [&](int u, auto form) {
    constexpr int kForm = decltype(form)::value;  // 0: no cap, 1: tanh of small values, 2: any
    float x0, x1, f0 = 1.f, f1 = 1.f;
    if constexpr (kForm > 0) {
      mul2(__uint_as_float(r[u]), __uint_as_float(r[u + 1]), a.cap_in, a.cap_in, x0, x1);
      if constexpr (kForm == 1) {
        tanh_small2(x0, x1, x0, x1);
        fma2v(-x0, -x1, x0, x1, 1.f, 1.f, f0, f1);
      } else {
        x0 = tanh_slope(x0, f0);
        x1 = tanh_slope(x1, f1);
      }
      fma2v(x0, x1, a.cap_out, a.cap_out, nl[u], nl[u + 1], x0, x1);
    } else {
      fma2v(__uint_as_float(r[u]), __uint_as_float(r[u + 1]), a.sl2, a.sl2, nl[u], nl[u + 1], x0, x1);
    }
    if constexpr (SHAPED) {
      x0 = fmaf(-s.slope, fabsf(s.p0 + (float)(c + u)), x0);
      x1 = fmaf(-s.slope, fabsf(s.p0 + (float)(c + u + 1)), x1);
    }
    p[u] = fast_ex2(x0);
    p[u + 1] = fast_ex2(x1);
    if constexpr (MASKED) {
      bool h0 = c + u < s.from || c + u >= s.to, h1 = c + u + 1 < s.from || c + u + 1 >= s.to;
      if (s.sdoc) {
        const int2 d = *reinterpret_cast<const int2*>(s.sdoc + c + u);
        h0 = h0 || d.x != s.doc;
        h1 = h1 || d.y != s.doc;
      }
      // the slope too: behind the last key it may come from NaN, and 0 NaN is NaN
      if (h0) p[u] = f0 = 0.f;
      if (h1) p[u + 1] = f1 = 0.f;
    }
    if constexpr (kForm > 0) {
      mul2(p[u], p[u + 1], f0, f1, pf[u], pf[u + 1]);
    } else {
      pf[u] = p[u];
      pf[u + 1] = p[u + 1];
    }
    if constexpr (SHAPED) {
      if (side) {
        if constexpr (REST)
          fma2v(pf[u], pf[u + 1], -1.f, -1.f, p[u], p[u + 1], f0, f1);
        else
          mul2(f0, f1, kSlopeScale, kSlopeScale, f0, f1);
        side[u / 2] = pack_f16x2(f0, f1);
      }
    }
  };
  if constexpr (SHAPED) {
    if (a.cap_out != 0.f) {
      if (small) {
#pragma unroll
        for (int u = 0; u < 16; u += 2) two(u, std::integral_constant<int, 1>());
      } else {
#pragma unroll
        for (int u = 0; u < 16; u += 2) two(u, std::integral_constant<int, 2>());
      }
      return;
    }
  }
#pragma unroll
  for (int u = 0; u < 16; u += 2) two(u, std::integral_constant<int, 0>());
}
// dS = pf (dP + nd) with nd = -delta. MASKED: dP of keys that do not exist may be anything.
template <bool MASKED>
__device__ __forceinline__ void score_grads(const uint32_t (&r)[16], const float (&nd)[16], const float* pf,
                                            float (&ds)[16]) {
#pragma unroll
  for (int u = 0; u < 16; u += 2) {
    float x0, x1;
    add2(__uint_as_float(r[u]), __uint_as_float(r[u + 1]), nd[u], nd[u + 1], x0, x1);
    mul2(x0, x1, pf[u], pf[u + 1], ds[u], ds[u + 1]);
    if constexpr (MASKED) {
      if (pf[u] == 0.f) ds[u] = 0.f;
      if (pf[u + 1] == 0.f) ds[u + 1] = 0.f;
    }
  }
}
template <typename T>
__device__ __forceinline__ void pack16(const float* f, uint32_t* pk) {
#pragma unroll
  for (int u = 0; u < 8; ++u) pk[u] = Elem<T>::pack(f[2 * u], f[2 * u + 1]);
}

// Half `side` of the columns of one row of an accumulator: to the output (scaled), or to
// the FP32 part. BACK: `back` takes the row's own factor out first.
template <typename T, int NB, bool WIDE, bool BACK>
__device__ __forceinline__ void store_row(uint32_t tacc, int side, bool have, bool in, int D, float scale, T* dst,
                                          bool wide, float* part, float back) {
#pragma unroll 1
  for (int c = side * NB * 32; c < (side + 1) * NB * 32; c += 32) {
    if (c >= D) break;
    uint32_t r[32];
    if (have) {
      tmem_ld_32x32b_x32(tacc + c, r);
      tmem_ld_wait_regs(r);
    } else {
#pragma unroll
      for (int u = 0; u < 32; ++u) r[u] = 0u;
    }
    if (!in) continue;
    if constexpr (BACK) {
#pragma unroll
      for (int u = 0; u < 32; ++u) r[u] = __float_as_uint(__uint_as_float(r[u]) * back);
    }
    if (part) {
      store_part32(part + c, r, D - c);
    } else {
      float f[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) f[u] = __uint_as_float(r[u]) * scale;
      store_row32<WIDE, T>(dst + c, f, D - c, wide);
    }
  }
}
// Tensor memory of both kernels: two score regions of 128 columns, two accumulators, and
// the packed P and dS that the products take as A operands.
//   head_dim <= 64: accumulators of 64 columns leave room for P and dS of their own, so
//     the scores of the next step are issued before this step's sums
//   head_dim <= 128: P and dS lie over their scores, each warp's 32 columns packed into the
//     first 16 of them, so that no warp writes where another still reads
template <int NB>
struct Tmem {
  static constexpr bool kApart = NB == 1;
  static constexpr uint32_t kS = 0, kDp = 128, kAcc0 = 256, kAcc1 = NB == 1 ? 320 : 384;
  static constexpr uint32_t kP = NB == 1 ? 384 : kS, kDs = NB == 1 ? 448 : kDp;
  // first packed column of scores [16 k, +16)
  static constexpr __host__ __device__ uint32_t packed(uint32_t k) {
    return NB == 1 ? 8 * k : (k >> 1) * 32 + (k & 1) * 8;
  }
};

constexpr size_t kTailBytes = kDocRing * 512 + kRing * sizeof(Record) + 512;  // documents, records, barriers

template <int NB>
constexpr size_t kDkvSmem = 1024 + (size_t)6 * NB * kBlockBytes + 2048 + kTailBytes;
template <int NB>
constexpr size_t kDqSmem = 1024 + (size_t)6 * NB * kBlockBytes + 2048 + kTailBytes;

// d = x y^T over the head dimension (nd steps of 16), both K-major; x and y as desc_k().
template <int NB>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t x, uint32_t y, int nd, uint32_t idesc, uint64_t* bar) {
  mma_ss<false>(d, x, y, idesc);
#pragma unroll
  for (int n = 1; n < 4 * NB; ++n) {
    const uint32_t o = (n >> 2) * (kBlockBytes >> 4) + (n & 3) * 2;
    if (n < nd) mma_ss<true>(d, x + o, y + o, idesc);
  }
  umma_commit(bar);
}
// d = or += x y, x packed P or dS, y 128 rows MN-major as desc_mn().
template <int NB>
__device__ __forceinline__ void issue_sum(uint32_t d, uint32_t x, uint32_t y, uint32_t idesc, bool more) {
  if (more)
    mma_ts<true>(d, x, y, idesc);
  else
    mma_ts<false>(d, x, y, idesc);
#pragma unroll
  for (int k = 1; k < 8; ++k) mma_ts<true>(d, x + Tmem<NB>::packed(k), y + k * 128, idesc);
}

// The walk of a dkv CTA over (head of the group, query tile).
struct HeadWalk {
  KeyTiles v;
  TileWalk<KeyTiles> w;
  int hh, steps;
  __device__ __forceinline__ HeadWalk(const KeyTiles& tiles, int G, const Part& part) : v(tiles), w(tiles), hh(0) {
    steps = INT32_MAX;
    if (part.slot >= 0) {
      const int count = w.count();
      const int64_t total = (int64_t)count * G, first = part.begin(total);
      steps = part.steps(total);
      if (steps > 0) {
        hh = (int)(first / count);
        w.skip((int)(first % count));
      }
    }
  }
  __device__ __forceinline__ int step(int G, bool& whole) {
    if (steps <= 0) return -1;
    int t = w.next(whole);
    while (t < 0) {
      if (hh + 1 >= G || v.tiles() == 0) {
        steps = 0;
        return -1;
      }
      ++hh;
      w.fetch(0);
      t = w.next(whole);
      if (t < 0) {  // no query tile sees these keys, in any head
        steps = 0;
        return -1;
      }
    }
    --steps;
    return t;
  }
};

template <typename T, int NB, bool SHAPED>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkv_kernel(const __grid_constant__ GradMaps maps, const __grid_constant__ GradArgs g) {
  constexpr bool f16 = Elem<T>::kF16;
  constexpr int kBytes = NB * kBlockBytes;
  const AttnArgs& a = g.f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + kBytes;
  uint8_t* sQ = sV + kBytes;       // [2]
  uint8_t* sDo = sQ + 2 * kBytes;  // [2]
  float* sstat = reinterpret_cast<float*>(sDo + 2 * kBytes);  // [2][-lse 128 | -delta 128]
  int32_t* sdocs = reinterpret_cast<int32_t*>(sstat + 512);  // [kDocRing][128]
  Record* recs = reinterpret_cast<Record*>(sdocs + kDocRing * kTile);
  uint64_t* bars = reinterpret_cast<uint64_t*>(recs + kRing);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;   // [2]
  uint64_t* q_empty = bars + 3;  // [2]
  uint64_t* s_full = bars + 5;
  uint64_t* dp_full = bars + 6;
  uint64_t* acc_done = bars + 7;
  uint64_t* p_full = bars + 8;
  uint64_t* ds_full = bars + 9;
  uint64_t* rec_full = bars + 10;   // [kRing]
  uint64_t* rec_empty = bars + 14;  // [kRing], the computing warps and the two MMA warps
  uint64_t* doc_full = bars + 18;   // [kDocRing]
  uint64_t* pv_done = bars + 18 + kDocRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 19 + kDocRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* do_top = tmem_slot + 2;  // FP16: bits of the largest |dO| of the key head's queries
  const RecordRing ring{recs, rec_full, rec_empty, abort_flag, a.err};
  const DocRing docs{sdocs, doc_full, abort_flag, a.err};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Part own(a.parts, blockIdx.x);
  const int heads = a.B * a.KV;
  const int kt = own.item / heads;  // the first key tiles first (with a causal mask they have the longest walks)
  const int b = own.item % heads / a.KV, kv = own.item % heads % a.KV;
  const int j0 = kt * kTile;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kDocRing; ++i) mbar_init(&doc_full[i], 1);
    for (int i = 0; i < 18; ++i) {
      const bool both = i == 3 || i == 4 || i == 7;  // released by both MMA warps
      mbar_init(bars + i, i >= 14 ? kComputeWarps + 2 : i == 8 || i == 9 ? kComputeWarps : both ? 2 : 1);
    }
    mbar_init(pv_done, 1);
    *abort_flag = 0;
    *do_top = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.d_o);
  }
  if (warp == 17) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  using Tm = Tmem<NB>;
  const uint32_t tS = tmem + Tm::kS, tDp = tmem + Tm::kDp, tDk = tmem + Tm::kAcc0, tDv = tmem + Tm::kAcc1;
  const uint32_t tP = tmem + Tm::kP, tDs = tmem + Tm::kDs;
  pdl_wait();
  pdl_trigger();

  const int nk = keys_of(a, b), off = nk - a.Nq, pre = prefix_of(a, b);
  if (warp == 16) {
    HeadWalk walk(KeyTiles(a, b, kt, g.qblocks, off, nk, pre), a.G, own);
    bool ok = a.hold_spins == 0 || mbar_wait(kv_full, 0, abort_flag, a.err, (uint32_t)a.hold_spins), whole;
    ok = __all_sync(0xffffffffu, ok);
    int t = 0;
    for (int tile; ok && (tile = walk.step(a.G, whole)) >= 0; ++t) {
      if (lane == 0) {
        const int i0 = tile * kTile, s = t & 1, h = kv * a.G + walk.hh;
        Record rec = {tile, whole ? kWhole : 0, 0, nk, pre, 0, b, h, i0, own.slot, {0, 0}};
        rec.flags |= walk.w.one_doc(tile, rec.doc);
        ok = ring.put(t, rec);
        if (ok && a.q_pad) {
          if (reads_docs(rec.flags))
            docs.load(t, a.q_pad + ((int64_t)b * g.qblocks + tile) * kTile);
          else
            docs.skip(t);
        }
        if (t == 0) {
          mbar_arrive_expect_tx(kv_full, 2 * kBytes);
          for (int c = 0; c < NB; ++c) {
            tma_load_4d(sK + c * kBlockBytes, &maps.k, kv_full, c * 64, kv, j0, b);
            tma_load_4d(sV + c * kBlockBytes, &maps.v, kv_full, c * 64, kv, j0, b);
          }
        }
        ok = ok && (t < 2 || mbar_wait(&q_empty[s], ((t >> 1) - 1) & 1, abort_flag, a.err));
        if (ok) {
          mbar_arrive_expect_tx(&q_full[s], 2 * kBytes + 1024);
          for (int c = 0; c < NB; ++c) {
            tma_load_4d(sQ + s * kBytes + c * kBlockBytes, &maps.q, &q_full[s], c * 64, h, i0, b);
            tma_load_4d(sDo + s * kBytes + c * kBlockBytes, &maps.d_o, &q_full[s], c * 64, h, i0, b);
          }
          const int64_t at = ((int64_t)b * a.H + h) * g.qpad + i0;
          bulk_load(sstat + s * 256, g.nlse + at, 512, &q_full[s]);
          bulk_load(sstat + s * 256 + 128, g.ndelta + at, 512, &q_full[s]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0 && ok) ring.end(t);
  } else if (warp >= 17) {
    // warp 17: S^T = K Q^T and dV += P^T dO; warp 18: dP^T = V dO^T and dK += dS^T Q
    const bool ds = warp == 18;
    const int nd = (a.D + 15) >> 4;
    const uint32_t id_s = idesc_f16(128, 128, f16, false, false);
    const uint32_t id_o = idesc_f16(128, nd * 16, f16, false, true);
    constexpr uint32_t kStage = kBytes >> 4;  // from one stage's descriptor to the other's
    const uint32_t x0 = desc_k(smem_u32(ds ? sV : sK)), y0 = desc_k(smem_u32(ds ? sDo : sQ));
    const uint32_t y0t = desc_mn(smem_u32(ds ? sQ : sDo), kBlockBytes);
    const uint32_t tScore = ds ? tDp : tS, tOp = ds ? tDs : tP, tAcc = ds ? tDk : tDv;
    uint64_t* const score_full = ds ? dp_full : s_full;
    uint64_t* const op_full = ds ? ds_full : p_full;
    auto next_scores = [&](int tt) {
      if (!mbar_wait(&q_full[tt & 1], (tt >> 1) & 1, abort_flag, a.err)) return false;
      tc_fence_after();
      issue_scores<NB>(tScore, x0, y0 + (tt & 1) * kStage, nd, id_s, score_full);
      return true;
    };
    bool ok = true;
    int t = 0;
    bool have = ring.get(0).x >= 0;
    if (have && lane == 0) ok = mbar_wait(kv_full, 0, abort_flag, a.err) && next_scores(0);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    for (; have && ok; ++t) {
      const bool more = ring.get(t + 1).x >= 0;
      if (lane == 0) {
        ok = mbar_wait(op_full, t & 1, abort_flag, a.err);
        tc_fence_after();
        if (Tm::kApart && ok && more) ok = next_scores(t + 1);
        if (ok) {
          issue_sum<NB>(tAcc, tOp, y0t + (t & 1) * kStage, id_o, t > 0);
          umma_commit(&q_empty[t & 1]);
          if (Tm::kApart && !ds) umma_commit(pv_done);
          if (!more) umma_commit(acc_done);
        }
        // over P^T or dS^T, whose product was issued before
        if (!Tm::kApart && ok && more) ok = next_scores(t + 1);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      have = more;
    }
  } else {
    const int q4 = warp & 3, cq = warp >> 2, c0 = cq * 32;  // lane quarter, column quarter
    const int row = q4 * 32 + lane, j = j0 + row;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tSr = tS + lane_off + c0, tDpr = tDp + lane_off + c0;
    const uint32_t tPr = tP + lane_off + Tm::packed(c0 / 16), tDsr = tDs + lane_off + Tm::packed(c0 / 16);
    ScoreTerms st;
    st.to = kTile;
    st.doc = a.k_doc && j < a.Nk ? a.k_doc[(int64_t)b * a.Nk + j] : 0;
    [[maybe_unused]] float ds_mul = 1.f;  // the CTA's factor of dS, without P's
    if constexpr (f16) {
      const int n = a.G * g.qblocks * 4;
      const uint32_t* const norms =
          reinterpret_cast<const uint32_t*>(g.do_max) + ((int64_t)b * a.H + kv * a.G) * g.qblocks * 4;
      uint32_t top = 0;
      for (int i = threadIdx.x; i < n; i += 32 * kComputeWarps) top = max(top, norms[i]);
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) atomicMax(do_top, top);
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kComputeWarps) : "memory");
      ds_mul = ds_factor(__uint_as_float(*do_top) * g.v_max[((int64_t)b * a.KV + kv) * a.ktiles + kt]) * g.v_scale;
    }
    bool alive = true;
    int t = 0;
    for (;; ++t) {
      const Record* const rec = ring.at(t);
      if (!(alive = rec != nullptr) || (rec->flags & kEnd)) break;
      const int flags = rec->flags;
      const bool whole = flags & kWhole;
      const int i0 = rec->i0, s = t & 1;
      if (SHAPED) st.slope = a.slopes ? a.slopes[rec->head] * kLog2e : 0.f;
      st.p0 = (float)(i0 + off - j);
      // queries of this tile from column `from` on see the key (none when it does not exist)
      st.from = j >= nk || ((flags & kOneDoc) && rec->doc != st.doc) ? kTile : a.causal && j >= pre ? j - off - i0 : 0;
      const float* stat = sstat + s * 256 + c0;
      st.sdoc = nullptr;
      if (a.q_pad && reads_docs(flags)) {
        st.sdoc = docs.get(t, alive);
        if (!alive) break;
      }
      if (!(alive = mbar_wait_all(&q_full[s], (t >> 1) & 1, abort_flag, a.err) &&
                    mbar_wait_all(s_full, t & 1, abort_flag, a.err)))
        break;
      tc_fence_after();
      if (!whole && cq < 2) {
        // queries that see nothing count as zeros in the sums, whatever they hold: S of this
        // tile is done, and dP is waited for before dO is touched
        const bool dead = i0 + row < a.Nq && sstat[s * 256 + row] == -INFINITY;
        if (__any_sync(0xffffffffu, dead)) {
          if (cq && !(alive = mbar_wait_all(dp_full, t & 1, abort_flag, a.err))) break;
          if (dead) {
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              uint4* z = reinterpret_cast<uint4*>((cq ? sDo : sQ) + s * kBytes + c * kBlockBytes + row * 128);
#pragma unroll
              for (int y = 0; y < 8; ++y) z[y] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_async_smem();
        }
      }
      float pf[32];
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 16) {
        uint32_t q[16];
        float nl[16], p[16];
        tmem_ld_x16(tSr + e, q);
#pragma unroll
        for (int u = 0; u < 16; u += 4) {
          const float4 v = *reinterpret_cast<const float4*>(stat + e + u);
          nl[u] = v.x;
          nl[u + 1] = v.y;
          nl[u + 2] = v.z;
          nl[u + 3] = v.w;
        }
        tmem_ld_wait_16(q);
        if (whole)
          probabilities<SHAPED, false>(a, st, q, c0 + e, nl, p, pf + e);
        else
          probabilities<SHAPED, true>(a, st, q, c0 + e, nl, p, pf + e);
        pack16<T>(p, pk + e / 2);
        if (!Tm::kApart) tmem_st_x8(tPr + e / 2, pk + e / 2);  // over scores already read
      }
      if (Tm::kApart) {
        // P's columns are free once the last step's product is done
        if (t > 0 && !(alive = mbar_wait_all(pv_done, (t - 1) & 1, abort_flag, a.err))) break;
        tc_fence_after();
        tmem_st_x16(tPr, pk);
      }
      tmem_store_wait();
      tc_fence_before();
      mbar_arrive_warp(p_full);
      if (!(alive = mbar_wait_all(dp_full, t & 1, abort_flag, a.err))) break;
      tc_fence_after();
#pragma unroll
      for (int e = 0; e < 32; e += 16) {
        uint32_t q[16];
        float nd[16], ds[16];
        tmem_ld_x16(tDpr + e, q);
#pragma unroll
        for (int u = 0; u < 16; u += 4) {
          const float4 v = *reinterpret_cast<const float4*>(stat + 128 + e + u);
          nd[u] = v.x;
          nd[u + 1] = v.y;
          nd[u + 2] = v.z;
          nd[u + 3] = v.w;
        }
        tmem_ld_wait_16(q);
        if (whole)
          score_grads<false>(q, nd, pf + e, ds);
        else
          score_grads<true>(q, nd, pf + e, ds);
        if constexpr (f16) {
#pragma unroll
          for (int u = 0; u < 16; u += 2) mul2(ds[u], ds[u + 1], ds_mul, ds_mul, ds[u], ds[u + 1]);
        }
        pack16<T>(ds, pk + e / 2);
        if (!Tm::kApart) tmem_st_x8(tDsr + e / 2, pk + e / 2);
      }
      if (Tm::kApart) {
        // dS's columns are free once the last step's dS product is done
        if (t > 0 && !(alive = mbar_wait_all(&q_empty[s ^ 1], ((t - 1) >> 1) & 1, abort_flag, a.err))) break;
        tc_fence_after();
        tmem_st_x16(tDsr, pk);
      }
      tmem_store_wait();
      tc_fence_before();
      mbar_arrive_warp(ds_full);
      ring.done(t);
    }
    if (alive && t > 0) alive = mbar_wait_all(acc_done, 0, abort_flag, a.err);
    tc_fence_after();
    if (alive) {
      // two warps of a lane quarter write dK, two dV, half of the columns each
      const int which = cq >> 1;
      const int64_t* os = which ? g.s1 : g.s0;
      T* dst = static_cast<T*>(which ? g.out1 : g.out0) + b * os[0] + j * os[1] + kv * os[2];
      float* part = nullptr;
      if (own.slot >= 0) part = g.part + ((which * g.slots + own.slot) * kTile + j - j0) * a.D;
      store_row<T, NB, !SHAPED, f16>((which ? tDv : tDk) + lane_off, cq & 1, t > 0, j < a.Nk, a.D, which ? g.v_scale : g.out_scale,
                       dst, wide_rows(which ? g.out1 : g.out0, which ? g.s1 : g.s0, a.D), part,
                       which ? 1.f : 1.f / ds_mul);
    }
  }
  settle(abort_flag);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// A unit of dq work: a part of 128 queries of one head, the last query tiles first.
struct DqUnit {
  Part part;
  int b, h, i0, i1, qt;
  __device__ __forceinline__ DqUnit(const GradArgs& g, int u) : part(g.f.parts, u) {
    const AttnArgs& a = g.f;
    const int heads = a.B * a.H, at = part.item % heads;
    qt = g.qblocks - 1 - part.item / heads;
    b = at / a.H;
    h = at % a.H;
    i0 = qt * kTile;
    i1 = min(a.Nq, i0 + kTile) - 1;
  }
};
struct DqWalk : TileWalk<RowTiles> {
  int steps;
  __device__ __forceinline__ DqWalk(const GradArgs& g, const DqUnit& u, int off, int nk, int pre)
      : TileWalk<RowTiles>(RowTiles(g.f, u.b, u.i0, u.i1, off, nk, pre,
                                    g.f.q_range + ((int64_t)u.b * g.qblocks + u.qt) * 2)) {
    steps = INT32_MAX;
    if (u.part.slot >= 0) {
      const int n = count();
      steps = u.part.steps(n);
      if (steps > 0) skip((int)u.part.begin(n));
    }
  }
  __device__ __forceinline__ int step(bool& whole) { return steps-- > 0 ? next(whole) : -1; }
};

// The end of a dq unit, one query row per thread: dQ = scale (dS K - e P K) and the
// corrected delta, or (given `part`) the parts of a cut item; BACK as in store_row(). Out of line: its registers
// would compete with the loop's. All by value, as in the forward kernel.
template <typename T, int NB, bool WIDE, bool BACK>
__device__ __noinline__ void store_dq(T* dst, bool wide, float* part, float* part_k, float* row_e, int D, float scale,
                                      int side, uint32_t tDq, uint32_t tPk, bool some, bool valid, float e,
                                      float back) {
  if (part) {
    store_row<T, NB, WIDE, BACK>(tDq, side, some, valid, D, 1.f, dst, wide, part, back);
    store_row<T, NB, WIDE, false>(tPk, side, some, valid, D, 1.f, dst, wide, part_k, 1.f);
    if (valid && side == 0) *row_e = e;
    return;
  }
#pragma unroll 1
  for (int c = side * NB * 32; c < (side + 1) * NB * 32; c += 16) {
    if (c >= D) break;
    uint32_t r[16], q[16];
    if (some) {
      tmem_ld_x16(tDq + c, r);
      tmem_ld_x16(tPk + c, q);
      tmem_ld_wait_16(r);
      tmem_ld_wait_16(q);
    }
    if (!valid) continue;
    uint32_t w[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      float f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float d = __uint_as_float(r[2 * y + x]);
        f[x] = some ? scale * fmaf(-e, __uint_as_float(q[2 * y + x]), BACK ? d * back : d) : 0.f;
      }
      w[y] = Elem<T>::pack(f[0], f[1]);
    }
    if (WIDE && wide) {
      st_global_v8(dst + c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    } else {
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
      if (c + 8 < D) *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// CTAs take over units as in the forward kernel; t counts steps and n units with steps.
template <typename T, int NB, bool SHAPED>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_kernel(const __grid_constant__ GradMaps maps, const __grid_constant__ GradArgs g) {
  constexpr bool f16 = Elem<T>::kF16;
  constexpr int kBytes = NB * kBlockBytes;
  const AttnArgs& a = g.f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sDo = sQ + kBytes;
  uint8_t* sK = sDo + kBytes;     // [2]
  uint8_t* sV = sK + 2 * kBytes;  // [2]
  float* srow = reinterpret_cast<float*>(sV + 2 * kBytes);  // [4][128] the column quarters' row sums
  int32_t* sdocs = reinterpret_cast<int32_t*>(srow + 4 * kTile);  // [kDocRing][128]
  Record* recs = reinterpret_cast<Record*>(sdocs + kDocRing * kTile);
  uint64_t* bars = reinterpret_cast<uint64_t*>(recs + kRing);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* kv_full = bars + 2;   // [2]
  uint64_t* kv_empty = bars + 4;  // [2]
  uint64_t* s_full = bars + 6;
  uint64_t* dp_full = bars + 7;
  uint64_t* acc_done = bars + 8;
  uint64_t* p_full = bars + 9;
  uint64_t* ds_full = bars + 10;
  uint64_t* rec_full = bars + 11;   // [kRing]
  uint64_t* rec_empty = bars + 15;  // [kRing], the computing warps and the two MMA warps
  uint64_t* next_bar = bars + 19;
  uint8_t* next_unit = reinterpret_cast<uint8_t*>(bars + 20);  // 16 bytes
  uint64_t* doc_full = bars + 22;  // [kDocRing]
  uint64_t* pv_done = bars + 22 + kDocRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 23 + kDocRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* left = reinterpret_cast<int*>(tmem_slot + 2);  // computing warps that are through
  const RecordRing ring{recs, rec_full, rec_empty, abort_flag, a.err};
  const DocRing docs{sdocs, doc_full, abort_flag, a.err};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDocRing; ++i) mbar_init(&doc_full[i], 1);
    for (int i = 0; i < 20; ++i) {
      const bool both = i == 1 || i == 4 || i == 5 || i == 8;  // released by both MMA warps
      mbar_init(bars + i, i == 9 || i == 10 ? kComputeWarps : i >= 15 && i < 19 ? kComputeWarps + 2 : both ? 2 : 1);
    }
    mbar_init(pv_done, 1);
    *abort_flag = 0;
    *left = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.d_o);
  }
  if (warp == 17) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  using Tm = Tmem<NB>;
  const uint32_t tS = tmem + Tm::kS, tDp = tmem + Tm::kDp, tDq = tmem + Tm::kAcc0, tPk = tmem + Tm::kAcc1;
  const uint32_t tP = tmem + Tm::kP, tDs = tmem + Tm::kDs;
  pdl_wait();
  pdl_trigger();

  if (warp == 16) {
    int t = 0, n = 0, r = 0, asked = 0;
    bool ok = a.hold_spins == 0 || mbar_wait(next_bar, 0, abort_flag, a.err, (uint32_t)a.hold_spins);
    ok = __all_sync(0xffffffffu, ok);
    for (int x = blockIdx.x; x >= 0 && ok;) {
      const DqUnit u(g, x);
      const int nk = keys_of(a, u.b), pre = prefix_of(a, u.b), kv = u.h / a.G;
      DqWalk walk(g, u, nk - a.Nq, nk, pre);
      bool whole, whole_next;
      int j = walk.step(whole), after;
      int first = kFirst;
      do {
        after = j >= 0 ? walk.step(whole_next) : -1;
        if (lane == 0) {
          Record rec = {j, first | (after < 0 ? kLast : 0) | (j >= 0 && whole ? kWhole : 0), x, nk, pre, 0, u.b, u.h, u.i0,
                        u.part.slot, {0, 0}};
          if (j >= 0) rec.flags |= walk.one_doc(j, rec.doc);
          ok = ring.put(r, rec);
          if (after < 0) {
            // at the unit's end: a unit asked for early would wait behind a long one
            mbar_arrive_expect_tx(next_bar, 16);
            ask_unit(next_unit, next_bar);
          }
          if (ok && a.k_pad) {
            if (j >= 0 && reads_docs(rec.flags))
              docs.load(r, a.k_pad + ((int64_t)u.b * a.ktiles + j) * kTile);
            else
              docs.skip(r);
          }
          if (j >= 0) {
            if (first && (ok = ok && (n == 0 || mbar_wait(q_empty, (n - 1) & 1, abort_flag, a.err)))) {
              mbar_arrive_expect_tx(q_full, 2 * kBytes);
              for (int c = 0; c < NB; ++c) {
                tma_load_4d(sQ + c * kBlockBytes, &maps.q, q_full, c * 64, u.h, u.i0, u.b);
                tma_load_4d(sDo + c * kBlockBytes, &maps.d_o, q_full, c * 64, u.h, u.i0, u.b);
              }
            }
            const int s = t & 1;
            ok = ok && (t < 2 || mbar_wait(&kv_empty[s], ((t >> 1) - 1) & 1, abort_flag, a.err));
            if (ok) {
              mbar_arrive_expect_tx(&kv_full[s], 2 * kBytes);
              for (int c = 0; c < NB; ++c) {
                tma_load_4d(sK + s * kBytes + c * kBlockBytes, &maps.k, &kv_full[s], c * 64, kv, j * kTile, u.b);
                tma_load_4d(sV + s * kBytes + c * kBlockBytes, &maps.v, &kv_full[s], c * 64, kv, j * kTile, u.b);
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++r;
        if (j >= 0) {
          ++t;
          n += first ? 1 : 0;
        }
        first = 0;
        j = after;
        whole = whole_next;
      } while (j >= 0 && ok);
      if (lane == 0) {
        ok = mbar_wait(next_bar, asked & 1, abort_flag, a.err) && ok;
        x = ok ? asked_unit(next_unit) : -1;
        fence_async_smem();  // read before the next answer is written
      }
      ++asked;
      x = __shfl_sync(0xffffffffu, x, 0);
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0 && ok) ring.end(r);
  } else if (warp >= 17) {
    // warp 17: S = Q K^T and the sum of P K; warp 18: dP = dO V^T and the sum of dS K.
    // Steps follow one another across units: while one is summed, the scores of the next
    // are issued, whichever unit it belongs to. Only one record is looked ahead: one
    // without a tile is not waited past, since the ring moves on only with this step.
    const bool ds = warp == 18;
    const int nd = (a.D + 15) >> 4;
    const uint32_t id_s = idesc_f16(128, 128, f16, false, false);
    const uint32_t id_o = idesc_f16(128, nd * 16, f16, false, true);
    constexpr uint32_t kStage = kBytes >> 4;  // from one stage's descriptor to the other's
    const uint32_t x0 = desc_k(smem_u32(ds ? sDo : sQ)), y0 = desc_k(smem_u32(ds ? sV : sK));
    const uint32_t k0t = desc_mn(smem_u32(sK), kBlockBytes);
    const uint32_t tScore = ds ? tDp : tS, tOp = ds ? tDs : tP, tAcc = ds ? tDq : tPk;
    uint64_t* const score_full = ds ? dp_full : s_full;
    uint64_t* const op_full = ds ? ds_full : p_full;
    int n = -1, t = 0;
    bool ok = true, issued = false;
    // the scores of step tt of unit nn
    auto next_scores = [&](int tt, int nn, int flags) {
      if ((flags & kFirst) && !mbar_wait(q_full, nn & 1, abort_flag, a.err)) return false;
      if (!mbar_wait(&kv_full[tt & 1], (tt >> 1) & 1, abort_flag, a.err)) return false;
      tc_fence_after();
      issue_scores<NB>(tScore, x0, y0 + (tt & 1) * kStage, nd, id_s, score_full);
      if (flags & kLast) umma_commit(q_empty);
      return true;
    };
    int2 cur = ring.get(0);  // tile, flags
    for (int r = 1; !(cur.y & kEnd) && ok; ++r) {
      const int2 nx = ring.get(r);
      if (cur.x < 0) {
        cur = nx;
        continue;
      }
      const bool more = nx.x >= 0;
      if (!issued) {
        if (cur.y & kFirst) ++n;
        if (lane == 0) ok = next_scores(t, n, cur.y);
      }
      if (more && (nx.y & kFirst)) ++n;
      if (lane == 0 && ok) {
        ok = mbar_wait(op_full, t & 1, abort_flag, a.err);
        tc_fence_after();
        if (Tm::kApart && ok && more) ok = next_scores(t + 1, n, nx.y);
        if (ok) {
          issue_sum<NB>(tAcc, tOp, k0t + (t & 1) * kStage, id_o, !(cur.y & kFirst));
          umma_commit(&kv_empty[t & 1]);
          if (Tm::kApart && !ds) umma_commit(pv_done);
          if (cur.y & kLast) umma_commit(acc_done);
        }
        // over P or dS, whose product was issued before
        if (!Tm::kApart && ok && more) ok = next_scores(t + 1, n, nx.y);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      issued = more;
      ++t;
      cur = nx;
    }
  } else {
    const int q4 = warp & 3, cq = warp >> 2, c0 = cq * 32;  // lane quarter, column quarter
    const int row = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tSr = tS + lane_off + c0, tDpr = tDp + lane_off + c0;
    const uint32_t tPr = tP + lane_off + Tm::packed(c0 / 16), tDsr = tDs + lane_off + Tm::packed(c0 / 16);
    int t = 0, n = 0;
    bool alive = true;
    ScoreTerms st;
    st.from = 0;
    int nk = 0, lim = 0, pos = 0;
    float nlse = 0.f, ndelta = 0.f;
    [[maybe_unused]] float ds_mul = 1.f;  // the row's factor of dS, without P's
    const bool wide = wide_rows(g.out0, g.s0, a.D);
    float e0 = 0.f, e1 = 0.f;  // the row's sum of P (dP - delta) over this half's columns
    for (int r = 0;; ++r) {
      const Record* const rec = ring.at(r);
      if (!rec || (rec->flags & kEnd)) break;
      const int flags = rec->flags, tile = rec->tile;
      const bool whole = flags & kWhole;
      if (flags & kFirst) {
        const int i = rec->i0 + row;
        const int64_t at = ((int64_t)rec->b * a.H + rec->head) * g.qpad + i;
        nk = rec->nk;
        pos = i + nk - a.Nq;
        lim = a.causal ? min(nk, max(pos + 1, rec->pre)) : nk;
        nlse = g.nlse[at];
        ndelta = g.ndelta[at];
        if constexpr (f16) {
          const float norm = g.do_norm[at];
          const uint32_t* const vm =
              reinterpret_cast<const uint32_t*>(g.v_max) + ((int64_t)rec->b * a.KV + rec->head / a.G) * a.ktiles;
          uint32_t v = 0;
          for (int k = lane; k < a.ktiles; k += 32) v = max(v, vm[k]);
          v = __reduce_max_sync(0xffffffffu, v);
          ds_mul = ds_factor(norm * __uint_as_float(v)) * g.v_scale;
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(norm));
          if (cq == 0 && lane == 0)
            g.do_max[(((int64_t)rec->b * a.H + rec->head) * g.qblocks + rec->i0 / kTile) * 4 + q4] = __uint_as_float(most);
        }
        st.doc = a.q_doc && i < a.Nq ? a.q_doc[(int64_t)rec->b * a.Nq + i] : 0;
        if (SHAPED) st.slope = a.slopes ? a.slopes[rec->head] * kLog2e : 0.f;
        e0 = e1 = 0.f;
      }
      const bool some = tile >= 0;
      if (some) {
        const int j0 = tile * kTile;
        st.sdoc = nullptr;
        if (a.k_pad && reads_docs(flags)) {
          st.sdoc = docs.get(r, alive);
          if (!alive) break;
        }
        if (!(alive = mbar_wait_all(s_full, t & 1, abort_flag, a.err))) break;
        tc_fence_after();
        st.to = (flags & kOneDoc) && rec->doc != st.doc ? 0 : lim - j0;
        st.p0 = (float)(j0 - pos);
        // With a cap dS needs P times the slope, and e needs P; both in FP32 would spill. BF16:
        // P, and the slope as FP16 pairs, off by 2^-11 of itself, an eighth of dS's own
        // rounding. FP16, whose dS is rounded no more than that: P times the slope, and the
        // rest of P as FP16 pairs, which go into nothing but e, the small correction
        // (head_dim 80: 203 us instead of 197 backward; BF16 would pay 8 of 190).
        constexpr bool kRest = f16 && SHAPED;
        float p[32];
        [[maybe_unused]] uint32_t side[SHAPED ? 16 : 1];
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          uint32_t q[16];
          float nl[16], other[16];
          tmem_ld_x16(tSr + e, q);
#pragma unroll
          for (int y = 0; y < 16; ++y) nl[y] = nlse;
          tmem_ld_wait_16(q);
          float *const all = kRest ? other : p + e, *const pf = kRest ? p + e : other;
          if (whole)
            probabilities<SHAPED, false, kRest>(a, st, q, c0 + e, nl, all, pf, SHAPED ? side + e / 2 : nullptr);
          else
            probabilities<SHAPED, true, kRest>(a, st, q, c0 + e, nl, all, pf, SHAPED ? side + e / 2 : nullptr);
          pack16<T>(pf, pk + e / 2);
          if (!Tm::kApart) tmem_st_x8(tPr + e / 2, pk + e / 2);  // over scores already read
        }
        if (Tm::kApart) {
          // P's columns are free once the last step's product is done
          if (t > 0 && !(alive = mbar_wait_all(pv_done, (t - 1) & 1, abort_flag, a.err))) break;
          tc_fence_after();
          tmem_st_x16(tPr, pk);
        }
        if (!whole && j0 + kTile > nk && nk < a.Nk) {
          // keys behind the last one count as zeros in the sums, whatever they hold (S of this tile is done)
          if (cq == 0 && j0 + row >= nk) {
#pragma unroll
            for (int c = 0; c < NB; ++c) {
              uint4* k = reinterpret_cast<uint4*>(sK + (t & 1) * kBytes + c * kBlockBytes + row * 128);
#pragma unroll
              for (int y = 0; y < 8; ++y) k[y] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_async_smem();
        }
        tmem_store_wait();
        tc_fence_before();
        mbar_arrive_warp(p_full);
        if (!(alive = mbar_wait_all(dp_full, t & 1, abort_flag, a.err))) break;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          uint32_t q[16];
          float nd[16], ds[16];
          tmem_ld_x16(tDpr + e, q);
#pragma unroll
          for (int y = 0; y < 16; ++y) nd[y] = ndelta;
          tmem_ld_wait_16(q);
          if constexpr (kRest) {
#pragma unroll
            for (int y = 0; y < 16; y += 2) {
              const uint32_t r = side[(e + y) / 2];
              float x0, x1, p0, p1;
              add2(__uint_as_float(q[y]), __uint_as_float(q[y + 1]), ndelta, ndelta, x0, x1);
              add2(p[e + y], p[e + y + 1], Elem<__half>::lo(r), Elem<__half>::hi(r), p0, p1);
              // dP of keys that do not exist may be anything
              if (!whole && p0 == 0.f) x0 = 0.f;
              if (!whole && p1 == 0.f) x1 = 0.f;
              fma2v(x0, x1, p0, p1, e0, e1, e0, e1);
              mul2(x0, x1, p[e + y], p[e + y + 1], ds[y], ds[y + 1]);
            }
          } else {
            if (whole)
              score_grads<false>(q, nd, p + e, ds);
            else
              score_grads<true>(q, nd, p + e, ds);
#pragma unroll
            for (int y = 0; y < 16; y += 2) add2(e0, e1, ds[y], ds[y + 1], e0, e1);
            if constexpr (SHAPED) {
#pragma unroll
              for (int y = 0; y < 16; y += 2)
                mul2(ds[y], ds[y + 1], Elem<__half>::lo(side[(e + y) / 2]), Elem<__half>::hi(side[(e + y) / 2]), ds[y],
                     ds[y + 1]);
            }
          }
          if constexpr (f16) {
#pragma unroll
            for (int y = 0; y < 16; y += 2) mul2(ds[y], ds[y + 1], ds_mul, ds_mul, ds[y], ds[y + 1]);
          }
          pack16<T>(ds, pk + e / 2);
          if (!Tm::kApart) tmem_st_x8(tDsr + e / 2, pk + e / 2);
        }
        if (Tm::kApart) {
          // dS's columns are free once the last step's dS product is done
          if (t > 0 && !(alive = mbar_wait_all(&kv_empty[(t - 1) & 1], ((t - 1) >> 1) & 1, abort_flag, a.err))) break;
          tc_fence_after();
          tmem_st_x16(tDsr, pk);
        }
        tmem_store_wait();
        tc_fence_before();
        mbar_arrive_warp(ds_full);
        ++t;
      }
      if (flags & kLast) {
        // the row sums of the four column quarters meet
        asm volatile("bar.sync 1, 512;" ::: "memory");
        srow[cq * kTile + row] = e0 + e1;
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (some && !(alive = mbar_wait_all(acc_done, n & 1, abort_flag, a.err))) break;
        n += some;
        tc_fence_after();
        // the accumulators are free for the next unit once they have been read: these threads
        // arrive at p_full only after that
        if (cq < 2) {
          const float e = (srow[row] + srow[kTile + row]) + (srow[2 * kTile + row] + srow[3 * kTile + row]);
          const int b = rec->b, h = rec->head, i = rec->i0 + row;
          const int64_t at = (int64_t)rec->slot * kTile + row;
          const bool part = rec->slot >= 0, valid = i < a.Nq;
          const float err = e * g.v_scale;
          if (valid && !part && cq == 0) g.ndelta[((int64_t)b * a.H + h) * g.qpad + i] = ndelta - err;
          // dS carries the row's factor, in BF16 kSlopeScale where it took the cap's slope
          store_dq<T, NB, !SHAPED, f16 || SHAPED>(static_cast<T*>(g.out0) + b * g.s0[0] + i * g.s0[1] + h * g.s0[2], wide,
                          part ? g.part + at * a.D : nullptr, g.part + (g.slots * kTile + at) * a.D, g.part_e + at, a.D,
                          g.out_scale, cq, tDq + lane_off, tPk + lane_off, some, valid, err,
                          f16 ? 1.f / ds_mul : 1.f / kSlopeScale);
        }
        tc_fence_before();
      }
      ring.done(r);
    }
    leave_barrier(abort_flag, left, kComputeWarps, 1);
  }
  settle(abort_flag);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// out = scale * sum of the parts of the cut items, in order; eight head dimensions per
// thread. For dQ (part_e given) the parts are dS K, and behind them P K, which the summed
// row error e multiplies; delta is corrected by e.
struct JoinArgs {
  Parts parts;
  const float* part;    // [2][slots][128][D]: dK and dV, or dS K and P K
  const float* part_e;  // [slots][128], or null
  float* ndelta;        // [B][heads][qpad]
  void* out[2];
  int64_t s[2][3], slots;
  float scale[2];
  int32_t sets, B, heads, rows, tiles, D;
};
template <typename T>
__global__ void __launch_bounds__(256) attn_grad_join_kernel(const __grid_constant__ JoinArgs a) {
  pdl_wait();
  pdl_trigger();
  const uint32_t vecs = (uint32_t)a.D / 8;
  const int64_t n = (int64_t)a.sets * a.parts.count * kTile * vecs;
  for (int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x) {
    const uint32_t at_row = (uint32_t)x / vecs;  // the plan keeps parts far below 2^32
    const int d = (int)((uint32_t)x - at_row * vecs) * 8, row = (int)(at_row % kTile), nth = (int)(at_row / kTile);
    const int set = nth >= a.parts.count, item = a.parts.first + nth - (set ? a.parts.count : 0);
    const int grp = a.parts.group_of_item(item), parts = a.parts.parts[grp];
    const int each = a.B * a.heads, b = item % each / a.heads, h = item % each % a.heads;
    const int i = (a.part_e ? a.tiles - 1 - item / each : item / each) * kTile + row;
    if (i >= a.rows) continue;
    const int64_t at = ((int64_t)a.parts.slot[grp] + (int64_t)(item - a.parts.item[grp]) * parts) * kTile + row;
    const int64_t step = (int64_t)kTile * a.D;
    float f[8];
    auto sum = [&](const float* q, float (&o)[8]) {
#pragma unroll
      for (int u = 0; u < 8; ++u) o[u] = 0.f;
#pragma unroll 4
      for (int z = 0; z < parts; ++z) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(q + z * step));
        const float4 w = __ldcg(reinterpret_cast<const float4*>(q + z * step) + 1);
        o[0] += v.x;
        o[1] += v.y;
        o[2] += v.z;
        o[3] += v.w;
        o[4] += w.x;
        o[5] += w.y;
        o[6] += w.z;
        o[7] += w.w;
      }
    };
    const float* p = a.part + at * a.D + d;
    sum(p + set * a.slots * step, f);
    if (a.part_e) {
      float e = 0.f, k[8];
      for (int z = 0; z < parts; ++z) e += __ldcg(a.part_e + at + (int64_t)z * kTile);
      sum(p + a.slots * step, k);
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] = fmaf(-e, k[u], f[u]);
      if (d == 0) a.ndelta[((int64_t)b * a.heads + h) * a.tiles * kTile + i] -= e;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] *= a.scale[set];
    const int64_t* s = a.s[set];
    *reinterpret_cast<uint4*>(static_cast<T*>(a.out[set]) + b * s[0] + i * s[1] + h * s[2] + d) = pack_vec<T, 8>(f);
  }
}

// ------------------------------------------------------------------ host side

struct GradPlan {
  int qblocks, ktiles, qpad;
  Cut dkv, dq;
  size_t rows_bytes, part_bytes;
  size_t do_max_bytes, v_max_bytes;  // FP16 (which has do_norm's rows too), else 0
};
// Time in steps of one SM, which holds one CTA: units start longest first and the last ones
// end about half the longest unit's steps after the average (of the cut ones where the rest
// are full rounds). Measured: a step takes 2.0 us at head_dim 64, 2.6 at 128, 1.3 more for
// capped scores, beginning and ending a unit 2.9 us more. Parts cost one more launch and
// their FP32 rows, written and joined at 2 TB/s.
Cut plan_cut(const sd_attention_cfg& c, int64_t items, double steps, double least, double total) {
  const double step_us = (c.head_dim <= 64 ? 2.0 : 2.6) + (c.softcap > 0.f ? 1.3 : 0.0);
  const double extra = 2.9 / step_us;
  Cut best;
  double best_t = 0;
  auto offer = [&](const Cut& cut, double longest) {
    longest = std::ceil(longest) + extra;
    const double units = (double)cut.units;
    double t = units <= kSms ? longest : std::max((total + extra * units) / kSms + 0.5 * longest, longest);
    if (cut.slots) t += (5.0 + cut.slots * kTile * c.head_dim * 16.0 / 2.0e6) / step_us;
    if (best_t == 0 || t < best_t) {
      best_t = t;
      best = cut;
    }
  };
  offer(cut_even(items, 1), steps);
  // whole items with a causal mask, two or fewer for each SM: a long one meets a short one
  if (c.causal && items > kSms && items <= 2 * kSms) {
    const double second = steps - (steps - least) * kSms / items;
    best_t = std::max(std::max(steps, 2 * second), total / kSms) + extra;
  }
  for (int s = 2; s <= kMaxSplits && 2 * s <= steps && items * s <= 16 * kSms; ++s) {
    offer(cut_even(items, s), steps / s);
    const int64_t rest = items % kSms;
    if (!c.causal && items > kSms && rest && rest * s <= 2 * kSms) offer(cut_last(items, rest, s), steps / s);
    if (c.causal && s <= kGroups) offer(cut_levels(items, s, steps, least), steps / s);
  }
  return best;
}
GradPlan plan_grad(const sd_attention_cfg& c) {
  GradPlan p;
  p.qblocks = (c.q_len + kTile - 1) / kTile;
  p.ktiles = (c.k_len + kTile - 1) / kTile;
  p.qpad = p.qblocks * kTile;
  const int64_t dkv_items = (int64_t)c.batch * c.kv_heads * p.ktiles, dq_items = (int64_t)c.batch * c.heads * p.qblocks;
  const double walk = (double)(c.heads / c.kv_heads) * p.qblocks, nq = c.q_len, nk = c.k_len;
  // with a causal mask the first key tiles see all queries, the last query tiles all keys
  const double seen = !c.causal ? 1.0 : nq <= nk ? 1.0 - nq / (2.0 * std::max(nk, 1.0)) : nk / (2.0 * nq);
  const double past = c.causal ? std::max(0.0, 1.0 - nk / std::max(nq, 1.0)) : 1.0;
  const double before = c.causal ? std::max(0.0, 1.0 - nq / std::max(nk, 1.0)) : 1.0;
  p.dkv = plan_cut(c, dkv_items, walk, walk * past, dkv_items * walk * seen);
  p.dq = plan_cut(c, dq_items, p.ktiles, p.ktiles * before, (double)dq_items * p.ktiles * seen);
  p.rows_bytes = up256((size_t)c.batch * c.heads * p.qpad * 4);
  const bool f16 = c.dtype == SD_DTYPE_F16;
  p.do_max_bytes = f16 ? up256((size_t)c.batch * c.heads * p.qblocks * 16) : 0;
  p.v_max_bytes = f16 ? up256((size_t)c.batch * c.kv_heads * p.ktiles * 4) : 0;
  p.part_bytes = up256(std::max((size_t)p.dkv.slots * 2 * kTile * c.head_dim * 4,
                                (size_t)p.dq.slots * kTile * (2 * c.head_dim + 1) * 4));
  return p;
}

template <typename T>
sd_status join(AttnCall& c, JoinArgs& j) {
  const int64_t n = (int64_t)j.sets * j.parts.count * kTile * (j.D / 8);
  const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, (int64_t)c.dev.sms * 8);
  return launched(launch_pdl(attn_grad_join_kernel<T>, dim3(blocks), dim3(256), 0, c.st, j));
}

template <typename T, int NB>
sd_status backward(AttnCall& c) {
  constexpr bool f16 = Elem<T>::kF16;
  const sd_attention_cfg& s = *c.cfg;
  const GradPlan p = plan_grad(s);
  GradArgs g;
  memset(&g, 0, sizeof(g));
  g.f = c.args;
  g.f.o = const_cast<void*>(c.o);
  g.qpad = p.qpad;
  g.qblocks = p.qblocks;
  g.nlse = reinterpret_cast<float*>(c.ws);
  g.ndelta = reinterpret_cast<float*>(c.ws + p.rows_bytes);
  uint8_t* w = c.ws + 2 * p.rows_bytes;
  if (f16) {
    g.do_norm = reinterpret_cast<float*>(w);
    g.do_max = reinterpret_cast<float*>(w += p.rows_bytes);
    g.v_max = reinterpret_cast<float*>(w += p.do_max_bytes);
    w += p.v_max_bytes;
  }
  g.part = reinterpret_cast<float*>(w);
  g.v = c.v;
  for (int i = 0; i < 3; ++i) g.vs[i] = c.vs[i];
  g.lse = c.lse;
  g.d_o = c.d_o;
  g.shift = f16 ? 15.f : 0.f;
  g.v_scale = exp2f(-g.shift);
  g.out_scale = c.args.sl2 / kLog2e * g.v_scale;

  // a map has no empty dimension: without queries (or keys) no tile of it is visited
  const void* any = s.q_len ? c.q : c.k;
  const int nq = std::max(s.q_len, 1), nk = std::max(s.k_len, 1);
  const int64_t unit[3] = {8 * ((s.head_dim + 7) / 8), 8 * ((s.head_dim + 7) / 8), 8 * ((s.head_dim + 7) / 8)};
  GradMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!attn_map(&maps.q, f16, s.q_len ? c.q : any, s.q_len ? c.qs : unit, s.batch, nq, s.heads, s.head_dim, 1, kTile) ||
      !attn_map(&maps.d_o, f16, s.q_len ? c.d_o : any, s.q_len ? c.os : unit, s.batch, nq, s.heads, s.head_dim, 1,
                kTile) ||
      !attn_map(&maps.k, f16, s.k_len ? c.k : any, s.k_len ? c.ks : unit, s.batch, nk, s.kv_heads, s.head_dim, 1,
                kTile) ||
      !attn_map(&maps.v, f16, s.k_len ? c.v : any, s.k_len ? c.vs : unit, s.batch, nk, s.kv_heads, s.head_dim, 1, kTile))
    return SD_ERR_LAUNCH;

  if (g.f.k_doc) OP_TRY(attn_doc_ranges(g.f, kTile, c.st));
  const double pairs = (double)s.batch * s.heads * s.q_len * s.k_len;
  const double act = 2.0 * s.batch * s.head_dim;
  if (s.q_len) {
    const int64_t rows = (int64_t)s.batch * s.heads * p.qpad;
    sdp::Scope sc("attn_delta", sdp::F_OTHER, 0, act * (2.0 * s.q_len * s.heads + (f16 ? s.k_len * s.kv_heads : 0)), c.st);
    int lanes = 0;
    while (8 << lanes < s.head_dim) ++lanes;
    const int64_t per = 4 * (256 >> lanes);
    g.row_ctas = (rows + per - 1) / per;
    const int64_t ctas = g.row_ctas + (f16 ? (int64_t)s.batch * s.kv_heads * p.ktiles : 0);
    OP_TRY(launched(launch_pdl(attn_delta_kernel<T>, dim3((unsigned)ctas), dim3(256), 0, c.st, g, lanes)));
  }
  if (!s.q_len) OP_TRY(launched(cudaMemsetAsync(c.args.err, 0, sizeof(int), c.st)));
  JoinArgs j;
  memset(&j, 0, sizeof(j));
  j.part = g.part;
  j.B = s.batch;
  j.D = s.head_dim;
  const bool shaped = g.f.cap_out != 0.f || g.f.slopes;
  if (s.q_len) {
    // dq first: it corrects delta
    g.f.parts = j.parts = p.dq.parts;
    g.f.hold_spins = injected_spins();
    g.slots = j.slots = p.dq.slots;
    g.part_e = g.part + (size_t)2 * g.slots * kTile * s.head_dim;
    for (int i = 0; i < 3; ++i) g.s0[i] = j.s[0][i] = c.qs[i];
    g.out0 = j.out[0] = c.dq;
    auto* kernel = shaped ? attn_dq_kernel<T, NB, true> : attn_dq_kernel<T, NB, false>;
    if (shaped)
      OP_TRY((allow_smem<attn_dq_kernel<T, NB, true>>(kDqSmem<NB>, c.dev.index)));
    else
      OP_TRY((allow_smem<attn_dq_kernel<T, NB, false>>(kDqSmem<NB>, c.dev.index)));
    {
      sdp::Scope sc("attn_dq", sdp::F_ATTN, 2.0 * pairs * s.head_dim,
                    act * (3.0 * s.q_len * s.heads + 2.0 * s.k_len * s.kv_heads), c.st);
      OP_TRY(launched(launch_pdl(kernel, dim3((unsigned)p.dq.units), dim3(kThreads),
                                 kDqSmem<NB>, c.st, maps, g)));
    }
    if (g.slots) {
      j.scale[0] = g.out_scale;
      j.sets = 1;
      j.heads = s.heads;
      j.rows = s.q_len;
      j.tiles = p.qblocks;
      j.part_e = g.part_e;
      j.ndelta = g.ndelta;
      sdp::Scope sc("attn_grad_join", sdp::F_OTHER, 0, 0, c.st);
      OP_TRY(join<T>(c, j));
    }
  }
  if (s.k_len) {
    g.f.parts = j.parts = p.dkv.parts;
    g.f.hold_spins = injected_spins();
    g.slots = j.slots = p.dkv.slots;
    for (int i = 0; i < 3; ++i) {
      g.s0[i] = j.s[0][i] = c.ks[i];
      g.s1[i] = j.s[1][i] = c.vs[i];
    }
    g.out0 = j.out[0] = c.dk;
    g.out1 = j.out[1] = c.dv;
    auto* kernel = shaped ? attn_dkv_kernel<T, NB, true> : attn_dkv_kernel<T, NB, false>;
    if (shaped)
      OP_TRY((allow_smem<attn_dkv_kernel<T, NB, true>>(kDkvSmem<NB>, c.dev.index)));
    else
      OP_TRY((allow_smem<attn_dkv_kernel<T, NB, false>>(kDkvSmem<NB>, c.dev.index)));
    {
      sdp::Scope sc("attn_dkv", sdp::F_ATTN, 8.0 * pairs * s.head_dim,
                    act * (2.0 * s.q_len * s.heads + 4.0 * s.k_len * s.kv_heads), c.st);
      OP_TRY(launched(launch_pdl(kernel, dim3((unsigned)p.dkv.units), dim3(kThreads),
                                 kDkvSmem<NB>, c.st, maps, g)));
    }
    if (g.slots) {
      j.scale[0] = g.out_scale;
      j.scale[1] = g.v_scale;
      j.sets = 2;
      j.part_e = nullptr;
      j.heads = s.kv_heads;
      j.rows = s.k_len;
      j.tiles = p.ktiles;
      sdp::Scope sc("attn_grad_join", sdp::F_OTHER, 0, 0, c.st);
      OP_TRY(join<T>(c, j));
    }
  }
  return SD_OK;
}

}  // namespace

size_t attn_grad_space(const sd_attention_cfg& c) {
  const GradPlan p = plan_grad(c);
  return (c.dtype == SD_DTYPE_F16 ? 3 : 2) * p.rows_bytes + p.do_max_bytes + p.v_max_bytes + p.part_bytes;
}

template <typename T>
sd_status attn_backward(AttnCall& c) {
  return c.cfg->head_dim > 64 ? backward<T, 2>(c) : backward<T, 1>(c);
}
template sd_status attn_backward<__half>(AttnCall&);
template sd_status attn_backward<__nv_bfloat16>(AttnCall&);

}  // namespace sdo
