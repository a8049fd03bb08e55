// Gradients of the attention operator. With P = exp(s - lse) recomputed tile by tile,
//   delta_i = sum_d dO_id O_id,  dP = dO V^T,  dS = P (dP - delta) (1 - tanh^2),
//   dV = P^T dO,  dK = scale dS^T Q (both summed over the heads that share a key head),
//   dQ = scale dS K.
//
// Bound by the tensor cores (10 D operations a pair in five products). Two kernels
// recompute S and dP each, seven products in all, so that every gradient is
// accumulated by one CTA in a fixed order: no atomics, results repeat bit for bit.
//   attn_dkv_kernel  a CTA owns 128 keys of one key head and walks the (head, query
//                    tile) pairs that may see them: S^T = K Q^T and dP^T = V dO^T
//                    have the keys as rows, so P^T and dS^T go from registers to
//                    TMEM as A operands of dV += P^T dO and dK += dS^T Q, and no
//                    transposed copy of anything is made
//   attn_dq_kernel   a CTA owns 128 queries of one head and walks the key tiles
// Few CTAs and a long walk: the walk is split and FP32 parts are joined in order.
//
// 320 threads, one CTA per SM: warps 0-7 turn scores into P and dS (two warps per
// TMEM lane quarter, half of the columns each), warp 8 loads by TMA, one thread of
// warp 9 issues the products. P and dS are rounded to the inputs' type (the tensor
// core takes no other); everything else is FP32. For FP16 inputs P carries a
// factor 2^shift (taken out of the results again) that keeps the small
// probabilities of long sequences above FP16's subnormals.
#include <string.h>

#include <algorithm>

#include "attention_op.cuh"
#include "profile.h"

namespace sdo {
namespace {

constexpr int kThreads = 320;
constexpr int kCompute = 256;
constexpr int kSms = 148;
constexpr int kMaxSplits = 32;

struct GradArgs {
  AttnArgs f;
  int32_t qpad;         // query rows of lse2 and delta: a multiple of 128
  int32_t qblocks;      // 128-query tiles
  float* lse2;          // [B][H][qpad] log2-domain sums, +inf where a row sees nothing or does not exist
  float* delta;         // [B][H][qpad]
  const float* lse;
  const void* d_o;
  float out_scale, v_scale;  // factors of dQ and dK, of dV
  float shift;
  int64_t s0[3], s1[3];      // output strides: dQ, or dK and dV
  void *out0, *out1;
  float* part;               // [splits][...] FP32 parts
};

struct __align__(64) GradMaps {
  CUtensorMap q, k, v, d_o;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// lse in log2 units and delta, 16 lanes per query row; rows up to qpad.
template <typename T>
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ GradArgs g) {
  pdl_wait();
  pdl_trigger();
  const AttnArgs& a = g.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
  const int sub = threadIdx.x & 15;
  const int64_t r = blockIdx.x * (int64_t)16 + (threadIdx.x >> 4);
  if (r >= (int64_t)a.B * a.H * g.qpad) return;
  const int i = (int)(r % g.qpad), h = (int)(r / g.qpad % a.H), b = (int)(r / g.qpad / a.H);
  float s = 0.f;
  if (i < a.Nq && sub * 8 < a.D) {
    const int64_t at = b * a.os[0] + i * a.os[1] + h * a.os[2] + sub * 8;
    float x[8], y[8];
    unpack_vec<T, 8>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.o) + at), x);
    unpack_vec<T, 8>(*reinterpret_cast<const uint4*>(static_cast<const T*>(g.d_o) + at), y);
#pragma unroll
    for (int u = 0; u < 8; ++u) s = fmaf(x[u], y[u], s);
  }
  const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(mask, s, o);
  if (sub == 0) {
    const float lse = i < a.Nq ? g.lse[((int64_t)b * a.H + h) * a.Nq + i] : -INFINITY;
    g.lse2[r] = lse == -INFINITY ? INFINITY : fmaf(lse, kLog2e, -g.shift);
    g.delta[r] = s;
  }
}

// Marks the tiles that the CTA visits; `base` rows against tiles of 128 columns.
template <typename F>
__device__ __forceinline__ void list_tiles(TileBits* tiles, int ntiles, int warp, int lane, F&& f) {
  const int words = (ntiles + 31) >> 5;
  for (int w = warp; w < words; w += kThreads / 32) {
    const int t = w * 32 + lane;
    bool see = false, all = false;
    if (t < ntiles) f(t, see, all);
    const uint32_t ms = __ballot_sync(0xffffffffu, see), ma = __ballot_sync(0xffffffffu, see && all);
    if (lane == 0) {
      tiles->see[w] = ms;
      tiles->all[w] = ma;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int w = lane; w < words; w += 32) n += __popc(tiles->see[w]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) tiles->count = n;
  }
  __syncthreads();
}

// The score in log2 units and the cap's slope, without the bias.
__device__ __forceinline__ float score(const AttnArgs& a, float s, float& fac) {
  if (a.cap_out != 0.f) {
    const float t = tanh_acc(s * a.cap_in);
    fac = fmaf(-t, t, 1.f);
    return a.cap_out * t;
  }
  fac = 1.f;
  return s * a.sl2;
}

// One row of an accumulator: to the output (scaled), or to the FP32 part.
template <typename T, int NB>
__device__ __forceinline__ void store_row(uint32_t tacc, bool have, bool in, int D, float scale, T* dst, float* part) {
#pragma unroll 1
  for (int c = 0; c < NB * 64; c += 32) {
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
    if (part) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c + 4 * u < D)
          __stcg(reinterpret_cast<float4*>(part + c) + u,
                 make_float4(__uint_as_float(r[4 * u]), __uint_as_float(r[4 * u + 1]), __uint_as_float(r[4 * u + 2]),
                             __uint_as_float(r[4 * u + 3])));
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + 8 * u < D)
          *reinterpret_cast<uint4*>(dst + c + 8 * u) = make_uint4(
              Elem<T>::pack(__uint_as_float(r[8 * u]) * scale, __uint_as_float(r[8 * u + 1]) * scale),
              Elem<T>::pack(__uint_as_float(r[8 * u + 2]) * scale, __uint_as_float(r[8 * u + 3]) * scale),
              Elem<T>::pack(__uint_as_float(r[8 * u + 4]) * scale, __uint_as_float(r[8 * u + 5]) * scale),
              Elem<T>::pack(__uint_as_float(r[8 * u + 6]) * scale, __uint_as_float(r[8 * u + 7]) * scale));
    }
  }
}

constexpr size_t kTailBytes = sizeof(TileBits) + 512 + 256;  // tile list, documents, barriers

template <int NB>
constexpr size_t kDkvSmem = 1024 + (size_t)6 * NB * kBlockBytes + 2048 + kTailBytes;
template <int NB>
constexpr size_t kDqSmem = 1024 + (size_t)6 * NB * kBlockBytes + kTailBytes;

// TMEM: S^T [0,128), dP^T [128,256), dK [256,384), dV [384,512). P^T and dS^T lie over
// their scores: columns [0,32) hold queries [0,64), columns [64,96) queries [64,128), so
// that the two warps of a lane quarter never write where the other still reads.
template <typename T, int NB>
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
  float* sstat = reinterpret_cast<float*>(sDo + 2 * kBytes);  // [2][lse2 128 | delta 128]
  TileBits* tiles = reinterpret_cast<TileBits*>(sstat + 512);
  int32_t* sdoc = reinterpret_cast<int32_t*>(tiles + 1);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sdoc) + 512);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;   // [2]
  uint64_t* q_empty = bars + 3;  // [2]
  uint64_t* s_full = bars + 5;
  uint64_t* dp_full = bars + 6;
  uint64_t* acc_done = bars + 7;
  uint64_t* p_full = bars + 8;
  uint64_t* ds_full = bars + 9;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 10);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int z = blockIdx.x % a.splits, item = blockIdx.x / a.splits;
  const int heads = a.B * a.KV;
  const int kt = item / heads;  // the first key tiles first (with a causal mask they have the longest walks)
  const int b = item % heads / a.KV, kv = item % heads % a.KV;
  const int j0 = kt * kTile;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 10; ++i) mbar_init(bars + i, i >= 8 ? kCompute : 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.d_o);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tDp = tmem + 128, tDk = tmem + 256, tDv = tmem + 384;
  pdl_wait();
  pdl_trigger();

  const int nk = keys_of(a, b), off = nk - a.Nq, pre = prefix_of(a, b);
  int32_t klo = 0, khi = 0;
  if (a.k_range) {
    klo = a.k_range[((int64_t)b * a.ktiles + kt) * 2];
    khi = a.k_range[((int64_t)b * a.ktiles + kt) * 2 + 1];
  }
  list_tiles(tiles, g.qblocks, warp, lane, [&](int t, bool& see, bool& all) {
    const int i0 = t * kTile, i1 = min(a.Nq, i0 + kTile) - 1;
    see = j0 < nk && (!a.causal || j0 <= max(i1 + off, pre - 1));
    all = j0 + kTile <= nk && (!a.causal || j0 + kTile - 1 <= max(i0 + off, pre - 1));
    if (see && a.q_range) {
      const int32_t lo = a.q_range[((int64_t)b * g.qblocks + t) * 2], hi = a.q_range[((int64_t)b * g.qblocks + t) * 2 + 1];
      see = lo <= khi && klo <= hi;
      all = all && lo == hi && klo == lo && khi == lo;
    }
  });
  const int count = tiles->count;
  const int64_t total = (int64_t)count * a.G;
  const int64_t first = total * z / a.splits;
  const int steps = (int)(total * (z + 1) / a.splits - first);
  // the walk over (head of the group, query tile)
  struct Walk {
    TileWalk w;
    int hh, left;
  };
  auto begin = [&](Walk& w) {
    w.hh = (int)(first / count);
    const int r = (int)(first % count);
    w.left = count - r;
    w.w.start(tiles, g.qblocks, r);
  };
  auto next = [&](Walk& w) {
    if (w.left == 0) {
      ++w.hh;
      w.left = count;
      w.w.start(tiles, g.qblocks, 0);
    }
    --w.left;
    return w.w.next();
  };

  if (warp == 8) {
    if (lane == 0 && steps > 0) {
      Walk w;
      begin(w);
      mbar_arrive_expect_tx(kv_full, 2 * kBytes);
      for (int c = 0; c < NB; ++c) {
        tma_load_4d(sK + c * kBlockBytes, &maps.k, kv_full, c * 64, kv, j0, b);
        tma_load_4d(sV + c * kBlockBytes, &maps.v, kv_full, c * 64, kv, j0, b);
      }
      for (int t = 0; t < steps; ++t) {
        const int i0 = next(w) * kTile, s = t & 1;
        const int h = kv * a.G + w.hh;
        if (t >= 2 && !mbar_wait(&q_empty[s], ((t >> 1) - 1) & 1, abort_flag, a.err)) break;
        mbar_arrive_expect_tx(&q_full[s], 2 * kBytes + 1024);
        for (int c = 0; c < NB; ++c) {
          tma_load_4d(sQ + s * kBytes + c * kBlockBytes, &maps.q, &q_full[s], c * 64, h, i0, b);
          tma_load_4d(sDo + s * kBytes + c * kBlockBytes, &maps.d_o, &q_full[s], c * 64, h, i0, b);
        }
        const int64_t at = ((int64_t)b * a.H + h) * g.qpad + i0;
        bulk_load(sstat + s * 256, g.lse2 + at, 512, &q_full[s]);
        bulk_load(sstat + s * 256 + 128, g.delta + at, 512, &q_full[s]);
      }
    }
  } else if (warp == 9) {
    if (lane == 0 && steps > 0) {
      const int nd = (a.D + 15) >> 4;
      const uint32_t id_s = idesc_f16(128, 128, f16, false, false);
      const uint32_t id_o = idesc_f16(128, nd * 16, f16, false, true);
      const uint32_t k0 = smem_u32(sK), v0 = smem_u32(sV);
      // S^T = K Q^T and dP^T = V dO^T
      auto scores = [&](uint32_t d, uint32_t x0, uint32_t y0, uint64_t* bar) {
        for (int n = 0; n < nd; ++n) {
          const uint32_t o = (n >> 2) * kBlockBytes + (n & 3) * 32;
          umma_bf16(d, umma_desc_k_sw128(x0 + o), umma_desc_k_sw128(y0 + o), id_s, n > 0);
        }
        umma_commit(bar);
      };
      // acc += A^T-form operand over the scores x 128 query rows of y
      auto accumulate = [&](uint32_t d, uint32_t x, uint32_t y0, bool more) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ts(d, x + (k >> 2) * 64 + (k & 3) * 8, umma_desc_mn(y0 + k * 2048, kBlockBytes), id_o,
                  (more || k > 0) ? 1u : 0u);
      };
      bool ok = mbar_wait(kv_full, 0, abort_flag, a.err) && mbar_wait(&q_full[0], 0, abort_flag, a.err);
      if (ok) {
        tc_fence_after();
        scores(tS, k0, smem_u32(sQ), s_full);
        scores(tDp, v0, smem_u32(sDo), dp_full);
      }
      for (int t = 0; t < steps && ok; ++t) {
        const int s = t & 1, s1 = s ^ 1;
        const bool more = t + 1 < steps;
        if (!(ok = mbar_wait(p_full, t & 1, abort_flag, a.err))) break;
        tc_fence_after();
        accumulate(tDv, tS, smem_u32(sDo + s * kBytes), t > 0);
        if (more) {
          if (!(ok = mbar_wait(&q_full[s1], ((t + 1) >> 1) & 1, abort_flag, a.err))) break;
          tc_fence_after();
          scores(tS, k0, smem_u32(sQ + s1 * kBytes), s_full);  // over P^T, whose product was issued before
        }
        if (!(ok = mbar_wait(ds_full, t & 1, abort_flag, a.err))) break;
        tc_fence_after();
        accumulate(tDk, tDp, smem_u32(sQ + s * kBytes), t > 0);
        umma_commit(&q_empty[s]);
        if (more) scores(tDp, v0, smem_u32(sDo + s1 * kBytes), dp_full);
      }
      if (ok) umma_commit(acc_done);
    }
  } else {
    const int q4 = warp & 3, half = warp >> 2;
    const int row = q4 * 32 + lane, j = j0 + row;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int doc = a.k_doc && j < a.Nk ? a.k_doc[(int64_t)b * a.Nk + j] : 0;
    Walk w;
    if (steps > 0) begin(w);
    bool alive = true;
    for (int t = 0; t < steps; ++t) {
      const int tile = next(w), i0 = tile * kTile, s = t & 1;
      const bool whole = w.w.whole(tile);
      const float slope = a.slopes ? a.slopes[kv * a.G + w.hh] * kLog2e : 0.f;
      const float* st = sstat + s * 256 + half * 64;
      const bool docs = !whole && a.q_doc;
      if (docs) {
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (half == 0) sdoc[row] = i0 + row < a.Nq ? a.q_doc[(int64_t)b * a.Nq + i0 + row] : 0;
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      if (!(alive = mbar_wait_all(&q_full[s], (t >> 1) & 1, abort_flag, a.err) &&
                    mbar_wait_all(s_full, t & 1, abort_flag, a.err)))
        break;
      tc_fence_after();
      // queries of this tile from column `from` on see the key (none when it does not exist)
      const int from = j >= nk ? kTile : a.causal && j >= pre ? j - off - i0 : 0;
      const float p0 = (float)(i0 + off - j);
      float pf[64];
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t r[32], pk[16];
        tmem_ld_32x32b_x32(tS + lane_off + half * 64 + c0, r);
        tmem_ld_wait_regs(r);
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
          const float4 ls = *reinterpret_cast<const float4*>(st + c0 + u);
          const float lv[4] = {ls.x, ls.y, ls.z, ls.w};
          int4 qd = make_int4(0, 0, 0, 0);
          if (docs) qd = *reinterpret_cast<const int4*>(sdoc + half * 64 + c0 + u);
          const int dv[4] = {qd.x, qd.y, qd.z, qd.w};
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = half * 64 + c0 + u + e;
            float fac;
            float x = score(a, __uint_as_float(r[u + e]), fac);
            if (a.slopes) x = fmaf(-slope, fabsf(p0 + (float)c), x);
            p[e] = fast_ex2(x - lv[e]);
            if (!whole && (c < from || (docs && dv[e] != doc))) p[e] = 0.f;
            pf[c0 + u + e] = p[e] * fac;
          }
          pk[u / 2] = Elem<T>::pack(p[0], p[1]);
          pk[u / 2 + 1] = Elem<T>::pack(p[2], p[3]);
        }
        // queries [64 half + c0, +32) as 16 packed columns; c0 = 32 goes over scores already read
        tmem_st_x16(tS + lane_off + half * 64 + c0 / 2, pk);
      }
      tmem_store_wait();
      tc_fence_before();
      mbar_arrive(p_full);
      if (!(alive = mbar_wait_all(dp_full, t & 1, abort_flag, a.err))) break;
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t r[32], pk[16];
        tmem_ld_32x32b_x32(tDp + lane_off + half * 64 + c0, r);
        tmem_ld_wait_regs(r);
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
          const float4 de = *reinterpret_cast<const float4*>(st + 128 + c0 + u);
          const float dl[4] = {de.x, de.y, de.z, de.w};
          float ds[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = pf[c0 + u + e];
            ds[e] = p * (__uint_as_float(r[u + e]) - dl[e]);
            if (!whole && p == 0.f) ds[e] = 0.f;  // dP of keys that do not exist may be anything
          }
          pk[u / 2] = Elem<T>::pack(ds[0], ds[1]);
          pk[u / 2 + 1] = Elem<T>::pack(ds[2], ds[3]);
        }
        tmem_st_x16(tDp + lane_off + half * 64 + c0 / 2, pk);
      }
      tmem_store_wait();
      tc_fence_before();
      mbar_arrive(ds_full);
    }
    if (alive && steps > 0) alive = mbar_wait_all(acc_done, 0, abort_flag, a.err);
    tc_fence_after();
    if (alive) {
      // half 0 writes dK, half 1 dV
      const int64_t* st = half ? g.s1 : g.s0;
      T* dst = static_cast<T*>(half ? g.out1 : g.out0) + b * st[0] + j * st[1] + kv * st[2];
      float* part = nullptr;
      if (a.splits > 1)
        part = g.part + ((((int64_t)z * 2 + half) * heads + b * a.KV + kv) * a.ktiles * kTile + j) * a.D;
      store_row<T, NB>((half ? tDv : tDk) + lane_off, steps > 0, j < a.Nk, a.D, half ? g.v_scale : g.out_scale, dst,
                       part);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// TMEM: S [0,128), dP [128,256) with dS over it, dQ [256,384).
template <typename T, int NB>
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
  TileBits* tiles = reinterpret_cast<TileBits*>(sV + 2 * kBytes);
  int32_t* sdoc = reinterpret_cast<int32_t*>(tiles + 1);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sdoc) + 512);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 1;   // [2]
  uint64_t* kv_empty = bars + 3;  // [2]
  uint64_t* s_full = bars + 5;
  uint64_t* dp_full = bars + 6;
  uint64_t* acc_done = bars + 7;
  uint64_t* s_free = bars + 8;
  uint64_t* ds_full = bars + 9;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 10);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int z = blockIdx.x % a.splits, item = blockIdx.x / a.splits;
  const int heads = a.B * a.H;
  const int qt = g.qblocks - 1 - item / heads;
  const int b = item % heads / a.H, h = item % heads % a.H, kv = h / a.G;
  const int i0 = qt * kTile, i1 = min(a.Nq, i0 + kTile) - 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 10; ++i) mbar_init(bars + i, i >= 8 ? kCompute : 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.d_o);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tDp = tmem + 128, tDq = tmem + 256;
  pdl_wait();
  pdl_trigger();

  const int nk = keys_of(a, b), off = nk - a.Nq, pre = prefix_of(a, b);
  const int lim_any = a.causal ? min(nk, max(i1 + off + 1, pre)) : nk;
  const int lim_all = a.causal ? min(nk, max(i0 + off + 1, pre)) : nk;
  int32_t qlo = 0, qhi = 0;
  if (a.q_range) {
    qlo = a.q_range[((int64_t)b * g.qblocks + qt) * 2];
    qhi = a.q_range[((int64_t)b * g.qblocks + qt) * 2 + 1];
  }
  list_tiles(tiles, a.ktiles, warp, lane, [&](int t, bool& see, bool& all) {
    see = t * kTile < lim_any;
    all = (t + 1) * kTile <= lim_all;
    if (see && a.k_range) {
      const int32_t lo = a.k_range[((int64_t)b * a.ktiles + t) * 2], hi = a.k_range[((int64_t)b * a.ktiles + t) * 2 + 1];
      see = lo <= qhi && qlo <= hi;
      all = all && lo == hi && qlo == lo && qhi == lo;
    }
  });
  const int first = (int)((int64_t)tiles->count * z / a.splits);
  const int steps = (int)((int64_t)tiles->count * (z + 1) / a.splits) - first;

  if (warp == 8) {
    if (lane == 0 && steps > 0) {
      TileWalk w;
      w.start(tiles, a.ktiles, first);
      mbar_arrive_expect_tx(q_full, 2 * kBytes);
      for (int c = 0; c < NB; ++c) {
        tma_load_4d(sQ + c * kBlockBytes, &maps.q, q_full, c * 64, h, i0, b);
        tma_load_4d(sDo + c * kBlockBytes, &maps.d_o, q_full, c * 64, h, i0, b);
      }
      for (int t = 0; t < steps; ++t) {
        const int j = w.next() * kTile, s = t & 1;
        if (t >= 2 && !mbar_wait(&kv_empty[s], ((t >> 1) - 1) & 1, abort_flag, a.err)) break;
        mbar_arrive_expect_tx(&kv_full[s], 2 * kBytes);
        for (int c = 0; c < NB; ++c) {
          tma_load_4d(sK + s * kBytes + c * kBlockBytes, &maps.k, &kv_full[s], c * 64, kv, j, b);
          tma_load_4d(sV + s * kBytes + c * kBlockBytes, &maps.v, &kv_full[s], c * 64, kv, j, b);
        }
      }
    }
  } else if (warp == 9) {
    if (lane == 0 && steps > 0) {
      const int nd = (a.D + 15) >> 4;
      const uint32_t id_s = idesc_f16(128, 128, f16, false, false);
      const uint32_t id_o = idesc_f16(128, nd * 16, f16, false, true);
      const uint32_t q0 = smem_u32(sQ), d0 = smem_u32(sDo);
      auto scores = [&](uint32_t d, uint32_t x0, uint32_t y0, uint64_t* bar) {
        for (int n = 0; n < nd; ++n) {
          const uint32_t o = (n >> 2) * kBlockBytes + (n & 3) * 32;
          umma_bf16(d, umma_desc_k_sw128(x0 + o), umma_desc_k_sw128(y0 + o), id_s, n > 0);
        }
        umma_commit(bar);
      };
      bool ok = mbar_wait(q_full, 0, abort_flag, a.err) && mbar_wait(&kv_full[0], 0, abort_flag, a.err);
      if (ok) {
        tc_fence_after();
        scores(tS, q0, smem_u32(sK), s_full);
        scores(tDp, d0, smem_u32(sV), dp_full);
      }
      for (int t = 0; t < steps && ok; ++t) {
        const int s = t & 1, s1 = s ^ 1;
        const bool more = t + 1 < steps;
        if (more) {
          if (!(ok = mbar_wait(s_free, t & 1, abort_flag, a.err) &&
                     mbar_wait(&kv_full[s1], ((t + 1) >> 1) & 1, abort_flag, a.err)))
            break;
          tc_fence_after();
          scores(tS, q0, smem_u32(sK + s1 * kBytes), s_full);
        }
        if (!(ok = mbar_wait(ds_full, t & 1, abort_flag, a.err))) break;
        tc_fence_after();
        const uint32_t k0 = smem_u32(sK + s * kBytes);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ts(tDq, tDp + (k >> 2) * 64 + (k & 3) * 8, umma_desc_mn(k0 + k * 2048, kBlockBytes), id_o,
                  (t > 0 || k > 0) ? 1u : 0u);
        umma_commit(&kv_empty[s]);
        if (more) scores(tDp, d0, smem_u32(sV + s1 * kBytes), dp_full);
      }
      if (ok) umma_commit(acc_done);
    }
  } else {
    const int q4 = warp & 3, half = warp >> 2;
    const int row = q4 * 32 + lane, i = i0 + row;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const bool valid = i < a.Nq;
    const int64_t at = ((int64_t)b * a.H + h) * g.qpad + i;
    const float lse2 = g.lse2[at], delta = g.delta[at];
    const int pos = i + off;
    const int lim = a.causal ? min(nk, max(pos + 1, pre)) : nk;
    const int doc = a.q_doc && valid ? a.q_doc[(int64_t)b * a.Nq + i] : 0;
    const float slope = a.slopes ? a.slopes[h] * kLog2e : 0.f;
    TileWalk w;
    if (steps > 0) w.start(tiles, a.ktiles, first);
    bool alive = true;
    for (int t = 0; t < steps; ++t) {
      const int tile = w.next(), j0 = tile * kTile, s = t & 1;
      const bool whole = w.whole(tile);
      const bool docs = !whole && a.k_doc;
      if (docs) {
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (half == 0) sdoc[row] = j0 + row < a.Nk ? a.k_doc[(int64_t)b * a.Nk + j0 + row] : 0;
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      if (!(alive = mbar_wait_all(s_full, t & 1, abort_flag, a.err))) break;
      tc_fence_after();
      const int lc = lim - j0;
      const float p0 = (float)(pos - j0);
      float pf[64];
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tS + lane_off + half * 64 + c0, r);
        tmem_ld_wait_regs(r);
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
          int4 kd = make_int4(0, 0, 0, 0);
          if (docs) kd = *reinterpret_cast<const int4*>(sdoc + half * 64 + c0 + u);
          const int dv[4] = {kd.x, kd.y, kd.z, kd.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = half * 64 + c0 + u + e;
            float fac;
            float x = score(a, __uint_as_float(r[u + e]), fac);
            if (a.slopes) x = fmaf(-slope, fabsf(p0 - (float)c), x);
            float p = fast_ex2(x - lse2) * fac;
            if (!whole && (c >= lc || (docs && dv[e] != doc))) p = 0.f;
            pf[c0 + u + e] = p;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(s_free);
      if (!whole && j0 + kTile > nk && nk < a.Nk) {
        // keys behind the last one count as zeros in dS K, whatever they hold (S of this tile is done)
        if (half == 0 && j0 + row >= nk) {
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            uint4* p = reinterpret_cast<uint4*>(sK + s * kBytes + c * kBlockBytes + row * 128);
#pragma unroll
            for (int u = 0; u < 8; ++u) p[u] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_async_smem();
      }
      if (!(alive = mbar_wait_all(dp_full, t & 1, abort_flag, a.err))) break;
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t r[32], pk[16];
        tmem_ld_32x32b_x32(tDp + lane_off + half * 64 + c0, r);
        tmem_ld_wait_regs(r);
#pragma unroll
        for (int u = 0; u < 32; u += 2) {
          float ds[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p = pf[c0 + u + e];
            ds[e] = p * (__uint_as_float(r[u + e]) - delta);
            if (!whole && p == 0.f) ds[e] = 0.f;  // dP of keys that do not exist may be anything
          }
          pk[u / 2] = Elem<T>::pack(ds[0], ds[1]);
        }
        tmem_st_x16(tDp + lane_off + half * 64 + c0 / 2, pk);
      }
      tmem_store_wait();
      tc_fence_before();
      mbar_arrive(ds_full);
    }
    if (alive && steps > 0) alive = mbar_wait_all(acc_done, 0, abort_flag, a.err);
    tc_fence_after();
    if (alive && half == 0) {
      T* dst = static_cast<T*>(g.out0) + b * g.s0[0] + i * g.s0[1] + h * g.s0[2];
      float* part = nullptr;
      if (a.splits > 1) part = g.part + (((int64_t)z * heads + b * a.H + h) * g.qpad + i) * a.D;
      store_row<T, NB>(tDq + lane_off, steps > 0, valid, a.D, g.out_scale, dst, part);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// out = scale * sum of the parts, in order; eight head dimensions per thread.
struct JoinArgs {
  const float* part;   // [splits][sets][B][heads][rows_pad][D]
  void* out[2];
  int64_t s[2][3];
  float scale[2];
  int32_t splits, sets, B, heads, rows, rows_pad, D;
};
template <typename T>
__global__ void __launch_bounds__(256) attn_grad_join_kernel(const __grid_constant__ JoinArgs a) {
  pdl_wait();
  pdl_trigger();
  const int vecs = a.D / 8;
  const int64_t n = (int64_t)a.sets * a.B * a.heads * a.rows * vecs;
  const int64_t stride = (int64_t)a.sets * a.B * a.heads * a.rows_pad * a.D;
  for (int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x) {
    const int d = (int)(x % vecs) * 8;
    const int64_t r = x / vecs;
    const int i = (int)(r % a.rows), h = (int)(r / a.rows % a.heads);
    const int b = (int)(r / a.rows / a.heads % a.B), set = (int)(r / a.rows / a.heads / a.B);
    const float* p = a.part + ((((int64_t)set * a.B + b) * a.heads + h) * a.rows_pad + i) * a.D + d;
    float f[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] = 0.f;
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + z * stride));
      const float4 w = __ldcg(reinterpret_cast<const float4*>(p + z * stride) + 1);
      f[0] += v.x;
      f[1] += v.y;
      f[2] += v.z;
      f[3] += v.w;
      f[4] += w.x;
      f[5] += w.y;
      f[6] += w.z;
      f[7] += w.w;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] *= a.scale[set];
    const int64_t* s = a.s[set];
    *reinterpret_cast<uint4*>(static_cast<T*>(a.out[set]) + b * s[0] + i * s[1] + h * s[2] + d) = pack_vec<T, 8>(f);
  }
}

// ------------------------------------------------------------------ host side

struct GradPlan {
  int qblocks, ktiles, qpad, dkv_splits, dq_splits;
  int64_t dkv_items, dq_items;
  size_t rows_bytes, part_bytes;
};
GradPlan plan_grad(const sd_attention_cfg& c) {
  GradPlan p;
  p.qblocks = (c.q_len + kTile - 1) / kTile;
  p.ktiles = (c.k_len + kTile - 1) / kTile;
  p.qpad = p.qblocks * kTile;
  p.dkv_items = (int64_t)c.batch * c.kv_heads * p.ktiles;
  p.dq_items = (int64_t)c.batch * c.heads * p.qblocks;
  // split a walk while every part keeps two tiles and all parts fit on the GPU at once
  const int64_t walk = (int64_t)(c.heads / c.kv_heads) * p.qblocks;
  auto splits = [](int64_t items, int64_t steps) {
    const int64_t s = std::min<int64_t>(std::min<int64_t>(kSms / std::max<int64_t>(items, 1), steps / 2), kMaxSplits);
    return (int)std::max<int64_t>(s, 1);
  };
  p.dkv_splits = splits(p.dkv_items, walk);
  p.dq_splits = splits(p.dq_items, p.ktiles);
  p.rows_bytes = up256((size_t)c.batch * c.heads * p.qpad * 4);
  const size_t dkv = p.dkv_splits > 1 ? (size_t)p.dkv_splits * 2 * p.dkv_items * kTile * c.head_dim * 4 : 0;
  const size_t dq = p.dq_splits > 1 ? (size_t)p.dq_splits * p.dq_items * kTile * c.head_dim * 4 : 0;
  p.part_bytes = up256(std::max(dkv, dq));
  return p;
}

template <typename T>
sd_status join(AttnCall& c, JoinArgs& j) {
  const int64_t n = (int64_t)j.sets * j.B * j.heads * j.rows * (j.D / 8);
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
  g.lse2 = reinterpret_cast<float*>(c.ws);
  g.delta = reinterpret_cast<float*>(c.ws + p.rows_bytes);
  g.part = reinterpret_cast<float*>(c.ws + 2 * p.rows_bytes);
  g.lse = c.lse;
  g.d_o = c.d_o;
  if (f16)
    while (s.k_len >> ((int)g.shift + 11)) g.shift += 1.f;  // P 2^shift <= 1024
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

  if (g.f.k_doc && s.k_len) OP_TRY(attn_doc_ranges(g.f.k_doc, s.batch, s.k_len, const_cast<int32_t*>(g.f.k_range), c.st));
  if (g.f.q_doc && s.q_len) OP_TRY(attn_doc_ranges(g.f.q_doc, s.batch, s.q_len, const_cast<int32_t*>(g.f.q_range), c.st));
  const double pairs = (double)s.batch * s.heads * s.q_len * s.k_len;
  const double act = 2.0 * s.batch * s.head_dim;
  if (s.q_len) {
    const int64_t rows = (int64_t)s.batch * s.heads * p.qpad;
    sdp::Scope sc("attn_delta", sdp::F_OTHER, 0, 2 * act * s.q_len * s.heads, c.st);
    OP_TRY(launched(launch_pdl(attn_delta_kernel<T>, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, c.st, g)));
  }
  if (!s.q_len) OP_TRY(launched(cudaMemsetAsync(c.args.err, 0, sizeof(int), c.st)));
  JoinArgs j;
  memset(&j, 0, sizeof(j));
  j.part = g.part;
  j.B = s.batch;
  j.D = s.head_dim;
  if (s.k_len) {
    g.f.splits = p.dkv_splits;
    for (int i = 0; i < 3; ++i) {
      g.s0[i] = j.s[0][i] = c.ks[i];
      g.s1[i] = j.s[1][i] = c.vs[i];
    }
    g.out0 = j.out[0] = c.dk;
    g.out1 = j.out[1] = c.dv;
    OP_TRY((allow_smem<attn_dkv_kernel<T, NB>>(kDkvSmem<NB>, c.dev.index)));
    {
      sdp::Scope sc("attn_dkv", sdp::F_ATTN, 8.0 * pairs * s.head_dim,
                    act * (2.0 * s.q_len * s.heads + 4.0 * s.k_len * s.kv_heads), c.st);
      OP_TRY(launched(launch_pdl(attn_dkv_kernel<T, NB>, dim3((unsigned)(p.dkv_items * p.dkv_splits)), dim3(kThreads),
                                 kDkvSmem<NB>, c.st, maps, g)));
    }
    if (p.dkv_splits > 1) {
      j.scale[0] = g.out_scale;
      j.scale[1] = g.v_scale;
      j.splits = p.dkv_splits;
      j.sets = 2;
      j.heads = s.kv_heads;
      j.rows = s.k_len;
      j.rows_pad = p.ktiles * kTile;
      sdp::Scope sc("attn_grad_join", sdp::F_OTHER, 0, 0, c.st);
      OP_TRY(join<T>(c, j));
    }
  }
  if (s.q_len) {
    g.f.splits = p.dq_splits;
    for (int i = 0; i < 3; ++i) g.s0[i] = j.s[0][i] = c.qs[i];
    g.out0 = j.out[0] = c.dq;
    OP_TRY((allow_smem<attn_dq_kernel<T, NB>>(kDqSmem<NB>, c.dev.index)));
    {
      sdp::Scope sc("attn_dq", sdp::F_ATTN, 2.0 * pairs * s.head_dim,
                    act * (3.0 * s.q_len * s.heads + 2.0 * s.k_len * s.kv_heads), c.st);
      OP_TRY(launched(launch_pdl(attn_dq_kernel<T, NB>, dim3((unsigned)(p.dq_items * p.dq_splits)), dim3(kThreads),
                                 kDqSmem<NB>, c.st, maps, g)));
    }
    if (p.dq_splits > 1) {
      j.scale[0] = g.out_scale;
      j.splits = p.dq_splits;
      j.sets = 1;
      j.heads = s.heads;
      j.rows = s.q_len;
      j.rows_pad = p.qpad;
      sdp::Scope sc("attn_grad_join", sdp::F_OTHER, 0, 0, c.st);
      OP_TRY(join<T>(c, j));
    }
  }
  return SD_OK;
}

}  // namespace

size_t attn_grad_space(const sd_attention_cfg& c) {
  const GradPlan p = plan_grad(c);
  return 2 * p.rows_bytes + p.part_bytes;
}

template <typename T>
sd_status attn_backward(AttnCall& c) {
  return c.cfg->head_dim > 64 ? backward<T, 2>(c) : backward<T, 1>(c);
}
template sd_status attn_backward<__half>(AttnCall&);
template sd_status attn_backward<__nv_bfloat16>(AttnCall&);

}  // namespace sdo
