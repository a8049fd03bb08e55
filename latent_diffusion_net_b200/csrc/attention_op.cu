// Attention with capped scores, a distance bias, documents, a prefix and key
// lengths: o = softmax(mask(cap(scale q k^T) - slope |p - j|)) v, one pass over the
// keys with a running maximum and sum. The backward kernels are in attention_grad.cu.
//
// Bound by the exponentials and the tensor cores for long sequences (4 D
// operations and one exponential a pair; three with a cap), by reading keys and
// values for single tokens.
//
// A CTA owns 128 query rows: kTile / G tokens with the G query heads that share a
// key head, so a key tile is read once for all of them. It lists the key tiles
// that its rows may see (length, causal limit with prefix, document ranges) as
// bits in shared memory and visits only those; tiles that every row sees whole
// skip the masks. Few rows and many keys: the visible tiles are split between CTAs
// and a second kernel joins the parts.
//
// 192 threads, two CTAs per SM:
//   warps 0-3  one query row per thread: S from TMEM into registers, cap, bias, mask,
//              running maximum (log2 domain), P = exp2(s - m) rounded to the inputs'
//              type (the tensor core takes no other; the row sum uses the unrounded
//              FP32 values) and written back to TMEM, where the second product
//              takes it as its A operand. O stays in TMEM and is rescaled only when
//              the maximum grew by more than 2^8.
//   warp 4     TMA: Q once, K and V tiles
//   warp 5     one thread issues S = Q K^T and O += P V
// TMEM (256 columns): head_dim <= 64: S [0,128), P [128,192), O [192,256), so S of the
// next tile is computed beside P of this one; head_dim <= 128: S [0,128) with P over its
// first half, O [128,256): there the two CTAs of an SM overlap each other instead.
#include "attention_op.cuh"

#include <string.h>

#include <algorithm>

#include "profile.h"

namespace sdo {
namespace {

constexpr int kThreads = 192;
constexpr int kSlots = 296;      // CTAs that fill 148 SMs
constexpr int kMaxSplits = 64;

template <int NB>
struct Shape {
  static constexpr int kStages = NB == 1 ? 2 : 1;
  static constexpr int kQBytes = NB * kBlockBytes;
  static constexpr uint32_t kP = NB == 1 ? 128 : 0;
  static constexpr uint32_t kO = NB == 1 ? 192 : 128;
  static constexpr size_t kSmem = 1024 + (size_t)(1 + 2 * kStages) * kQBytes + sizeof(TileBits) + 512 + 256;
};

struct __align__(64) FwdMaps {
  CUtensorMap q, k, v;
};

template <typename T, int NB>
__global__ void __launch_bounds__(kThreads, 2)
    attn_fwd_kernel(const __grid_constant__ FwdMaps maps, const __grid_constant__ AttnArgs a) {
  using Sh = Shape<NB>;
  constexpr int KS = Sh::kStages;
  constexpr bool f16 = Elem<T>::kF16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + Sh::kQBytes;
  uint8_t* sV = sK + KS * Sh::kQBytes;
  TileBits* tiles = reinterpret_cast<TileBits*>(sV + KS * Sh::kQBytes);
  int32_t* sdoc = reinterpret_cast<int32_t*>(tiles + 1);  // [128] documents of the current key tile
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sdoc) + 512);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;    // [KS]
  uint64_t* k_empty = bars + 3;   // [KS]
  uint64_t* v_full = bars + 5;    // [KS]
  uint64_t* v_empty = bars + 7;   // [KS]
  uint64_t* s_full = bars + 9;
  uint64_t* s_free = bars + 10;
  uint64_t* p_full = bars + 11;
  uint64_t* pv_done = bars + 12;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 13);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* doc_lo = reinterpret_cast<int32_t*>(tmem_slot + 2);
  int32_t* doc_hi = doc_lo + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // item: the last query tiles first (with a causal mask they are the longest)
  const int z = blockIdx.x % a.splits;
  const int item = blockIdx.x / a.splits;
  const int heads = a.B * a.KV;
  const int qt = a.qtiles - 1 - item / heads;
  const int b = item % heads / a.KV, kv = item % heads % a.KV;
  const int i0 = qt * a.tq, i1 = min(a.Nq, i0 + a.tq) - 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 13; ++i) mbar_init(bars + i, i == 10 || i == 11 ? 128 : 1);
    *abort_flag = 0;
    *doc_lo = INT32_MAX;
    *doc_hi = INT32_MIN;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 5) tmem_alloc(tmem_slot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tP = tmem + Sh::kP, tO = tmem + Sh::kO;
  pdl_wait();
  pdl_trigger();
  if (a.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;

  const int nk = keys_of(a, b), off = nk - a.Nq, pre = prefix_of(a, b);
  if (a.q_doc) {
    for (int i = i0 + (int)threadIdx.x; i <= i1; i += kThreads) {
      const int d = a.q_doc[(int64_t)b * a.Nq + i];
      atomicMin(doc_lo, d);
      atomicMax(doc_hi, d);
    }
    __syncthreads();
  }
  // the last key any row sees, and the last one that all rows see, but for documents
  const int lim_any = a.causal ? min(nk, max(i1 + off + 1, pre)) : nk;
  const int lim_all = a.causal ? min(nk, max(i0 + off + 1, pre)) : nk;
  {
    const int words = (a.ktiles + 31) >> 5;
    for (int w = warp; w < words; w += kThreads / 32) {
      const int j = w * 32 + lane;
      bool see = j < a.ktiles && j * kTile < lim_any;
      bool all = see && (j + 1) * kTile <= lim_all;
      if (see && a.k_range) {
        const int32_t lo = a.k_range[((int64_t)b * a.ktiles + j) * 2], hi = a.k_range[((int64_t)b * a.ktiles + j) * 2 + 1];
        see = lo <= *doc_hi && *doc_lo <= hi;
        all = all && lo == hi && *doc_lo == lo && *doc_hi == lo;
      }
      const uint32_t ms = __ballot_sync(0xffffffffu, see), ma = __ballot_sync(0xffffffffu, all);
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
  const int first = (int)((int64_t)tiles->count * z / a.splits);
  const int steps = (int)((int64_t)tiles->count * (z + 1) / a.splits) - first;

  if (warp == 4) {
    if (lane == 0 && steps > 0) {
      TileWalk walk;
      walk.start(tiles, a.ktiles, first);
      mbar_arrive_expect_tx(q_full, (uint32_t)(NB * 128 * a.tq * a.G));
      for (int c = 0; c < NB; ++c) tma_load_4d(sQ + c * kBlockBytes, &maps.q, q_full, c * 64, kv * a.G, i0, b);
      for (int t = 0; t < steps; ++t) {
        const int j = walk.next() * kTile, s = t % KS;
        const uint32_t ph = (t / KS - 1) & 1;
        if (t >= KS && !mbar_wait(&k_empty[s], ph, abort_flag, a.err)) break;
        mbar_arrive_expect_tx(&k_full[s], Sh::kQBytes);
        for (int c = 0; c < NB; ++c)
          tma_load_4d(sK + s * Sh::kQBytes + c * kBlockBytes, &maps.k, &k_full[s], c * 64, kv, j, b);
        if (t >= KS && !mbar_wait(&v_empty[s], ph, abort_flag, a.err)) break;
        mbar_arrive_expect_tx(&v_full[s], Sh::kQBytes);
        for (int c = 0; c < NB; ++c)
          tma_load_4d(sV + s * Sh::kQBytes + c * kBlockBytes, &maps.v, &v_full[s], c * 64, kv, j, b);
      }
    }
  } else if (warp == 5) {
    if (lane == 0 && steps > 0) {
      const int nd = (a.D + 15) >> 4;  // head dimension in steps of 16
      const uint32_t id_s = idesc_f16(128, 128, f16, false, false);
      const uint32_t id_o = idesc_f16(128, nd * 16, f16, false, true);
      const uint32_t q0 = smem_u32(sQ);
      bool ok = mbar_wait(q_full, 0, abort_flag, a.err);
      auto issue_s = [&](int t) {
        const int s = t % KS;
        if (!mbar_wait(&k_full[s], (t / KS) & 1, abort_flag, a.err)) return false;
        tc_fence_after();
        const uint32_t k0 = smem_u32(sK + s * Sh::kQBytes);
        for (int d = 0; d < nd; ++d) {
          const uint32_t o = (d >> 2) * kBlockBytes + (d & 3) * 32;
          umma_bf16(tS, umma_desc_k_sw128(q0 + o), umma_desc_k_sw128(k0 + o), id_s, d > 0);
        }
        umma_commit(&k_empty[s]);
        umma_commit(s_full);
        return true;
      };
      auto issue_pv = [&](int t) {
        const int s = t % KS;
        if (!mbar_wait(p_full, t & 1, abort_flag, a.err)) return false;
        if (!mbar_wait(&v_full[s], (t / KS) & 1, abort_flag, a.err)) return false;
        tc_fence_after();
        const uint32_t v0 = smem_u32(sV + s * Sh::kQBytes);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ts(tO, tP + 8 * k, umma_desc_mn(v0 + k * 2048, kBlockBytes), id_o, (t > 0 || k > 0) ? 1u : 0u);
        umma_commit(&v_empty[s]);
        umma_commit(pv_done);
        return true;
      };
      if constexpr (NB == 1) {
        // S of step t beside the softmax of step t - 1
        for (int t = 0; t <= steps && ok; ++t) {
          if (t < steps) ok = (t == 0 || mbar_wait(s_free, (t - 1) & 1, abort_flag, a.err)) && issue_s(t);
          if (ok && t > 0) ok = issue_pv(t - 1);
        }
      } else {
        for (int t = 0; t < steps && ok; ++t) ok = issue_s(t) && issue_pv(t);
      }
    }
  } else {
    const int row = threadIdx.x;
    const int i = i0 + row / a.G, h = kv * a.G + row % a.G;
    const bool valid = row < a.tq * a.G && i < a.Nq;
    const bool work = __any_sync(0xffffffffu, valid);  // a warp without rows only keeps the barriers going
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const int pos = i + off;
    const int lim = !valid ? 0 : a.causal ? min(nk, max(pos + 1, pre)) : nk;
    const int doc = a.q_doc && valid ? a.q_doc[(int64_t)b * a.Nq + i] : 0;
    const float slope = a.slopes && valid ? a.slopes[h] * kLog2e : 0.f;
    const bool scaled = a.cap_out != 0.f || a.slopes;  // the scores are in log2 units before the maximum
    const float mul = scaled ? 1.f : a.sl2;
    float m = -INFINITY, l = 0.f;
    TileWalk walk;
    if (steps > 0) walk.start(tiles, a.ktiles, first);
    bool alive = true;
    for (int t = 0; t < steps; ++t) {
      const int j = walk.next(), j0 = j * kTile;
      const bool whole = walk.whole(j);
      const int s = t % KS;
      if (!mbar_wait_all(s_full, t & 1, abort_flag, a.err)) {
        alive = false;
        break;
      }
      tc_fence_after();
      uint32_t sv[128];
      if (work) {
        tmem_ld_32x32b_x32(tS + lane_off, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld_32x32b_x32(tS + lane_off + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_ld_32x32b_x32(tS + lane_off + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
        tmem_ld_32x32b_x32(tS + lane_off + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
        tmem_ld_wait();
      }
      if constexpr (NB == 1) {
        tc_fence_before();
        mbar_arrive(s_free);
      }
      if (!whole && a.k_doc) {
        asm volatile("bar.sync 1, 128;" ::: "memory");
        sdoc[row] = j0 + row < a.Nk ? a.k_doc[(int64_t)b * a.Nk + j0 + row] : 0;
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
      if (!whole && j0 + kTile > nk && nk < a.Nk) {
        // values behind the last key count as zeros, whatever they hold
        if (!mbar_wait_all(&v_full[s], (t / KS) & 1, abort_flag, a.err)) {
          alive = false;
          break;
        }
        if (j0 + row >= nk) {
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            uint4* p = reinterpret_cast<uint4*>(sV + s * Sh::kQBytes + c * kBlockBytes + row * 128);
#pragma unroll
            for (int u = 0; u < 8; ++u) p[u] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_async_smem();
      }
      float alpha = 1.f;
      bool rescale = false;
      uint32_t pk[64];
      if (work) {
        if (a.cap_out != 0.f) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            sv[c] = __float_as_uint(a.cap_out * tanh_acc(__uint_as_float(sv[c]) * a.cap_in));
        } else if (scaled) {
#pragma unroll
          for (int c = 0; c < 128; ++c) sv[c] = __float_as_uint(__uint_as_float(sv[c]) * a.sl2);
        }
        if (a.slopes) {
          const float p0 = (float)(pos - j0);
#pragma unroll
          for (int c = 0; c < 128; ++c)
            sv[c] = __float_as_uint(fmaf(-slope, fabsf(p0 - (float)c), __uint_as_float(sv[c])));
        }
        if (!whole) {
          const int lc = lim - j0;
          if (a.k_doc) {
#pragma unroll
            for (int c = 0; c < 128; c += 4) {
              const int4 d = *reinterpret_cast<const int4*>(sdoc + c);
              if (c >= lc || d.x != doc) sv[c] = __float_as_uint(-INFINITY);
              if (c + 1 >= lc || d.y != doc) sv[c + 1] = __float_as_uint(-INFINITY);
              if (c + 2 >= lc || d.z != doc) sv[c + 2] = __float_as_uint(-INFINITY);
              if (c + 3 >= lc || d.w != doc) sv[c + 3] = __float_as_uint(-INFINITY);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= lc) sv[c] = __float_as_uint(-INFINITY);
          }
        }
        float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          m0 = max3f(m0, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
          m1 = max3f(m1, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
          m2 = max3f(m2, __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
          m3 = max3f(m3, __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
        }
        const float m_new = fmaxf(m, max3f(m0, m1, fmaxf(m2, m3)) * mul);
        if (m == -INFINITY) {
          m = m_new;  // nothing seen so far: O's row is zeros (or not written yet)
        } else if (m_new > m + 8.f) {
          alpha = fast_ex2(m - m_new);
          l *= alpha;
          m = m_new;
          rescale = true;
        }
        const float base = m == -INFINITY ? 0.f : -m;  // a row without keys: exp2(-inf) = 0 throughout
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          float x0, x1, x2, x3;
          fma2v(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), mul, mul, base, base, x0, x1);
          fma2v(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]), mul, mul, base, base, x2, x3);
          x0 = fast_ex2(x0);
          x1 = fast_ex2(x1);
          x2 = fast_ex2(x2);
          x3 = fast_ex2(x3);
          add2(l0, l1, x0, x1, l0, l1);
          add2(l2, l3, x2, x3, l2, l3);
          pk[c / 2] = Elem<T>::pack(x0, x1);
          pk[c / 2 + 1] = Elem<T>::pack(x2, x3);
        }
        l += (l0 + l1) + (l2 + l3);
      }
      // P and O are free once the previous product is done
      if (t > 0 && !mbar_wait_all(pv_done, (t - 1) & 1, abort_flag, a.err)) {
        alive = false;
        break;
      }
      tc_fence_after();
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
        for (int c = 0; c < 2 * NB; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tO + lane_off + c * 32, r);
          tmem_ld_wait_regs(r);
#pragma unroll
          for (int u = 0; u < 32; ++u) r[u] = __float_as_uint(__uint_as_float(r[u]) * alpha);
          tmem_st_x32(tO + lane_off + c * 32, r);
        }
      }
      if (work) {
        tmem_st_x32(tP + lane_off, pk);
        tmem_st_x32(tP + lane_off + 32, pk + 32);
      }
      tmem_store_wait();
      tc_fence_before();
      mbar_arrive(p_full);
    }
    if (alive && steps > 0) alive = mbar_wait_all(pv_done, (steps - 1) & 1, abort_flag, a.err);
    tc_fence_after();
    if (alive && work) {
      const bool part = a.splits > 1;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      T* dst = static_cast<T*>(a.o) + b * a.os[0] + i * a.os[1] + h * a.os[2];
      const int64_t slot = ((int64_t)item * a.splits + z) * kTile + row;
#pragma unroll 1
      for (int c = 0; c < NB * 64; c += 32) {
        if (c >= a.D) break;
        uint32_t r[32];
        if (steps > 0) {
          tmem_ld_32x32b_x32(tO + lane_off + c, r);
          tmem_ld_wait_regs(r);
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) r[u] = 0u;
        }
        if (valid && part && steps > 0) {
          float4* p = reinterpret_cast<float4*>(a.partial + slot * a.D + c);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (c + 4 * u < a.D)
              __stcg(p + u, make_float4(__uint_as_float(r[4 * u]), __uint_as_float(r[4 * u + 1]),
                                        __uint_as_float(r[4 * u + 2]), __uint_as_float(r[4 * u + 3])));
        } else if (valid && !part) {
          // a row whose mask leaves nothing has l = 0 and gets zeros
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (c + 8 * u < a.D)
              *reinterpret_cast<uint4*>(dst + c + 8 * u) = make_uint4(
                  Elem<T>::pack(__uint_as_float(r[8 * u]) * inv, __uint_as_float(r[8 * u + 1]) * inv),
                  Elem<T>::pack(__uint_as_float(r[8 * u + 2]) * inv, __uint_as_float(r[8 * u + 3]) * inv),
                  Elem<T>::pack(__uint_as_float(r[8 * u + 4]) * inv, __uint_as_float(r[8 * u + 5]) * inv),
                  Elem<T>::pack(__uint_as_float(r[8 * u + 6]) * inv, __uint_as_float(r[8 * u + 7]) * inv));
        }
      }
      if (valid && part) {
        a.partial_ml[slot * 2] = m;
        a.partial_ml[slot * 2 + 1] = l;
      } else if (valid && a.lse) {
        a.lse[((int64_t)b * a.H + h) * a.Nq + i] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, 256);
}

// Joins the parts of split items, one warp per query row: m = max m_z, o = sum
// 2^(m_z - m) O_z / sum 2^(m_z - m) l_z, over z in order.
template <typename T>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);
  if (r >= (int64_t)a.B * a.H * a.Nq) return;
  const int i = (int)(r % a.Nq), h = (int)(r / a.Nq % a.H), b = (int)(r / a.Nq / a.H);
  const int kv = h / a.G;
  const int64_t item = (int64_t)(a.qtiles - 1 - i / a.tq) * (a.B * a.KV) + b * a.KV + kv;
  const int64_t slot = item * a.splits * kTile + (i % a.tq) * a.G + h % a.G;
  float mz[2], lz[2];
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < 2; ++u) {  // at most 64 parts
    const int z = u * 32 + lane;
    mz[u] = -INFINITY;
    lz[u] = 0.f;
    if (z < a.splits) {
      const float2 v = *reinterpret_cast<const float2*>(a.partial_ml + (slot + (int64_t)z * kTile) * 2);
      mz[u] = v.x;
      lz[u] = v.y;
    }
    m = fmaxf(m, mz[u]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float w[2], l = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    w[u] = mz[u] == -INFINITY ? 0.f : fast_ex2(mz[u] - m);
    l += w[u] * lz[u];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const bool in = lane * 4 < a.D;
#pragma unroll 4
  for (int z = 0; z < a.splits; ++z) {
    const float f = __shfl_sync(0xffffffffu, z < 32 ? w[0] : w[1], z & 31);
    if (f != 0.f && in) {  // a part that saw no key holds no values
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.partial + (slot + (int64_t)z * kTile) * a.D) + lane);
      acc[0] = fmaf(f, v.x, acc[0]);
      acc[1] = fmaf(f, v.y, acc[1]);
      acc[2] = fmaf(f, v.z, acc[2]);
      acc[3] = fmaf(f, v.w, acc[3]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  if (in) {
    T* dst = static_cast<T*>(a.o) + b * a.os[0] + i * a.os[1] + h * a.os[2] + lane * 4;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(Elem<T>::pack(acc[0] * inv, acc[1] * inv), Elem<T>::pack(acc[2] * inv, acc[3] * inv));
  }
  if (lane == 0 && a.lse) a.lse[((int64_t)b * a.H + h) * a.Nq + i] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

__global__ void __launch_bounds__(128) attn_doc_range_kernel(const int32_t* doc, int len, int tiles, int32_t* range) {
  pdl_wait();
  pdl_trigger();
  const int64_t w = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);  // one warp per tile
  const int lane = threadIdx.x & 31;
  const int64_t b = w / tiles;
  const int tile = (int)(w % tiles);
  int lo = INT32_MAX, hi = INT32_MIN;
  for (int i = tile * kTile + lane; i < min(len, (tile + 1) * kTile); i += 32) {
    const int d = doc[b * len + i];
    lo = min(lo, d);
    hi = max(hi, d);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    range[w * 2] = lo;
    range[w * 2 + 1] = hi;
  }
}

// ------------------------------------------------------------------ host side

int tiles_of(int n) { return (n + kTile - 1) / kTile; }

struct FwdPlan {
  int tq, qtiles, ktiles, splits;
  int64_t items;
};
FwdPlan plan_forward(const sd_attention_cfg& c) {
  FwdPlan p;
  const int g = c.heads / c.kv_heads;
  p.tq = kTile / g;
  p.qtiles = (c.q_len + p.tq - 1) / p.tq;
  p.ktiles = tiles_of(c.k_len);
  p.items = (int64_t)c.batch * c.kv_heads * p.qtiles;
  // split while it leaves every part two tiles and all parts fit on the GPU at once
  int64_t s = std::min<int64_t>(std::min<int64_t>(kSlots / std::max<int64_t>(p.items, 1), p.ktiles / 2), kMaxSplits);
  p.splits = (int)std::max<int64_t>(s, 1);
  return p;
}

// Scratch after the header: document ranges of the key tiles and query tiles, then
// the forward's parts or what the backward needs.
size_t range_bytes(int batch, int len) { return up256((size_t)batch * tiles_of(len) * 8); }
size_t ranges_bytes(const sd_attention_cfg& c) { return range_bytes(c.batch, c.k_len) + range_bytes(c.batch, c.q_len); }
size_t parts_bytes(const sd_attention_cfg& c) {
  const FwdPlan p = plan_forward(c);
  return p.splits > 1 ? up256((size_t)p.items * p.splits * kTile * (c.head_dim + 2) * 4) : 0;
}

bool strides_ok(const int64_t* s, int batch, int tokens, int heads, int d, int64_t* out) {
  if (!s[0] && !s[1] && !s[2]) {
    out[2] = d;
    out[1] = (int64_t)heads * d;
    out[0] = out[1] * tokens;
    return out[0] < (int64_t)1 << 38;
  }
  const int n[3] = {batch, tokens, heads};
  for (int i = 0; i < 3; ++i) {
    out[i] = s[i];
    if (n[i] <= 1 && (s[i] <= 0 || s[i] % 8 || s[i] >= (int64_t)1 << 38)) out[i] = 8;  // never stepped
    else if (s[i] <= 0 || s[i] % 8 || s[i] >= (int64_t)1 << 38) return false;
  }
  return true;
}

sd_status check(const sd_attention_cfg* c, AttnCall* call) {
  if (!c) return SD_ERR_NULL_ARG;
  if (c->batch < 0 || c->q_len < 0 || c->k_len < 0 || c->heads <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 ||
      c->heads % c->kv_heads)
    return SD_ERR_BAD_SHAPE;
  // a given scale or cap within what FP32 products of scores can hold
  const auto sane = [](float f) { return f == 0.f || (f >= 1e-20f && f <= 1e20f); };
  if (!sane(c->scale) || !sane(c->softcap)) return SD_ERR_BAD_SHAPE;
  if (c->head_dim % 8 || c->head_dim > 128 || c->heads / c->kv_heads > kTile || c->q_len > 1 << 20 ||
      c->k_len > 1 << 20 || (c->dtype != SD_DTYPE_BF16 && c->dtype != SD_DTYPE_F16))
    return SD_ERR_UNSUPPORTED;
  // CTA and row counts within a grid's x extent
  if ((int64_t)c->batch * c->heads > 1 << 24 || (int64_t)c->batch * c->heads * std::max(c->q_len, 1) > (int64_t)1 << 32)
    return SD_ERR_UNSUPPORTED;
  if (!strides_ok(c->q_stride, c->batch, c->q_len, c->heads, c->head_dim, call->qs) ||
      !strides_ok(c->k_stride, c->batch, c->k_len, c->kv_heads, c->head_dim, call->ks) ||
      !strides_ok(c->v_stride, c->batch, c->k_len, c->kv_heads, c->head_dim, call->vs) ||
      !strides_ok(c->o_stride, c->batch, c->q_len, c->heads, c->head_dim, call->os))
    return SD_ERR_BAD_SHAPE;
  call->cfg = c;
  return SD_OK;
}

sd_status check_masks(const sd_attention_cfg& c, const sd_attention_masks* m) {
  if (!m) return SD_OK;
  if (m->prefix && !c.causal) return SD_ERR_BAD_SHAPE;
  if (!m->q_doc != !m->k_doc) return SD_ERR_NULL_ARG;
  for (const void* p : {(const void*)m->k_lens, (const void*)m->prefix, (const void*)m->q_doc, (const void*)m->k_doc,
                        (const void*)m->slopes})
    if (misaligned(p)) return SD_ERR_MISALIGNED;
  return SD_OK;
}

template <typename T, int NB>
sd_status forward(AttnCall& c, const FwdPlan& p) {
  constexpr bool f16 = Elem<T>::kF16;
  const sd_attention_cfg& g = *c.cfg;
  AttnArgs& a = c.args;
  FwdMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!attn_map(&maps.q, f16, c.q, c.qs, g.batch, g.q_len, g.heads, g.head_dim, (uint32_t)a.G, (uint32_t)p.tq) ||
      !attn_map(&maps.k, f16, c.k, c.ks, g.batch, g.k_len, g.kv_heads, g.head_dim, 1, kTile) ||
      !attn_map(&maps.v, f16, c.v, c.vs, g.batch, g.k_len, g.kv_heads, g.head_dim, 1, kTile))
    return SD_ERR_LAUNCH;
  OP_TRY((allow_smem<attn_fwd_kernel<T, NB>>(Shape<NB>::kSmem, c.dev.index)));
  const double pairs = (double)g.batch * g.heads * g.q_len * g.k_len;
  const double bytes = 2.0 * g.batch * g.head_dim * (2.0 * g.q_len * g.heads + 2.0 * g.k_len * g.kv_heads);
  sdp::Scope sc("attn_fwd", sdp::F_ATTN, 4.0 * pairs * g.head_dim, bytes, c.st, p.splits > 1 ? 2 : 1);
  OP_TRY(launched(launch_pdl(attn_fwd_kernel<T, NB>, dim3((unsigned)(p.items * p.splits)), dim3(kThreads),
                             Shape<NB>::kSmem, c.st, maps, a)));
  if (p.splits == 1) return SD_OK;
  const int64_t rows = (int64_t)g.batch * g.heads * g.q_len;
  return launched(launch_pdl(attn_join_kernel<T>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, c.st, a));
}

}  // namespace

bool attn_map(CUtensorMap* m, bool f16, const void* p, const int64_t* s, int batch, int tokens, int heads, int d,
              uint32_t box_heads, uint32_t box_tokens) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)heads, (uint64_t)tokens, (uint64_t)batch};
  const int64_t strides[3] = {s[2], s[1], s[0]};
  const uint32_t box[4] = {64, box_heads, box_tokens, 1};
  return encode_map(m, f16, p, 4, dims, strides, box);
}

sd_status attn_doc_ranges(const int32_t* doc, int batch, int len, int32_t* range, cudaStream_t st) {
  const int tiles = tiles_of(len);
  const int64_t warps = (int64_t)batch * tiles;
  sdp::Scope sc("attn_doc_range", sdp::F_OTHER, 0, 4.0 * batch * len, st);
  return launched(launch_pdl(attn_doc_range_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, doc, len, tiles,
                             range));
}

void attn_fill(AttnCall& c, const sd_attention_masks* m) {
  const sd_attention_cfg& g = *c.cfg;
  AttnArgs& a = c.args;
  memset(&a, 0, sizeof(a));
  a.B = g.batch;
  a.Nq = g.q_len;
  a.Nk = g.k_len;
  a.H = g.heads;
  a.KV = g.kv_heads;
  a.G = g.heads / g.kv_heads;
  a.D = g.head_dim;
  a.causal = g.causal != 0;
  const float scale = g.scale > 0.f ? g.scale : 1.f / sqrtf((float)g.head_dim);
  a.sl2 = scale * kLog2e;
  if (g.softcap > 0.f) {
    a.cap_in = scale / g.softcap;
    a.cap_out = g.softcap * kLog2e;
  }
  if (m) {
    a.k_lens = m->k_lens;
    a.prefix = m->prefix;
    a.q_doc = m->q_doc;
    a.k_doc = m->k_doc;
    a.slopes = m->slopes;
  }
  for (int i = 0; i < 3; ++i) a.os[i] = c.os[i];
  a.ktiles = tiles_of(g.k_len);
  a.err = reinterpret_cast<int*>(c.ws);
  a.k_range = a.k_doc ? reinterpret_cast<int32_t*>(c.ws + kOpHeader) : nullptr;
  a.q_range = a.k_doc ? reinterpret_cast<int32_t*>(c.ws + kOpHeader + range_bytes(g.batch, g.k_len)) : nullptr;
}

}  // namespace sdo

using namespace sdo;

extern "C" {

size_t sd_attention_workspace_size(const sd_attention_cfg* cfg) {
  AttnCall c;
  if (check(cfg, &c) != SD_OK) return 0;
  if (cfg->batch == 0) return kOpHeader;
  return kOpHeader + ranges_bytes(*cfg) + std::max(parts_bytes(*cfg), attn_grad_space(*cfg));
}

sd_status sd_attention_fwd(const sd_attention_cfg* cfg, const void* q, const void* k, const void* v,
                           const sd_attention_masks* masks, void* o, float* lse, void* workspace, size_t ws_bytes,
                           sd_stream_t stream) {
  AttnCall c;
  OP_TRY(check(cfg, &c));
  OP_TRY(check_masks(*cfg, masks));
  if (cfg->batch == 0 || cfg->q_len == 0) return SD_OK;
  if (!q || !o || (cfg->k_len > 0 && (!k || !v))) return SD_ERR_NULL_ARG;
  for (const void* p : {q, k, v, (const void*)o, (const void*)lse})
    if (misaligned(p)) return SD_ERR_MISALIGNED;
  OP_TRY(check_workspace(sd_attention_workspace_size(cfg), workspace, ws_bytes));
  OP_TRY(current_device(&c.dev));
  c.st = (cudaStream_t)stream;
  c.ws = static_cast<uint8_t*>(workspace);
  c.q = q;
  // without keys nothing is loaded: any readable address makes a map
  c.k = cfg->k_len ? k : q;
  c.v = cfg->k_len ? v : q;
  sd_attention_cfg shaped = *cfg;
  if (cfg->k_len == 0) {
    for (int i = 0; i < 3; ++i) c.ks[i] = c.vs[i] = 8 * ((cfg->head_dim + 7) / 8);
  }
  attn_fill(c, cfg->k_len ? masks : nullptr);
  const FwdPlan p = plan_forward(*cfg);
  AttnArgs& a = c.args;
  a.tq = p.tq;
  a.qtiles = p.qtiles;
  a.splits = p.splits;
  a.o = o;
  a.lse = lse;
  a.clear_err = 1;
  if (p.splits > 1) {
    a.partial = reinterpret_cast<float*>(c.ws + kOpHeader + ranges_bytes(*cfg));
    a.partial_ml = a.partial + (size_t)p.items * p.splits * kTile * cfg->head_dim;
  }
  if (cfg->k_len == 0) {
    shaped.k_len = 1;  // a map has no empty dimension; no tile of it is visited
    c.cfg = &shaped;
  }
  if (a.k_doc) OP_TRY(attn_doc_ranges(a.k_doc, cfg->batch, cfg->k_len, const_cast<int32_t*>(a.k_range), c.st));
  const bool wide = cfg->head_dim > 64;
  if (cfg->dtype == SD_DTYPE_F16) return wide ? forward<__half, 2>(c, p) : forward<__half, 1>(c, p);
  return wide ? forward<__nv_bfloat16, 2>(c, p) : forward<__nv_bfloat16, 1>(c, p);
}

sd_status sd_attention_bwd(const sd_attention_cfg* cfg, const void* q, const void* k, const void* v,
                           const sd_attention_masks* masks, const void* o, const float* lse, const void* d_o, void* dq,
                           void* dk, void* dv, void* workspace, size_t ws_bytes, sd_stream_t stream) {
  AttnCall c;
  OP_TRY(check(cfg, &c));
  OP_TRY(check_masks(*cfg, masks));
  if (cfg->batch == 0 || (cfg->q_len == 0 && cfg->k_len == 0)) return SD_OK;
  if ((cfg->q_len > 0 && (!q || !o || !lse || !d_o || !dq)) || (cfg->k_len > 0 && (!k || !v || !dk || !dv)))
    return SD_ERR_NULL_ARG;
  for (const void* p : {q, k, v, o, (const void*)lse, d_o, (const void*)dq, (const void*)dk, (const void*)dv})
    if (misaligned(p)) return SD_ERR_MISALIGNED;
  OP_TRY(check_workspace(sd_attention_workspace_size(cfg), workspace, ws_bytes));
  OP_TRY(current_device(&c.dev));
  c.st = (cudaStream_t)stream;
  c.ws = static_cast<uint8_t*>(workspace);
  c.q = q;
  c.k = k;
  c.v = v;
  c.o = o;
  c.d_o = d_o;
  c.lse = lse;
  c.dq = dq;
  c.dk = dk;
  c.dv = dv;
  attn_fill(c, masks);
  c.ws += kOpHeader + ranges_bytes(*cfg);
  return cfg->dtype == SD_DTYPE_F16 ? attn_backward<__half>(c) : attn_backward<__nv_bfloat16>(c);
}

}  // extern "C"
