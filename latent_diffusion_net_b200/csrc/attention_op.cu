// Attention with capped scores, a distance bias, documents, a prefix and key
// lengths: o = softmax(mask(cap(scale q k^T) - slope |p - j|)) v, one pass over the
// keys with a running maximum and sum. The backward kernels are in attention_grad.cu.
//
// Long sequences take 4 D operations and one exponential a pair (three with a cap), single
// tokens the reading of keys and values. Neither is reached: on 9216 tokens x 5 heads of 64 in
// three documents the exponential unit is busy 53 % of the time and the tensor pipe 18 %; a tile's steps follow one
// another, and one thread issues its twelve products.
//
// A unit of work is 128 query rows: kTile / G tokens with the G query heads that
// share a key head, so a key tile is read once for all of them. Its key tiles are
// found by vote, 32 at a time (length, causal limit with prefix, document ranges),
// and only those that some row may see are visited; tiles that every row sees whole
// skip the masks. Items that would leave SMs idle, or end long after the rest, are cut into
// parts that a second kernel joins: few rows and many keys, tiles beyond full rounds of
// the GPU, the longest of a causal mask's. The grid has one CTA per unit, and a CTA that
// runs takes over units of CTAs that have not been launched yet (cluster launch
// control), so the loads and the first product of a unit run beside the end of the
// one before and long units even out.
//
// 320 threads, two CTAs per SM:
//   warps 0-7  two threads per query row, 64 keys each: S from TMEM into registers, cap,
//              bias, mask, running maximum (log2 domain; the halves meet in shared
//              memory), P = exp2(s - m) rounded to the inputs' type (the tensor core
//              takes no other; the row sum uses the unrounded FP32 values) and
//              written back to TMEM, where the second product takes it as its A
//              operand. O stays in TMEM and is rescaled only when the maximum grew
//              by more than 2^8.
//   warp 8     TMA: Q once, K and V tiles
//   warp 9     one thread issues S = Q K^T and O += P V
// TMEM (256 columns): head_dim <= 64: S [0,128), P [128,192), O [192,256), so S of the
// next tile is computed beside P of this one; head_dim <= 128: S [0,128) with P over its
// first half, O [128,256): there the two CTAs of an SM overlap each other instead.
//
// Measured (BF16): 296 units of 64 key tiles 586 TFLOP/s at head_dim 64, 800 at 128, where
// the exponentials and the MMA issue take turns; 9216 tokens x 5 heads of 64 190 us (572);
// 4096 queries x 77 keys, 10 heads, batch 4 29 us, two thirds of it a unit's beginning and
// end; one FP16 query each on 4096 keys, 16 heads of 128 over 4 key heads, batch 8 24 us
// with the join (2.1 TB/s of keys and values: one stage of K and V at head_dim 128, so that a
// tile is asked for only when the one before is done, and the join's launch).
#include "attention_op.cuh"

#include <string.h>

#include <algorithm>

#include "profile.h"

namespace sdo {
namespace {

constexpr int kThreads = 320;
constexpr int kSoftmaxWarps = 8;
constexpr int kSms = 148;
constexpr int kMaxSplits = 64;

template <int NB>
struct Shape {
  static constexpr int kStages = NB == 1 ? 2 : 1;  // of Q, K and V each
  static constexpr int kBytes = NB * kBlockBytes;
  static constexpr uint32_t kP = NB == 1 ? 128 : 0;
  static constexpr uint32_t kO = NB == 1 ? 192 : 128;
  static constexpr size_t kSmem = 1024 + (size_t)3 * kStages * kBytes + kDocRing * 512 + 2048 + kRing * sizeof(Record) + 512;
};

struct __align__(64) FwdMaps {
  CUtensorMap q, k, v;
};

// A unit of work: a part of 128 query rows. The last query tiles come first (with
// a causal mask they are the longest).
struct Unit {
  Part part;
  int b, kv, i0, i1, qt;
  __device__ __forceinline__ Unit(const AttnArgs& a, int u) : part(a.parts, u) {
    const int heads = a.B * a.KV, at = part.item % heads;
    qt = a.qtiles - 1 - part.item / heads;
    b = at / a.KV;
    kv = at % a.KV;
    i0 = qt * a.tq;
    i1 = min(a.Nq, i0 + a.tq) - 1;
  }
  __device__ __forceinline__ const int32_t* docs(const AttnArgs& a) const {
    return a.q_range + ((int64_t)b * a.qtiles + qt) * 2;
  }
};
// The unit's walk and its number of steps (INT32_MAX: until the walk ends).
struct UnitWalk : TileWalk<RowTiles> {
  int steps;
  __device__ __forceinline__ UnitWalk(const AttnArgs& a, const Unit& u, int off, int nk, int pre)
      : TileWalk<RowTiles>(RowTiles(a, u.b, u.i0, u.i1, off, nk, pre, u.docs(a))) {
    steps = INT32_MAX;
    if (u.part.slot >= 0) {
      const int n = count();
      steps = u.part.steps(n);
      if (steps > 0) skip((int)u.part.begin(n));
    }
  }
  __device__ __forceinline__ int step(bool& whole) { return steps-- > 0 ? next(whole) : -1; }
};

// The end of a unit: one query row per thread, normalised to the output, or its part
// (given `part`) of a cut item. All by value: what a reference to the kernel's arguments
// reads comes from far away (77 keys: 5000 cycles a unit, half of its time).
template <typename T, int NB, bool WIDE>
__device__ __forceinline__ void store_rows(T* dst, float* part, float* ml, float* lse, int D, bool wide, int half,
                                        uint32_t tO, bool some, bool valid, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;  // l = 0: a row that sees no key; NaN stays NaN
#pragma unroll 1
  for (int k = 0; k < NB * 32; k += 32) {
    const int c = half * NB * 32 + k;
    if (c >= D) break;
    uint32_t r[32];
    if (some) {
      tmem_ld_32x32b_x32(tO + k, r);
      tmem_ld_wait_regs(r);
    } else {
#pragma unroll
      for (int q = 0; q < 32; ++q) r[q] = 0u;
    }
    if (valid && part && some) {
      store_part32(part + c, r, D - c);
    } else if (valid && !part) {
      // a row whose mask leaves nothing has l = 0 and gets zeros
      float f[32];
#pragma unroll
      for (int q = 0; q < 32; ++q) f[q] = __uint_as_float(r[q]) * inv;
      store_row32<WIDE, T>(dst + c, f, D - c, wide);
    }
  }
  if (half || !valid) return;
  if (part) {
    *reinterpret_cast<float2*>(ml) = make_float2(m, l);
  } else if (lse) {
    *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// SHAPED: the scores are capped or biased before the mask.
template <typename T, int NB, bool SHAPED>
__global__ void __launch_bounds__(kThreads, 2)
    attn_fwd_kernel(const __grid_constant__ FwdMaps maps, const __grid_constant__ AttnArgs a) {
  using Sh = Shape<NB>;
  constexpr int KS = Sh::kStages;
  constexpr bool f16 = Elem<T>::kF16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + KS * Sh::kBytes;
  uint8_t* sV = sK + KS * Sh::kBytes;
  int32_t* sdocs = reinterpret_cast<int32_t*>(sV + KS * Sh::kBytes);  // [kDocRing][128]
  float* smax = reinterpret_cast<float*>(sdocs + kDocRing * kTile);  // [2][2][128] the halves' row maxima, by step parity
  Record* recs = reinterpret_cast<Record*>(smax + 4 * kTile);
  uint64_t* bars = reinterpret_cast<uint64_t*>(recs + kRing);
  uint64_t* q_full = bars;        // [KS]
  uint64_t* q_empty = bars + 2;   // [KS]
  uint64_t* k_full = bars + 4;    // [KS]
  uint64_t* k_empty = bars + 6;   // [KS]
  uint64_t* v_full = bars + 8;    // [KS]
  uint64_t* v_empty = bars + 10;  // [KS]
  uint64_t* s_full = bars + 12;
  uint64_t* pv_done = bars + 13;
  uint64_t* s_free = bars + 14;
  uint64_t* p_full = bars + 15;
  uint64_t* rec_full = bars + 16;   // [kRing]
  uint64_t* rec_empty = bars + 20;  // [kRing], eight softmax warps and the MMA warp
  uint64_t* next_bar = bars + 24;
  uint8_t* next_unit = reinterpret_cast<uint8_t*>(bars + 26);  // 16 bytes
  uint64_t* doc_full = bars + 28;  // [kDocRing]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 28 + kDocRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* left = reinterpret_cast<int*>(tmem_slot + 2);  // [4] softmax warps of a row quarter that are through
  const RecordRing ring{recs, rec_full, rec_empty, abort_flag, a.err};
  const DocRing docs{sdocs, doc_full, abort_flag, a.err};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDocRing; ++i) mbar_init(&doc_full[i], 1);
    for (int i = 0; i < 25; ++i) mbar_init(bars + i, i == 14 || i == 15 ? kSoftmaxWarps : i >= 20 && i < 24 ? 9 : 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) left[i] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tP = tmem + Sh::kP, tO = tmem + Sh::kO;
  pdl_wait();
  pdl_trigger();
  if (a.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;

  // t counts steps and n units with steps since the kernel began: they give each
  // barrier's phase.
  if (warp == 8) {
    int t = 0, n = 0, r = 0, asked = 0;
    bool ok = a.hold_spins == 0 || mbar_wait(next_bar, 0, abort_flag, a.err, (uint32_t)a.hold_spins);
    ok = __all_sync(0xffffffffu, ok);
    for (int x = blockIdx.x; x >= 0 && ok;) {
      const Unit u(a, x);
      const int nk = keys_of(a, u.b), pre = prefix_of(a, u.b);
      UnitWalk walk(a, u, nk - a.Nq, nk, pre);
      bool whole, whole_next;
      int j = walk.step(whole), after;
      int first = kFirst;
      do {
        after = j >= 0 ? walk.step(whole_next) : -1;
        if (lane == 0) {
          Record rec = {j, first | (after < 0 ? kLast : 0) | (j >= 0 && whole ? kWhole : 0), x, nk, pre, 0, u.b,
                        u.kv, u.i0, u.part.slot, {0, 0}};
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
            if (first) {
              const int s = n % KS;
              ok = ok && (n < KS || mbar_wait(&q_empty[s], (n / KS - 1) & 1, abort_flag, a.err));
              if (ok) {
                mbar_arrive_expect_tx(&q_full[s], (uint32_t)(NB * 128 * a.tq * a.G));
                for (int c = 0; c < NB; ++c)
                  tma_load_4d(sQ + s * Sh::kBytes + c * kBlockBytes, &maps.q, &q_full[s], c * 64, u.kv * a.G, u.i0,
                              u.b);
              }
            }
            const int s = t % KS;
            const uint32_t ph = (t / KS - 1) & 1;
            ok = ok && (t < KS || mbar_wait(&k_empty[s], ph, abort_flag, a.err));
            if (ok) {
              mbar_arrive_expect_tx(&k_full[s], Sh::kBytes);
              for (int c = 0; c < NB; ++c)
                tma_load_4d(sK + s * Sh::kBytes + c * kBlockBytes, &maps.k, &k_full[s], c * 64, u.kv, j * kTile, u.b);
            }
            ok = ok && (t < KS || mbar_wait(&v_empty[s], ph, abort_flag, a.err));
            if (ok) {
              mbar_arrive_expect_tx(&v_full[s], Sh::kBytes);
              for (int c = 0; c < NB; ++c)
                tma_load_4d(sV + s * Sh::kBytes + c * kBlockBytes, &maps.v, &v_full[s], c * 64, u.kv, j * kTile, u.b);
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
  } else if (warp == 9) {
    const int nd = (a.D + 15) >> 4;  // head dimension in steps of 16
    const uint32_t id_s = idesc_f16(128, 128, f16, false, false);
    const uint32_t id_o = idesc_f16(128, nd * 16, f16, false, true);
    constexpr uint32_t kStage = Sh::kBytes >> 4;  // from one stage's descriptor to the next's
    const uint32_t q0 = desc_k(smem_u32(sQ)), k0 = desc_k(smem_u32(sK)), v0t = desc_mn(smem_u32(sV), kBlockBytes);
    auto issue_s = [&](int t, int n, bool first, bool last) {
      const int s = t % KS, sq = n % KS;
      if (first && !mbar_wait(&q_full[sq], (n / KS) & 1, abort_flag, a.err)) return false;
      if (!mbar_wait(&k_full[s], (t / KS) & 1, abort_flag, a.err)) return false;
      tc_fence_after();
      const uint32_t q = q0 + sq * kStage, k = k0 + s * kStage;
      mma_ss<false>(tS, q, k, id_s);
#pragma unroll
      for (int d = 1; d < 4 * NB; ++d) {
        const uint32_t o = (d >> 2) * (kBlockBytes >> 4) + (d & 3) * 2;
        if (d < nd) mma_ss<true>(tS, q + o, k + o, id_s);
      }
      umma_commit(&k_empty[s]);
      umma_commit(s_full);
      if (last) umma_commit(&q_empty[sq]);
      return true;
    };
    auto issue_pv = [&](int t, bool first) {
      const int s = t % KS;
      if (!mbar_wait(p_full, t & 1, abort_flag, a.err)) return false;
      if (!mbar_wait(&v_full[s], (t / KS) & 1, abort_flag, a.err)) return false;
      tc_fence_after();
      const uint32_t v = v0t + s * kStage;
      if (first)
        mma_ts<false>(tO, tP, v, id_o);
      else
        mma_ts<true>(tO, tP, v, id_o);
#pragma unroll
      for (int k = 1; k < 8; ++k) mma_ts<true>(tO, tP + 8 * k, v + k * 128, id_o);
      umma_commit(&v_empty[s]);
      umma_commit(pv_done);
      return true;
    };
    // NB = 1: S of a step beside the softmax of the one before, across units; that
    // step's PV product is pending meanwhile
    int t = 0, n = -1;
    bool ok = true, pending = false, pending_first = false;
    for (int r = 0; ok; ++r) {
      const int2 rec = ring.get(r);  // tile, flags
      if (rec.x >= 0) {
        const bool first = rec.y & kFirst, last = rec.y & kLast;
        n += first;
        if (lane == 0) {
          if constexpr (NB == 1) {
            ok = (t == 0 || mbar_wait(s_free, (t - 1) & 1, abort_flag, a.err)) && issue_s(t, n, first, last);
            if (ok && pending) ok = issue_pv(t - 1, pending_first);
          } else {
            ok = issue_s(t, n, first, last) && issue_pv(t, first);
          }
        }
        ++t;
        pending = NB == 1;
        pending_first = first;
      }
      if (pending && rec.x < 0) {
        // nothing to issue beside it: the next record has no tile, or there is none
        if (lane == 0) ok = issue_pv(t - 1, pending_first);
        pending = false;
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (rec.y & kEnd) break;
    }
  } else {
    const int q4 = warp & 3, half = warp >> 2;
    const int row = q4 * 32 + lane, row_i = row / a.G, row_h = row % a.G;  // token and head within the unit
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tSr = tS + lane_off + half * 64, tPr = tP + lane_off + half * 32;
    const uint32_t tOr = tO + lane_off + half * NB * 32;  // the columns of O this half rescales and stores
    const bool wide = wide_rows(a.o, a.os, a.D);
    const float mul = SHAPED ? 1.f : a.sl2;  // shaped scores are in log2 units before the maximum
    int t = 0;
    bool alive = true, valid = false, work = false, some = false;
    int nk = 0, pos = 0, lim = 0, doc = 0;
    float slope = 0.f, m = -INFINITY, l = 0.f;
    for (int r = 0;; ++r) {
      const Record* const rec = ring.at(r);
      if (!rec || (rec->flags & kEnd)) break;
      const int flags = rec->flags, tile = rec->tile;
      const bool first = flags & kFirst, whole = flags & kWhole;
      if (first) {
        const int i = rec->i0 + row_i;
        nk = rec->nk;
        valid = row < a.tq * a.G && i < a.Nq;
        work = __any_sync(0xffffffffu, valid);
        pos = i + nk - a.Nq;
        lim = !valid ? 0 : a.causal ? min(nk, max(pos + 1, rec->pre)) : nk;
        doc = a.q_doc && valid ? a.q_doc[(int64_t)rec->b * a.Nq + i] : 0;
        if (SHAPED) slope = a.slopes && valid ? a.slopes[rec->head * a.G + row_h] * kLog2e : 0.f;
        m = -INFINITY;
        l = 0.f;
      }
      some = tile >= 0;
      if (some) {
        const int j0 = tile * kTile;
        // what all softmax warps do together for a tile that not every row sees whole
        auto prepare_masks = [&]() {
          if (j0 + kTile > nk && nk < a.Nk) {
            // values behind the last key count as zeros, whatever they hold
            const int s = t % KS;
            if (!mbar_wait_all(&v_full[s], (t / KS) & 1, abort_flag, a.err)) return false;
            if (half == 0 && j0 + row >= nk) {
#pragma unroll
              for (int c = 0; c < NB; ++c) {
                uint4* p = reinterpret_cast<uint4*>(sV + s * Sh::kBytes + c * kBlockBytes + row * 128);
#pragma unroll
                for (int q = 0; q < 8; ++q) p[q] = make_uint4(0u, 0u, 0u, 0u);
              }
            }
            fence_async_smem();
          }
          return true;
        };
        if (!(alive = mbar_wait_all(s_full, t & 1, abort_flag, a.err))) break;
        tc_fence_after();
        if (!work) {
          // a warp without rows only keeps the barriers going (its rows of P and O are never read)
          if (NB == 1) mbar_arrive_warp(s_free);
          if (!whole && !(alive = prepare_masks())) break;
          // not ahead of the working warps by more than this tile: their arrivals share a phase
          if (!first && !(alive = mbar_wait_all(pv_done, (t - 1) & 1, abort_flag, a.err))) break;
          mbar_arrive_warp(p_full);
        } else {
          uint32_t sv[64];
          tmem_ld_32x32b_x32(tSr, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld_32x32b_x32(tSr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          if constexpr (NB == 1) {
            tc_fence_before();
            mbar_arrive_warp(s_free);
          }
          if constexpr (SHAPED) {
            if (a.cap_out != 0.f) {
              // the form is chosen by what may be seen: neither padding nor what the last call
              // left in the rows beyond tq * G takes part
              const int lc = whole && valid ? 64 : lim - j0 - half * 64;  // lim is 0 in those rows
              if (__any_sync(0xffffffffu, lc < 64)) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                  if (c >= lc) sv[c] = 0u;
              }
              float top = 0.f;
#pragma unroll
              for (int c = 0; c < 64; c += 2)
                top = max3f(top, fabsf(__uint_as_float(sv[c])), fabsf(__uint_as_float(sv[c + 1])));
              if (__all_sync(0xffffffffu, top * a.cap_in <= kTanhSmall)) {
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                  float x0, x1;
                  mul2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), a.cap_in, a.cap_in, x0, x1);
                  tanh_small2(x0, x1, x0, x1);
                  mul2(x0, x1, a.cap_out, a.cap_out, x0, x1);
                  sv[c] = __float_as_uint(x0);
                  sv[c + 1] = __float_as_uint(x1);
                }
              } else {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                  sv[c] = __float_as_uint(a.cap_out * tanh_acc(__uint_as_float(sv[c]) * a.cap_in));
              }
            } else {
#pragma unroll
              for (int c = 0; c < 64; ++c) sv[c] = __float_as_uint(__uint_as_float(sv[c]) * a.sl2);
            }
            if (a.slopes) {
              const float p0 = (float)(pos - j0 - half * 64);
#pragma unroll
              for (int c = 0; c < 64; ++c)
                sv[c] = __float_as_uint(fmaf(-slope, fabsf(p0 - (float)c), __uint_as_float(sv[c])));
            }
          }
          if (!whole) {
            if (!(alive = prepare_masks())) break;
            const int lc = (flags & kOneDoc) && rec->doc != doc ? 0 : lim - j0 - half * 64;
            if (__any_sync(0xffffffffu, lc < 64)) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (c >= lc) sv[c] = __float_as_uint(-INFINITY);
            }
            if (a.k_pad && reads_docs(flags)) {
              const int32_t* sdoc = docs.get(r, alive) + half * 64;
              if (!alive) break;
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                const int4 d = *reinterpret_cast<const int4*>(sdoc + c);
                if (d.x != doc) sv[c] = __float_as_uint(-INFINITY);
                if (d.y != doc) sv[c + 1] = __float_as_uint(-INFINITY);
                if (d.z != doc) sv[c + 2] = __float_as_uint(-INFINITY);
                if (d.w != doc) sv[c + 3] = __float_as_uint(-INFINITY);
              }
            }
          }
          float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
            m0 = max3f(m0, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            m1 = max3f(m1, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
            m2 = max3f(m2, __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
            m3 = max3f(m3, __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
          }
          // the row's two halves share a maximum (two buffers: one barrier of the two warps per step)
          m0 = max3f(m0, m1, fmaxf(m2, m3));
          float* const sm = smax + (t & 1) * 2 * kTile;
          sm[half * kTile + row] = m0;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q4) : "memory");
          const float m_new = fmaxf(m, fmaxf(m0, sm[(half ^ 1) * kTile + row]) * mul);
          float alpha = 1.f;
          bool rescale = false;
          if (m == -INFINITY) {
            m = m_new;  // nothing seen so far: O's row is zeros (or not written yet)
          } else if (m_new > m + 8.f) {
            alpha = fast_ex2(m - m_new);
            l *= alpha;
            m = m_new;
            rescale = true;
          }
          const float base = m == -INFINITY ? 0.f : -m;  // a row without keys: exp2(-inf) = 0 throughout
          uint32_t pk[32];
          float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
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
          // P and O are free once the previous product is done
          if (!first && !(alive = mbar_wait_all(pv_done, (t - 1) & 1, abort_flag, a.err))) break;
          tc_fence_after();
          if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
            for (int c = 0; c < NB * 32; c += 32) {
              uint32_t q[32];
              tmem_ld_32x32b_x32(tOr + c, q);
              tmem_ld_wait_regs(q);
#pragma unroll
              for (int y = 0; y < 32; ++y) q[y] = __float_as_uint(__uint_as_float(q[y]) * alpha);
              tmem_st_x32(tOr + c, q);
            }
          }
          tmem_st_x32(tPr, pk);
          tmem_store_wait();
          tc_fence_before();
          mbar_arrive_warp(p_full);
        }
        ++t;
      }
      if (flags & kLast) {
        if (some && !(alive = mbar_wait_all(pv_done, (t - 1) & 1, abort_flag, a.err))) break;
        tc_fence_after();
        if (work) {
          // the row sum of both halves
          float* const sm = smax + (t & 1) * 2 * kTile;
          sm[half * kTile + row] = l;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q4) : "memory");
          l += sm[(half ^ 1) * kTile + row];
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q4) : "memory");
          const int i = rec->i0 + row_i, h = rec->head * a.G + row_h, b = rec->b;
          const int64_t at = (int64_t)rec->slot * kTile + row;
          const bool part = rec->slot >= 0;
          store_rows<T, NB, !SHAPED>(static_cast<T*>(a.o) + b * a.os[0] + i * a.os[1] + h * a.os[2],
                            part ? a.partial + at * a.D : nullptr, a.partial_ml + at * 2,
                            a.lse ? a.lse + ((int64_t)b * a.H + h) * a.Nq + i : nullptr, a.D, wide, half, tOr, some,
                            valid, m, l);
        }
        tc_fence_before();
      }
      ring.done(r);
    }
    leave_barrier(abort_flag, left + q4, 2, 1 + q4);
  }
  settle(abort_flag);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 256);
}

// Joins the parts of cut items: m = max m_z, o = sum 2^(m_z - m) O_z / sum 2^(m_z - m) l_z,
// over z in order, U parts at a time whose loads are all under way at once (few parts: fewer
// registers and more rows on an SM). LANES lanes per query row, 16 bytes each.
template <typename T, int LANES, int U>
__global__ void __launch_bounds__(256, U <= 4 ? 4 : 2) attn_join_kernel(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % LANES, row = (int)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int item = a.parts.first + (int)blockIdx.y;
  const int g = a.parts.group_of_item(item), parts = a.parts.parts[g];
  const int heads = a.B * a.KV, qt = a.qtiles - 1 - item / heads, b = item % heads / a.KV, kv = item % heads % a.KV;
  const int i = qt * a.tq + row / a.G, h = kv * a.G + row % a.G;
  if (row >= a.tq * a.G || i >= a.Nq) return;
  const int64_t at = ((int64_t)a.parts.slot[g] + (int64_t)(item - a.parts.item[g]) * parts) * kTile + row;
  const float* pml = a.partial_ml + at * 2;
  const float* po = a.partial + at * a.D + lane * 4;
  const bool in = lane * 4 < a.D;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int z0 = 0; z0 < parts; z0 += U) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (z0 + u < parts) {
        ml[u] = __ldcg(reinterpret_cast<const float2*>(pml + (int64_t)(z0 + u) * kTile * 2));
        if (in) v[u] = __ldcg(reinterpret_cast<const float4*>(po + (int64_t)(z0 + u) * kTile * a.D));
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
    // a part that saw no key has l = 0 and holds no values. One whose scores are all NaN has
    // no maximum either, since a maximum passes NaN over: its l is NaN and has to stay
    const float base = top == -INFINITY ? 0.f : top, keep = fast_ex2(m - base);
    m = top;
    if (l != 0.f) {
      l *= keep;
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[x] *= keep;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ml[u].y != 0.f) {
        const float f = fast_ex2(ml[u].x - base);
        l = fmaf(f, ml[u].y, l);
        acc[0] = fmaf(f, v[u].x, acc[0]);
        acc[1] = fmaf(f, v[u].y, acc[1]);
        acc[2] = fmaf(f, v[u].z, acc[2]);
        acc[3] = fmaf(f, v[u].w, acc[3]);
      }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (in) {
    T* dst = static_cast<T*>(a.o) + b * a.os[0] + i * a.os[1] + h * a.os[2] + lane * 4;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(Elem<T>::pack(acc[0] * inv, acc[1] * inv), Elem<T>::pack(acc[2] * inv, acc[3] * inv));
  }
  if (lane == 0 && a.lse) a.lse[((int64_t)b * a.H + h) * a.Nq + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// One warp per tile: the key tiles of all sequences, then the query tiles.
struct DocArgs {
  const int32_t* doc[2];
  int32_t *range[2], *pad[2];
  int32_t len[2], width[2], tiles[2];
  int64_t total[2];
};
__global__ void __launch_bounds__(128) attn_doc_range_kernel(const __grid_constant__ DocArgs a) {
  pdl_wait();
  pdl_trigger();
  int64_t w = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);
  const int set = w >= a.total[0];
  if (set) w -= a.total[0];
  if (w >= a.total[set]) return;
  const int lane = threadIdx.x & 31, len = a.len[set], width = a.width[set];
  const int64_t b = w / a.tiles[set];
  const int tile = (int)(w % a.tiles[set]);
  int lo = INT32_MAX, hi = INT32_MIN;
  const int row = (len + kTile - 1) / kTile * kTile;
  for (int i = tile * width + lane; i < min(len, (tile + 1) * width); i += 32) {
    const int d = a.doc[set][b * len + i];
    lo = min(lo, d);
    hi = max(hi, d);
    a.pad[set][b * row + i] = d;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    a.range[set][w * 2] = lo;
    a.range[set][w * 2 + 1] = hi;
  }
}

// ------------------------------------------------------------------ host side

int tiles_of(int n) { return (n + kTile - 1) / kTile; }

struct FwdPlan {
  int tq, qtiles, ktiles;
  int64_t items;
  Cut cut;
};
FwdPlan plan_forward(const sd_attention_cfg& c) {
  FwdPlan p;
  const int g = c.heads / c.kv_heads;
  p.tq = kTile / g;
  p.qtiles = (c.q_len + p.tq - 1) / p.tq;
  p.ktiles = tiles_of(c.k_len);
  p.items = (int64_t)c.batch * c.kv_heads * p.qtiles;
  // Time in key tiles of one SM. Two CTAs share an SM and take turns (measured: 1.13 us a
  // tile and SM at head_dim 64, 1.52 at 128, 0.75 more for capped scores; a CTA alone needs
  // 1.45 of that). Beginning and ending a unit takes 2.2 us more. The last units end about
  // half the longest unit's tiles after the average (of the cut ones where the rest are full
  // rounds). Parts cost one more launch and their FP32 rows, written and joined at 2 TB/s,
  // 4 TB/s where the items are few (128 queries on 8192 keys: 16 parts 30 us, 8 parts 40).
  const double nq = c.q_len, nk = c.k_len, L = p.ktiles, N = (double)p.items;
  const double least = !c.causal ? L : std::max(0.0, L - nq / kTile);  // tiles of the shortest item
  const double total = N * (c.causal && nq > nk ? 0.5 * L * nk / nq : 0.5 * (L + least)) / kSms;
  const double tile_us = (c.head_dim <= 64 ? 1.13 : 1.52) + (c.softcap > 0.f ? 0.75 : 0.0);
  const double alone = 1.45, extra = 2.2 / tile_us;
  const double part_tiles = std::min<double>(p.tq, nq) * g * (c.head_dim + 2) * 8.0 / 2.0e6 / tile_us;
  double best = 0;
  // units of at most `longest` tiles, the 149th longest has `second`
  auto offer = [&](const Cut& cut, double longest, double second) {
    const double units = (double)cut.units;
    longest += extra, second += extra;
    double t = units <= kSms       ? alone * longest
               : units <= 2 * kSms ? 2 * second + alone * (longest - second)
                                   : std::max(total + extra * units / kSms + 0.5 * longest, alone * longest);
    if (cut.slots) t += 5.0 / tile_us + cut.slots * part_tiles * (N < kSms ? 0.5 : 1.0);
    if (best == 0 || t < best) {
      best = t;
      p.cut = cut;
    }
  };
  for (int s = 1; s <= std::min(kMaxSplits, std::max(p.ktiles, 1)); ++s) {
    const double at = c.causal ? std::max(0.0, 1.0 - kSms / (N * s)) : 1.0;
    offer(cut_even(p.items, s), std::ceil(L / s), std::ceil((least + (L - least) * at) / s));
    if (N * s > 16.0 * kSms) break;  // far from idle: parts only cost
  }
  if (!c.causal) {
    // the items beyond full rounds of the GPU in parts: they end together
    const int64_t rest = p.items % (2 * kSms);
    if (p.items > 2 * kSms && rest)
      for (int s = 2; s <= std::min(kMaxSplits, p.ktiles) && rest * s <= 2 * kSms; ++s)
        offer(cut_last(p.items, rest, s), std::ceil(L / s), std::ceil(L / s));
  } else if (N <= 16.0 * kSms) {
    // items in parts of at most 1/k of the longest: short ones whole
    for (int k = 2; k <= std::min(kGroups, p.ktiles); ++k)
      offer(cut_levels(p.items, k, L, least), std::ceil(L / k), std::ceil(L / k));
  }
  return p;
}

// Scratch after the header: the documents' ranges and padded rows, then the forward's
// parts or what the backward needs.
struct DocSpace {
  size_t q_range, k_pad, q_pad, bytes;  // k_range comes first
};
DocSpace doc_space(const sd_attention_cfg& c) {
  DocSpace s;
  const size_t b = (size_t)c.batch;
  s.q_range = up256(b * tiles_of(c.k_len) * 8);
  s.k_pad = s.q_range + up256(b * std::max(plan_forward(c).qtiles, tiles_of(c.q_len)) * 8);
  s.q_pad = s.k_pad + b * tiles_of(c.k_len) * kTile * 4;
  s.bytes = s.q_pad + b * tiles_of(c.q_len) * kTile * 4;
  return s;
}
size_t ranges_bytes(const sd_attention_cfg& c) { return doc_space(c).bytes; }
size_t parts_bytes(const sd_attention_cfg& c) {
  return up256((size_t)plan_forward(c).cut.slots * kTile * (c.head_dim + 2) * 4);
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
  if ((int64_t)c->batch * c->heads > 1 << 24 || (int64_t)c->batch * c->heads * std::max(c->q_len, 1) > (int64_t)1 << 32 ||
      (int64_t)c->batch * c->kv_heads * std::max(c->k_len, 1) > (int64_t)1 << 36)
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
  const bool shaped = a.cap_out != 0.f || a.slopes;
  if (shaped)
    OP_TRY((allow_smem<attn_fwd_kernel<T, NB, true>>(Shape<NB>::kSmem, c.dev.index)));
  else
    OP_TRY((allow_smem<attn_fwd_kernel<T, NB, false>>(Shape<NB>::kSmem, c.dev.index)));
  a.hold_spins = injected_spins();
  auto* kernel = shaped ? attn_fwd_kernel<T, NB, true> : attn_fwd_kernel<T, NB, false>;
  const double pairs = (double)g.batch * g.heads * g.q_len * g.k_len;
  const double bytes = 2.0 * g.batch * g.head_dim * (2.0 * g.q_len * g.heads + 2.0 * g.k_len * g.kv_heads);
  sdp::Scope sc("attn_fwd", sdp::F_ATTN, 4.0 * pairs * g.head_dim, bytes, c.st, p.cut.slots ? 2 : 1);
  OP_TRY(launched(launch_pdl(kernel, dim3((unsigned)p.cut.units), dim3(kThreads),
                             Shape<NB>::kSmem, c.st, maps, a)));
  if (!p.cut.slots) return SD_OK;
  constexpr int kLanes = NB == 1 ? 16 : 32;
  const int rows = std::min(p.tq, g.q_len) * a.G, per = 256 / kLanes;  // of an item
  const int most = *std::max_element(p.cut.parts.parts, p.cut.parts.parts + p.cut.parts.n);
  auto* join = most <= 4 ? attn_join_kernel<T, kLanes, 4> : attn_join_kernel<T, kLanes, 8>;
  return launched(
      launch_pdl(join, dim3((rows + per - 1) / per, p.cut.parts.count), dim3(256), 0, c.st, a));
}

}  // namespace

bool attn_map(CUtensorMap* m, bool f16, const void* p, const int64_t* s, int batch, int tokens, int heads, int d,
              uint32_t box_heads, uint32_t box_tokens) {
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)heads, (uint64_t)tokens, (uint64_t)batch};
  const int64_t strides[3] = {s[2], s[1], s[0]};
  const uint32_t box[4] = {64, box_heads, box_tokens, 1};
  return encode_map(m, f16, p, 4, dims, strides, box);
}

sd_status attn_doc_ranges(const AttnArgs& a, int tq, cudaStream_t st) {
  DocArgs d;
  d.doc[0] = a.k_doc;
  d.doc[1] = a.q_doc;
  d.range[0] = const_cast<int32_t*>(a.k_range);
  d.range[1] = const_cast<int32_t*>(a.q_range);
  d.pad[0] = const_cast<int32_t*>(a.k_pad);
  d.pad[1] = const_cast<int32_t*>(a.q_pad);
  d.len[0] = a.Nk;
  d.len[1] = a.Nq;
  d.width[0] = kTile;
  d.width[1] = tq;
  for (int i = 0; i < 2; ++i) {
    d.tiles[i] = std::max(1, (d.len[i] + d.width[i] - 1) / d.width[i]);
    d.total[i] = d.len[i] ? (int64_t)a.B * d.tiles[i] : 0;
  }
  sdp::Scope sc("attn_doc_range", sdp::F_OTHER, 0, 4.0 * a.B * (a.Nk + a.Nq), st);
  const int64_t warps = d.total[0] + d.total[1];
  return launched(launch_pdl(attn_doc_range_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, d));
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
  if (a.k_doc) {
    const DocSpace d = doc_space(g);
    uint8_t* w = c.ws + kOpHeader;
    a.k_range = reinterpret_cast<int32_t*>(w);
    a.q_range = reinterpret_cast<int32_t*>(w + d.q_range);
    a.k_pad = reinterpret_cast<int32_t*>(w + d.k_pad);
    a.q_pad = reinterpret_cast<int32_t*>(w + d.q_pad);
  }
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
  a.parts = p.cut.parts;
  a.o = o;
  a.lse = lse;
  a.clear_err = 1;
  if (p.cut.slots) {
    a.partial = reinterpret_cast<float*>(c.ws + kOpHeader + ranges_bytes(*cfg));
    a.partial_ml = a.partial + (size_t)p.cut.slots * kTile * cfg->head_dim;
  }
  if (cfg->k_len == 0) {
    shaped.k_len = 1;  // a map has no empty dimension; no tile of it is visited
    c.cfg = &shaped;
  }
  if (a.k_doc) OP_TRY(attn_doc_ranges(a, p.tq, c.st));
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
