// Gated feed-forward block and its gradients:
//   [v | z] = x w1^T + b1,  h = v act(z),  y = h w2^T + b2;
//   dh = dy w2,  dv = dh act(z),  dz = dh v act'(z),  dpre = [dv | dz],
//   dx = dpre w1,  dw1 = dpre^T x,  dw2 = dy^T h,  db1, db2 = column sums of dpre, dy.
//
// Bound by the tensor cores (6 and 12 tokens d d_hidden operations forward and
// backward), or by reading the weights when there are few tokens.
//
// ff_gemm_kernel computes every product with one main loop: a CTA pair owns
// 256 x bn tiles (tcgen05.mma.cta_group::2, FP32 accumulators double-buffered in
// TMEM), operands come by TMA with the 128-byte swizzle either K-major or
// MN-major, so none of the six products needs a transposed copy of anything:
//   forward 1   A = x K-major,      B = w1 K-major, half a tile of value rows and
//               half of gate rows (one CTA of the pair loads each), so the
//               epilogue holds v and z of the same hidden column
//   forward 2   A = h K-major,      B = w2 K-major
//   dh          A = dy K-major,     B = w2 MN-major; the epilogue turns dh into
//               dv, dz and h from the saved v and z
//   dx          A = dpre K-major,   B = w1 MN-major
//   dw1, dw2    A = dpre, dy MN-major, B = x, h MN-major (the reduction runs over
//               the tokens), split over the tokens where the weights have few tiles
#include <string.h>

#include <algorithm>

#include "op_tma.cuh"
#include "profile.h"

namespace sdo {
namespace {

// Warp 0 TMA, warp 1 MMA, the others epilogue: sixteen for the gate and its gradient, whose
// activations bounded them with eight (9216 x 320 x 1280: forward 22 instead of 29 us,
// backward 131 instead of 135), eight elsewhere.
template <int EPI>
constexpr int kEpiWarps = EPI == 0 ? 8 : 16;
template <int EPI>
constexpr int kThreads = 64 + 32 * kEpiWarps<EPI>;
constexpr int kSubA = 128 * 64 * 2;  // one CTA's 128 rows x 64 reduction elements
constexpr int kRingBytes = 196608;
constexpr int kColBytes = 2 * 4 * 256 * 2 * 4;  // EPI_GATE_GRAD: column sums [2][4 row quarters][2][256]
constexpr int kSmemBytes = 1024 + kRingBytes + 256 + 2 * 256 * 4 + kColBytes;
constexpr int kPairs = 74;        // CTA pairs the plan assumes (148 SMs)
constexpr int kMaxSplits = 16;
constexpr size_t kSplitBytes = size_t(64) << 20;

enum Epi { EPI_PLAIN = 0, EPI_GATE = 1, EPI_GATE_GRAD = 2 };

struct FfMaps {
  CUtensorMap a, b, pre;
};

struct FfArgs {
  int32_t M, N;           // output rows and columns (hidden columns for the gated epilogues)
  int32_t kb;             // 64-wide blocks of the reduction
  int32_t kb_split;       // blocks of one split (even)
  int32_t splits, tiles_n, units;
  int32_t bn, step_n;     // MMA width of a tile; output columns of a tile (bn, or bn/2 when gated)
  int32_t a_mn, b_mn;     // operand stored MN-major
  int32_t gate_row;       // first gate row of B (EPI_GATE)
  int32_t stages, sub_bytes, b_bytes;
  uint32_t idesc;
  int32_t act;
  const void* bias;       // [N], or [2N] for EPI_GATE
  void* out;              // EPI_PLAIN: [M][N]; else h [M][N]
  void* pre;              // EPI_GATE: [M][2N] out or null; EPI_GATE_GRAD: [M][2N] in
  void* dpre;             // EPI_GATE_GRAD: [M][2N] out
  float* partial;         // EPI_PLAIN with splits: [splits][M][N]
  float* colsum;          // EPI_GATE_GRAD: [M / 128][2N] column sums of dpre, or null
  int* err;
  int32_t clear_err;
  int32_t hold_spins;     // tests only: the loading thread first waits, this long, for what never comes
};

// 16 elements of T, packed, to consecutive places, and back; n as below.
template <typename T>
__device__ __forceinline__ void put16(T* p, const uint32_t (&w)[8], int n, bool wide) {
  if (wide && n >= 16) {
    st_global_v8(p, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    if (n > 8) *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&f)[16], int n, bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = Elem<T>::pack(f[2 * j], f[2 * j + 1]);
  put16<T>(p, w, n, wide);
}
template <typename T>
__device__ __forceinline__ void load16(const T* p, uint32_t (&r)[8], int n, bool wide) {
  if (wide && n >= 16) {
    ld_global_v8(p, r);
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint4 b = n > 8 ? *reinterpret_cast<const uint4*>(p + 8) : make_uint4(0u, 0u, 0u, 0u);
    r[0] = a.x;
    r[1] = a.y;
    r[2] = a.z;
    r[3] = a.w;
    r[4] = b.x;
    r[5] = b.y;
    r[6] = b.z;
    r[7] = b.w;
  }
}
// Sums of 8 columns over the warp's 32 rows (one row per lane): lanes 4j to 4j + 3 get
// column j. Halves of the columns change places, so it takes 9 exchanges, not 40.
__device__ __forceinline__ float column_sum8(float (&a)[8], int lane) {
#pragma unroll
  for (int w = 4; w > 0; w >>= 1) {
    const bool up = lane & (4 * w);
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? a[i] : a[i + w], keep = up ? a[i + w] : a[i];
      a[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * w);
    }
  }
  const float s = a[0] + __shfl_xor_sync(0xffffffffu, a[0], 2);
  return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

// 32 FP32 values to 32 consecutive elements of T, `n` of them inside (n a multiple of 8).
// A thread stores a row piece of its own, so a warp's instruction touches 32 rows: 32-byte
// accesses where rows start on 32-byte boundaries (`wide`) fill whole sectors.
template <typename T>
__device__ __forceinline__ void store32(T* p, const float (&f)[32], int n, bool wide) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = Elem<T>::pack(f[16 * i + 2 * j], f[16 * i + 2 * j + 1]);
    if (wide && 16 * i + 16 <= n) {
      st_global_v8(p + 16 * i, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    } else {
      if (16 * i < n) *reinterpret_cast<uint4*>(p + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
      if (16 * i + 8 < n) *reinterpret_cast<uint4*>(p + 16 * i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}
template <typename T, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<EPI>, 1)
    ff_gemm_kernel(const __grid_constant__ FfMaps maps, const __grid_constant__ FfArgs args) {
  constexpr int kEpiThreads = 32 * kEpiWarps<EPI>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingBytes);  // [stages <= 8]
  uint64_t* empty = full + 8;
  uint64_t* acc_full = empty + 8;   // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2], used in the even CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* ecols = reinterpret_cast<float*>(smem + kRingBytes + 256);  // [2][256]
  float* csums = ecols + 512;                                        // [2][4][2][256]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = pair_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int stages = args.stages, sub_bytes = args.sub_bytes;
  const int stage_bytes = 2 * sub_bytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) pair_tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  pair_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  if (args.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *args.err = 0;

  if (warp == 0) {
    if (lane == 0) {
      const int half = args.bn >> 1;
      const int bblocks = (half + 63) >> 6;
      int s = 0;
      uint32_t ph = 0, q = 0;
      bool ok = args.hold_spins == 0 || mbar_wait(&full[0], 0, abort_flag, args.err, (uint32_t)args.hold_spins);
      for (int u = pair; u < args.units && ok; u += npairs) {
        const int z = u % args.splits, rest = u / args.splits;
        const int m0 = ((rest / args.tiles_n) * 2 + (int)rank) * 128;
        const int n0 = (rest % args.tiles_n) * args.step_n;
        const int brow = EPI == EPI_GATE ? (rank ? args.gate_row + n0 : n0) : n0 + (int)rank * half;
        const int hi = min(args.kb, (z + 1) * args.kb_split);
        if (EPI == EPI_GATE_GRAD) {
          // the epilogue's v and z of this tile, on their way to L2 during its main loop
          for (int c = 0; c < args.bn && n0 + c < args.N; c += 64) {
            tma_prefetch_2d(&maps.pre, n0 + c, m0);
            tma_prefetch_2d(&maps.pre, args.N + n0 + c, m0);
          }
        }
        for (int kb = z * args.kb_split; kb < hi; kb += 2) {
          if (q >= (uint32_t)stages && !mbar_wait(&empty[s], ph ^ 1, abort_flag, args.err)) {
            ok = false;
            break;
          }
          const int nsub = min(2, hi - kb);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * nsub * (kSubA + args.b_bytes)));
          for (int h = 0; h < nsub; ++h) {
            uint8_t* da = smem + s * stage_bytes + h * sub_bytes;
            uint8_t* db = da + kSubA;
            const int k = (kb + h) * 64;
            if (args.a_mn) {
              pair_load_2d(da, &maps.a, &full[s], m0, k);
              pair_load_2d(da + 8192, &maps.a, &full[s], m0 + 64, k);
            } else {
              pair_load_2d(da, &maps.a, &full[s], k, m0);
            }
            if (args.b_mn) {
              for (int i = 0; i < bblocks; ++i) pair_load_2d(db + i * 8192, &maps.b, &full[s], brow + i * 64, k);
            } else {
              pair_load_2d(db, &maps.b, &full[s], k, brow);
            }
          }
          ++q;
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // descriptor steps of 16 reduction elements: 32 bytes K-major, 2048 bytes MN-major
      const uint32_t a_step = args.a_mn ? 128 : 2, b_step = args.b_mn ? 128 : 2;
      const uint32_t a0 = smem_u32(smem), b0 = a0 + kSubA;
      const uint32_t a_base = args.a_mn ? desc_mn(a0, 8192) : desc_k(a0);
      const uint32_t b_base = args.b_mn ? desc_mn(b0, 8192) : desc_k(b0);
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = pair; u < args.units && ok; u += npairs, ++it) {
        const int z = u % args.splits;
        const int hi = min(args.kb, (z + 1) * args.kb_split);
        const int b = it & 1;
        if (!mbar_wait(&acc_empty[b], ((it >> 1) & 1) ^ 1, abort_flag, args.err)) break;
        tc_fence_after();
        const uint32_t tacc = tmem + (uint32_t)(b * 256);
        uint32_t acc = 0;
        for (int kb = z * args.kb_split; kb < hi; kb += 2) {
          if (!mbar_wait(&full[s], ph, abort_flag, args.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int nsub = min(2, hi - kb);
          for (int h = 0; h < nsub; ++h) {
            const uint32_t o = (uint32_t)(s * stage_bytes + h * sub_bytes) >> 4;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              pair_mma(tacc, a_base + o + k * a_step, b_base + o + k * b_step, args.idesc, acc);
              acc = 1;
            }
          }
          pair_commit(&empty[s]);
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok) pair_commit(&acc_full[b]);
      }
    }
  } else {
    const int et = threadIdx.x - 64;
    const int half = (warp - 2) >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t empty_addr[2] = {pair_addr(smem_u32(&acc_empty[0]), 0), pair_addr(smem_u32(&acc_empty[1]), 0)};
    const int M = args.M, N = args.N, bn = args.bn, step_n = args.step_n, act = args.act;
    const T* const bias = static_cast<const T*>(args.bias);
    T* const out = static_cast<T*>(args.out);
    T* const pre = static_cast<T*>(args.pre);
    T* const dpre = static_cast<T*>(args.dpre);
    float* const partial = args.partial;
    const bool wide = N % 16 == 0 && ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(pre) |
                                       reinterpret_cast<uintptr_t>(dpre)) & 31) == 0;
    int it = 0;
    for (int u = pair; u < args.units; u += npairs, ++it) {
      const int z = u % args.splits, rest = u / args.splits;
      const int n0 = (rest % args.tiles_n) * step_n;
      const int64_t grow = ((rest / args.tiles_n) * 2 + (int)rank) * (int64_t)128 + row;
      const int b = it & 1;
      float* const ecol = ecols + b * 256;
      if (bias) {
        // this tile's biases, while its main loop runs; the buffer was last read two tiles ago
        for (int c = et; c < bn; c += kEpiThreads) {
          int n = n0 + c;
          bool in = n < N;
          if (EPI == EPI_GATE) {
            const int j = c < step_n ? c : c - step_n;
            in = n0 + j < N;
            n = n0 + j + (c < step_n ? 0 : N);
          }
          ecol[c] = in ? Elem<T>::to_f(bias[n]) : 0.f;
        }
        asm volatile("bar.sync 2, %0;" ::"n"(kEpiThreads) : "memory");
      }
      const bool in = grow < M;
      // the saved v and z of this row's first chunk while the main loop runs, each further
      // chunk's once the one before is computed
      [[maybe_unused]] uint32_t pv[8], pz[8];
      auto load_pre = [&](int c) {
        const int left = N - (n0 + c);
        if (in && c < step_n && left > 0) {
          load16<T>(pre + grow * 2 * N + n0 + c, pv, left, wide);
          load16<T>(pre + grow * 2 * N + N + n0 + c, pz, left, wide);
        }
      };
      if (EPI == EPI_GATE_GRAD) load_pre(half * 16);
      if (!mbar_wait_all(&acc_full[b], (it >> 1) & 1, abort_flag, args.err)) {
        // other warps may have got through, and wait for this one at the barriers
        asm volatile("bar.sync 3, %0;" ::"n"(kEpiThreads) : "memory");
        continue;
      }
      tc_fence_after();
      const uint32_t tacc = tmem + (uint32_t)(b * 256) + lane_off;
      if constexpr (EPI == EPI_GATE_GRAD) {
        float* const cs = csums + b * 2048 + q4 * 512;
        for (int c = half * 16; c < step_n && n0 + c < N; c += 64) {
          const int left = N - (n0 + c);
          uint32_t r[16], of[8], oz[8], oh[8];
          tmem_ld_x16(tacc + c, r);
          tmem_ld_wait_16(r);
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            float zv[8], d[8], a8[8], f[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const int w = (i + j) / 2;
              zv[j] = Elem<T>::lo(pz[w]);
              zv[j + 1] = Elem<T>::hi(pz[w]);
              // dz = dh v act'(z)
              mul2(__uint_as_float(r[i + j]), __uint_as_float(r[i + j + 1]), Elem<T>::lo(pv[w]), Elem<T>::hi(pv[w]), d[j],
                   d[j + 1]);
            }
            act_grad_vec<8>(zv, d, a8, act);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const int w = (i + j) / 2;
              float h0, h1;
              mul2(__uint_as_float(r[i + j]), __uint_as_float(r[i + j + 1]), a8[j], a8[j + 1], f[j], f[j + 1]);
              mul2(Elem<T>::lo(pv[w]), Elem<T>::hi(pv[w]), a8[j], a8[j + 1], h0, h1);
              of[w] = Elem<T>::pack(f[j], f[j + 1]);
              oz[w] = Elem<T>::pack(d[j], d[j + 1]);
              oh[w] = Elem<T>::pack(h0, h1);
            }
            if (args.colsum) {
              if (!in) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = d[j] = 0.f;
              }
              const float sv = column_sum8(f, lane), sz = column_sum8(d, lane);
              if (!(lane & 3)) {
                cs[c + i + (lane >> 2)] = sv;
                cs[256 + c + i + (lane >> 2)] = sz;
              }
            }
          }
          if (in) {
            put16<T>(dpre + grow * 2 * N + n0 + c, of, left, wide);
            put16<T>(dpre + grow * 2 * N + N + n0 + c, oz, left, wide);
            if (out) put16<T>(out + grow * N + n0 + c, oh, left, wide);
          }
          load_pre(c + 64);
        }
      }
      if constexpr (EPI == EPI_GATE) {
        for (int c = half * 16; c < step_n; c += 64) {
          const int left = N - (n0 + c);  // columns of this chunk inside the output
          if (left <= 0) break;
          uint32_t r[16], r2[16];
          tmem_ld_x16(tacc + c, r);
          tmem_ld_x16(tacc + step_n + c, r2);
          tmem_ld_wait_16(r);
          tmem_ld_wait_16(r2);
          float f[16], g[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f[i] = __uint_as_float(r[i]);
            g[i] = __uint_as_float(r2[i]);
          }
          if (bias) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 bv = *reinterpret_cast<const float4*>(ecol + c + i);
              const float4 bz = *reinterpret_cast<const float4*>(ecol + step_n + c + i);
              add2(f[i], f[i + 1], bv.x, bv.y, f[i], f[i + 1]);
              add2(f[i + 2], f[i + 3], bv.z, bv.w, f[i + 2], f[i + 3]);
              add2(g[i], g[i + 1], bz.x, bz.y, g[i], g[i + 1]);
              add2(g[i + 2], g[i + 3], bz.z, bz.w, g[i + 2], g[i + 3]);
            }
          }
          if (pre && in) {
            store16<T>(pre + grow * 2 * N + n0 + c, f, left, wide);
            store16<T>(pre + grow * 2 * N + N + n0 + c, g, left, wide);
          }
          act_vec<16>(g, act);
#pragma unroll
          for (int i = 0; i < 16; i += 2) mul2(f[i], f[i + 1], g[i], g[i + 1], f[i], f[i + 1]);
          if (in) store16<T>(out + grow * N + n0 + c, f, left, wide);
        }
      }
      if constexpr (EPI == EPI_PLAIN) {
        for (int c = half * 32; c < step_n; c += 64) {
          const int left = N - (n0 + c);  // columns of this chunk inside the output
          if (left <= 0) break;
          uint32_t r[32];
          tmem_ld_32x32b_x32(tacc + c, r);
          tmem_ld_wait_regs(r);
          if (partial) {
            if (in) {
              // N is a multiple of 8 and the parts start on 256 bytes (scratch()): whole 32-byte sectors
              float* p = partial + ((int64_t)z * M + grow) * N + n0 + c;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (8 * i < left)
                  st_global_v8(p + 8 * i, r[8 * i], r[8 * i + 1], r[8 * i + 2], r[8 * i + 3], r[8 * i + 4],
                               r[8 * i + 5], r[8 * i + 6], r[8 * i + 7]);
            }
          } else {
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
            if (bias) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 bv = *reinterpret_cast<const float4*>(ecol + c + i);
                add2(f[i], f[i + 1], bv.x, bv.y, f[i], f[i + 1]);
                add2(f[i + 2], f[i + 3], bv.z, bv.w, f[i + 2], f[i + 3]);
              }
            }
            if (in) store32<T>(out + grow * N + n0 + c, f, left, wide);
          }
        }
      }
      // this warp's TMEM reads are done; the even CTA's MMA warp may reuse the accumulator
      // once all epilogue warps of both CTAs have said so
      tc_fence_before();
      asm volatile("bar.sync 3, %0;" ::"n"(kEpiThreads) : "memory");
      if (et == 0) pair_arrive(empty_addr[b]);
      if (EPI == EPI_GATE_GRAD && args.colsum && et < step_n && n0 + et < N && grow - row < M) {
        // the four row quarters in order; this buffer is written again two tiles from now
        const float* c = csums + b * 2048 + et;
        float* o = args.colsum + (grow - row) / 128 * 2 * N + n0 + et;
        o[0] = (c[0] + c[512]) + (c[1024] + c[1536]);
        o[N] = (c[256] + c[768]) + (c[1280] + c[1792]);
      }
    }
  }

  settle(abort_flag);
  tc_fence_before();
  pair_sync();
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ few tokens
// Bound by reading the weights: a warp per weight row (or a few, which share the
// tokens' values), each lane 16 bytes at a time, several loads under way, FP32 sums
// joined across the warp.
// What an earlier kernel may still be writing when one of these starts (x, h, FP32 parts) is
// read by plain loads behind pdl_wait(): no __restrict__ and no read-only path, which are
// for memory that nobody writes while the kernel lives.
constexpr int kSmallThreads = 256;
constexpr int kSmallTokens = 4;  // 5 to 8 tokens took 29 to 30 us at 1280 x 5120, the tensor cores 24

// acc[r][m] += row r's 8 weights times token m's 8 values (even and odd elements apart as
// packed FP32 where there are several tokens). All tokens' values are asked for at once
// and without a branch, else their latencies would add up: rows past the last token
// repeat it and are not stored.
template <typename T, int MT, int R>
__device__ __forceinline__ void dot_step(const uint4 (&w)[R], const T* x, int64_t ld, int M, bool in,
                                         float (&acc)[R][MT][2]) {
  uint4 xv[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xv[m] = in ? *reinterpret_cast<const uint4*>(x + min(m, M - 1) * ld) : make_uint4(0u, 0u, 0u, 0u);
  float f[R][8];
#pragma unroll
  for (int r = 0; r < R; ++r) unpack_vec<T, 8>(w[r], f[r]);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float v[8];
    unpack_vec<T, 8>(xv[m], v);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (MT == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[r][m][j & 1] = fmaf(f[r][j], v[j], acc[r][m][j & 1]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          fma2v(f[r][j], f[r][j + 1], v[j], v[j + 1], acc[r][m][0], acc[r][m][1], acc[r][m][0], acc[r][m][1]);
      }
    }
  }
}
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// h = v act(z) (and pre = [v | z]): a warp reads the value and gate rows of C hidden columns.
template <typename T, int MT, int C>
__global__ void __launch_bounds__(kSmallThreads) ff_small_up_kernel(const T* x, const T* w1, const T* b1, T* pre, T* h,
                                                                    int M, int D, int F, int act, int* err) {
  constexpr int R = 2 * C;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *err = 0;
  const int lane = threadIdx.x & 31;
  const int j0 = (blockIdx.x * (kSmallThreads / 32) + (threadIdx.x >> 5)) * C;  // F is a multiple of C
  if (j0 >= F) return;
  const uint4* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    w[r] = reinterpret_cast<const uint4*>(w1 + (int64_t)((r < C ? 0 : F) + j0 + r % C) * D);
  float acc[R][MT][2];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m][0] = acc[r][m][1] = 0.f;
  constexpr int U = 8 / R;
  for (int i0 = lane; i0 < D / 8; i0 += 32 * U) {
    uint4 v[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
        v[u][r] = i0 + 32 * u < D / 8 ? w[r][i0 + 32 * u] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      dot_step<T, MT, R>(v[u], x + (int64_t)(i0 + 32 * u) * 8, D, M, i0 + 32 * u < D / 8, acc);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = j0 + c;
    const float bv = b1 ? Elem<T>::to_f(b1[j]) : 0.f, bz = b1 ? Elem<T>::to_f(b1[F + j]) : 0.f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float v = lane_sum(acc[c][m][0] + acc[c][m][1]) + bv;
      const float z = lane_sum(acc[C + c][m][0] + acc[C + c][m][1]) + bz;
      if (m < M && lane == 0) {
        h[(int64_t)m * F + j] = Elem<T>::from_f(v * act_f(z, act));
        if (pre) {
          pre[(int64_t)m * 2 * F + j] = Elem<T>::from_f(v);
          pre[(int64_t)m * 2 * F + F + j] = Elem<T>::from_f(z);
        }
      }
    }
  }
}

// y = h w2^T + b2: four warps share the rows of R output columns, a quarter of the
// reduction each. The first weights are asked for before the wait for h: no kernel of the
// call writes them, and the kernel before this one started only after everything ahead
// of the call had finished.
template <typename T, int MT, int R>
__global__ void __launch_bounds__(kSmallThreads) ff_small_down_kernel(const T* h, const T* w2, const T* b2, T* y, int M,
                                                                      int F, int N) {
  __shared__ float red[kSmallThreads / 32][R][MT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & 3;
  const int n0 = (blockIdx.x * (kSmallThreads / 128) + (warp >> 2)) * R;  // N is a multiple of R
  const int per = (F / 8 + 3) / 4, lo = part * per, hi = n0 < N ? min(F / 8, lo + per) : 0;
  const uint4* w = reinterpret_cast<const uint4*>(w2 + (int64_t)min(n0, N - R) * F);
  const int64_t row = F / 8;
  float acc[R][MT][2];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m][0] = acc[r][m][1] = 0.f;
  constexpr int U = 5;
  uint4 v[U][R];
  auto ask = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
        v[u][r] = i0 + 32 * u < hi ? __ldg(w + r * row + i0 + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
  };
  ask(lo + lane);
  pdl_wait();
  pdl_trigger();
  for (int i0 = lo + lane; i0 < hi; i0 += 32 * U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      dot_step<T, MT, R>(v[u], h + (int64_t)(i0 + 32 * u) * 8, F, M, i0 + 32 * u < hi, acc);
    ask(i0 + 32 * U);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float s = lane_sum(acc[r][m][0] + acc[r][m][1]);
      if (lane == 0) red[warp][r][m] = s;
    }
  __syncthreads();
  if (part == 0 && n0 < N && lane < R * MT) {
    const int r = lane / MT, m = lane % MT;
    float s = red[warp][r][m];
    for (int p = 1; p < 4; ++p) s += red[warp + p][r][m];
    if (m < M) y[(int64_t)m * N + n0 + r] = Elem<T>::from_f(s + (b2 ? Elem<T>::to_f(b2[n0 + r]) : 0.f));
  }
}

// out = sum of the splits (in order) + bias, 8 columns per thread.
template <typename T>
__global__ void __launch_bounds__(256) ff_join_kernel(const float* partial, int splits, int64_t M, int N,
                                                      const T* bias, T* out) {
  pdl_wait();
  pdl_trigger();
  const int64_t vecs = M * N / 8, stride = M * N;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * blockDim.x) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
    // eight parts at a time, all asked for before the first is added
    for (int z = 0; z < splits; z += 8) {
      float4 u[8], w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (z + k < splits) {
          const float4* p = reinterpret_cast<const float4*>(partial + (z + k) * stride + i * 8);
          u[k] = __ldcg(p);
          w[k] = __ldcg(p + 1);
        }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (z + k >= splits) break;
        f[0] += u[k].x;
        f[1] += u[k].y;
        f[2] += u[k].z;
        f[3] += u[k].w;
        f[4] += w[k].x;
        f[5] += w[k].y;
        f[6] += w[k].z;
        f[7] += w[k].w;
      }
    }
    if (bias) {
      float b[8];
      unpack_vec<T, 8>(*reinterpret_cast<const uint4*>(bias + i * 8 % N), b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += b[j];
    }
    *reinterpret_cast<uint4*>(out + i * 8) = pack_vec<T, 8>(f);
  }
}

// Column sums of dy [rows][n] for db2: a CTA sums 256 columns over a share of the rows
// into an FP32 part.
template <typename T>
__global__ void __launch_bounds__(256) ff_colsum_kernel(const T* m, int n, int64_t rows, int64_t chunk_rows,
                                                        float* part, int* clear_err) {
  __shared__ float red[8][256];
  pdl_wait();
  pdl_trigger();
  if (clear_err && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *clear_err = 0;
  const int c0 = (int)blockIdx.x * 256;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = c0 + tx * 8;
  const int64_t r0 = blockIdx.y * chunk_rows, r1 = min(rows, r0 + chunk_rows);
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.f;
  if (c < n) {
#pragma unroll 4
    for (int64_t r = r0 + ty; r < r1; r += 8) {
      float f[8];
      unpack_vec<T, 8>(*reinterpret_cast<const uint4*>(m + r * n + c), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += f[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) red[ty][tx * 8 + j] = s[j];
  __syncthreads();
  if (c0 + (int)threadIdx.x < n) {
    float t = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) t += red[y][threadIdx.x];
    part[(int64_t)blockIdx.y * n + c0 + threadIdx.x] = t;
  }
}

// db1 and db2 from their parts, 32 columns per CTA: eight slices of the parts, then the
// slices in order.
struct BiasJoin {
  const float* part[2];  // [parts][n]
  void* out[2];
  int32_t n[2], blocks[2];
  int64_t parts[2];
};
template <typename T>
__global__ void __launch_bounds__(256) ff_bias_join_kernel(const __grid_constant__ BiasJoin a) {
  __shared__ float red[8][32];
  pdl_wait();
  pdl_trigger();
  const int which = (int)blockIdx.x >= a.blocks[0];
  const int n = a.n[which], tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = ((int)blockIdx.x - (which ? a.blocks[0] : 0)) * 32 + tx;
  float s = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int64_t p = ty; p < a.parts[which]; p += 8) s += a.part[which][p * n + c];
  }
  red[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < n) {
#pragma unroll
    for (int y = 1; y < 8; ++y) s += red[y][tx];
    static_cast<T*>(a.out[which])[c] = Elem<T>::from_f(s);
  }
}

// ------------------------------------------------------------------ host side

struct Product {
  int64_t M, K;
  int N;
  bool gated;  // B holds value and gate rows (EPI_GATE)
  bool may_split, a_mn, b_mn;
};
struct Plan {
  int bn, splits, kb_split;
};

// Tile width and number of splits with the least predicted time, in cycles of one
// SM: a 64-wide block costs the slower of its MMAs (2 bn cycles, 4 x 80 to issue them)
// and its operands' arrival (50 bytes a cycle), a tile about 1500 cycles more for
// filling the pipeline and its last epilogue, and a split product the writing and
// joining of its FP32 parts.
Plan plan_product(const Product& p) {
  const int widths[] = {256, 192, 160, 128, 96, 64};
  const int64_t kb = (p.K + 63) / 64, pairs_m = (p.M + 255) / 256;
  Plan best{0, 1, 0};
  double best_cost = 0;
  // reduction blocks of a part for each number of splits, 0 where it would leave none or few
  int64_t pers[kMaxSplits + 1];
  for (int sp = 1; sp <= (p.may_split ? kMaxSplits : 1); ++sp) {
    int64_t per = ((uint32_t)kb + sp - 1) / (uint32_t)sp;
    per = (per + 1) / 2 * 2;
    const bool use = sp == 1 || (per >= 4 && ((uint32_t)kb + per - 1) / (uint32_t)per == (uint32_t)sp);
    pers[sp] = use ? per : 0;
  }
  for (int bn : widths) {
    if (p.gated && bn % 64) continue;  // each half whole 32-column chunks
    const int step = p.gated ? bn / 2 : bn;
    const int64_t tiles = pairs_m * ((p.N + step - 1) / step);
    // more splits than fill the GPU four times only cost
    const int most = !p.may_split ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, 4 * kPairs / tiles));
    for (int sp = 1; sp <= most; ++sp) {
      const int64_t per = pers[sp];
      if (!per) continue;
      if (sp > 1 && (size_t)sp * p.M * p.N * 4 > kSplitBytes) break;
      const int64_t rounds = (tiles * sp + kPairs - 1) / kPairs;
      const double b_bytes = p.b_mn ? (bn / 2 + 63) / 64 * 8192.0 : bn * 64.0;
      const double block = std::max(std::max(2.0 * bn, 320.0), (kSubA + b_bytes) / 50.0);
      double cost = rounds * (per * block + 1500.0);
      if (sp > 1) cost += 4000.0 + 1.9 * 2.0 * sp * p.M * p.N * 4 / 4000.0;
      if (best.bn == 0 || cost < best_cost) {
        best = Plan{bn, sp, (int)per};
        best_cost = cost;
      }
    }
  }
  return best;
}

size_t split_bytes(const Product& p) {
  const Plan g = plan_product(p);
  return g.splits > 1 ? (size_t)g.splits * p.M * p.N * 4 : 0;
}

int pairs_available(const Device& dev) { return std::min(kPairs, dev.sms / 2); }

struct Call {
  const sd_gated_ff_cfg* cfg;
  Device dev;
  cudaStream_t st;
  int* err;
  float* partial;
  bool first = true;  // the next launch clears the error word
};

// One product of A and B (16-bit, row-major in memory: [M or K rows][...]).
template <typename T, int EPI>
sd_status product(Call& c, const char* name, const Product& p, const void* A, const void* B, FfArgs a) {
  constexpr bool f16 = Elem<T>::kF16;
  const Plan g = plan_product(p);
  FfMaps maps;
  memset(&maps, 0, sizeof(maps));
  const uint64_t M = (uint64_t)p.M, K = (uint64_t)p.K, rows_b = (uint64_t)p.N * (p.gated ? 2 : 1);
  const uint64_t da[2] = {p.a_mn ? M : K, p.a_mn ? K : M}, db[2] = {p.b_mn ? rows_b : K, p.b_mn ? K : rows_b};
  const int64_t sa[1] = {(int64_t)da[0]}, sb[1] = {(int64_t)db[0]};
  const uint32_t ba[2] = {64, p.a_mn ? 64u : 128u}, bb[2] = {64, p.b_mn ? 64u : (uint32_t)g.bn / 2};
  if (!encode_map(&maps.a, f16, A, 2, da, sa, ba) || !encode_map(&maps.b, f16, B, 2, db, sb, bb)) return SD_ERR_LAUNCH;
  if (EPI == EPI_GATE_GRAD) {
    const uint64_t dp[2] = {2 * (uint64_t)p.N, M};
    const int64_t sp[1] = {2 * (int64_t)p.N};
    const uint32_t bp[2] = {64, 128};
    if (!encode_map(&maps.pre, f16, a.pre, 2, dp, sp, bp)) return SD_ERR_LAUNCH;
  }
  a.M = (int32_t)p.M;
  a.N = p.N;
  a.kb = (int32_t)((p.K + 63) / 64);
  a.kb_split = g.kb_split;
  a.splits = g.splits;
  a.bn = g.bn;
  a.step_n = p.gated ? g.bn / 2 : g.bn;
  a.tiles_n = (p.N + a.step_n - 1) / a.step_n;
  const int64_t units = (p.M + 255) / 256 * a.tiles_n * g.splits;
  if (units > INT32_MAX) return SD_ERR_UNSUPPORTED;
  a.units = (int32_t)units;
  a.a_mn = p.a_mn;
  a.b_mn = p.b_mn;
  a.gate_row = p.N;
  a.b_bytes = p.b_mn ? (g.bn / 2 + 63) / 64 * 8192 : g.bn * 64;
  a.sub_bytes = kSubA + (a.b_bytes + 1023) / 1024 * 1024;
  a.stages = std::min(8, kRingBytes / (2 * a.sub_bytes));
  a.idesc = idesc_f16(256, g.bn, f16, p.a_mn, p.b_mn);
  a.act = c.cfg->act;
  a.err = c.err;
  a.clear_err = c.first;
  a.hold_spins = injected_spins();
  c.first = false;
  const void* bias = a.bias;
  if (g.splits > 1) {
    a.partial = c.partial;
    a.bias = nullptr;
  }
  OP_TRY((allow_smem<ff_gemm_kernel<T, EPI>>(kSmemBytes, c.dev.index)));
  const int pairs = std::min(a.units, pairs_available(c.dev));
  const double flops = 2.0 * p.M * p.N * p.K * (p.gated ? 2 : 1);
  const double bytes = 2.0 * (p.M * (double)p.K + p.K * (double)rows_b + p.M * (double)p.N);
  sdp::Scope sc(name, sdp::F_GEMM, flops, bytes, c.st, g.splits > 1 ? 2 : 1);
  OP_TRY(launched(launch_pdl(ff_gemm_kernel<T, EPI>, dim3(2 * pairs), dim3(kThreads<EPI>), kSmemBytes, c.st, maps, a)));
  if (g.splits == 1) return SD_OK;
  const int64_t vecs = p.M * p.N / 8;
  const int threads = vecs < 256 * (int64_t)c.dev.sms ? 64 : 256;  // few vectors: over all SMs
  const unsigned blocks = (unsigned)std::min<int64_t>((vecs + threads - 1) / threads, (int64_t)c.dev.sms * 8);
  return launched(launch_pdl(ff_join_kernel<T>, dim3(blocks), dim3(threads), 0, c.st, (const float*)c.partial, g.splits,
                             p.M, p.N, static_cast<const T*>(bias), static_cast<T*>(a.out)));
}

sd_status check(const sd_gated_ff_cfg* c) {
  if (!c) return SD_ERR_NULL_ARG;
  if (c->tokens < 0 || c->d_in <= 0 || c->d_hidden <= 0 || c->d_out <= 0) return SD_ERR_BAD_SHAPE;
  if (c->d_in % 8 || c->d_hidden % 8 || c->d_out % 8) return SD_ERR_UNSUPPORTED;
  if ((c->dtype != SD_DTYPE_BF16 && c->dtype != SD_DTYPE_F16) || c->act < SD_ACT_NONE || c->act > SD_ACT_GELU)
    return SD_ERR_UNSUPPORTED;
  if (c->tokens > (int64_t)1 << 30 || c->d_in > 1 << 20 || c->d_hidden > 1 << 20 || c->d_out > 1 << 20)
    return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

Product p_up(const sd_gated_ff_cfg& c) { return {c.tokens, c.d_in, c.d_hidden, true, false, false, false}; }
Product p_down(const sd_gated_ff_cfg& c) { return {c.tokens, c.d_hidden, c.d_out, false, true, false, false}; }
Product p_dh(const sd_gated_ff_cfg& c) { return {c.tokens, c.d_out, c.d_hidden, false, false, false, true}; }
Product p_dx(const sd_gated_ff_cfg& c) { return {c.tokens, 2 * (int64_t)c.d_hidden, c.d_in, false, true, false, true}; }
Product p_dw1(const sd_gated_ff_cfg& c) { return {2 * (int64_t)c.d_hidden, c.tokens, c.d_in, false, true, true, true}; }
Product p_dw2(const sd_gated_ff_cfg& c) { return {c.d_out, c.tokens, c.d_hidden, false, true, true, true}; }

// Scratch, from the first 256-byte boundary behind the header: a workspace starts on any
// 16-byte boundary, and the FP32 parts are written 32 bytes at a time.
struct Space {
  size_t h, dpre, partial, colsum, colsum2, total;
  int chunks;
};
uint8_t* scratch(void* workspace) {
  return reinterpret_cast<uint8_t*>(up256(reinterpret_cast<uintptr_t>(workspace) + kOpHeader));
}
Space plan_space(const sd_gated_ff_cfg& c) {
  Space s;
  s.h = 0;
  s.dpre = s.h + up256((size_t)c.tokens * c.d_hidden * 2);
  s.partial = s.dpre + up256((size_t)c.tokens * c.d_hidden * 4);
  size_t parts = 0;
  for (const Product& p : {p_down(c), p_dx(c), p_dw1(c), p_dw2(c)}) parts = std::max(parts, split_bytes(p));
  s.colsum = s.partial + up256(parts);
  // db1: a part for every 128 tokens; db2: enough parts to fill the GPU
  const int blocks = (c.d_out + 255) / 256;
  s.chunks = (int)std::max<int64_t>(1, std::min<int64_t>((c.tokens + 63) / 64, (592 + blocks - 1) / blocks));
  s.colsum2 = s.colsum + up256((size_t)((c.tokens + 127) / 128) * 2 * c.d_hidden * 4);
  s.total = kOpHeader + 240 + s.colsum2 + up256((size_t)s.chunks * c.d_out * 4);
  return s;
}

template <typename T, int MT>
sd_status forward_small(Call& c, const Space& s, uint8_t* ws, const void* w1, const void* b1, const void* w2,
                        const void* b2, const void* x, void* pre, void* y) {
  // one token: as many warps as can be; more: rows that share the tokens' values
  constexpr int C = MT == 1 ? 1 : 2, R = MT == 1 ? 1 : 2;
  const sd_gated_ff_cfg& g = *c.cfg;
  const int M = (int)g.tokens, D = g.d_in, F = g.d_hidden, N = g.d_out;
  const auto t = [](const void* p) { return static_cast<const T*>(p); };
  T* h = reinterpret_cast<T*>(ws + s.h);
  {
    const int per = kSmallThreads / 32 * C;
    sdp::Scope sc("ff_small_up", sdp::F_GEMV, 4.0 * M * D * F, 4.0 * D * F, c.st);
    OP_TRY(launched(launch_pdl(ff_small_up_kernel<T, MT, C>, dim3((unsigned)((F + per - 1) / per)), dim3(kSmallThreads), 0,
                               c.st, t(x), t(w1), t(b1), static_cast<T*>(pre), h, M, D, F, (int)g.act, c.err)));
  }
  const int per = kSmallThreads / 128 * R;
  sdp::Scope sc("ff_small_down", sdp::F_GEMV, 2.0 * M * N * F, 2.0 * N * F, c.st);
  return launched(launch_pdl(ff_small_down_kernel<T, MT, R>, dim3((unsigned)((N + per - 1) / per)), dim3(kSmallThreads), 0,
                             c.st, (const T*)h, t(w2), t(b2), static_cast<T*>(y), M, F, N));
}

template <typename T>
sd_status forward(Call& c, const Space& s, uint8_t* ws, const void* w1, const void* b1, const void* w2, const void* b2,
                  const void* x, void* pre, void* y) {
  // up to kSmallTokens tokens the weights' bytes are all that counts (see the kernels)
  if (c.cfg->tokens == 1) return forward_small<T, 1>(c, s, ws, w1, b1, w2, b2, x, pre, y);
  if (c.cfg->tokens == 2) return forward_small<T, 2>(c, s, ws, w1, b1, w2, b2, x, pre, y);
  if (c.cfg->tokens <= kSmallTokens) return forward_small<T, kSmallTokens>(c, s, ws, w1, b1, w2, b2, x, pre, y);
  FfArgs a;
  memset(&a, 0, sizeof(a));
  a.bias = b1;
  a.out = ws + s.h;
  a.pre = pre;
  OP_TRY((product<T, EPI_GATE>(c, "ff_up_gate", p_up(*c.cfg), x, w1, a)));
  memset(&a, 0, sizeof(a));
  a.bias = b2;
  a.out = y;
  return product<T, EPI_PLAIN>(c, "ff_down", p_down(*c.cfg), ws + s.h, w2, a);
}

template <typename T>
sd_status backward(Call& c, const Space& s, uint8_t* ws, const void* w1, const void* w2, const void* x, const void* pre,
                   const void* dy, void* dx, void* dw1, void* db1, void* dw2, void* db2) {
  const sd_gated_ff_cfg& g = *c.cfg;
  FfArgs a;
  if (dx || dw1 || db1 || dw2) {
    memset(&a, 0, sizeof(a));
    a.pre = const_cast<void*>(pre);
    a.dpre = ws + s.dpre;
    a.out = dw2 ? ws + s.h : nullptr;
    a.colsum = db1 ? reinterpret_cast<float*>(ws + s.colsum) : nullptr;
    OP_TRY((product<T, EPI_GATE_GRAD>(c, "ff_dh_gate", p_dh(g), dy, w2, a)));
  }
  memset(&a, 0, sizeof(a));
  if (dx) {
    a.out = dx;
    OP_TRY((product<T, EPI_PLAIN>(c, "ff_dx", p_dx(g), ws + s.dpre, w1, a)));
  }
  if (dw1) {
    a.out = dw1;
    OP_TRY((product<T, EPI_PLAIN>(c, "ff_dw1", p_dw1(g), ws + s.dpre, x, a)));
  }
  if (dw2) {
    a.out = dw2;
    OP_TRY((product<T, EPI_PLAIN>(c, "ff_dw2", p_dw2(g), dy, ws + s.h, a)));
  }
  if (db2) {
    const int64_t rows = (g.tokens + s.chunks - 1) / s.chunks;
    sdp::Scope sc("ff_colsum", sdp::F_OTHER, 0, 2.0 * g.tokens * g.d_out, c.st);
    OP_TRY(launched(launch_pdl(ff_colsum_kernel<T>, dim3((g.d_out + 255) / 256, (unsigned)((g.tokens + rows - 1) / rows)),
                               dim3(256), 0, c.st, static_cast<const T*>(dy), g.d_out, g.tokens, rows,
                               reinterpret_cast<float*>(ws + s.colsum2), c.first ? c.err : nullptr)));
    c.first = false;
  }
  if (db1 || db2) {
    BiasJoin j;
    memset(&j, 0, sizeof(j));
    const int64_t rows = (g.tokens + s.chunks - 1) / s.chunks;
    j.part[0] = reinterpret_cast<const float*>(ws + s.colsum);
    j.part[1] = reinterpret_cast<const float*>(ws + s.colsum2);
    j.out[0] = db1;
    j.out[1] = db2;
    j.n[0] = 2 * g.d_hidden;
    j.n[1] = g.d_out;
    j.parts[0] = (g.tokens + 127) / 128;
    j.parts[1] = (g.tokens + rows - 1) / rows;
    for (int i = 0; i < 2; ++i) j.blocks[i] = j.out[i] ? (j.n[i] + 31) / 32 : 0;
    sdp::Scope sc("ff_bias_join", sdp::F_OTHER, 0, 4.0 * (j.parts[0] * j.n[0] + j.parts[1] * j.n[1]), c.st);
    OP_TRY(launched(
        launch_pdl(ff_bias_join_kernel<T>, dim3((unsigned)(j.blocks[0] + j.blocks[1])), dim3(256), 0, c.st, j)));
  }
  return SD_OK;
}

}  // namespace
}  // namespace sdo

using namespace sdo;

extern "C" {

size_t sd_gated_ff_workspace_size(const sd_gated_ff_cfg* cfg) {
  if (check(cfg) != SD_OK) return 0;
  if (cfg->tokens == 0) return kOpHeader;
  return plan_space(*cfg).total;
}

sd_status sd_gated_ff_fwd(const sd_gated_ff_cfg* cfg, const void* w1, const void* b1, const void* w2, const void* b2,
                          const void* x, void* pre, void* y, void* workspace, size_t ws_bytes, sd_stream_t stream) {
  OP_TRY(check(cfg));
  if (cfg->tokens == 0) return SD_OK;
  if (!w1 || !w2 || !x || !y) return SD_ERR_NULL_ARG;
  for (const void* p : {w1, b1, w2, b2, x, (const void*)pre, (const void*)y})
    if (misaligned(p)) return SD_ERR_MISALIGNED;
  const Space s = plan_space(*cfg);
  OP_TRY(check_workspace(s.total, workspace, ws_bytes));
  Call c{cfg};
  OP_TRY(current_device(&c.dev));
  uint8_t* ws = scratch(workspace);
  c.st = (cudaStream_t)stream;
  c.err = static_cast<int*>(workspace);
  c.partial = reinterpret_cast<float*>(ws + s.partial);
  return cfg->dtype == SD_DTYPE_F16 ? forward<__half>(c, s, ws, w1, b1, w2, b2, x, pre, y)
                                    : forward<__nv_bfloat16>(c, s, ws, w1, b1, w2, b2, x, pre, y);
}

sd_status sd_gated_ff_bwd(const sd_gated_ff_cfg* cfg, const void* w1, const void* w2, const void* x, const void* pre,
                          const void* dy, void* dx, void* dw1, void* db1, void* dw2, void* db2, void* workspace,
                          size_t ws_bytes, sd_stream_t stream) {
  OP_TRY(check(cfg));
  for (const void* p : {w1, w2, x, pre, dy, (const void*)dx, (const void*)dw1, (const void*)db1, (const void*)dw2,
                        (const void*)db2})
    if (misaligned(p)) return SD_ERR_MISALIGNED;
  if (cfg->tokens == 0) {
    Device dev;
    OP_TRY(current_device(&dev));
    const size_t di = cfg->d_in, f = cfg->d_hidden, dout = cfg->d_out;
    const std::pair<void*, size_t> zero[] = {{dw1, 2 * f * di}, {db1, 2 * f}, {dw2, dout * f}, {db2, dout}};
    for (const auto& z : zero)
      if (z.first) OP_TRY(launched(cudaMemsetAsync(z.first, 0, z.second * 2, (cudaStream_t)stream)));
    return SD_OK;
  }
  if (!dx && !dw1 && !db1 && !dw2 && !db2) return SD_OK;
  if (!w1 || !w2 || !x || !pre || !dy) return SD_ERR_NULL_ARG;
  const Space s = plan_space(*cfg);
  OP_TRY(check_workspace(s.total, workspace, ws_bytes));
  Call c{cfg};
  OP_TRY(current_device(&c.dev));
  uint8_t* ws = scratch(workspace);
  c.st = (cudaStream_t)stream;
  c.err = static_cast<int*>(workspace);
  c.partial = reinterpret_cast<float*>(ws + s.partial);
  return cfg->dtype == SD_DTYPE_F16
             ? backward<__half>(c, s, ws, w1, w2, x, pre, dy, dx, dw1, db1, dw2, db2)
             : backward<__nv_bfloat16>(c, s, ws, w1, w2, x, pre, dy, dx, dw1, db1, dw2, db2);
}

}  // extern "C"
