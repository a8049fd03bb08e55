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

constexpr int kThreads = 320;     // warp 0 TMA, warp 1 MMA, warps 2-9 epilogue
constexpr int kEpiThreads = 256;
constexpr int kSubA = 128 * 64 * 2;  // one CTA's 128 rows x 64 reduction elements
constexpr int kRingBytes = 196608;
constexpr int kSmemBytes = 1024 + kRingBytes + 256 + 2 * 256 * 4;
constexpr int kPairs = 74;        // CTA pairs the plan assumes (148 SMs)
constexpr int kMaxSplits = 16;
constexpr size_t kSplitBytes = size_t(64) << 20;

enum Epi { EPI_PLAIN = 0, EPI_GATE = 1, EPI_GATE_GRAD = 2 };

struct FfMaps {
  CUtensorMap a, b;
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
  int* err;
  int32_t clear_err;
};

// 32 FP32 values to 32 consecutive elements of T, `n` of them inside (n a multiple of 8).
template <typename T>
__device__ __forceinline__ void store32(T* p, const float (&f)[32], int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (8 * i < n)
      *reinterpret_cast<uint4*>(p + 8 * i) =
          make_uint4(Elem<T>::pack(f[8 * i], f[8 * i + 1]), Elem<T>::pack(f[8 * i + 2], f[8 * i + 3]),
                     Elem<T>::pack(f[8 * i + 4], f[8 * i + 5]), Elem<T>::pack(f[8 * i + 6], f[8 * i + 7]));
  }
}
template <typename T>
__device__ __forceinline__ void load32(const T* p, uint32_t (&r)[16], int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = 8 * i < n ? *reinterpret_cast<const uint4*>(p + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
    r[4 * i] = v.x;
    r[4 * i + 1] = v.y;
    r[4 * i + 2] = v.z;
    r[4 * i + 3] = v.w;
  }
}

template <typename T, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ff_gemm_kernel(const __grid_constant__ FfMaps maps, const __grid_constant__ FfArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingBytes);  // [stages <= 8]
  uint64_t* empty = full + 8;
  uint64_t* acc_full = empty + 8;   // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2], used in the even CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* ecols = reinterpret_cast<float*>(smem + kRingBytes + 256);  // [2][256]

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
      bool ok = true;
      for (int u = pair; u < args.units && ok; u += npairs) {
        const int z = u % args.splits, rest = u / args.splits;
        const int m0 = ((rest / args.tiles_n) * 2 + (int)rank) * 128;
        const int n0 = (rest % args.tiles_n) * args.step_n;
        const int brow = EPI == EPI_GATE ? (rank ? args.gate_row + n0 : n0) : n0 + (int)rank * half;
        const int hi = min(args.kb, (z + 1) * args.kb_split);
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
      // encoded descriptor steps of 16 reduction elements: 32 bytes K-major, 2048 bytes MN-major
      const uint64_t a_step = args.a_mn ? 128 : 2, b_step = args.b_mn ? 128 : 2;
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
            const uint32_t a = smem_u32(smem + s * stage_bytes + h * sub_bytes);
            const uint64_t adesc = args.a_mn ? umma_desc_mn(a, 8192) : umma_desc_k_sw128(a);
            const uint64_t bdesc = args.b_mn ? umma_desc_mn(a + kSubA, 8192) : umma_desc_k_sw128(a + kSubA);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              pair_umma(tacc, adesc + k * a_step, bdesc + k * b_step, args.idesc, acc);
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
      if (!mbar_wait_all(&acc_full[b], (it >> 1) & 1, abort_flag, args.err)) break;
      tc_fence_after();
      const uint32_t tacc = tmem + (uint32_t)(b * 256) + lane_off;
      const bool in = grow < M;
      for (int c = half * 32; c < step_n; c += 64) {
        const int left = N - (n0 + c);  // columns of this chunk inside the output
        if (left <= 0) break;
        uint32_t r[32];
        tmem_ld_32x32b_x32(tacc + c, r);
        float f[32];
        if (EPI == EPI_GATE) {
          uint32_t r2[32];
          tmem_ld_32x32b_x32(tacc + step_n + c, r2);
          tmem_ld_wait_regs(r);
          tmem_ld_wait_regs(r2);
          float g[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            f[i] = __uint_as_float(r[i]);
            g[i] = __uint_as_float(r2[i]);
          }
          if (bias) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              f[i] += ecol[c + i];
              g[i] += ecol[step_n + c + i];
            }
          }
          if (pre && in) {
            store32<T>(pre + grow * 2 * N + n0 + c, f, left);
            store32<T>(pre + grow * 2 * N + N + n0 + c, g, left);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] *= act_f(g[i], act);
          if (in) store32<T>(out + grow * N + n0 + c, f, left);
        } else if (EPI == EPI_GATE_GRAD) {
          uint32_t v[16], zz[16];
          if (in) {
            load32<T>(pre + grow * 2 * N + n0 + c, v, left);
            load32<T>(pre + grow * 2 * N + N + n0 + c, zz, left);
          }
          tmem_ld_wait_regs(r);
          float dz[32], h[32];
          if (in) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float vv = i & 1 ? Elem<T>::hi(v[i >> 1]) : Elem<T>::lo(v[i >> 1]);
              const float zv = i & 1 ? Elem<T>::hi(zz[i >> 1]) : Elem<T>::lo(zz[i >> 1]);
              float a, d;
              act_grad_f(zv, act, a, d);
              const float dh = __uint_as_float(r[i]);
              f[i] = dh * a;
              dz[i] = dh * vv * d;
              h[i] = vv * a;
            }
            store32<T>(dpre + grow * 2 * N + n0 + c, f, left);
            store32<T>(dpre + grow * 2 * N + N + n0 + c, dz, left);
            if (out) store32<T>(out + grow * N + n0 + c, h, left);
          }
        } else {
          tmem_ld_wait_regs(r);
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
          if (partial) {
            if (in) {
              float* p = partial + ((int64_t)z * M + grow) * N + n0 + c;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (4 * i < left)
                  __stcg(reinterpret_cast<float4*>(p + 4 * i),
                         make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]));
            }
          } else {
            if (bias) {
#pragma unroll
              for (int i = 0; i < 32; ++i) f[i] += ecol[c + i];
            }
            if (in) store32<T>(out + grow * N + n0 + c, f, left);
          }
        }
      }
      // this warp's TMEM reads are done; the even CTA's MMA warp may reuse the accumulator
      // once all epilogue warps of both CTAs have said so
      tc_fence_before();
      asm volatile("bar.sync 3, %0;" ::"n"(kEpiThreads) : "memory");
      if (et == 0) pair_arrive(empty_addr[b]);
    }
  }

  tc_fence_before();
  pair_sync();
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc(tmem, 512);
}

// out = sum of the splits (in order) + bias, 8 columns per thread.
template <typename T>
__global__ void __launch_bounds__(256) ff_join_kernel(const float* __restrict__ partial, int splits, int64_t M, int N,
                                                      const T* __restrict__ bias, T* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t vecs = M * N / 8, stride = M * N;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * blockDim.x) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
#pragma unroll 4
    for (int z = 0; z < splits; ++z) {
      const float4* p = reinterpret_cast<const float4*>(partial + z * stride + i * 8);
      const float4 u = __ldcg(p), w = __ldcg(p + 1);
      f[0] += u.x;
      f[1] += u.y;
      f[2] += u.z;
      f[3] += u.w;
      f[4] += w.x;
      f[5] += w.y;
      f[6] += w.z;
      f[7] += w.w;
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

// Column sums of up to two [rows][n] matrices (db1 and db2 in one launch): a CTA
// sums 256 columns over a share of the rows into FP32 shares; a second kernel adds
// the shares in order.
struct ColSum {
  const void* m[2];
  void* out[2];
  float* part[2];  // [chunks][n]
  int32_t n[2], blocks[2];
  int64_t rows, chunk_rows;
  int32_t chunks;
};

template <typename T>
__global__ void __launch_bounds__(256) ff_colsum_kernel(const __grid_constant__ ColSum a) {
  __shared__ float red[8][256];
  pdl_wait();
  pdl_trigger();
  const int which = (int)blockIdx.x >= a.blocks[0];
  const int n = a.n[which];
  const int c0 = ((int)blockIdx.x - (which ? a.blocks[0] : 0)) * 256;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = c0 + tx * 8;
  const int64_t r0 = blockIdx.y * a.chunk_rows, r1 = min(a.rows, r0 + a.chunk_rows);
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.f;
  if (c < n) {
    const T* m = static_cast<const T*>(a.m[which]) + c;
#pragma unroll 4
    for (int64_t r = r0 + ty; r < r1; r += 8) {
      float f[8];
      unpack_vec<T, 8>(*reinterpret_cast<const uint4*>(m + r * n), f);
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
    a.part[which][(int64_t)blockIdx.y * n + c0 + threadIdx.x] = t;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) ff_colsum_join_kernel(const __grid_constant__ ColSum a) {
  pdl_wait();
  pdl_trigger();
  const int which = (int)blockIdx.x >= a.blocks[0];
  const int n = a.n[which];
  const int c = ((int)blockIdx.x - (which ? a.blocks[0] : 0)) * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.f;
#pragma unroll 8
  for (int p = 0; p < a.chunks; ++p) s += a.part[which][(int64_t)p * n + c];
  static_cast<T*>(a.out[which])[c] = Elem<T>::from_f(s);
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
// SM: a 64-wide block costs the slower of its MMAs (2 bn cycles, 4 x 54 at least)
// and its operands' arrival (50 bytes a cycle), a tile about 1500 cycles more for
// filling the pipeline and its last epilogue, and a split product the writing and
// joining of its FP32 parts.
Plan plan_product(const Product& p) {
  const int widths[] = {256, 224, 192, 160, 128, 96, 64};
  const int64_t kb = (p.K + 63) / 64, pairs_m = (p.M + 255) / 256;
  Plan best{0, 1, 0};
  double best_cost = 0;
  for (int bn : widths) {
    if (p.gated && bn % 64) continue;  // each half whole 32-column chunks
    const int step = p.gated ? bn / 2 : bn;
    const int64_t tiles = pairs_m * ((p.N + step - 1) / step);
    for (int sp = 1; sp <= (p.may_split ? kMaxSplits : 1); ++sp) {
      int64_t per = (kb + sp - 1) / sp;
      per = (per + 1) / 2 * 2;
      if (sp > 1 && ((kb + per - 1) / per != sp || per < 4)) continue;
      if (sp > 1 && (size_t)sp * p.M * p.N * 4 > kSplitBytes) break;
      const int64_t rounds = (tiles * sp + kPairs - 1) / kPairs;
      const double b_bytes = p.b_mn ? (bn / 2 + 63) / 64 * 8192.0 : bn * 64.0;
      const double block = std::max(std::max(2.0 * bn, 216.0), (kSubA + b_bytes) / 50.0);
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
  OP_TRY(launched(launch_pdl(ff_gemm_kernel<T, EPI>, dim3(2 * pairs), dim3(kThreads), kSmemBytes, c.st, maps, a)));
  if (g.splits == 1) return SD_OK;
  const int64_t vecs = p.M * p.N / 8;
  const unsigned blocks = (unsigned)std::min<int64_t>((vecs + 255) / 256, (int64_t)c.dev.sms * 8);
  return launched(launch_pdl(ff_join_kernel<T>, dim3(blocks), dim3(256), 0, c.st, (const float*)c.partial, g.splits,
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

struct Space {
  size_t h, dpre, partial, colsum, total;
  int chunks;
};
Space plan_space(const sd_gated_ff_cfg& c) {
  Space s;
  s.h = kOpHeader;
  s.dpre = s.h + up256((size_t)c.tokens * c.d_hidden * 2);
  s.partial = s.dpre + up256((size_t)c.tokens * c.d_hidden * 4);
  size_t parts = 0;
  for (const Product& p : {p_down(c), p_dx(c), p_dw1(c), p_dw2(c)}) parts = std::max(parts, split_bytes(p));
  s.colsum = s.partial + up256(parts);
  const int blocks = (2 * c.d_hidden + 255) / 256 + (c.d_out + 255) / 256;
  s.chunks = (int)std::max<int64_t>(1, std::min<int64_t>((c.tokens + 63) / 64, (592 + blocks - 1) / blocks));
  s.total = s.colsum + up256((size_t)s.chunks * (2 * (size_t)c.d_hidden + c.d_out) * 4);
  return s;
}

template <typename T>
sd_status forward(Call& c, const Space& s, uint8_t* ws, const void* w1, const void* b1, const void* w2, const void* b2,
                  const void* x, void* pre, void* y) {
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
  if (db1 || db2) {
    ColSum cs;
    memset(&cs, 0, sizeof(cs));
    float* part = reinterpret_cast<float*>(ws + s.colsum);
    cs.m[0] = ws + s.dpre;
    cs.m[1] = dy;
    cs.out[0] = db1;
    cs.out[1] = db2;
    cs.part[0] = part;
    cs.part[1] = part + (size_t)s.chunks * 2 * g.d_hidden;
    cs.n[0] = 2 * g.d_hidden;
    cs.n[1] = g.d_out;
    cs.blocks[0] = db1 ? (cs.n[0] + 255) / 256 : 0;
    cs.blocks[1] = db2 ? (cs.n[1] + 255) / 256 : 0;
    cs.rows = g.tokens;
    cs.chunk_rows = (g.tokens + s.chunks - 1) / s.chunks;
    cs.chunks = (int)((g.tokens + cs.chunk_rows - 1) / cs.chunk_rows);
    const unsigned blocks = (unsigned)(cs.blocks[0] + cs.blocks[1]);
    const double bytes = 2.0 * g.tokens * ((db1 ? cs.n[0] : 0) + (db2 ? cs.n[1] : 0));
    sdp::Scope sc("ff_colsum", sdp::F_OTHER, 0, bytes, c.st, 2);
    OP_TRY(launched(launch_pdl(ff_colsum_kernel<T>, dim3(blocks, cs.chunks), dim3(256), 0, c.st, cs)));
    OP_TRY(launched(launch_pdl(ff_colsum_join_kernel<T>, dim3(blocks), dim3(256), 0, c.st, cs)));
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
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  c.st = (cudaStream_t)stream;
  c.err = reinterpret_cast<int*>(ws);
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
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  c.st = (cudaStream_t)stream;
  c.err = reinterpret_cast<int*>(ws);
  c.partial = reinterpret_cast<float*>(ws + s.partial);
  return cfg->dtype == SD_DTYPE_F16
             ? backward<__half>(c, s, ws, w1, w2, x, pre, dy, dx, dw1, db1, dw2, db2)
             : backward<__nv_bfloat16>(c, s, ws, w1, w2, x, pre, dy, dx, dw1, db1, dw2, db2);
}

}  // extern "C"
