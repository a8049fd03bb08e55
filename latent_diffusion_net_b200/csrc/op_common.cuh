// Shared pieces of the standalone operators (group norm, gated feed-forward,
// attention): element types, activations with their derivatives, the tcgen05
// forms they need beyond common.cuh, and the host-side checks.
#pragma once

#include "common.cuh"
#include "sd_api.h"

namespace sdo {

using namespace sdk;

// ------------------------------------------------------------------ element types
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr bool kF16 = false;
  static __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float lo(uint32_t v) { return bf16lo(v); }
  static __device__ __forceinline__ float hi(uint32_t v) { return bf16hi(v); }
};
template <>
struct Elem<__half> {
  static constexpr bool kF16 = true;
  static __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
  static __device__ __forceinline__ float lo(uint32_t v) {
    return __low2float(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ float hi(uint32_t v) {
    return __high2float(*reinterpret_cast<const __half2*>(&v));
  }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to_f(float v) { return v; }
  static __device__ __forceinline__ float from_f(float v) { return v; }
};

// V consecutive elements as FP32: one 16-byte access when V fills it, else element by element.
template <typename T, int V>
__device__ __forceinline__ void unpack_vec(const uint4& raw, float (&f)[V]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = Elem<T>::lo(w[i]);
      f[2 * i + 1] = Elem<T>::hi(w[i]);
    }
  } else {
    f[0] = __uint_as_float(raw.x);
    f[1] = __uint_as_float(raw.y);
    f[2] = __uint_as_float(raw.z);
    f[3] = __uint_as_float(raw.w);
  }
}
template <typename T, int V>
__device__ __forceinline__ uint4 pack_vec(const float (&f)[V]) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(Elem<T>::pack(f[0], f[1]), Elem<T>::pack(f[2], f[3]), Elem<T>::pack(f[4], f[5]),
                      Elem<T>::pack(f[6], f[7]));
  else
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// ------------------------------------------------------------------ activations
// 2^x and 1/x as one instruction each: relative errors near 2^-22, and what the rounding of
// x adds to 2^x. Far below half a step of the 16-bit types; FP32 outputs are within 1e-6 of
// their own size, but for the far tail of the normal distribution (below).
__device__ __forceinline__ float fast_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 1 / (1 + e^-z); e^-z overflows to infinity below z = -88, where the result is 0.
__device__ __forceinline__ float sigmoid_f(float z) { return fast_rcp(1.f + fast_ex2(-kLog2e * z)); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2). With u = |z| / sqrt 2,
// Phi(-|z|) = erfc(u) / 2 = e w(t) with t = 1 / (1 + u / 2), w a polynomial fitted to
// erfc(u) e^(u^2) / 2 on 0 <= u <= 6.2 for the least relative error (4e-7): one reciprocal
// and one exponential, which the derivative uses too, and no cancellation for negative z. The
// exponent's FP32 rounding leaves 3e-6 relative at z = -8, where Phi is 6e-16.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = fast_rcp(fmaf(fabsf(z), 0.35355339f, 1.f));
  e = fast_ex2(z * z * (-0.5f * kLog2e));
  float w = fmaf(0.04765096f, t, -0.19102928f);
  w = fmaf(w, t, 0.21266575f);
  w = fmaf(w, t, 0.0058340114f);
  w = fmaf(w, t, 0.14584327f);
  w = fmaf(w, t, 0.13779275f);
  w = fmaf(w, t, 0.14124271f);
  const float q = w * t * e;
  return z < 0.f ? q : 1.f - q;
}

__device__ __forceinline__ float act_f(float z, int act) {
  if (act == SD_ACT_SILU) return z * sigmoid_f(z);
  if (act == SD_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  return z;
}
// a = act(z), d = act'(z)
__device__ __forceinline__ void act_grad_f(float z, int act, float& a, float& d) {
  if (act == SD_ACT_SILU) {
    const float s = sigmoid_f(z);
    a = z * s;
    d = s + a * (1.f - s);
  } else if (act == SD_ACT_GELU) {
    float e;
    const float cdf = normal_cdf(z, e);
    a = z * cdf;
    d = fmaf(z * 0.39894228040143268f, e, cdf);
  } else {
    a = z;
    d = 1.f;
  }
}

// (y0, y1) = (a0 * b0, a1 * b1)
__device__ __forceinline__ void mul2(float a0, float a1, float b0, float b1, float& y0, float& y1) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%2, %3};\n\t"
      "mov.b64 q, {%4, %5};\n\t"
      "mul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(y0), "=f"(y1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// normal_cdf of two values, the same arithmetic in packed FP32.
__device__ __forceinline__ void normal_cdf2(float z0, float z1, float& c0, float& c1, float& e0, float& e1) {
  float t0, t1, w0, w1, q0, q1;
  fma2v(fabsf(z0), fabsf(z1), 0.35355339f, 0.35355339f, 1.f, 1.f, t0, t1);
  t0 = fast_rcp(t0);
  t1 = fast_rcp(t1);
  mul2(z0, z1, z0, z1, e0, e1);
  mul2(e0, e1, -0.5f * kLog2e, -0.5f * kLog2e, e0, e1);
  e0 = fast_ex2(e0);
  e1 = fast_ex2(e1);
  fma2v(t0, t1, 0.04765096f, 0.04765096f, -0.19102928f, -0.19102928f, w0, w1);
  fma2v(w0, w1, t0, t1, 0.21266575f, 0.21266575f, w0, w1);
  fma2v(w0, w1, t0, t1, 0.0058340114f, 0.0058340114f, w0, w1);
  fma2v(w0, w1, t0, t1, 0.14584327f, 0.14584327f, w0, w1);
  fma2v(w0, w1, t0, t1, 0.13779275f, 0.13779275f, w0, w1);
  fma2v(w0, w1, t0, t1, 0.14124271f, 0.14124271f, w0, w1);
  mul2(w0, w1, t0, t1, w0, w1);
  mul2(w0, w1, e0, e1, w0, w1);
  fma2v(w0, w1, -1.f, -1.f, 1.f, 1.f, q0, q1);
  c0 = z0 < 0.f ? w0 : q0;
  c1 = z1 < 0.f ? w1 : q1;
}

// The activations on V values at once: the same arithmetic as act_f and act_grad_f
// with the multiply-adds as packed pairs (half the instructions); the activation is
// chosen once for all V.
template <int V>
__device__ __forceinline__ void act_vec(float (&z)[V], int act) {
  if constexpr (V % 2) {
    for (int j = 0; j < V; ++j) z[j] = act_f(z[j], act);
  } else if (act == SD_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      float e0, e1;
      mul2(z[j], z[j + 1], -kLog2e, -kLog2e, e0, e1);
      e0 = fast_ex2(e0);
      e1 = fast_ex2(e1);
      add2(e0, e1, 1.f, 1.f, e0, e1);
      mul2(z[j], z[j + 1], fast_rcp(e0), fast_rcp(e1), z[j], z[j + 1]);
    }
  } else if (act == SD_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      float c0, c1, e0, e1;
      normal_cdf2(z[j], z[j + 1], c0, c1, e0, e1);
      mul2(z[j], z[j + 1], c0, c1, z[j], z[j + 1]);
    }
  }
}
// d *= act'(z); a = act(z) (both may be unused)
template <int V>
__device__ __forceinline__ void act_grad_vec(const float (&z)[V], float (&d)[V], float (&a)[V], int act) {
  if constexpr (V % 2) {
    for (int j = 0; j < V; ++j) {
      float s;
      act_grad_f(z[j], act, a[j], s);
      d[j] *= s;
    }
  } else if (act == SD_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      float e0, e1, q0, q1;
      mul2(z[j], z[j + 1], -kLog2e, -kLog2e, e0, e1);
      e0 = fast_ex2(e0);
      e1 = fast_ex2(e1);
      add2(e0, e1, 1.f, 1.f, e0, e1);
      e0 = fast_rcp(e0);  // s
      e1 = fast_rcp(e1);
      mul2(z[j], z[j + 1], e0, e1, a[j], a[j + 1]);
      fma2v(e0, e1, -1.f, -1.f, 1.f, 1.f, q0, q1);
      fma2v(a[j], a[j + 1], q0, q1, e0, e1, q0, q1);  // s + z s (1 - s)
      mul2(d[j], d[j + 1], q0, q1, d[j], d[j + 1]);
    }
  } else if (act == SD_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      float c0, c1, e0, e1;
      normal_cdf2(z[j], z[j + 1], c0, c1, e0, e1);
      mul2(z[j], z[j + 1], c0, c1, a[j], a[j + 1]);
      mul2(e0, e1, 0.39894228040143268f, 0.39894228040143268f, e0, e1);
      fma2v(z[j], z[j + 1], e0, e1, c0, c1, c0, c1);
      mul2(d[j], d[j + 1], c0, c1, d[j], d[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) a[j] = z[j];
  }
}

// ------------------------------------------------------------------ host side
struct Device {
  int index, sms;
};
// The current device's index and SM count; SD_ERR_NOT_SM100 off compute capability 10.0.
sd_status current_device(Device* d);

// Polls of the wait that sd_debug_inject_timeout asks the next tensor-core kernel to give up; 0
// for none (api.cpp).
int injected_spins();

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace bytes before an operator's own scratch: word 0 holds the device error
// flags, which the first kernel of every call clears.
constexpr size_t kOpHeader = 256;

inline sd_status check_workspace(size_t need, const void* ws, size_t ws_bytes) {
  if (!ws) return SD_ERR_NULL_ARG;
  if (misaligned(ws)) return SD_ERR_MISALIGNED;
  if (ws_bytes < need) return SD_ERR_WORKSPACE_TOO_SMALL;
  return SD_OK;
}

// Raises a kernel's shared-memory limit once per device (the attribute belongs to
// the device's copy of the kernel).
template <auto kernel>
inline sd_status allow_smem(size_t bytes, int device) {
  static unsigned long long done = 0;  // one bit per device; a race sets the same value again
  if ((__atomic_load_n(&done, __ATOMIC_RELAXED) >> device) & 1) return SD_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return SD_ERR_LAUNCH;
  }
  __atomic_fetch_or(&done, 1ull << device, __ATOMIC_RELAXED);
  return SD_OK;
}

inline sd_status launched(cudaError_t e) {
  if (e == cudaSuccess) return SD_OK;
  (void)cudaGetLastError();
  return SD_ERR_LAUNCH;
}

#define OP_TRY(x)                      \
  do {                                 \
    const sd_status _s = (x);          \
    if (_s != SD_OK) return _s;        \
  } while (0)

}  // namespace sdo
