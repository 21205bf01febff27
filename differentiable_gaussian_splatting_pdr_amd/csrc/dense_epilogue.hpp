// dense_epilogue.hpp -- what the matrix-product kernels do with their fp32
// sums before storing: bias, activation and residual of a projection, the
// gated product and its gradient, the Newton-Schulz polynomial's update.
//
// Everything here is computed in fp32 and rounded once, when it is stored.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pdr_dense.h"

namespace pdr {
namespace dense {

constexpr int kF32 = PDR_FMT_F32, kF16 = PDR_FMT_F16, kBf16 = PDR_FMT_BF16;

__host__ __device__ inline int fmt_bytes(int fmt) { return fmt == kF32 ? 4 : 2; }

enum EpiKind { kEpiLinear = 0, kEpiGated = 1, kEpiGatedGrad = 2, kEpiPoly = 3 };

struct Epi {
  // result, [rows][ldy] of format fmt; columns [N, store_n) are written too
  // (their sums are zero: operands read zeros beyond their ends)
  void *y;
  long long ldy, batch_y;
  int fmt, store_n;
  int vec;  // every row of every tensor here starts on 16 bytes
  // kEpiLinear: y = act(scale sum + bias) + res; slope = act'(scale sum + bias)
  const void *bias;
  int bias_fmt;
  const void *res;  // format fmt
  long long ldr;
  int act;
  void *slope;  // format slope_fmt, or null
  int slope_fmt;
  long long ld_slope;
  // binary exponents of the scales of fp32 operands split into fp16 planes (null: 0)
  const int *exp_a, *exp_b;
  // kEpiGated: gate and up sums kept for the gradient, fp32 [rows][2][ld_gu] (null: not kept)
  // kEpiGatedGrad: reads them; y = [dg | du], du at column up_at
  float *gu;
  long long ld_gu;
  long long up_at;
  // kEpiPoly: y = alpha sum + beta c, c and y in one or two fp16 planes (lo: null with one)
  float alpha, beta;
  const void *c, *c_lo;
  long long ldc, batch_c;
  void *y_lo;
};

// ---------------------------------------------------------------- formats

__device__ __forceinline__ float bf16_to_f(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ float f16_to_f(uint16_t h) {
  return (float)__builtin_bit_cast(_Float16, h);
}
__device__ __forceinline__ uint16_t f_to_f16(float v) {
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}
__device__ __forceinline__ uint16_t f_to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
template <int FMT>
__device__ __forceinline__ float to_f(uint16_t h) {
  return FMT == kBf16 ? bf16_to_f(h) : f16_to_f(h);
}

__device__ __forceinline__ float load1(const void *p, int fmt, long long at) {
  if (fmt == kF32) return ((const float *)p)[at];
  const uint16_t h = ((const uint16_t *)p)[at];
  return fmt == kBf16 ? bf16_to_f(h) : f16_to_f(h);
}
__device__ __forceinline__ void store1(void *p, int fmt, long long at, float v) {
  if (fmt == kF32)
    ((float *)p)[at] = v;
  else
    ((uint16_t *)p)[at] = fmt == kBf16 ? f_to_bf16(v) : f_to_f16(v);
}

// 8 values from element `at` on; `n`: how many of them exist; `vec`: 16-byte
// accesses are allowed if all do.  Values that do not exist read as 0.
__device__ __forceinline__ void load8(const void *p, int fmt, long long at, int n, int vec,
                                      float v[8]) {
  if (vec && n >= 8) {
    if (fmt == kF32) {
      const float4 a = *(const float4 *)((const float *)p + at);
      const float4 b = *(const float4 *)((const float *)p + at + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *(const uint4 *)((const uint16_t *)p + at);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t h = (uint16_t)(w[i >> 1] >> ((i & 1) * 16));
        v[i] = fmt == kBf16 ? bf16_to_f(h) : f16_to_f(h);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? load1(p, fmt, at + i) : 0.f;
  }
}
__device__ __forceinline__ void store8(void *p, int fmt, long long at, int n, int vec,
                                       const float v[8]) {
  if (vec && n >= 8) {
    if (fmt == kF32) {
      *(float4 *)((float *)p + at) = make_float4(v[0], v[1], v[2], v[3]);
      *(float4 *)((float *)p + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t a = fmt == kBf16 ? f_to_bf16(v[2 * i]) : f_to_f16(v[2 * i]);
        const uint16_t b = fmt == kBf16 ? f_to_bf16(v[2 * i + 1]) : f_to_f16(v[2 * i + 1]);
        w[i] = a | ((uint32_t)b << 16);
      }
      *(uint4 *)((uint16_t *)p + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store1(p, fmt, at + i, v[i]);
  }
}

// ------------------------------------------------------------- activations

// y = act(z) and, where wanted, its slope.  An infinity or NaN gives what the
// formula gives.
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case PDR_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case PDR_ACT_SILU: return z / (1.f + expf(-z));
    case PDR_ACT_GELU: return z * (0.5f * (1.f + erff(z * 0.70710678f)));
    default: return z;
  }
}
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case PDR_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case PDR_ACT_SILU: {
      const float p = 1.f / (1.f + expf(-z));
      return p * (1.f + z * (1.f - p));
    }
    case PDR_ACT_GELU:
      return 0.5f * (1.f + erff(z * 0.70710678f)) + z * (0.39894228f * expf(-0.5f * z * z));
    default: return 1.f;
  }
}

// --------------------------------------------------------------- epilogues

__device__ __forceinline__ void store_partial(float *p, int m, int n, int N, const float v[8]) {
  const int left = N - n;
  if (left <= 0) return;
  store8(p, kF32, (long long)m * N + n, left, (N & 3) == 0, v);
}

__device__ __forceinline__ int epi_exp(const Epi &e) { return e.exp_a ? -(*e.exp_a + *e.exp_b) : 0; }

// 8 consecutive columns n.. of row m.  N: columns that exist in the product.
template <int KIND>
__device__ __forceinline__ void epi_apply(const Epi &e, int batch, int m, int n, int N,
                                          const float sum[8]) {
  const int left = e.store_n - n;
  if (left <= 0) return;
  float v[8];
  if constexpr (KIND == kEpiLinear) {
    const int s = epi_exp(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ldexpf(sum[i], s);
    if (e.bias) {
      float b[8];
      load8(e.bias, e.bias_fmt, n, N - n, e.vec, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += b[i];
    }
    if (e.act != PDR_ACT_NONE) {
      if (e.slope) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = act_slope(e.act, v[i]);
        store8(e.slope, e.slope_fmt, (long long)m * e.ld_slope + n, left, e.vec, d);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = activate(e.act, v[i]);
    }
    if (e.res) {
      float r[8];
      load8(e.res, e.fmt, (long long)m * e.ldr + n, left, e.vec, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    store8(e.y, e.fmt, batch * e.batch_y + (long long)m * e.ldy + n, left, e.vec, v);
  } else if constexpr (KIND == kEpiGatedGrad) {
    const int s = epi_exp(e);
    float gate[8], up[8], d[8];
    const long long at = (long long)m * 2 * e.ld_gu + n;
    load8(e.gu, kF32, at, left, e.vec, gate);
    load8(e.gu, kF32, at + e.ld_gu, left, e.vec, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // columns past N are stored as zeros whatever w_out's rows hold beyond
      const float dh = n + i < N ? ldexpf(sum[i], s) : 0.f;
      v[i] = dh * up[i] * act_slope(e.act, gate[i]);
      d[i] = dh * activate(e.act, gate[i]);
    }
    store8(e.y, e.fmt, (long long)m * e.ldy + n, left, e.vec, v);
    store8(e.y, e.fmt, (long long)m * e.ldy + e.up_at + n, left, e.vec, d);
  } else if constexpr (KIND == kEpiPoly) {
    const long long at = batch * e.batch_y + (long long)m * e.ldy + n;
    const long long at_c = batch * e.batch_c + (long long)m * e.ldc + n;
    float c[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (e.c) load8(e.c, kF16, at_c, left, e.vec, c);
    if (e.c_lo) {
      float lo[8];
      load8(e.c_lo, kF16, at_c, left, e.vec, lo);
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] += lo[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e.alpha * sum[i] + e.beta * c[i];
    store8(e.y, e.fmt, at, left, e.vec, v);
    if (e.y_lo) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] -= f16_to_f(f_to_f16(v[i]));
      store8(e.y_lo, kF16, at, left, e.vec, v);
    }
  }
}

// 8 gate sums and the 8 up sums of the same columns.
__device__ __forceinline__ void epi_gated(const Epi &e, int m, int n, const float sum_g[8],
                                          const float sum_u[8]) {
  const int left = e.store_n - n;
  if (left <= 0) return;
  const int s = epi_exp(e);
  float gate[8], up[8], h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gate[i] = ldexpf(sum_g[i], s);
    up[i] = ldexpf(sum_u[i], s);
    h[i] = activate(e.act, gate[i]) * up[i];
  }
  if (e.gu) {
    const long long at = (long long)m * 2 * e.ld_gu + n;
    store8(e.gu, kF32, at, left, e.vec, gate);
    store8(e.gu, kF32, at + e.ld_gu, left, e.vec, up);
  }
  store8(e.y, e.fmt, (long long)m * e.ldy + n, left, e.vec, h);
}

}  // namespace dense
}  // namespace pdr
