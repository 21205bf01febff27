// dense_epilogue.hpp -- what the matrix-product kernels do with their fp32
// sums before storing: bias, activation and residual of a projection, the
// gated product and its gradient, the Newton-Schulz polynomial's update.
//
// Everything here is computed in fp32 and rounded once, when it is stored.
#pragma once

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
  long long batch_y;
  int ldy, fmt, store_n;
  int vec;  // every row of every tensor here starts on 16 bytes
  // kEpiLinear: y = act(sum + bias) + res; slope = act'(sum + bias)
  const void *bias;
  int bias_fmt;
  const void *res;  // format fmt
  int ldr;
  int act;
  void *slope;  // slope_scale times it, format slope_fmt, or null
  int slope_fmt, ld_slope;
  float slope_scale;
  // kEpiGated: gate and up sums kept for the gradient, fp32 [rows][2][ld_gu] (null: not kept)
  // kEpiGatedGrad: reads them; y = [dg | du], du at column up_at
  float *gu;
  int ld_gu, up_at;
  // kEpiPoly: y = alpha sum + beta c, c and y in one or two fp16 planes (lo: null with one)
  float alpha, beta;
  const void *c, *c_lo;
  int ldc;
  long long batch_c;
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

// W values from element `at` on: 8 with 16-byte accesses, or 1.
template <int W>
__device__ __forceinline__ void load_w(const void *p, int fmt, long long at, float v[W]) {
  if constexpr (W == 1) {
    v[0] = load1(p, fmt, at);
  } else if (fmt == kF32) {
    const float4 a = *(const float4 *)((const float *)p + at);
    const float4 b = *(const float4 *)((const float *)p + at + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *(const uint4 *)((const uint16_t *)p + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if (fmt == kBf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = bf16_to_f((uint16_t)(w[i >> 1] >> ((i & 1) * 16)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = f16_to_f((uint16_t)(w[i >> 1] >> ((i & 1) * 16)));
    }
  }
}
template <int W>
__device__ __forceinline__ void store_w(void *p, int fmt, long long at, const float v[W]) {
  if constexpr (W == 1) {
    store1(p, fmt, at, v[0]);
  } else if (fmt == kF32) {
    *(float4 *)((float *)p + at) = make_float4(v[0], v[1], v[2], v[3]);
    *(float4 *)((float *)p + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    uint32_t w[4];
    if (fmt == kBf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * i], v[2 * i + 1]}), b2));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * i], v[2 * i + 1]}), h2));
    }
    *(uint4 *)((uint16_t *)p + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// The same where only n of the 8 values may exist and rows may start anywhere
// (`vec`: they start on 16 bytes).  Values that do not exist read as 0.
__device__ __forceinline__ void load8(const void *p, int fmt, long long at, int n, int vec,
                                      float v[8]) {
  if (vec && n >= 8) {
    load_w<8>(p, fmt, at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? load1(p, fmt, at + i) : 0.f;
  }
}
__device__ __forceinline__ void store8(void *p, int fmt, long long at, int n, int vec,
                                       const float v[8]) {
  if (vec && n >= 8) {
    store_w<8>(p, fmt, at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store1(p, fmt, at + i, v[i]);
  }
}

// ------------------------------------------------------------- activations

// exp2 and reciprocal as the hardware has them (1 ulp): of sigmoid, the error
// is below 2^-22 of 1.  An infinity or NaN gives what the formula gives.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}
// Phi(z) and phi(z) of the normal distribution from one exponential, by
// Abramowitz and Stegun 7.1.26: erfc(x) = t (a1 + t (a2 + ...)) exp(-x^2) with
// t = 1 / (1 + 0.3275911 x), x = |z| / sqrt 2; |error| < 1.5e-7.
__device__ __forceinline__ float normal_cdf(float z, float *pdf) {
  const float t = __builtin_amdgcn_rcpf(1.f + 0.23164189f * fabsf(z));
  const float e = __builtin_amdgcn_exp2f(-0.72134752f * z * z);
  const float half = 0.5f * t * e *
                     (0.254829592f +
                      t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
  *pdf = 0.39894228f * e;
  return z < 0.f ? half : 1.f - half;
}

// act(z) of W values in place; with `slope`, act'(z) there.
template <int W>
__device__ __forceinline__ void activate(int act, float v[W], float *slope) {
  if (act == PDR_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float z = v[i], p = sigmoid(z);
      v[i] = z * p;
      if (slope) slope[i] = p * (1.f + z * (1.f - p));
    }
  } else if (act == PDR_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float pdf;
      const float z = v[i], cdf = normal_cdf(z, &pdf);
      v[i] = z * cdf;
      if (slope) slope[i] = cdf + z * pdf;
    }
  } else if (act == PDR_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float z = v[i];
      v[i] = z > 0.f ? z : (z != z ? z : 0.f);
      if (slope) slope[i] = z > 0.f ? 1.f : 0.f;
    }
  } else if (slope) {
#pragma unroll
    for (int i = 0; i < W; ++i) slope[i] = 1.f;
  }
}

// --------------------------------------------------------------- epilogues

__device__ __forceinline__ long long place(int row, int ld) { return (long long)row * ld; }

// Which memory accesses an epilogue makes, where that is known at compile
// time.  Stores and loads return in one order: a load that may or may not have
// been issued makes the compiler wait for every store before it.
enum EpiFlags {
  kReads = 1,  // kEpiLinear: a residual; kEpiPoly: c
  kWide = 2,   // y is fp32
  kKeeps = 4,  // kEpiLinear: slope; kEpiGated: gu; kEpiPoly: two planes
  kAsked = 8,  // none of it is known: the struct is asked
};
__device__ __forceinline__ int epi_flags(int kind, const Epi &e) {
  const bool reads = kind == kEpiLinear ? e.res != nullptr : e.c != nullptr;
  const bool keeps = kind == kEpiLinear  ? e.slope != nullptr
                     : kind == kEpiGated ? e.gu != nullptr
                                         : e.y_lo != nullptr;
  return (reads ? kReads : 0) | (e.fmt == kF32 ? kWide : 0) | (keeps ? kKeeps : 0);
}
template <int F>
struct Flags {
  static constexpr int value = F;
};
template <int FLAGS>
__device__ __forceinline__ int y_fmt(const Epi &e) {
  if constexpr (FLAGS == kAsked) return e.fmt;
  if constexpr ((FLAGS & kWide) != 0) return kF32;
  return e.fmt == kBf16 ? kBf16 : kF16;
}
template <int FLAGS>
__device__ __forceinline__ bool flag(const Epi &e, int kind, int which) {
  if constexpr (FLAGS == kAsked) return (epi_flags(kind, e) & which) != 0;
  return (FLAGS & which) != 0;
}

// What an epilogue does for W columns n.. of several rows: fetch() what a row
// needs from memory, then finish() it.  What belongs to the columns is fetched
// once, here.  The columns [0, N) exist in the product, [0, store_n) are stored.
template <int KIND, int W, int FLAGS>
struct Columns;

template <int W, int FLAGS>
struct Columns<kEpiLinear, W, FLAGS> {
  float bias[W];
  long long at_y;
  int n;
  struct Row {
    float res[W];
  };
  __device__ __forceinline__ Columns(const Epi &e, int batch, int n_, int) : n(n_) {
    at_y = batch * e.batch_y + n;
    if (e.bias) {
      load_w<W>(e.bias, e.bias_fmt, n, bias);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) bias[i] = 0.f;
    }
  }
  __device__ __forceinline__ void fetch(const Epi &e, int m, Row &r) const {
    if (flag<FLAGS>(e, kEpiLinear, kReads)) load_w<W>(e.res, y_fmt<FLAGS>(e), place(m, e.ldr) + n, r.res);
  }
  __device__ __forceinline__ void finish(const Epi &e, int m, float v[W], const Row &r) const {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += bias[i];
    if (flag<FLAGS>(e, kEpiLinear, kKeeps)) {
      float d[W];
      activate<W>(e.act, v, d);
#pragma unroll
      for (int i = 0; i < W; ++i) d[i] *= e.slope_scale;
      store_w<W>(e.slope, e.slope_fmt, place(m, e.ld_slope) + n, d);
    } else {
      activate<W>(e.act, v, nullptr);
    }
    if (flag<FLAGS>(e, kEpiLinear, kReads)) {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] += r.res[i];
    }
    store_w<W>(e.y, y_fmt<FLAGS>(e), at_y + place(m, e.ldy), v);
  }
};

template <int W, int FLAGS>
struct Columns<kEpiGatedGrad, W, FLAGS> {
  int n, exist;
  struct Row {
    float gate[W], up[W];
  };
  __device__ __forceinline__ Columns(const Epi &, int, int n_, int N) : n(n_) {
    exist = N - n;
  }
  __device__ __forceinline__ void fetch(const Epi &e, int m, Row &r) const {
    const long long at = place(m, 2 * e.ld_gu) + n;
    load_w<W>(e.gu, kF32, at, r.gate);
    load_w<W>(e.gu, kF32, at + e.ld_gu, r.up);
  }
  __device__ __forceinline__ void finish(const Epi &e, int m, float v[W], const Row &r) const {
    float a[W], slope[W];
#pragma unroll
    for (int i = 0; i < W; ++i) a[i] = r.gate[i];
    activate<W>(e.act, a, slope);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      // columns past N are stored as zeros whatever w_out's rows hold beyond
      const float dh = i < exist ? v[i] : 0.f;
      v[i] = dh * r.up[i] * slope[i];
      a[i] = dh * a[i];
    }
    const long long at = place(m, e.ldy) + n;
    store_w<W>(e.y, y_fmt<FLAGS>(e), at, v);
    store_w<W>(e.y, y_fmt<FLAGS>(e), at + e.up_at, a);
  }
};

template <int W, int FLAGS>
struct Columns<kEpiPoly, W, FLAGS> {
  long long at_y, at_c;
  struct Row {
    float c[W], lo[W];
  };
  __device__ __forceinline__ Columns(const Epi &e, int batch, int n, int) {
    at_y = batch * e.batch_y + n;
    at_c = batch * e.batch_c + n;
  }
  __device__ __forceinline__ void fetch(const Epi &e, int m, Row &r) const {
    if (!flag<FLAGS>(e, kEpiPoly, kReads)) return;
    load_w<W>(e.c, kF16, at_c + place(m, e.ldc), r.c);
    // with one plane c is read twice, from the cache, rather than perhaps
    load_w<W>(e.c_lo ? e.c_lo : e.c, kF16, at_c + place(m, e.ldc), r.lo);
  }
  __device__ __forceinline__ void finish(const Epi &e, int m, float v[W], const Row &r) const {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= e.alpha;
    if (flag<FLAGS>(e, kEpiPoly, kReads)) {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] += e.beta * (e.c_lo ? r.c[i] + r.lo[i] : r.c[i]);
    }
    const long long at = at_y + place(m, e.ldy);
    store_w<W>(e.y, y_fmt<FLAGS>(e), at, v);
    if (flag<FLAGS>(e, kEpiPoly, kKeeps)) {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] -= f16_to_f(f_to_f16(v[i]));
      store_w<W>(e.y_lo, kF16, at, v);
    }
  }
};

// v: W gate sums, then the W up sums of the same columns.
template <int W, int FLAGS>
struct Columns<kEpiGated, W, FLAGS> {
  int n;
  struct Row {};
  __device__ __forceinline__ Columns(const Epi &, int, int n_, int) : n(n_) {}
  __device__ __forceinline__ void fetch(const Epi &, int, Row &) const {}
  __device__ __forceinline__ void finish(const Epi &e, int m, float v[2 * W], const Row &) const {
    if (flag<FLAGS>(e, kEpiGated, kKeeps)) {
      const long long at = place(m, 2 * e.ld_gu) + n;
      store_w<W>(e.gu, kF32, at, v);
      store_w<W>(e.gu, kF32, at + e.ld_gu, v + W);
    }
    activate<W>(e.act, v, nullptr);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= v[W + i];
    store_w<W>(e.y, y_fmt<FLAGS>(e), place(m, e.ldy) + n, v);
  }
};

// ------------------------------------------- from a wave's sums staged in LDS

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Column c of row r of a wave's staged rows of COLS sums: 16-byte chunks are
// moved by the row, so that rows of one chunk fall on different banks.
template <int COLS>
__device__ __forceinline__ const char *staged(const char *mine, int r, int c) {
  return mine + r * (COLS * 4) + ((((c >> 2) ^ (r & (COLS >= 64 ? 15 : 7)))) << 4) + (c & 3) * 4;
}

// The epilogue of `rows` staged rows m0.. and their columns n0..,
// W columns of a row to a lane at a time.  A gated product's staged columns
// are 8 gate sums, the 8 up sums of the same columns, and so on.  The next
// rows are fetched before the present ones are stored.  FLIP: the columns of
// the FLIP staged rows are the result's rows, and its columns the staged rows.
template <int KIND, int COLS, int W, int FLAGS, int FLIP>
__device__ __forceinline__ void finish_rows(const Epi &e, const char *mine, int lane, int batch,
                                            int m0, int rows, int n0, int N) {
  constexpr bool DUAL = KIND == kEpiGated;
  constexpr int kOut = DUAL ? COLS / 2 : FLIP ? FLIP : COLS;  // columns of the result
  constexpr int kLanes = kOut / W < 64 ? kOut / W : 64;
  constexpr int kRows = 64 / kLanes, kAtOnce = W == 1 ? 4 : 2;
#pragma unroll 1
  for (int c = (lane % kLanes) * W; c < kOut; c += kLanes * W) {
    if (n0 + c >= e.store_n) continue;
    const Columns<KIND, W, FLAGS> cols(e, batch, n0 + c, N);
    typename Columns<KIND, W, FLAGS>::Row row[kAtOnce], next[kAtOnce];
    auto fetch = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int r = r0 + u * kRows;
        cols.fetch(e, m0 + (r < rows ? r : rows - 1), next[u]);
      }
    };
    fetch(lane / kLanes);
    // what the columns need is there, so that nothing in the loop waits for it
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
#pragma unroll 1
    for (int r0 = lane / kLanes; r0 < rows; r0 += kRows * kAtOnce) {
      float v[kAtOnce][DUAL ? 2 * W : W];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) row[u] = next[u];
      fetch(r0 + kRows * kAtOnce);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        // a row past the last is read (the staged rows go on) and not used
        const int r = r0 + u * kRows;
#pragma unroll
        for (int k = 0; k < (DUAL ? 2 : 1); ++k) {
          const int s = DUAL ? (c >> 3) * 16 + (c & 7) + k * 8 : c;
          if constexpr (FLIP != 0) {
#pragma unroll
            for (int i = 0; i < W; ++i) v[u][i] = *(const float *)staged<COLS>(mine, s + i, r);
          } else if constexpr (W == 1) {
            v[u][k] = *(const float *)staged<COLS>(mine, r, s);
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const f32x4 w = *(const f32x4 *)staged<COLS>(mine, r, s + x * 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[u][k * 8 + x * 4 + i] = w[i];
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (r0 + u * kRows < rows) cols.finish(e, m0 + r0 + u * kRows, v[u], row[u]);
    }
  }
}

template <int KIND, int COLS, int W, int FLIP>
__device__ __forceinline__ void finish_flags(const Epi &e, const char *mine, int lane, int batch,
                                             int m0, int rows, int n0, int N) {
  const int f = epi_flags(KIND, e);
  auto with = [&](auto flags) {
    finish_rows<KIND, COLS, W, decltype(flags)::value, FLIP>(e, mine, lane, batch, m0, rows, n0, N);
  };
  if constexpr (KIND == kEpiGatedGrad) {
    (f & kWide) ? with(Flags<kWide>()) : with(Flags<0>());
  } else if constexpr (KIND == kEpiGated) {
    if (f & kWide)
      (f & kKeeps) ? with(Flags<kWide | kKeeps>()) : with(Flags<kWide>());
    else
      (f & kKeeps) ? with(Flags<kKeeps>()) : with(Flags<0>());
  } else {
    switch (f) {
      case 0: return with(Flags<0>());
      case 1: return with(Flags<1>());
      case 2: return with(Flags<2>());
      case 3: return with(Flags<3>());
      case 4: return with(Flags<4>());
      case 5: return with(Flags<5>());
      case 6: return with(Flags<6>());
      default: return with(Flags<7>());
    }
  }
}

template <int KIND, int COLS, int FLIP = 0>
__device__ __forceinline__ void finish_staged(const Epi &e, const char *mine, int lane, int batch,
                                              int m0, int rows, int n0, int N) {
  if (rows <= 0) return;
  if (e.vec)
    finish_flags<KIND, COLS, 8, FLIP>(e, mine, lane, batch, m0, rows, n0, N);
  else if constexpr (KIND == kEpiLinear || KIND == kEpiPoly)  // the others write rows of their own
    finish_flags<KIND, COLS, 1, FLIP>(e, mine, lane, batch, m0, rows, n0, N);
}

// The sums themselves, as one part of a contraction that is cut: rows m0..
// and columns n0.. of a part's N columns.  FLIP: as above.
template <int COLS, int FLIP>
__device__ __forceinline__ void store_staged(const char *mine, int lane, float *part, int m0,
                                             int rows, int n0, int N) {
  constexpr int kLanes = (FLIP ? FLIP : COLS) / 4, kRows = 64 / kLanes;
  const int c = (lane % kLanes) * 4;
  const int left = N - n0 - c;
  if (left <= 0) return;
#pragma unroll 2
  for (int r = lane / kLanes; r < rows; r += kRows) {
    f32x4 w;
    if constexpr (FLIP != 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *(const float *)staged<COLS>(mine, c + i, r);
    } else {
      w = *(const f32x4 *)staged<COLS>(mine, r, c);
    }
    float *to = part + (long long)(m0 + r) * N + n0 + c;
    if ((N & 3) == 0) {
      *(f32x4 *)to = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) to[i] = w[i];
    }
  }
}

}  // namespace dense
}  // namespace pdr
