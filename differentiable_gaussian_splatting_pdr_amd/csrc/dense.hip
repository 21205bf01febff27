// dense.hip -- the operators of include/pdr_dense.h: argument checks, the
// passes around the products (layout of operands, slopes, norms) and the
// order of launches.
#include <math.h>
#include <stdint.h>

#include "dense_internal.hpp"
#include "pdr_dense.h"

using namespace pdr::dense;

namespace {

constexpr int kThreads = 256;
constexpr int kAmaxBlocks = 256;

// ------------------------------------------------------------------ kernels

// Copy a 16-bit matrix to rows of ldd elements (a multiple of 8), zeros after
// each row's end.  One thread per 8 values.
__global__ __launch_bounds__(kThreads) void k_repack(const uint16_t *__restrict__ src, long long ld,
                                                     long long rows, int cols,
                                                     uint16_t *__restrict__ dst, int ldd) {
  const int groups = ldd / 8;
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long r = at / groups;
  if (r >= rows) return;
  const int c = (int)(at - r * groups) * 8;
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) w[i >> 1] |= (uint32_t)src[r * ld + c + i] << ((i & 1) * 16);
  *(uint4 *)(dst + r * ldd + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest finite magnitude of an fp32 matrix, one value per workgroup.
__global__ __launch_bounds__(kThreads) void k_amax(const float *__restrict__ src, long long ld,
                                                   long long rows, int cols,
                                                   float *__restrict__ part) {
  const int groups = (cols + 7) / 8;
  const long long total = rows * groups;
  float best = 0.f;
  for (long long at = (long long)blockIdx.x * kThreads + threadIdx.x; at < total;
       at += (long long)gridDim.x * kThreads) {
    const long long r = at / groups;
    const int c = (int)(at - r * groups) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) {
        const float a = fabsf(src[r * ld + c + i]);
        if (a < INFINITY) best = fmaxf(best, a);
      }
  }
  __shared__ float red[kThreads];
  red[threadIdx.x] = best;
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] = fmaxf(red[threadIdx.x], red[threadIdx.x + s]);
    __syncthreads();
  }
  if (threadIdx.x == 0) part[blockIdx.x] = red[0];
}

// Split an fp32 matrix into fp16 planes hi + lo under the scale 2^e that
// brings its largest value to [2^14, 2^15); e goes to *exp.
__global__ __launch_bounds__(kThreads) void k_split(const float *__restrict__ src, long long ld,
                                                    long long rows, int cols,
                                                    const float *__restrict__ part,
                                                    uint16_t *__restrict__ hi,
                                                    uint16_t *__restrict__ lo, int ldd,
                                                    int *__restrict__ exp) {
  __shared__ float red[kThreads];
  red[threadIdx.x] = part[threadIdx.x];
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] = fmaxf(red[threadIdx.x], red[threadIdx.x + s]);
    __syncthreads();
  }
  const float amax = red[0];
  const int e = amax > 0.f ? 14 - ilogbf(amax) : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *exp = e;
  const int groups = ldd / 8;
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long r = at / groups;
  if (r >= rows) return;
  const int c = (int)(at - r * groups) * 8;
  float h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = c + i < cols ? ldexpf(src[r * ld + c + i], e) : 0.f;
    h[i] = f16_to_f(f_to_f16(v));
    l[i] = fabsf(v) < INFINITY ? v - h[i] : 0.f;
  }
  store8(hi, kF16, r * ldd + c, 8, 1, h);
  store8(lo, kF16, r * ldd + c, 8, 1, l);
}

// dz = dy * slope (slope null: dz = dy), rounded to the products' format, and
// the sums of dz over this workgroup's rows.  A workgroup takes kDzRows rows
// and 256 columns (32 threads of 8 columns, 8 rows at a time).
constexpr int kDzRows = 256;
__global__ __launch_bounds__(kThreads) void k_dz(const void *__restrict__ dy, int dy_fmt,
                                                 long long lddy, const void *__restrict__ slope,
                                                 int slope_fmt, long long ld_slope, long long M,
                                                 int N, void *__restrict__ dz, int dz_fmt,
                                                 long long ld_dz, float *__restrict__ colsum,
                                                 int vec) {
  const int n = (blockIdx.y * 32 + (threadIdx.x & 31)) * 8;
  const int ty = threadIdx.x >> 5;
  const long long m0 = (long long)blockIdx.x * kDzRows;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n < N) {
    for (int i = ty; i < kDzRows && m0 + i < M; i += 8) {
      const long long m = m0 + i;
      float v[8], s[8];
      load8(dy, dy_fmt, m * lddy + n, N - n, vec, v);
      if (slope) {
        load8(slope, slope_fmt, m * ld_slope + n, N - n, 1, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= s[j];
      }
      if (dz) store8(dz, dz_fmt, m * ld_dz + n, 8, 1, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
    }
  }
  if (!colsum) return;
  __shared__ float red[8][256];
#pragma unroll
  for (int j = 0; j < 8; ++j) red[ty][(threadIdx.x & 31) * 8 + j] = sum[j];
  __syncthreads();
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c < N) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][threadIdx.x];
    colsum[(long long)blockIdx.x * N + c] = t;
  }
}

// dbias[n] = sum of the row blocks' sums.
__global__ __launch_bounds__(kThreads) void k_colsum(const float *__restrict__ part, int blocks,
                                                     int N, void *__restrict__ out, int fmt) {
  const int n = blockIdx.x * 32 + (threadIdx.x & 31), ty = threadIdx.x >> 5;
  float s = 0.f;
  if (n < N)
    for (int b = ty; b < blocks; b += 8) s += part[(long long)b * N + n];
  __shared__ float red[8][32];
  red[ty][threadIdx.x & 31] = s;
  __syncthreads();
  if (ty == 0 && n < N) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][threadIdx.x];
    store1(out, fmt, n, t);
  }
}

// Sums of squares of a batch's matrices (fp64: the square of any fp32 value is
// in range), kNormBlocks partial sums per matrix.
constexpr int kNormBlocks = 128;
__global__ __launch_bounds__(kThreads) void k_squares(const void *__restrict__ g, int fmt,
                                                      long long ld, long long batch_g, long long m,
                                                      int n, int vec, double *__restrict__ part) {
  const int groups = (n + 7) / 8;
  const long long total = m * groups;
  double s = 0.0;
  for (long long at = (long long)blockIdx.x * kThreads + threadIdx.x; at < total;
       at += (long long)kNormBlocks * kThreads) {
    const long long r = at / groups;
    const int c = (int)(at - r * groups) * 8;
    float v[8];
    load8(g, fmt, blockIdx.y * batch_g + r * ld + c, n - c, vec, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (double)v[i] * (double)v[i];
  }
  __shared__ double red[kThreads];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int h = kThreads / 2; h > 0; h >>= 1) {
    if (threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) part[blockIdx.y * kNormBlocks + blockIdx.x] = red[0];
}

// x = g / (|g| + eps) 2^shift in fp16 planes (lo null: one), or in format
// `fmt_out` with no planes; rows of ldx elements, zeros after each row's end.
__global__ __launch_bounds__(kThreads) void k_normalise(
    const void *__restrict__ g, int fmt, long long ld, long long batch_g, long long m, int n, int vec,
    const double *__restrict__ part, float eps, int shift, void *__restrict__ x,
    void *__restrict__ x_lo, int fmt_out, long long ldx, long long batch_x, int cols_out, int vec_out) {
  __shared__ double red[kNormBlocks];
  if (threadIdx.x < kNormBlocks) red[threadIdx.x] = part[blockIdx.y * kNormBlocks + threadIdx.x];
  __syncthreads();
  for (int h = kNormBlocks / 2; h > 0; h >>= 1) {
    if (threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
    __syncthreads();
  }
  const double scale = ldexp(1.0 / (sqrt(red[0]) + (double)eps), shift);
  const int groups = (cols_out + 7) / 8;
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long r = at / groups;
  if (r >= m) return;
  const int c = (int)(at - r * groups) * 8;
  float v[8], lo[8];
  load8(g, fmt, blockIdx.y * batch_g + r * ld + c, n - c, vec, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a zero matrix with eps = 0 stays zero rather than 0 * inf
    const float t = v[i] == 0.f ? 0.f : (float)((double)v[i] * scale);
    v[i] = t;
    lo[i] = t - f16_to_f(f_to_f16(t));
  }
  const long long to = blockIdx.y * batch_x + r * ldx + c;
  store8(x, fmt_out, to, cols_out - c, vec_out, v);
  if (x_lo) store8(x_lo, kF16, to, cols_out - c, vec_out, lo);
}

// ------------------------------------------------------------------- set-up

bool good_fmt(int f) { return f == kF32 || f == kF16 || f == kBf16; }
bool good_len(long long n) { return n >= 0 && n <= 0x7fffffffLL - 256; }
// A matrix of this many rows and columns: its pointer and row distance.
bool good_mat(const void *p, long long ld, long long rows, long long cols, int fmt) {
  if (rows == 0 || cols == 0) return true;
  if (!p || ((uintptr_t)p & (uintptr_t)(fmt_bytes(fmt) - 1))) return false;
  return ld >= cols && ld <= kMaxLd;
}
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// The workspace: a first walk with no base counts bytes, a second one with
// the caller's memory launches.
struct Walk {
  char *base = nullptr;
  size_t at = 0, high = 0;
  hipStream_t st = nullptr;
  bool run = false;
  hipError_t err = hipSuccess;

  void *take(size_t bytes) {
    void *p = base + at;
    at += (bytes + 255) / 256 * 256;
    if (at > high) high = at;
    return p;
  }
  void done(hipError_t e) {
    if (err == hipSuccess) err = e;
  }
  bool go() const { return run && err == hipSuccess; }
};

// A matrix as the products read it: one 16-bit plane, or two of a split fp32.
struct Planes {
  const uint16_t *hi = nullptr, *lo = nullptr;
  const int *exp = nullptr;
  long long ld = 0;
};

int product_fmt(int fmt) { return fmt == kBf16 ? kBf16 : kF16; }

Planes lay_out(Walk &w, const void *p, int fmt, long long ld, long long rows, long long cols,
               bool summed_along_row) {
  Planes r;
  if (rows == 0 || cols == 0) {
    r.ld = round8(cols > 0 ? cols : 1);
    return r;
  }
  if (fmt != kF32 && aligned16(p) && (ld & 7) == 0 && (!summed_along_row || (cols & 7) == 0)) {
    r.hi = (const uint16_t *)p;
    r.ld = ld;
    return r;
  }
  const long long ldd = round8(cols);
  const unsigned blocks = (unsigned)((rows * (ldd / 8) + kThreads - 1) / kThreads);
  uint16_t *hi = (uint16_t *)w.take((size_t)(rows * ldd) * 2);
  r.hi = hi;
  r.ld = ldd;
  if (fmt != kF32) {
    if (w.go()) {
      hipLaunchKernelGGL(k_repack, dim3(blocks), dim3(kThreads), 0, w.st, (const uint16_t *)p, ld,
                         rows, (int)cols, hi, (int)ldd);
      w.done(hipGetLastError());
    }
    return r;
  }
  uint16_t *lo = (uint16_t *)w.take((size_t)(rows * ldd) * 2);
  float *part = (float *)w.take(kAmaxBlocks * sizeof(float));
  int *exp = (int *)w.take(sizeof(int));
  r.lo = lo;
  r.exp = exp;
  if (w.go()) {
    hipLaunchKernelGGL(k_amax, dim3(kAmaxBlocks), dim3(kThreads), 0, w.st, (const float *)p, ld, rows,
                       (int)cols, part);
    hipLaunchKernelGGL(k_split, dim3(blocks), dim3(kThreads), 0, w.st, (const float *)p, ld, rows,
                       (int)cols, part, hi, lo, (int)ldd, exp);
    w.done(hipGetLastError());
  }
  return r;
}

// Add the product of two matrices, offset by so many elements, to the
// segments: one, or three with split operands.
void add_product(GemmArgs &g, const Planes &a, long long off_a, const Planes &b, long long off_b) {
  auto add = [&](const uint16_t *pa, const uint16_t *pb) {
    g.a[g.segs] = pa ? pa + off_a : nullptr;
    g.b[g.segs] = pb ? pb + off_b : nullptr;
    ++g.segs;
  };
  add(a.hi, b.hi);
  if (a.lo && b.lo) {
    add(a.hi, b.lo);
    add(a.lo, b.hi);
  }
  g.lda = a.ld;
  g.ldb = b.ld;
}

GemmArgs product(long long M, long long N, long long K) {
  GemmArgs g = {};
  g.M = (int)M;
  g.N = (int)N;
  g.K = g.ka = g.kb = (int)K;
  g.batches = 1;
  g.epi.store_n = (int)N;
  return g;
}

void multiply(Walk &w, const GemmArgs &g, int fmt, bool a_mc, bool b_mc, EpiKind kind) {
  const size_t keep = w.at;
  void *ws = w.take(gemm_scratch_bytes(g, kind));
  if (w.go())
    w.done(product_fmt(fmt) == kBf16 ? launch_gemm_bf16(g, a_mc, b_mc, kind, ws, w.st)
                                     : launch_gemm_f16(g, a_mc, b_mc, kind, ws, w.st));
  w.at = keep;  // the next launch on this stream may use it again
}

void set_out(Epi &e, void *y, int fmt, long long ldy) {
  e.y = y;
  e.fmt = fmt;
  e.ldy = (int)ldy;
  e.vec = aligned16(y) && (ldy & 7) == 0;
}

// ------------------------------------------------------------------- linear

int check_linear(const pdr_linear *p, bool backward) {
  if (!p || !good_fmt(p->fmt) || (p->out_fmt != p->fmt && p->out_fmt != kF32)) return PDR_ERR_INVALID_ARG;
  if (p->activation < PDR_ACT_NONE || p->activation > PDR_ACT_GELU) return PDR_ERR_INVALID_ARG;
  if (!good_len(p->M) || !good_len(p->N) || !good_len(p->K)) return PDR_ERR_INVALID_ARG;
  if (!good_mat(p->x, p->ldx, p->M, p->K, p->fmt) || !good_mat(p->w, p->ldw, p->N, p->K, p->fmt))
    return PDR_ERR_INVALID_ARG;
  if (p->slope && !aligned16(p->slope)) return PDR_ERR_INVALID_ARG;
  if (!backward) {
    if (!good_mat(p->y, p->ldy, p->M, p->N, p->out_fmt)) return PDR_ERR_INVALID_ARG;
    if (p->res && !good_mat(p->res, p->ldr, p->M, p->N, p->out_fmt)) return PDR_ERR_INVALID_ARG;
    if ((uintptr_t)p->bias & (uintptr_t)(fmt_bytes(p->fmt) - 1)) return PDR_ERR_INVALID_ARG;
    return PDR_OK;
  }
  if (!good_mat(p->dy, p->lddy, p->M, p->N, p->out_fmt)) return PDR_ERR_INVALID_ARG;
  if (p->dx && !good_mat(p->dx, p->lddx, p->M, p->K, p->fmt)) return PDR_ERR_INVALID_ARG;
  if (p->dw && !good_mat(p->dw, p->lddw, p->N, p->K, p->fmt)) return PDR_ERR_INVALID_ARG;
  if ((uintptr_t)p->dbias & (uintptr_t)(fmt_bytes(p->fmt) - 1)) return PDR_ERR_INVALID_ARG;
  if (p->activation != PDR_ACT_NONE && p->M && p->N && !p->slope) return PDR_ERR_INVALID_ARG;
  return PDR_OK;
}

int slope_fmt(int fmt) { return fmt == kBf16 ? kF16 : kF32; }

void linear_forward(Walk &w, const pdr_linear &p) {
  const Planes x = lay_out(w, p.x, p.fmt, p.ldx, p.M, p.K, true);
  const Planes wt = lay_out(w, p.w, p.fmt, p.ldw, p.N, p.K, true);
  GemmArgs g = product(p.M, p.N, round8(p.K));
  add_product(g, x, 0, wt, 0);
  set_out(g.epi, p.y, p.out_fmt, p.ldy);
  g.epi.exp_a = x.exp;
  g.epi.exp_b = wt.exp;
  g.epi.bias = p.bias;
  g.epi.bias_fmt = p.fmt;
  g.epi.res = p.res;
  g.epi.ldr = (int)p.ldr;
  g.epi.vec = g.epi.vec && (!p.bias || aligned16(p.bias)) && (!p.res || (aligned16(p.res) && (p.ldr & 7) == 0));
  g.epi.act = p.activation;
  g.epi.slope = p.slope;
  g.epi.slope_fmt = slope_fmt(p.fmt);
  g.epi.ld_slope = (int)round8(p.N);
  multiply(w, g, p.fmt, false, false, kEpiLinear);
}

void linear_backward(Walk &w, const pdr_linear &p) {
  const bool act = p.activation != PDR_ACT_NONE;
  const bool products = p.dx || p.dw;
  // dz in its own rows unless it is dy itself
  const void *dz = p.dy;
  long long ld_dz = p.lddy;
  const bool write = products && p.M && p.N && (act || p.out_fmt != p.fmt);
  void *buf = nullptr;
  if (write) {
    ld_dz = round8(p.N);
    dz = buf = w.take((size_t)(p.M * ld_dz) * fmt_bytes(p.fmt));
  }
  const int row_blocks = (int)((p.M + kDzRows - 1) / kDzRows);
  float *part = p.dbias ? (float *)w.take((size_t)row_blocks * p.N * sizeof(float)) : nullptr;
  if ((write || p.dbias) && p.N && w.go()) {
    if (row_blocks)
      hipLaunchKernelGGL(k_dz, dim3((unsigned)row_blocks, (unsigned)((p.N + 255) / 256)),
                         dim3(kThreads), 0, w.st, p.dy, p.out_fmt, p.lddy, act ? p.slope : nullptr,
                         slope_fmt(p.fmt), round8(p.N), p.M, (int)p.N, buf, p.fmt, ld_dz, part,
                         aligned16(p.dy) && (p.lddy & 7) == 0);
    if (p.dbias)
      hipLaunchKernelGGL(k_colsum, dim3((unsigned)((p.N + 31) / 32)), dim3(kThreads), 0, w.st, part,
                         row_blocks, (int)p.N, p.dbias, p.fmt);
    w.done(hipGetLastError());
  }
  if (!products) return;
  const Planes z = lay_out(w, dz, p.fmt, ld_dz, p.M, write ? round8(p.N) : p.N, p.dx != nullptr);
  if (p.dx) {
    const size_t keep = w.at;
    const Planes wt = lay_out(w, p.w, p.fmt, p.ldw, p.N, p.K, false);
    GemmArgs g = product(p.M, p.K, round8(p.N));
    g.kb = (int)p.N;
    add_product(g, z, 0, wt, 0);
    set_out(g.epi, p.dx, p.fmt, p.lddx);
    g.epi.exp_a = z.exp;
    g.epi.exp_b = wt.exp;
    multiply(w, g, p.fmt, false, true, kEpiLinear);
    w.at = keep;
  }
  if (p.dw) {
    const Planes x = lay_out(w, p.x, p.fmt, p.ldx, p.M, p.K, false);
    GemmArgs g = product(p.N, p.K, p.M);
    add_product(g, z, 0, x, 0);
    set_out(g.epi, p.dw, p.fmt, p.lddw);
    g.epi.exp_a = z.exp;
    g.epi.exp_b = x.exp;
    multiply(w, g, p.fmt, true, true, kEpiLinear);
  }
}

// -------------------------------------------------------------- gated block

int check_gated(const pdr_gated_mlp *p, bool backward) {
  if (!p || !good_fmt(p->fmt)) return PDR_ERR_INVALID_ARG;
  if (p->activation < PDR_ACT_NONE || p->activation > PDR_ACT_GELU) return PDR_ERR_INVALID_ARG;
  if (!good_len(p->M) || !good_len(p->D) || !good_len(p->F) || !good_len(p->O)) return PDR_ERR_INVALID_ARG;
  if (2 * round8(p->F) > kMaxLd) return PDR_ERR_INVALID_ARG;
  if (!good_mat(p->x, p->ldx, p->M, p->D, p->fmt) ||
      !good_mat(p->w_in, p->ld_in, 2 * p->F, p->D, p->fmt) ||
      !good_mat(p->w_out, p->ld_out, p->O, p->F, p->fmt))
    return PDR_ERR_INVALID_ARG;
  if (p->M && p->F && (!p->h || !aligned16(p->h))) return PDR_ERR_INVALID_ARG;
  if (!aligned16(p->gu)) return PDR_ERR_INVALID_ARG;
  if (!backward) {
    if (!good_mat(p->y, p->ldy, p->M, p->O, p->fmt)) return PDR_ERR_INVALID_ARG;
    if (p->res && !good_mat(p->res, p->ldr, p->M, p->O, p->fmt)) return PDR_ERR_INVALID_ARG;
    return PDR_OK;
  }
  if (!good_mat(p->dy, p->lddy, p->M, p->O, p->fmt)) return PDR_ERR_INVALID_ARG;
  if (p->dx && !good_mat(p->dx, p->lddx, p->M, p->D, p->fmt)) return PDR_ERR_INVALID_ARG;
  if (p->dw_in && !good_mat(p->dw_in, p->ldd_in, 2 * p->F, p->D, p->fmt)) return PDR_ERR_INVALID_ARG;
  if (p->dw_out && !good_mat(p->dw_out, p->ldd_out, p->O, p->F, p->fmt)) return PDR_ERR_INVALID_ARG;
  if ((p->dx || p->dw_in) && p->M && p->F && !p->gu) return PDR_ERR_INVALID_ARG;
  return PDR_OK;
}

void gated_forward(Walk &w, const pdr_gated_mlp &p) {
  const long long Fp = round8(p.F);
  {
    const size_t keep = w.at;
    const Planes x = lay_out(w, p.x, p.fmt, p.ldx, p.M, p.D, true);
    const Planes wi = lay_out(w, p.w_in, p.fmt, p.ld_in, 2 * p.F, p.D, true);
    GemmArgs g = product(p.M, p.F, round8(p.D));
    add_product(g, x, 0, wi, 0);
    g.up_at = p.F * wi.ld;
    set_out(g.epi, p.h, p.fmt, Fp);
    g.epi.store_n = (int)Fp;
    g.epi.exp_a = x.exp;
    g.epi.exp_b = wi.exp;
    g.epi.act = p.activation;
    g.epi.gu = (float *)p.gu;
    g.epi.ld_gu = (int)Fp;
    multiply(w, g, p.fmt, false, false, kEpiGated);
    w.at = keep;
  }
  const Planes h = lay_out(w, p.h, p.fmt, Fp, p.M, Fp, true);
  const Planes wo = lay_out(w, p.w_out, p.fmt, p.ld_out, p.O, p.F, true);
  GemmArgs g = product(p.M, p.O, Fp);
  add_product(g, h, 0, wo, 0);
  set_out(g.epi, p.y, p.fmt, p.ldy);
  g.epi.exp_a = h.exp;
  g.epi.exp_b = wo.exp;
  g.epi.res = p.res;
  g.epi.ldr = (int)p.ldr;
  g.epi.vec = g.epi.vec && (!p.res || (aligned16(p.res) && (p.ldr & 7) == 0));
  multiply(w, g, p.fmt, false, false, kEpiLinear);
}

void gated_backward(Walk &w, const pdr_gated_mlp &p) {
  const long long Fp = round8(p.F);
  const bool through = p.dx || p.dw_in;
  const Planes dy = lay_out(w, p.dy, p.fmt, p.lddy, p.M, p.O, through);
  if (p.dw_out) {
    const size_t keep = w.at;
    const Planes h = lay_out(w, p.h, p.fmt, Fp, p.M, Fp, false);
    GemmArgs g = product(p.O, p.F, p.M);
    add_product(g, dy, 0, h, 0);
    set_out(g.epi, p.dw_out, p.fmt, p.ldd_out);
    g.epi.exp_a = dy.exp;
    g.epi.exp_b = h.exp;
    multiply(w, g, p.fmt, true, true, kEpiLinear);
    w.at = keep;
  }
  if (!through) return;
  void *dgu = w.take((size_t)(p.M * 2 * Fp) * fmt_bytes(p.fmt));
  {
    const size_t keep = w.at;
    const Planes wo = lay_out(w, p.w_out, p.fmt, p.ld_out, p.O, p.F, false);
    GemmArgs g = product(p.M, p.F, round8(p.O));
    g.kb = (int)p.O;
    add_product(g, dy, 0, wo, 0);
    set_out(g.epi, dgu, p.fmt, 2 * Fp);
    g.epi.store_n = (int)Fp;
    g.epi.up_at = (int)Fp;
    g.epi.exp_a = dy.exp;
    g.epi.exp_b = wo.exp;
    g.epi.act = p.activation;
    g.epi.gu = (float *)p.gu;
    g.epi.ld_gu = (int)Fp;
    multiply(w, g, p.fmt, false, true, kEpiGatedGrad);
    w.at = keep;
  }
  const Planes d = lay_out(w, dgu, p.fmt, 2 * Fp, p.M, 2 * Fp, true);
  if (p.dx) {
    const size_t keep = w.at;
    const Planes wi = lay_out(w, p.w_in, p.fmt, p.ld_in, 2 * p.F, p.D, false);
    GemmArgs g = product(p.M, p.D, Fp);
    g.kb = (int)p.F;
    add_product(g, d, 0, wi, 0);
    add_product(g, d, Fp, wi, p.F * wi.ld);
    set_out(g.epi, p.dx, p.fmt, p.lddx);
    g.epi.exp_a = d.exp;
    g.epi.exp_b = wi.exp;
    multiply(w, g, p.fmt, false, true, kEpiLinear);
    w.at = keep;
  }
  if (p.dw_in) {
    const Planes x = lay_out(w, p.x, p.fmt, p.ldx, p.M, p.D, false);
    GemmArgs g = product(p.F, p.D, p.M);
    add_product(g, d, 0, x, 0);
    g.batches = 2;  // the gate rows, then the up rows
    g.batch_a = Fp;
    set_out(g.epi, p.dw_in, p.fmt, p.ldd_in);
    g.epi.batch_y = p.F * p.ldd_in;
    g.epi.vec = g.epi.vec && (g.epi.batch_y * fmt_bytes(p.fmt)) % 16 == 0;
    g.epi.exp_a = d.exp;
    g.epi.exp_b = x.exp;
    multiply(w, g, p.fmt, true, true, kEpiLinear);
  }
}

// ------------------------------------------------------------ orthogonalize

int check_ortho(const pdr_orthogonalize_args *p) {
  if (!p || !good_fmt(p->fmt) || p->steps < 0) return PDR_ERR_INVALID_ARG;
  if (!good_len(p->batch) || p->batch > 65535 || !good_len(p->m) || !good_len(p->n)) return PDR_ERR_INVALID_ARG;
  if (round8(p->m) > kMaxLd || round8(p->n) > kMaxLd) return PDR_ERR_INVALID_ARG;
  const long long rows = p->batch ? p->m : 0;
  if (!good_mat(p->g, p->ldg, rows, p->n, p->fmt) || !good_mat(p->x, p->ldx, rows, p->n, p->fmt))
    return PDR_ERR_INVALID_ARG;
  if (!isfinite(p->a) || !isfinite(p->b) || !isfinite(p->c) || !isfinite(p->eps) || p->eps < 0.f)
    return PDR_ERR_INVALID_ARG;
  return PDR_OK;
}

// Powers of two that keep the iterates' entries well inside fp16's normal
// range: X's entries are at most a singular value (< 8) and about 1/sqrt(n),
// those of A and B at most (b + c) and about 1/n.
constexpr int kShiftX = 12, kShiftA = 10;

void orthogonalize(Walk &w, const pdr_orthogonalize_args &p) {
  const bool two = p.fmt != kBf16, tall = p.m > p.n;
  const long long s = tall ? p.n : p.m, sp = round8(s), np = round8(p.n);
  const size_t x_bytes = (size_t)(p.batch * p.m * np) * 2, a_bytes = (size_t)(p.batch * s * sp) * 2;
  double *part = (double *)w.take((size_t)p.batch * kNormBlocks * sizeof(double));
  if (p.batch == 0 || p.m == 0 || p.n == 0) return;
  const int vec_g = aligned16(p.g) && (p.ldg & 7) == 0 && (p.batch_g & 7) == 0;
  const int vec_x = aligned16(p.x) && (p.ldx & 7) == 0 && (p.batch_x & 7) == 0;
  auto normalise = [&](void *x, void *lo, int shift, int fmt, long long ldx, long long batch_x,
                       long long cols, int vec) {
    const long long threads = p.m * ((cols + 7) / 8);
    if (!w.go()) return;
    hipLaunchKernelGGL(k_squares, dim3(kNormBlocks, (unsigned)p.batch), dim3(kThreads), 0, w.st, p.g,
                       p.fmt, p.ldg, p.batch_g, p.m, (int)p.n, vec_g, part);
    hipLaunchKernelGGL(k_normalise,
                       dim3((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)p.batch),
                       dim3(kThreads), 0, w.st, p.g, p.fmt, p.ldg, p.batch_g, p.m, (int)p.n, vec_g,
                       part, p.eps, shift, x, lo, fmt, ldx, batch_x, (int)cols, vec);
    w.done(hipGetLastError());
  };
  if (p.steps == 0) {
    normalise(p.x, nullptr, 0, p.fmt, p.ldx, p.batch_x, p.n, vec_x);
    return;
  }
  auto planes = [&](size_t bytes, long long ld) {
    Planes q;
    q.hi = (const uint16_t *)w.take(bytes);
    if (two) q.lo = (const uint16_t *)w.take(bytes);
    q.ld = ld;
    return q;
  };
  Planes x[2] = {planes(x_bytes, np), p.steps > 1 ? planes(x_bytes, np) : Planes()};
  const Planes a = planes(a_bytes, sp), b = planes(a_bytes, sp);
  normalise((void *)x[0].hi, (void *)x[0].lo, kShiftX, kF16, np, p.m * np, np, 1);

  auto to = [](Epi &e, const Planes &y, long long batch) {
    set_out(e, (void *)y.hi, kF16, y.ld);
    e.y_lo = (void *)y.lo;
    e.batch_y = batch;
  };
  auto plus = [](Epi &e, float beta, const Planes &c, long long batch) {
    e.beta = beta;
    e.c = c.hi;
    e.c_lo = c.lo;
    e.ldc = (int)c.ld;
    e.batch_c = batch;
  };
  for (int i = 0; i < p.steps; ++i) {
    const Planes &xi = x[i & 1], &xo = x[(i + 1) & 1];
    {  // A = X X^T or X^T X
      GemmArgs g = product(s, s, tall ? p.m : np);
      add_product(g, xi, 0, xi, 0);
      g.batches = (int)p.batch;
      g.batch_a = g.batch_b = p.m * np;
      to(g.epi, a, s * sp);
      g.epi.store_n = (int)sp;
      g.epi.alpha = ldexpf(1.f, kShiftA - 2 * kShiftX);
      multiply(w, g, kF16, tall, tall, kEpiPoly);
    }
    {  // B = b A + c A A; A is symmetric, so its rows serve as its columns
      GemmArgs g = product(s, s, sp);
      add_product(g, a, 0, a, 0);
      g.batches = (int)p.batch;
      g.batch_a = g.batch_b = s * sp;
      to(g.epi, b, s * sp);
      g.epi.store_n = (int)sp;
      g.epi.alpha = ldexpf(p.c, -kShiftA);
      plus(g.epi, p.b, a, s * sp);
      multiply(w, g, kF16, false, false, kEpiPoly);
    }
    // X <- a X + B X, or a X + X B
    const bool last = i + 1 == p.steps;
    GemmArgs g = product(p.m, p.n, sp);
    g.batches = (int)p.batch;
    if (tall) {
      add_product(g, xi, 0, b, 0);
      g.batch_a = p.m * np;
      g.batch_b = s * sp;
    } else {
      add_product(g, b, 0, xi, 0);
      g.kb = (int)s;
      g.batch_a = s * sp;
      g.batch_b = p.m * np;
    }
    const int down = last ? kShiftX : 0;
    if (last) {
      set_out(g.epi, p.x, p.fmt, p.ldx);
      g.epi.batch_y = p.batch_x;
      g.epi.vec = vec_x;
    } else {
      to(g.epi, xo, p.m * np);
      g.epi.store_n = (int)np;
    }
    g.epi.alpha = ldexpf(1.f, -kShiftA - down);
    plus(g.epi, ldexpf(p.a, -down), xi, p.m * np);
    multiply(w, g, kF16, false, !tall, kEpiPoly);
  }
}

template <class Desc, class Op>
long long bytes_of(const Desc &d, Op op) {
  Walk w;
  op(w, d);
  return (long long)w.high;
}

template <class Desc, class Op>
int run_in(const Desc &d, Op op, void *workspace, size_t bytes, void *stream) {
  const long long need = bytes_of(d, op);
  if (need > 0 && (!workspace || ((uintptr_t)workspace & 255u) || bytes < (size_t)need))
    return PDR_ERR_WORKSPACE;
  Walk w;
  w.base = (char *)workspace;
  w.st = (hipStream_t)stream;
  w.run = true;
  op(w, d);
  return w.err == hipSuccess ? PDR_OK : PDR_ERR_HIP;
}

}  // namespace

extern "C" {

long long pdr_dense_kept_ld(long long n) { return n < 0 ? PDR_ERR_INVALID_ARG : round8(n); }

long long pdr_linear_forward_workspace_bytes(const pdr_linear *p) {
  const int rc = check_linear(p, false);
  return rc != PDR_OK ? rc : bytes_of(*p, linear_forward);
}
int pdr_linear_forward(const pdr_linear *p, void *workspace, size_t workspace_bytes, void *stream) {
  const int rc = check_linear(p, false);
  return rc != PDR_OK ? rc : run_in(*p, linear_forward, workspace, workspace_bytes, stream);
}
long long pdr_linear_backward_workspace_bytes(const pdr_linear *p) {
  const int rc = check_linear(p, true);
  return rc != PDR_OK ? rc : bytes_of(*p, linear_backward);
}
int pdr_linear_backward(const pdr_linear *p, void *workspace, size_t workspace_bytes, void *stream) {
  const int rc = check_linear(p, true);
  return rc != PDR_OK ? rc : run_in(*p, linear_backward, workspace, workspace_bytes, stream);
}

long long pdr_gated_mlp_forward_workspace_bytes(const pdr_gated_mlp *p) {
  const int rc = check_gated(p, false);
  return rc != PDR_OK ? rc : bytes_of(*p, gated_forward);
}
int pdr_gated_mlp_forward(const pdr_gated_mlp *p, void *workspace, size_t workspace_bytes,
                          void *stream) {
  const int rc = check_gated(p, false);
  return rc != PDR_OK ? rc : run_in(*p, gated_forward, workspace, workspace_bytes, stream);
}
long long pdr_gated_mlp_backward_workspace_bytes(const pdr_gated_mlp *p) {
  const int rc = check_gated(p, true);
  return rc != PDR_OK ? rc : bytes_of(*p, gated_backward);
}
int pdr_gated_mlp_backward(const pdr_gated_mlp *p, void *workspace, size_t workspace_bytes,
                           void *stream) {
  const int rc = check_gated(p, true);
  return rc != PDR_OK ? rc : run_in(*p, gated_backward, workspace, workspace_bytes, stream);
}

long long pdr_orthogonalize_workspace_bytes(const pdr_orthogonalize_args *p) {
  const int rc = check_ortho(p);
  return rc != PDR_OK ? rc : bytes_of(*p, orthogonalize);
}
int pdr_orthogonalize(const pdr_orthogonalize_args *p, void *workspace, size_t workspace_bytes,
                      void *stream) {
  const int rc = check_ortho(p);
  return rc != PDR_OK ? rc : run_in(*p, orthogonalize, workspace, workspace_bytes, stream);
}

}  // extern "C"

// How a product is cut into workgroups: 256x256 tiles, one workgroup on a
// compute unit, or 128x128 tiles, two; and the contraction in one part or in
// several, which a second kernel joins.  The choice is the least of an
// estimate in microseconds whose constants are fits to measured products
// (bf16, M x N x K, this card): a step is 64 contraction values of every
// workgroup in flight.
//   128: 2048x2048x2048 (256 workgroups) 22.9, 1024x1024x4096 (64) 34.2,
//        4096x2048x2048 (512) 34.0, 8192x1024x2816 (512) 43.7
//   256: 8192x1024x512 (128) 23.9, 16384x1024x1024 (256) 36.7,
//        16384x2048x11264 (512, two rounds) 582; the same in 128 tiles: 687
//   parts: 2048x2048x11264 in 256 tiles: one part 210, four 91.9;
//        1024x1024x4096 in 128 tiles: one 34.2, four 21.6
namespace pdr {
namespace dense {

namespace {

double tiles_us(bool large, double workgroups, double steps) {
  const double slots = large ? 256.0 : 512.0;
  const double rounds = floor(workgroups / slots), rest = workgroups - rounds * slots;
  const double full = large ? 1.5 * steps + 9.0 : 0.9 * steps + 5.0;
  double last = 0.0;
  if (rest > 0.0) {
    if (large)
      last = (rest > 128.0 ? 1.5 : 1.2) * steps + 9.0;
    else
      last = rest > 256.0 ? full : 0.46 * steps + 4.0;
  }
  return rounds * full + last;
}

}  // namespace

TilePlan plan_tiles(const GemmArgs &g, EpiKind kind) {
  const int steps = (g.K + kBK - 1) / kBK * g.segs;
  const double batches = g.batches > 0 ? g.batches : 1;
  const double sums = batches * (double)g.M * (double)g.N;
  const int most = kind == kEpiGated ? 1 : steps / 2 > 32 ? 32 : steps / 2 > 1 ? steps / 2 : 1;
  TilePlan best = {};
  double least = 0.0;
  for (int large = 0; large < 2; ++large) {
    const int bm = large ? 256 : 128, bn = kind == kEpiGated ? bm / 2 : bm;
    TilePlan p;
    p.large = large != 0;
    p.tiles_m = (g.M + bm - 1) / bm;
    p.tiles_n = (g.epi.store_n + bn - 1) / bn;
    for (p.splits = 1; p.splits <= most; ++p.splits) {
      double us = tiles_us(p.large, batches * p.tiles_m * p.tiles_n * p.splits,
                           (double)((steps + p.splits - 1) / p.splits));
      // the parts are written and read once, at 4.6 TB/s
      if (p.splits > 1) us += 3.0 + 8.0 * sums * p.splits / 4.6e6;
      if (least == 0.0 || us < least) {
        least = us;
        best = p;
      }
    }
  }
  return best;
}

size_t gemm_scratch_bytes(const GemmArgs &g, EpiKind kind) {
  const TilePlan p = plan_tiles(g, kind);
  return p.splits > 1 ? (size_t)p.splits * (size_t)g.batches * (size_t)g.M * (size_t)g.N * 4 : 0;
}

}  // namespace dense
}  // namespace pdr
