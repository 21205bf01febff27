// dense.hip -- the operators of include/pdr_dense.h: argument checks, the
// passes around the products (layout of operands, slopes, norms) and the
// order of launches.
#include <math.h>
#include <stdint.h>

#include "dense_internal.hpp"
#include "pdr_common.hpp"
#include "pdr_dense.h"

using namespace pdr;
using namespace pdr::dense;

namespace {

constexpr int kThreads = 256;
constexpr int kParts = 1024;  // workgroups of a pass that reduces, at most

// ------------------------------------------------------------------ kernels
//
// The passes around the products are bound by memory (4.6 TB/s for a copy on
// this card): 8 values to a thread in 16-byte accesses where rows allow, a few
// rows in flight to a thread, and enough workgroups (about a thousand) to
// cover the latency.  k_dz of 16384 x 2048 bf16 (200 MB) takes 38.5 us, 5.2 TB/s;
// k_split of 5120 x 1024 fp32 (52 MB) 11 us; k_squares and k_normalise of
// 11264 x 2048 bf16 10 and 26 us.

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kThreads];
  red[threadIdx.x] = v;
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  return red[0];
}

// Values as sums of bf16 values, each the rest's nearest: two hold fp16's 11
// bits (and 16 of an fp32 value), three hold 24 bits, over fp32's own range (a
// rest below bf16's smallest step, 2^-133, is lost: the last bits of values
// below 2^-110).
constexpr int kMaxPlanes = 3;
__device__ __forceinline__ void store_planes(uint16_t *const *plane, int planes, long long at,
                                             float v[8]) {
#pragma unroll
  for (int k = 0; k < kMaxPlanes; ++k) {
    if (k >= planes) return;
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = bf16_to_f(f_to_bf16(v[i]));
      // a finite value that rounds to infinity is cut short; an infinity or a NaN has no rest
      const bool finite = fabsf(v[i]) < INFINITY;
      if (finite && fabsf(h[i]) == INFINITY) h[i] = __uint_as_float(__float_as_uint(v[i]) & 0xffff0000u);
      v[i] = finite ? v[i] - h[i] : 0.f;
    }
    store_w<8>(plane[k], kBf16, at, h);
  }
}

// Matrices to lay out for the products, several to a launch: workgroups
// [first, first of the next) of a pass work on one matrix.
constexpr int kMaxPrep = 6;
struct Prep {
  const void *src;
  long long ld;
  int fmt, rows, cols, vec;
  FastDiv groups;               // by the groups of 8 of a row
  uint16_t *plane[kMaxPlanes];  // rows of ldd elements (a multiple of 8), zeros after each row's end
  int planes, ldd;
  unsigned first;
};
struct PrepBatch {
  Prep item[kMaxPrep];
  int count;
};
__device__ __forceinline__ int prep_of(const PrepBatch &b, unsigned block) {
  int i = 0;
  while (i + 1 < b.count && block >= b.item[i + 1].first) ++i;
  return i;
}

// Copy 16-bit matrices.  One thread per 8 values.
__global__ __launch_bounds__(kThreads) void k_repack(PrepBatch b) {
  const Prep &p = b.item[prep_of(b, blockIdx.x)];
  const uint32_t at = (blockIdx.x - p.first) * kThreads + threadIdx.x;
  const uint32_t r = fdiv(at, p.groups);
  if (r >= (uint32_t)p.rows) return;
  const int c = (int)(at - r * p.groups.d) * 8;
  const uint16_t *src = (const uint16_t *)p.src + r * p.ld + c;
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < p.cols) w[i >> 1] |= (uint32_t)src[i] << ((i & 1) * 16);
  *(uint4 *)(p.plane[0] + (long long)r * p.ldd + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Split fp32 (or fp16) matrices into bf16 planes.  One thread per 8 values.
__global__ __launch_bounds__(kThreads) void k_split(PrepBatch b) {
  const Prep &p = b.item[prep_of(b, blockIdx.x)];
  const uint32_t at = (blockIdx.x - p.first) * kThreads + threadIdx.x;
  const uint32_t r = fdiv(at, p.groups);
  if (r >= (uint32_t)p.rows) return;
  const int c = (int)(at - r * p.groups.d) * 8;
  float v[8];
  load8(p.src, p.fmt, r * p.ld + c, p.cols - c, p.vec, v);
  store_planes(p.plane, p.planes, (long long)r * p.ldd + c, v);
}

// dz = dy * slope (no slope: dz = dy), rounded to the products' format or in
// bf16 planes, and the sums of dz over this workgroup's rows.  A workgroup
// takes `rows` rows and TX * 8 columns.
struct DzArgs {
  const void *dy, *slope;
  uint16_t *plane[kMaxPlanes];
  int planes;     // 0: only the sums; 1: dz in dz_fmt (16 bits)
  float *colsum;  // [row block][N], or null
  long long lddy, ld_slope, ld_dz;
  int dy_fmt, slope_fmt, dz_fmt;
  float slope_down;  // 1 / the scale that the slope is kept under
  int M, N, rows, vec;
};
template <int TX, bool SLOPE>
__global__ __launch_bounds__(kThreads) void k_dz(DzArgs a) {
  constexpr int TY = kThreads / TX, kAtOnce = 4;
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int n = (blockIdx.y * TX + tx) * 8;
  // unsigned: the last workgroup's rows may end, and a thread's last step go, past 2^31
  const uint32_t rows = (uint32_t)a.rows, m0 = blockIdx.x * rows;
  const uint32_t m1 = m0 + rows < (uint32_t)a.M ? m0 + rows : (uint32_t)a.M;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n < a.N) {
    for (uint32_t m = m0 + ty; m < m1; m += TY * kAtOnce) {
      float v[kAtOnce][8], s[kAtOnce][8];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const uint32_t r = m + u * TY < m1 ? m + u * TY : m;
        load8(a.dy, a.dy_fmt, r * a.lddy + n, a.N - n, a.vec, v[u]);
        if constexpr (SLOPE) load_w<8>(a.slope, a.slope_fmt, r * a.ld_slope + n, s[u]);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (m + u * TY >= m1) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // past N the slope's rows hold nothing that was written
          if constexpr (SLOPE) v[u][j] = n + j < a.N ? v[u][j] * (s[u][j] * a.slope_down) : 0.f;
          sum[j] += v[u][j];
        }
        const long long at = (m + u * TY) * a.ld_dz + n;
        if (a.planes == 1)
          store_w<8>(a.plane[0], a.dz_fmt, at, v[u]);
        else if (a.planes)
          store_planes(a.plane, a.planes, at, v[u]);
      }
    }
  }
  if (!a.colsum) return;
  __shared__ float red[TY][TX * 8 + 1];
#pragma unroll
  for (int j = 0; j < 8; ++j) red[ty][tx * 8 + j] = sum[j];
  __syncthreads();
  for (int c = threadIdx.x; c < TX * 8; c += kThreads) {
    if (blockIdx.y * TX * 8 + c >= a.N) break;
    float t = 0.f;
    for (int i = 0; i < TY; ++i) t += red[i][c];
    a.colsum[(long long)blockIdx.x * a.N + blockIdx.y * TX * 8 + c] = t;
  }
}

// dbias[n] = sum of the row blocks' sums; 8 columns to a workgroup.
__global__ __launch_bounds__(kThreads) void k_colsum(const float *__restrict__ part, int blocks,
                                                     int N, void *__restrict__ out, int fmt) {
  const int n = blockIdx.x * 8 + (threadIdx.x & 7), ty = threadIdx.x >> 3;
  float s = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int b = ty; b < blocks; b += 32) s += part[(long long)b * N + n];
  }
  __shared__ float red[32][8];
  red[ty][threadIdx.x & 7] = s;
  __syncthreads();
  if (ty == 0 && n < N) {
    float t = 0.f;
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x];
    store1(out, fmt, n, t);
  }
}

// Sums of squares of a batch's matrices (fp64: the square of any fp32 value is
// in range), gridDim.x partial sums per matrix.
__global__ __launch_bounds__(kThreads) void k_squares(const void *__restrict__ g, int fmt,
                                                      long long ld, long long batch_g, int m, int n,
                                                      int vec, FastDiv groups,
                                                      double *__restrict__ part) {
  const uint32_t total = (uint32_t)m * groups.d;
  double s = 0.0;
#pragma unroll 4
  for (uint32_t at = blockIdx.x * kThreads + threadIdx.x; at < total; at += gridDim.x * kThreads) {
    const uint32_t r = fdiv(at, groups);
    const int c = (int)(at - r * groups.d) * 8;
    float v[8];
    load8(g, fmt, blockIdx.y * batch_g + r * ld + c, n - c, vec, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (double)v[i] * (double)v[i];
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// x = g / (|g| + eps) 2^shift in fp16 planes (lo null: one), or in format
// `fmt_out` with no planes; rows of ldx elements, zeros after each row's end.
struct NormaliseArgs {
  const void *g;
  const double *part;
  void *x, *x_lo;
  long long ld, batch_g, ldx, batch_x;
  int fmt, fmt_out, parts, m, n, cols_out, vec, vec_out, shift;
  float eps;
  FastDiv groups;
};
__global__ __launch_bounds__(kThreads) void k_normalise(NormaliseArgs a) {
  const uint32_t at = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t r = fdiv(at, a.groups);
  const int c = (int)(at - r * a.groups.d) * 8;
  const bool mine = r < (uint32_t)a.m;
  float v[8], lo[8];
  if (mine) load8(a.g, a.fmt, blockIdx.y * a.batch_g + r * a.ld + c, a.n - c, a.vec, v);
  double s = 0.0;
  for (int i = threadIdx.x; i < a.parts; i += kThreads) s += a.part[blockIdx.y * a.parts + i];
  s = block_sum(s);
  if (!mine) return;
  // 1 / (|g| + eps) as a power of two and a value in [1/2, 1), in this order: no
  // fp32 input leaves fp32's range on the way up or loses bits on the way down,
  // also where its own values are subnormal
  int e;
  const float f = (float)frexp(1.0 / (sqrt(s) + (double)a.eps), &e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a zero matrix with eps = 0 stays zero rather than 0 * inf
    const float t = v[i] == 0.f ? 0.f : ldexpf(v[i], e + a.shift) * f;
    v[i] = t;
    lo[i] = t - f16_to_f(f_to_f16(t));
  }
  const long long to = blockIdx.y * a.batch_x + r * a.ldx + c;
  store8(a.x, a.fmt_out, to, a.cols_out - c, a.vec_out, v);
  if (a.x_lo) store8(a.x_lo, kF16, to, a.cols_out - c, a.vec_out, lo);
}

// ------------------------------------------------------------------- set-up

bool good_fmt(int f) { return f == kF32 || f == kF16 || f == kBf16; }
bool good_len(long long n) { return n >= 0 && n <= 0x7fffffffLL - 256; }
// Passes index a matrix by 8 values in 31 bits.
bool good_size(long long rows, long long cols) {
  return rows * ((cols + 7) / 8) <= 0x7fffffffLL - kThreads;
}
// A matrix of this many rows and columns: its pointer and row distance.
bool good_mat(const void *p, long long ld, long long rows, long long cols, int fmt) {
  if (rows == 0 || cols == 0) return true;
  if (!good_size(rows, cols)) return false;
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
  PrepBatch repack = {}, split = {};  // laid out by flush(), before the next product
  pdr_dense_product *out = nullptr;   // if asked for: the first `most` products
  int most = 0, products = 0;

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
  void note(const pdr_dense_product &p) {
    if (products < most) out[products] = p;
    ++products;
  }
  void add(PrepBatch &b, const Prep &p) {
    if (b.count == kMaxPrep) flush();
    b.item[b.count++] = p;
  }
  void flush();
};

// A matrix as the products read it: 16-bit planes whose sum it is.
struct Planes {
  const uint16_t *p[kMaxPlanes] = {nullptr, nullptr, nullptr};
  int count = 1;
  long long ld = 0;
};

// The planes of a matrix of this format, and their format.
int planes_of(int fmt) { return fmt == kF32 ? 3 : 1; }
int product_fmt(int fmt) { return fmt == kF16 ? kF16 : kBf16; }

unsigned blocks_for(long long threads) { return (unsigned)((threads + kThreads - 1) / kThreads); }
unsigned parts_for(long long threads) {
  const long long b = (threads + kThreads - 1) / kThreads;
  return (unsigned)(b < 1 ? 1 : b < kParts ? b : kParts);
}

void Walk::flush() {
  if (go()) {
    unsigned blocks = 0;
    for (int i = 0; i < repack.count; ++i) {
      Prep &p = repack.item[i];
      p.first = blocks;
      blocks += blocks_for((long long)p.rows * p.groups.d);
    }
    if (blocks) hipLaunchKernelGGL(k_repack, dim3(blocks), dim3(kThreads), 0, st, repack);
    blocks = 0;
    for (int i = 0; i < split.count; ++i) {
      Prep &p = split.item[i];
      p.first = blocks;
      blocks += blocks_for((long long)p.rows * p.groups.d);
    }
    if (blocks) hipLaunchKernelGGL(k_split, dim3(blocks), dim3(kThreads), 0, st, split);
    done(hipGetLastError());
  }
  repack.count = split.count = 0;
}

// Planes of this many rows and columns in the workspace.
Planes take_planes(Walk &w, int count, long long rows, long long cols) {
  Planes r;
  r.count = count;
  r.ld = round8(cols);
  for (int k = 0; k < count; ++k) r.p[k] = (const uint16_t *)w.take((size_t)(rows * r.ld) * 2);
  return r;
}

// A matrix of format fmt in so many planes: itself, where it can be read in
// place, or laid out in the workspace.
Planes lay_out(Walk &w, const void *p, int fmt, int planes, long long ld, long long rows,
               long long cols, bool summed_along_row) {
  Planes r;
  if (rows == 0 || cols == 0) {
    r.ld = round8(cols > 0 ? cols : 1);
    return r;
  }
  if (planes == 1 && aligned16(p) && (ld & 7) == 0 && (!summed_along_row || (cols & 7) == 0)) {
    r.p[0] = (const uint16_t *)p;
    r.ld = ld;
    return r;
  }
  r = take_planes(w, planes, rows, cols);
  Prep m = {};
  m.src = p;
  m.ld = ld;
  m.fmt = fmt;
  m.rows = (int)rows;
  m.cols = (int)cols;
  m.vec = aligned16(p) && (ld & 7) == 0;
  m.groups = make_fastdiv((uint32_t)(r.ld / 8));
  m.ldd = (int)r.ld;
  m.planes = r.count;
  for (int k = 0; k < r.count; ++k) m.plane[k] = (uint16_t *)r.p[k];
  w.add(planes > 1 ? w.split : w.repack, m);
  return r;
}

// Add the product of two matrices, offset by so many elements, to the
// segments: of the planes' products those that matter (with three planes, whose
// values are 2^-8 of each other's or less: six, down to 2^-16; the others are
// at most 2^-23 of the product of two values), smallest first.
void add_product(GemmArgs &g, const Planes &a, long long off_a, const Planes &b, long long off_b) {
  const int most = a.count > b.count ? a.count : b.count;
  for (int order = most - 1; order >= 0; --order)
    for (int i = 0; i <= order; ++i) {
      const int j = order - i;
      if (i >= a.count || j >= b.count) continue;
      g.a[g.segs] = a.p[i] ? a.p[i] + off_a : nullptr;
      g.b[g.segs] = b.p[j] ? b.p[j] + off_b : nullptr;
      ++g.segs;
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
  w.flush();
  if (w.out) {
    const TilePlan t = plan_tiles(g, kind);
    w.note({g.M, g.N, (long long)g.K * g.segs, product_fmt(fmt), a_mc, b_mc, kind, g.batches, t.tile,
            t.groups, t.splits, t.lower});
  }
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

// A bf16 projection's slopes are kept in fp16, under a scale: they lie in
// (-0.14, 1.14), and those of units that are nearly off (silu at -20: -4e-8)
// keep fp16's 11 bits down to 2^-29.
int slope_fmt(int fmt) { return fmt == kBf16 ? kF16 : kF32; }
float slope_scale(int fmt) { return fmt == kBf16 ? 32768.f : 1.f; }

// Few rows: the kernel for them, which lays nothing out.
void multiply_few(Walk &w, const void *x, long long ldx, const void *wt, long long ldw,
                  long long up_at, long long M, long long N, long long K, const Epi &epi, int fmt,
                  bool gated) {
  if (w.out) w.note({M, N, K, fmt, 0, 0, gated ? kEpiGated : kEpiLinear, 1, 0, 1, 1, 0});
  if (!w.go()) return;
  SkinnyArgs a = {x, wt, ldx, ldw, up_at, (int)M, (int)N, (int)K, epi};
  w.done(launch_skinny(a, fmt, gated, w.st));
}

void linear_forward(Walk &w, const pdr_linear &p) {
  Epi e = {};
  e.store_n = (int)p.N;
  set_out(e, p.y, p.out_fmt, p.ldy);
  e.bias = p.bias;
  e.bias_fmt = p.fmt;
  e.res = p.res;
  e.ldr = (int)p.ldr;
  e.vec = e.vec && (!p.bias || aligned16(p.bias)) && (!p.res || (aligned16(p.res) && (p.ldr & 7) == 0));
  e.act = p.activation;
  e.slope = p.activation != PDR_ACT_NONE ? p.slope : nullptr;
  e.slope_fmt = slope_fmt(p.fmt);
  e.slope_scale = slope_scale(p.fmt);
  e.ld_slope = (int)round8(p.N);
  if (p.M <= kSkinnyRows)
    return multiply_few(w, p.x, p.ldx, p.w, p.ldw, 0, p.M, p.N, p.K, e, p.fmt, false);
  const Planes x = lay_out(w, p.x, p.fmt, planes_of(p.fmt), p.ldx, p.M, p.K, true);
  const Planes wt = lay_out(w, p.w, p.fmt, planes_of(p.fmt), p.ldw, p.N, p.K, true);
  GemmArgs g = product(p.M, p.N, round8(p.K));
  add_product(g, x, 0, wt, 0);
  g.epi = e;
  multiply(w, g, p.fmt, false, false, kEpiLinear);
}

void linear_backward(Walk &w, const pdr_linear &p) {
  const bool act = p.activation != PDR_ACT_NONE;
  const bool products = p.dx || p.dw;
  // fp32 gradients of an fp16 projection may be anywhere in fp32's range (a mean
  // loss gives 1 / numel), which fp16 does not hold: dz has two bf16 planes, 16
  // bits, and so have the other operands, which they hold exactly.  Three
  // products instead of one; a scale to one dz in fp16 would cost small rows
  // their bits where another is large.
  const int planes = p.fmt == kF16 && p.out_fmt == kF32 ? 2 : planes_of(p.fmt);
  const int in = planes > 1 ? kBf16 : p.fmt;
  // dz as the products read it, unless it is dy itself
  Planes z;
  const bool write = products && p.M && p.N && (act || p.out_fmt != p.fmt || planes > 1);
  if (write) z = take_planes(w, planes, p.M, p.N);
  // threads across a row's 8s, and rows to a workgroup for about kParts of them
  const int tx = p.N <= 8 ? 1 : p.N <= 64 ? 8 : 32, ty = kThreads / tx;
  const long long col_blocks = (p.N + tx * 8 - 1) / (tx * 8);
  long long rows = (p.M * col_blocks + kParts - 1) / kParts;
  rows = rows < ty ? ty : (rows + ty - 1) / ty * ty;
  const long long row_blocks = p.M ? (p.M + rows - 1) / rows : 0;
  float *part = p.dbias ? (float *)w.take((size_t)(row_blocks * p.N) * sizeof(float)) : nullptr;
  if ((write || p.dbias) && p.N && w.go()) {
    DzArgs a = {};
    a.dy = p.dy;
    a.slope = act ? p.slope : nullptr;
    a.planes = write ? z.count : 0;
    for (int k = 0; k < a.planes; ++k) a.plane[k] = (uint16_t *)z.p[k];
    a.colsum = part;
    a.lddy = p.lddy;
    a.ld_slope = round8(p.N);
    a.ld_dz = z.ld;
    a.dy_fmt = p.out_fmt;
    a.slope_fmt = slope_fmt(p.fmt);
    a.slope_down = 1.f / slope_scale(p.fmt);
    a.dz_fmt = in;
    a.M = (int)p.M;
    a.N = (int)p.N;
    a.rows = (int)rows;
    a.vec = aligned16(p.dy) && (p.lddy & 7) == 0;
    const dim3 grid((unsigned)row_blocks, (unsigned)col_blocks);
    auto run = [&](auto with_slope, auto without) {
      if (a.slope)
        hipLaunchKernelGGL(with_slope, grid, dim3(kThreads), 0, w.st, a);
      else
        hipLaunchKernelGGL(without, grid, dim3(kThreads), 0, w.st, a);
    };
    if (row_blocks) {
      if (tx == 1)
        run(k_dz<1, true>, k_dz<1, false>);
      else if (tx == 8)
        run(k_dz<8, true>, k_dz<8, false>);
      else
        run(k_dz<32, true>, k_dz<32, false>);
    }
    if (p.dbias)
      hipLaunchKernelGGL(k_colsum, dim3((unsigned)((p.N + 7) / 8)), dim3(kThreads), 0, w.st, part,
                         (int)row_blocks, (int)p.N, p.dbias, p.fmt);
    w.done(hipGetLastError());
  }
  if (!products) return;
  if (!write) z = lay_out(w, p.dy, p.fmt, planes, p.lddy, p.M, p.N, p.dx != nullptr);
  const Planes wt = p.dx ? lay_out(w, p.w, p.fmt, planes, p.ldw, p.N, p.K, false) : Planes();
  const Planes x = p.dw ? lay_out(w, p.x, p.fmt, planes, p.ldx, p.M, p.K, false) : Planes();
  if (p.dx) {
    GemmArgs g = product(p.M, p.K, round8(p.N));
    g.kb = (int)p.N;
    add_product(g, z, 0, wt, 0);
    set_out(g.epi, p.dx, p.fmt, p.lddx);
    multiply(w, g, in, false, true, kEpiLinear);
  }
  if (p.dw) {
    GemmArgs g = product(p.N, p.K, p.M);
    add_product(g, z, 0, x, 0);
    set_out(g.epi, p.dw, p.fmt, p.lddw);
    multiply(w, g, in, true, true, kEpiLinear);
  }
}

// -------------------------------------------------------------- gated block

int check_gated(const pdr_gated_mlp *p, bool backward) {
  if (!p || !good_fmt(p->fmt)) return PDR_ERR_INVALID_ARG;
  if (p->activation < PDR_ACT_NONE || p->activation > PDR_ACT_GELU) return PDR_ERR_INVALID_ARG;
  if (!good_len(p->M) || !good_len(p->D) || !good_len(p->F) || !good_len(p->O)) return PDR_ERR_INVALID_ARG;
  if (2 * round8(p->F) > kMaxLd) return PDR_ERR_INVALID_ARG;
  // h and [dg | du] of fp32 are laid out anew for the products
  if (p->fmt == kF32 && !good_size(p->M, (backward ? 2 : 1) * round8(p->F))) return PDR_ERR_INVALID_ARG;
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
  Epi in = {}, out = {};
  in.store_n = (int)Fp;
  set_out(in, p.h, p.fmt, Fp);
  in.act = p.activation;
  in.gu = (float *)p.gu;
  in.ld_gu = (int)Fp;
  out.store_n = (int)p.O;
  set_out(out, p.y, p.fmt, p.ldy);
  out.res = p.res;
  out.ldr = (int)p.ldr;
  out.vec = out.vec && (!p.res || (aligned16(p.res) && (p.ldr & 7) == 0));
  if (p.M <= kSkinnyRows) {
    multiply_few(w, p.x, p.ldx, p.w_in, p.ld_in, p.F * p.ld_in, p.M, p.F, p.D, in, p.fmt, true);
    return multiply_few(w, p.h, Fp, p.w_out, p.ld_out, 0, p.M, p.O, p.F, out, p.fmt, false);
  }
  const Planes wo = lay_out(w, p.w_out, p.fmt, planes_of(p.fmt), p.ld_out, p.O, p.F, true);
  {
    const size_t keep = w.at;
    const Planes x = lay_out(w, p.x, p.fmt, planes_of(p.fmt), p.ldx, p.M, p.D, true);
    const Planes wi = lay_out(w, p.w_in, p.fmt, planes_of(p.fmt), p.ld_in, 2 * p.F, p.D, true);
    GemmArgs g = product(p.M, p.F, round8(p.D));
    add_product(g, x, 0, wi, 0);
    g.up_at = p.F * wi.ld;
    g.epi = in;
    multiply(w, g, p.fmt, false, false, kEpiGated);
    w.at = keep;
  }
  const Planes h = lay_out(w, p.h, p.fmt, planes_of(p.fmt), Fp, p.M, Fp, true);
  GemmArgs g = product(p.M, p.O, Fp);
  add_product(g, h, 0, wo, 0);
  g.epi = out;
  multiply(w, g, p.fmt, false, false, kEpiLinear);
}

void gated_backward(Walk &w, const pdr_gated_mlp &p) {
  const long long Fp = round8(p.F);
  const bool through = p.dx || p.dw_in;
  const Planes dy = lay_out(w, p.dy, p.fmt, planes_of(p.fmt), p.lddy, p.M, p.O, through);
  const Planes x = p.dw_in ? lay_out(w, p.x, p.fmt, planes_of(p.fmt), p.ldx, p.M, p.D, false) : Planes();
  const Planes wi = p.dx ? lay_out(w, p.w_in, p.fmt, planes_of(p.fmt), p.ld_in, 2 * p.F, p.D, false) : Planes();
  const Planes wo = through ? lay_out(w, p.w_out, p.fmt, planes_of(p.fmt), p.ld_out, p.O, p.F, false) : Planes();
  if (p.dw_out) {
    const size_t keep = w.at;
    const Planes h = lay_out(w, p.h, p.fmt, planes_of(p.fmt), Fp, p.M, Fp, false);
    GemmArgs g = product(p.O, p.F, p.M);
    add_product(g, dy, 0, h, 0);
    set_out(g.epi, p.dw_out, p.fmt, p.ldd_out);
    multiply(w, g, p.fmt, true, true, kEpiLinear);
    w.at = keep;
  }
  if (!through) return;
  void *dgu = w.take((size_t)(p.M * 2 * Fp) * fmt_bytes(p.fmt));
  {
    GemmArgs g = product(p.M, p.F, round8(p.O));
    g.kb = (int)p.O;
    add_product(g, dy, 0, wo, 0);
    set_out(g.epi, dgu, p.fmt, 2 * Fp);
    g.epi.store_n = (int)Fp;
    g.epi.up_at = (int)Fp;
    g.epi.act = p.activation;
    g.epi.gu = (float *)p.gu;
    g.epi.ld_gu = (int)Fp;
    multiply(w, g, p.fmt, false, true, kEpiGatedGrad);
  }
  const Planes d = lay_out(w, dgu, p.fmt, planes_of(p.fmt), 2 * Fp, p.M, 2 * Fp, true);
  if (p.dx) {
    GemmArgs g = product(p.M, p.D, Fp);
    g.kb = (int)p.F;
    add_product(g, d, 0, wi, 0);
    add_product(g, d, Fp, wi, p.F * wi.ld);
    set_out(g.epi, p.dx, p.fmt, p.lddx);
    multiply(w, g, p.fmt, false, true, kEpiLinear);
  }
  if (p.dw_in) {
    GemmArgs g = product(p.F, p.D, p.M);
    add_product(g, d, 0, x, 0);
    g.batches = 2;  // the gate rows, then the up rows
    g.batch_a = Fp;
    set_out(g.epi, p.dw_in, p.fmt, p.ldd_in);
    g.epi.batch_y = p.F * p.ldd_in;
    g.epi.vec = g.epi.vec && (g.epi.batch_y * fmt_bytes(p.fmt)) % 16 == 0;
    multiply(w, g, p.fmt, true, true, kEpiLinear);
  }
}

// ------------------------------------------------------------ orthogonalize

int g_fmt(const pdr_orthogonalize_args &p) { return p.g_f32 ? kF32 : p.fmt; }

// Powers of two that keep the iterates' entries well inside fp16's normal
// range: X's entries are at most a singular value and about 1/sqrt(n), those
// of A and B = b A + c A^2 at most theirs and about 1/n.
constexpr int kShiftX = 12, kShiftA = 10;
constexpr double kMostX = 15.0, kMostA = 60.0;  // times the shifts: below 65504, with room for roundings

// The largest of |f| over [0, most], at its ends or where its slope is zero.
template <class F>
double largest(F f, double most, double at0, double at1) {
  double r = fabs(f(most));
  for (double t : {at0, at1})
    if (t > 0.0 && t < most) r = fmax(r, fabs(f(t)));
  return r;
}
// Whether the iterates stay in range from singular values in [0, 1] on.
bool stays_in_range(const pdr_orthogonalize_args &p) {
  const double a = p.a, b = p.b, c = p.c;
  double top = 1.0;
  for (int i = 0; i < p.steps; ++i) {
    const double t = top * top;
    auto poly = [&](double x) { return b * x + c * x * x; };
    if (t > kMostA || !(largest(poly, t, -b / (2.0 * c), 0.0) <= kMostA)) return false;
    if (i + 1 == p.steps) break;  // the result has its own format
    auto next = [&](double x) { return sqrt(x) * (a + x * (b + c * x)); };  // of the square
    const double root = sqrt(9.0 * b * b - 20.0 * a * c);  // NaN: no such place
    const double at0 = c != 0.0 ? (-3.0 * b + root) / (10.0 * c) : -a / (3.0 * b);
    const double at1 = c != 0.0 ? (-3.0 * b - root) / (10.0 * c) : 0.0;
    top = largest(next, t, at0, at1);
    if (!(top <= kMostX)) return false;
  }
  return true;
}

int check_ortho(const pdr_orthogonalize_args *p) {
  if (!p || !good_fmt(p->fmt) || p->steps < 0) return PDR_ERR_INVALID_ARG;
  if (!good_len(p->batch) || p->batch > 65535 || !good_len(p->m) || !good_len(p->n)) return PDR_ERR_INVALID_ARG;
  if (round8(p->m) > kMaxLd || round8(p->n) > kMaxLd) return PDR_ERR_INVALID_ARG;
  const long long rows = p->batch ? p->m : 0;
  if (!good_mat(p->g, p->ldg, rows, p->n, g_fmt(*p)) || !good_mat(p->x, p->ldx, rows, p->n, p->fmt))
    return PDR_ERR_INVALID_ARG;
  if (!isfinite(p->a) || !isfinite(p->b) || !isfinite(p->c) || !isfinite(p->eps) || p->eps < 0.f)
    return PDR_ERR_INVALID_ARG;
  if (!stays_in_range(*p)) return PDR_ERR_INVALID_ARG;
  return PDR_OK;
}

void orthogonalize(Walk &w, const pdr_orthogonalize_args &p) {
  const bool two = p.fmt != kBf16, tall = p.m > p.n;
  const long long s = tall ? p.n : p.m, sp = round8(s), np = round8(p.n);
  const size_t x_bytes = (size_t)(p.batch * p.m * np) * 2, a_bytes = (size_t)(p.batch * s * sp) * 2;
  const int parts = (int)parts_for(p.m * ((p.n + 7) / 8) / 4);
  double *part = (double *)w.take((size_t)p.batch * kParts * sizeof(double));
  if (p.batch == 0 || p.m == 0 || p.n == 0) return;
  const int vec_g = aligned16(p.g) && (p.ldg & 7) == 0 && (p.batch_g & 7) == 0;
  const int vec_x = aligned16(p.x) && (p.ldx & 7) == 0 && (p.batch_x & 7) == 0;
  auto normalise = [&](void *x, void *lo, int shift, int fmt, long long ldx, long long batch_x,
                       long long cols, int vec) {
    if (!w.go()) return;
    hipLaunchKernelGGL(k_squares, dim3((unsigned)parts, (unsigned)p.batch), dim3(kThreads), 0, w.st,
                       p.g, g_fmt(p), p.ldg, p.batch_g, (int)p.m, (int)p.n, vec_g,
                       make_fastdiv((uint32_t)((p.n + 7) / 8)), part);
    NormaliseArgs a = {};
    a.g = p.g;
    a.part = part;
    a.x = x;
    a.x_lo = lo;
    a.ld = p.ldg;
    a.batch_g = p.batch_g;
    a.ldx = ldx;
    a.batch_x = batch_x;
    a.fmt = g_fmt(p);
    a.fmt_out = fmt;
    a.parts = parts;
    a.m = (int)p.m;
    a.n = (int)p.n;
    a.cols_out = (int)cols;
    a.vec = vec_g;
    a.vec_out = vec;
    a.shift = shift;
    a.eps = p.eps;
    a.groups = make_fastdiv((uint32_t)((cols + 7) / 8));
    hipLaunchKernelGGL(k_normalise, dim3(blocks_for(p.m * ((cols + 7) / 8)), (unsigned)p.batch),
                       dim3(kThreads), 0, w.st, a);
    w.done(hipGetLastError());
  };
  if (p.steps == 0) {
    normalise(p.x, nullptr, 0, p.fmt, p.ldx, p.batch_x, p.n, vec_x);
    return;
  }
  auto planes = [&](size_t bytes, long long ld) {
    Planes q;
    q.count = two ? 2 : 1;
    for (int k = 0; k < q.count; ++k) q.p[k] = (const uint16_t *)w.take(bytes);
    q.ld = ld;
    return q;
  };
  Planes x[2] = {planes(x_bytes, np), p.steps > 1 ? planes(x_bytes, np) : Planes()};
  const Planes a = planes(a_bytes, sp), b = planes(a_bytes, sp);
  normalise((void *)x[0].p[0], (void *)x[0].p[1], kShiftX, kF16, np, p.m * np, np, 1);

  auto to = [](Epi &e, const Planes &y, long long batch) {
    set_out(e, (void *)y.p[0], kF16, y.ld);
    e.y_lo = (void *)y.p[1];
    e.batch_y = batch;
  };
  auto plus = [](Epi &e, float beta, const Planes &c, long long batch) {
    e.beta = beta;
    e.c = c.p[0];
    e.c_lo = c.p[1];
    e.ldc = (int)c.ld;
    e.batch_c = batch;
  };
  for (int i = 0; i < p.steps; ++i) {
    const Planes &xi = x[i & 1], &xo = x[(i + 1) & 1];
    {  // A = X X^T or X^T X
      GemmArgs g = product(s, s, tall ? p.m : np);
      add_product(g, xi, 0, xi, 0);
      g.symmetric = 1;
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
      g.symmetric = 1;
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
int products_of(const Desc &d, Op op, pdr_dense_product *out, int most) {
  if (most < 0 || (most > 0 && !out)) return PDR_ERR_INVALID_ARG;
  pdr_dense_product none;
  Walk w;
  w.out = out ? out : &none;
  w.most = most;
  op(w, d);
  return w.products;
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

int pdr_linear_products(const pdr_linear *p, int backward, pdr_dense_product *out, int most) {
  const int rc = check_linear(p, backward != 0);
  return rc != PDR_OK ? rc : products_of(*p, backward ? linear_backward : linear_forward, out, most);
}
int pdr_gated_mlp_products(const pdr_gated_mlp *p, int backward, pdr_dense_product *out, int most) {
  const int rc = check_gated(p, backward != 0);
  return rc != PDR_OK ? rc : products_of(*p, backward ? gated_backward : gated_forward, out, most);
}
int pdr_orthogonalize_products(const pdr_orthogonalize_args *p, pdr_dense_product *out, int most) {
  const int rc = check_ortho(p);
  return rc != PDR_OK ? rc : products_of(*p, orthogonalize, out, most);
}

}  // extern "C"

// How a product is cut into workgroups: 256x256 tiles, one workgroup on a
// compute unit; 128x128 or 64x64 tiles, two workgroups, or one whose groups of
// waves share the contraction; and the contraction in one part or in several,
// which a second kernel joins.  The choice is the least of an estimate in
// microseconds whose constants are fits to measured products (bf16, M x N x K,
// this card): a step is 64 contraction values of every workgroup in flight.
//   64:  512x512x512 (64 workgroups) 6.2, 1024x1024x1024 (256) 8.3,
//        2048x1024x1024 (512) 10.9; in 128 tiles: 9.0, 12.7, 12.8
//   64, four groups: 512x512x4096 (64) 14.3, 1024x1024x4096 (256) 18.7; with
//        one group 19.0, 20.7
//   128: 4096x2048x2048 (512) 34.4, 8192x1024x2816 (512) 44.3; in 64 tiles:
//        60.1, 81.1
//   128, two groups: 2048x2048x2048 (256) 21.9, 2816x1024x8192 (176) 51.8,
//        2048x2048x11264 (256) 80.1 (91.0 with both operands mc); with one
//        group 22.9, 63.4, 92.5 (108.7)
//   256: 8192x1024x512 (128) 25.8, 16384x1024x1024 (256) 38.0,
//        16384x2048x11264 (512, two rounds) 582; in 128 tiles: 15.3, 37.3, 687
//   16384x2048x2048 with gelu, its slope and a residual: 194 in 256 tiles, 166
//        in 128 tiles; with nothing: 132 (114 at its best), 150 (123)
//   parts: 512x512x4096 in 64 tiles: one 19.0, four 13.1
//   a symmetric result's lower tiles alone: 2048x2048x11264 (mc, mc), three
//        parts, 88, all tiles 133; 2048x2048x2048 32.1, all tiles 31
namespace pdr {
namespace dense {

namespace {

struct TileCost {
  int tile, groups;
  double slots, fixed;     // workgroups in a round, microseconds of one beside its steps
  double full, half, few;  // microseconds of a step with over 1/2 of the slots taken, over 1/4, fewer
};
constexpr TileCost kCosts[] = {
    {64, 1, 512, 3.0, 0.43, 0.28, 0.25}, {64, 4, 256, 4.0, 0.20, 0.15, 0.13},
    {128, 1, 512, 5.0, 0.90, 0.57, 0.45}, {128, 2, 256, 7.0, 0.48, 0.42, 0.36},
    {256, 1, 256, 9.0, 1.50, 1.30, 1.20},
};

double tiles_us(const TileCost &c, double workgroups, double steps, double slow) {
  const double rounds = floor(workgroups / c.slots), rest = workgroups - rounds * c.slots;
  const double fixed = c.fixed + slow;
  double us = rounds * (c.full * steps + fixed);
  if (rest > 0.0)
    us += (rest > c.slots / 2 ? c.full : rest > c.slots / 4 ? c.half : c.few) * steps + fixed;
  return us;
}

}  // namespace

TilePlan plan_tiles(const GemmArgs &g, EpiKind kind) {
  const int steps = (g.K + kBK - 1) / kBK * g.segs;
  const double batches = g.batches > 0 ? g.batches : 1;
  const double sums = batches * (double)g.M * (double)g.N;
  const int most = kind == kEpiGated ? 1 : steps / 2 > 32 ? 32 : steps / 2 > 1 ? steps / 2 : 1;
  TilePlan best = {};
  double least = 0.0;
  for (const TileCost &c : kCosts) {
    const int bm = c.tile;
    const int bn = kind == kEpiGated ? bm / 2 : bm;
    TilePlan p;
    p.tile = bm;
    p.groups = c.groups;
    p.tiles_m = (g.M + bm - 1) / bm;
    p.tiles_n = (g.epi.store_n + bn - 1) / bn;
    // What an epilogue adds to a round: rows that do not begin on 16 bytes are
    // stored value by value; activations and a residual take time that only
    // two workgroups on a compute unit hide behind each other's products.
    double slow = 0.0;
    if (kind == kEpiLinear) {
      if (!(g.epi.vec && (g.epi.store_n & 7) == 0)) slow += bm == 256 ? 40.0 : bm == 128 ? 12.0 : 4.0;
      const int more = (g.epi.act != PDR_ACT_NONE) + 2 * (g.epi.slope != nullptr) + 2 * (g.epi.res != nullptr);
      slow += more * (bm == 256 ? 5.0 : bm == 128 ? 1.0 : 0.5);
    }
    for (int lower = 0; lower <= (g.symmetric ? 1 : 0); ++lower) {
      p.lower = lower != 0;
      p.tiles = lower ? p.tiles_m * (p.tiles_m + 1) / 2 : p.tiles_m * p.tiles_n;
      if ((long long)p.tiles * 256 * p.groups >= 1LL << 32) continue;  // more threads than a launch holds
      // storing a tile on both sides
      const double mirror = lower ? bm == 256 ? 14.0 : bm == 128 ? 4.0 : 2.0 : 0.0;
      for (p.splits = 1; p.splits <= most; ++p.splits) {
        if (p.splits > 1 && (long long)g.M * g.epi.store_n >= 1LL << 31) break;  // nor would the second kernel's
        double us = tiles_us(c, batches * p.tiles * p.splits,
                             (double)((steps + p.splits - 1) / p.splits),
                             mirror + (p.splits > 1 ? 0.0 : slow));
        // the parts are written and read once, at 4.6 TB/s
        if (p.splits > 1) us += 5.0 + 8.0 * sums * p.splits / 4.6e6;
        if (least == 0.0 || us < least) {
          least = us;
          best = p;
        }
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
