// norm.hip -- layer norm and dropout: passes that are bound by memory, so
// each value is read once and written once.
#include "norm.hpp"

namespace pdr {
namespace norm {

namespace {

using dense::fmt_bytes;
using dense::kBf16;
using dense::kF16;
using dense::kF32;

constexpr int kThreads = 256;

// ------------------------------------------------------------------ layer norm
//
// A row is held in the registers of LANES lanes, CH groups of 8 values each, so
// that mean and variance are two sums over what is there (the second of centred
// values: no cancellation) and nothing is read twice.  With 16-byte accesses a
// group is 8 neighbouring columns; otherwise its values are LANES columns apart,
// so that a wave's accesses still follow one another.
template <int LANES, int CH, bool VEC>
__device__ __forceinline__ int column(int j, int e, int l) {
  return VEC ? (j * LANES + l) * 8 + e : (j * 8 + e) * LANES + l;
}

template <int FMT, int LANES, int CH, bool VEC>
struct Row {
  float v[CH * 8];
  // zeros past the end
  __device__ __forceinline__ void load(const void *p, long long at, int cols, int l) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if constexpr (VEC) {
        if (column<LANES, CH, VEC>(j, 0, l) < cols) {
          dense::load_w<8>(p, FMT, at + column<LANES, CH, VEC>(j, 0, l), v + j * 8);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j * 8 + e] = 0.f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = column<LANES, CH, VEC>(j, e, l);
          v[j * 8 + e] = c < cols ? dense::load1(p, FMT, at + c) : 0.f;
        }
      }
    }
  }
  __device__ __forceinline__ void store(void *p, long long at, int cols, int l) const {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if constexpr (VEC) {
        if (column<LANES, CH, VEC>(j, 0, l) < cols)
          dense::store_w<8>(p, FMT, at + column<LANES, CH, VEC>(j, 0, l), v + j * 8);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = column<LANES, CH, VEC>(j, e, l);
          if (c < cols) dense::store1(p, FMT, at + c, v[j * 8 + e]);
        }
      }
    }
  }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) v[i] = x;
  }
};

// A row on its way: as it is in memory, so that the next row's loads are in flight
// while this one is worked on (16-byte accesses; others are loaded when opened).
template <int FMT, int LANES, int CH, bool VEC>
struct Ahead {
  static constexpr int kPieces = FMT == kF32 ? 2 : 1, kSize = FMT == kF32 ? 4 : 2;
  uint4 raw[VEC ? CH * kPieces : 1];
  const void *p;
  long long at;
  __device__ __forceinline__ void load(const void *p_, long long at_, int cols, int l) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = column<LANES, CH, VEC>(j, 0, l);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          raw[j * kPieces + i] = c < cols ? *(const uint4 *)((const char *)p_ + (at_ + c) * kSize + i * 16)
                                          : make_uint4(0, 0, 0, 0);
      }
    } else {
      p = p_;
      at = at_;
    }
  }
  __device__ __forceinline__ void open(Row<FMT, LANES, CH, VEC> &row, int cols, int l) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < CH * 8; ++i) {
        const uint4 w = raw[i * kSize / 16];
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
        const uint32_t word = words[i * kSize / 4 % 4];
        row.v[i] = FMT == kF32 ? __uint_as_float(word) : dense::to_f<FMT>((uint16_t)(word >> (i % 2 * 16)));
      }
    } else {
      row.load(p, at, cols, l);
    }
  }
};

// Sums of N values over the LANES lanes of a row, for all of them.  `red` has
// room for two calls: each uses the half that the one before did not.
template <int LANES, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*red)[4][3], int &turn) {
#pragma unroll
  for (int w = (LANES < 64 ? LANES : 64) / 2; w > 0; w >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] += __shfl_xor(s[n], w);
  if constexpr (LANES > 64) {
    const int wave = threadIdx.x >> 6;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) red[turn][wave][n] = s[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
      s[n] = (red[turn][0][n] + red[turn][1][n]) + (red[turn][2][n] + red[turn][3][n]);
  }
}

// From the mean square of values whose mean is `off`.
__device__ __forceinline__ float rstd_of(float square, float off, float eps) {
  const float var = fmaf(-off, off, square);
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

//
// Bound by memory: 16384 x 2048 bf16 28 us, 4.8 TB/s (a copy reaches 4.7).
template <int FMT, int LANES, int CH, bool VEC>
__global__ __launch_bounds__(kThreads) void k_norm(Norm a) {
  using R = Row<FMT, LANES, CH, VEC>;
  constexpr int kRows = kThreads / LANES;
  __shared__ float red[2][4][3];
  int turn = 0;
  const int l = threadIdx.x % LANES;
  R w, b;
  w.fill(1.f);
  b.fill(0.f);
  if (a.weight) w.load(a.weight, 0, a.cols, l);
  if (a.bias) b.load(a.bias, 0, a.cols, l);
  const long long step = (long long)gridDim.x * kRows;
  for (long long first = (long long)blockIdx.x * kRows; first < a.rows; first += step) {
    const long long r = first + threadIdx.x / LANES;
    const bool there = r < a.rows;
    R x;
    x.load(a.x, (there ? r : a.rows - 1) * a.ldx, a.cols, l);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) s[0] += x.v[i];
    row_sum<LANES, 1>(s, red, turn);
    const float mean = s[0] * a.by_cols;
    float c[2] = {0.f, 0.f};  // of centred values: their sum is what rounding left of the mean
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) {
      const bool in = column<LANES, CH, VEC>(i / 8, i % 8, l) < a.cols;
      x.v[i] = in ? x.v[i] - mean : 0.f;
      c[0] += x.v[i];
      c[1] = fmaf(x.v[i], x.v[i], c[1]);
    }
    row_sum<LANES, 2>(c, red, turn);
    const float off = c[0] * a.by_cols, rstd = rstd_of(c[1] * a.by_cols, off, a.eps);
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) x.v[i] = fmaf((x.v[i] - off) * rstd, w.v[i], b.v[i]);
    if (!there) continue;
    x.store(a.y, r * a.ldy, a.cols, l);
    if (a.stats && l == 0) *(float2 *)(a.stats + 2 * r) = make_float2(mean, rstd);
  }
}

// dx of rows, and this workgroup's sums of dy xh and dy over its rows: each lane
// meets the same columns in every row.  At most 512 workgroups, so that their sums stay
// few, which leaves 8 waves to a compute unit: the next row is fetched ahead (16384 x 2048
// bf16: 42 us, 4.8 TB/s, 54 without, and 5 to add the workgroups' sums).
template <int FMT, int LANES, int CH, bool VEC>
__global__ __launch_bounds__(kThreads) void k_norm_backward(Norm a) {
  using R = Row<FMT, LANES, CH, VEC>;
  constexpr int kRows = kThreads / LANES, kCols = LANES * CH * 8;
  __shared__ float red[2][4][3];
  __shared__ float sums[kRows][kCols];
  int turn = 0;
  const int l = threadIdx.x % LANES;
  R w, dw, db;
  w.fill(1.f);
  if (a.weight) w.load(a.weight, 0, a.cols, l);
  dw.fill(0.f);
  db.fill(0.f);
  const long long step = (long long)gridDim.x * kRows;
  // (a row of several waves is a workgroup's: all of them go round as often)
  long long r = (long long)blockIdx.x * kRows + threadIdx.x / LANES;
  Ahead<FMT, LANES, CH, VEC> next_x, next_g;
  float2 next_st = make_float2(0.f, 0.f);
  auto fetch = [&](long long row) {
    next_x.load(a.x, row * a.ldx, a.cols, l);
    next_g.load(a.dy, row * a.lddy, a.cols, l);
    next_st = *(const float2 *)(a.stats + 2 * row);
  };
  if (r < a.rows) fetch(r);
  for (; r < a.rows; r += step) {
    R x, g;
    next_x.open(x, a.cols, l);
    next_g.open(g, a.cols, l);
    const float2 st = next_st;
    if (r + step < a.rows) fetch(r + step);
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) {
      const bool in = column<LANES, CH, VEC>(i / 8, i % 8, l) < a.cols;
      x.v[i] = in ? (x.v[i] - st.x) * st.y : 0.f;
      const float gw = g.v[i] * w.v[i];
      s[0] += gw;
      s[1] = fmaf(gw, x.v[i], s[1]);
      s[2] += x.v[i];
    }
    row_sum<LANES, 3>(s, red, turn);
    // xh without what the mean's rounding left in it
    const float off = s[2] * a.by_cols, m = s[0] * a.by_cols, mx = fmaf(-off, m, s[1] * a.by_cols);
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) {
      x.v[i] -= off;
      dw.v[i] = fmaf(g.v[i], x.v[i], dw.v[i]);
      db.v[i] += g.v[i];
      g.v[i] = (g.v[i] * w.v[i] - m - x.v[i] * mx) * st.y;
    }
    if (a.dx) g.store(a.dx, r * a.lddx, a.cols, l);
  }
  if (!a.part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const R &from = which ? db : dw;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CH * 8; ++i)
      sums[threadIdx.x / LANES][column<LANES, CH, VEC>(i / 8, i % 8, l)] = from.v[i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
      float t = 0.f;
      for (int i = 0; i < kRows; ++i) t += sums[i][c];
      a.part[((long long)which * gridDim.x + blockIdx.x) * a.cols + c] = t;
    }
  }
}

// Rows too long for registers: a workgroup goes over one row several times, from
// the caches.  Columns are counted in 32 bits: rows end at kMaxCols, so that a step
// behind the end does not leave them.
__global__ __launch_bounds__(kThreads) void k_norm_long(Norm a) {
  __shared__ float red[2][4][3];
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float s[1] = {0.f};
    for (int c = threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
      float v[8];
      dense::load8(a.x, a.fmt, r * a.ldx + c, a.cols - c, a.vec, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[i];
    }
    row_sum<256, 1>(s, red, turn);
    const float mean = s[0] * a.by_cols;
    float sq[2] = {0.f, 0.f};
    for (int c = threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
      float v[8];
      dense::load8(a.x, a.fmt, r * a.ldx + c, a.cols - c, a.vec, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = c + i < a.cols ? v[i] - mean : 0.f;
        sq[0] += d;
        sq[1] = fmaf(d, d, sq[1]);
      }
    }
    row_sum<256, 2>(sq, red, turn);
    const float off = sq[0] * a.by_cols, rstd = rstd_of(sq[1] * a.by_cols, off, a.eps);
    for (int c = threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
      float v[8], w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, b[8] = {};
      dense::load8(a.x, a.fmt, r * a.ldx + c, a.cols - c, a.vec, v);
      if (a.weight) dense::load8(a.weight, a.fmt, c, a.cols - c, a.vec, w);
      if (a.bias) dense::load8(a.bias, a.fmt, c, a.cols - c, a.vec, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf((v[i] - mean - off) * rstd, w[i], b[i]);
      dense::store8(a.y, a.fmt, r * a.ldy + c, a.cols - c, a.vec, v);
    }
    if (a.stats && threadIdx.x == 0) *(float2 *)(a.stats + 2 * r) = make_float2(mean, rstd);
  }
}

// dx, and each row's offset for the columns' sums.
__global__ __launch_bounds__(kThreads) void k_norm_long_backward(Norm a) {
  __shared__ float red[2][4][3];
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float2 st = *(const float2 *)(a.stats + 2 * r);
    float s[3] = {0.f, 0.f, 0.f};
    for (int pass = 0; pass < 2; ++pass) {
      const float off = s[2] * a.by_cols, m = s[0] * a.by_cols, mx = fmaf(-off, m, s[1] * a.by_cols);
      for (int c = threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
        float x[8], g[8], w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        dense::load8(a.x, a.fmt, r * a.ldx + c, a.cols - c, a.vec, x);
        dense::load8(a.dy, a.fmt, r * a.lddy + c, a.cols - c, a.vec, g);
        if (a.weight) dense::load8(a.weight, a.fmt, c, a.cols - c, a.vec, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = c + i < a.cols;
          x[i] = in ? (x[i] - st.x) * st.y : 0.f;
          g[i] = in ? g[i] * w[i] : 0.f;
          if (pass == 0) {
            s[0] += g[i];
            s[1] = fmaf(g[i], x[i], s[1]);
            s[2] += x[i];
          } else {
            g[i] = (g[i] - m - (x[i] - off) * mx) * st.y;
          }
        }
        if (pass == 1) dense::store8(a.dx, a.fmt, r * a.lddx + c, a.cols - c, a.vec, g);
      }
      if (pass == 0) row_sum<256, 3>(s, red, turn);
    }
    if (a.offs && threadIdx.x == 0) a.offs[r] = s[2] * a.by_cols;
  }
}

// The offsets alone, where dx is not wanted: x is read once more (4096 x 16384 bf16, of which
// part is in the caches: 15 us of 141; the pass above without its second half takes 41).
__global__ __launch_bounds__(kThreads) void k_norm_offsets(Norm a) {
  __shared__ float red[2][4][3];
  int turn = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float2 st = *(const float2 *)(a.stats + 2 * r);
    float s[1] = {0.f};
    if (a.vec) {
#pragma unroll 2
      for (int c = threadIdx.x * 8; c < a.cols; c += kThreads * 8) {
        float x[8];
        dense::load8(a.x, a.fmt, r * a.ldx + c, 8, true, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += (x[i] - st.x) * st.y;
      }
    } else {
#pragma unroll 8
      for (int c = threadIdx.x; c < a.cols; c += kThreads)
        s[0] += (dense::load1(a.x, a.fmt, r * a.ldx + c) - st.x) * st.y;
    }
    row_sum<256, 1>(s, red, turn);
    if (threadIdx.x == 0) a.offs[r] = s[0] * a.by_cols;
  }
}

// Sums of dy xh and dy over a block of rows: a column to a thread.  xh is without what
// the mean's rounding left in it, as elsewhere: with it, rows 1e4 deviations from zero
// would all be off to one side (2000 rows: dweight by 0.4 of 64).
__global__ __launch_bounds__(kThreads) void k_norm_columns(Norm a, int rows_each) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.cols) return;
  const long long r0 = (long long)blockIdx.y * rows_each;
  const long long r1 = r0 + rows_each < a.rows ? r0 + rows_each : a.rows;
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (long long r = r0; r < r1; ++r) {
    const float2 st = *(const float2 *)(a.stats + 2 * r);
    const float g = dense::load1(a.dy, a.fmt, r * a.lddy + c);
    const float xh = (dense::load1(a.x, a.fmt, r * a.ldx + c) - st.x) * st.y;
    dw = fmaf(g, xh - (a.offs ? a.offs[r] : 0.f), dw);
    db += g;
  }
  a.part[(long long)blockIdx.y * a.cols + c] = dw;
  a.part[((long long)gridDim.y + blockIdx.y) * a.cols + c] = db;
}

// dweight and dbias: the sums of the blocks' sums; 32 columns to a workgroup, and the
// next 32 of as many workgroups as there are.
__global__ __launch_bounds__(kThreads) void k_norm_join(Norm a, int blocks) {
  const int ty = threadIdx.x >> 5, which = blockIdx.y;
  void *const out = which ? a.dbias : a.dweight;
  if (!out) return;
  const float *const part = a.part + (long long)which * blocks * a.cols;
  __shared__ float red[8][32];
  for (int first = blockIdx.x * 32; first < a.cols; first += gridDim.x * 32) {
    const int c = first + (threadIdx.x & 31);
    float s = 0.f;
    if (c < a.cols) {
#pragma unroll 8
      for (int i = ty; i < blocks; i += 8) s += part[(long long)i * a.cols + c];
    }
    __syncthreads();
    red[ty][threadIdx.x & 31] = s;
    __syncthreads();
    if (ty == 0 && c < a.cols) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t += red[i][threadIdx.x];
      dense::store1(out, a.fmt, c, t);
    }
  }
}

constexpr int kLongRow = 8192;

// Which lanes hold a row: as few as have room for it.
template <class F>
void by_shape(const Norm &a, F go) {
  if (a.cols <= 64)
    go(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  else if (a.cols <= 256)
    go(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  else if (a.cols <= 512)
    go(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  else if (a.cols <= 1024)
    go(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  else if (a.cols <= 2048)
    go(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
  else if (a.cols <= 4096)
    go(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  else
    go(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
}
template <class F>
void by_format(const Norm &a, F go) {
  if (a.fmt == kBf16)
    go(std::integral_constant<int, kBf16>());
  else if (a.fmt == kF16)
    go(std::integral_constant<int, kF16>());
  else
    go(std::integral_constant<int, kF32>());
}

unsigned workgroups(long long units, long long most) {
  return (unsigned)(units < 1 ? 1 : units < most ? units : most);
}

}  // namespace

hipError_t launch_norm(const Norm &a, hipStream_t st) {
  if (!a.rows || !a.cols) return hipSuccess;
  if (a.cols > kLongRow) {
    hipLaunchKernelGGL(k_norm_long, dim3(workgroups(a.rows, 4096)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
  by_format(a, [&](auto fmt) {
    by_shape(a, [&](auto lanes, auto ch) {
      constexpr int F = decltype(fmt)::value, LN = decltype(lanes)::value, CH = decltype(ch)::value;
      const dim3 grid(workgroups((a.rows + kThreads / LN - 1) / (kThreads / LN), 2048));
      if (a.vec)
        hipLaunchKernelGGL((k_norm<F, LN, CH, true>), grid, dim3(kThreads), 0, st, a);
      else
        hipLaunchKernelGGL((k_norm<F, LN, CH, false>), grid, dim3(kThreads), 0, st, a);
    });
  });
  return hipGetLastError();
}

// Workgroups of the backward, each of which leaves sums of all columns.
int norm_blocks(long long rows, long long cols) {
  if (cols > kLongRow) return (int)workgroups((rows + 63) / 64, 256);
  int lanes = 64;
  Norm a = {};
  a.cols = (int)cols;
  by_shape(a, [&](auto l, auto) { lanes = decltype(l)::value; });
  const int per = kThreads / lanes;
  return (int)workgroups((rows + per - 1) / per, 512);
}

long long norm_offsets(long long rows, long long cols) { return cols > kLongRow ? rows : 0; }

hipError_t launch_norm_backward(const Norm &a, hipStream_t st) {
  if (!a.cols) return hipSuccess;
  const int blocks = a.rows ? norm_blocks(a.rows, a.cols) : 0;
  if (a.rows && a.cols > kLongRow) {
    if (a.dx)
      hipLaunchKernelGGL(k_norm_long_backward, dim3(workgroups(a.rows, 4096)), dim3(kThreads), 0, st, a);
    else if (a.offs)
      hipLaunchKernelGGL(k_norm_offsets, dim3(workgroups(a.rows, 4096)), dim3(kThreads), 0, st, a);
    if (a.part)
      hipLaunchKernelGGL(k_norm_columns, dim3((unsigned)((a.cols + kThreads - 1) / kThreads), (unsigned)blocks),
                         dim3(kThreads), 0, st, a, (int)((a.rows + blocks - 1) / blocks));
  } else if (a.rows) {
    by_format(a, [&](auto fmt) {
      by_shape(a, [&](auto lanes, auto ch) {
        constexpr int F = decltype(fmt)::value, LN = decltype(lanes)::value, CH = decltype(ch)::value;
        if (a.vec)
          hipLaunchKernelGGL((k_norm_backward<F, LN, CH, true>), dim3(blocks), dim3(kThreads), 0, st, a);
        else
          hipLaunchKernelGGL((k_norm_backward<F, LN, CH, false>), dim3(blocks), dim3(kThreads), 0, st, a);
      });
    });
  }
  if (a.dweight || a.dbias)
    // (a launch has fewer than 2^32 threads)
    hipLaunchKernelGGL(k_norm_join, dim3(workgroups((a.cols + 31) / 32, 1 << 20), 2), dim3(kThreads), 0, st, a, blocks);
  return hipGetLastError();
}

// --------------------------------------------------------------------- dropout
//
// Which elements stay is 16 bits of a counter-based generator for each, drawn
// again wherever it is needed: Philox 4x32 with 10 rounds (Salmon, Moraes, Dror
// and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), one block of 128
// bits for 8 elements.  16 bits make p a multiple of 2^-16 and the generator's 20
// wide products serve eight elements.

namespace {

struct Bits {
  uint32_t w[4];
  __device__ __forceinline__ Bits(uint64_t block, uint64_t offset, uint64_t seed) {
    uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32);
    uint32_t x2 = (uint32_t)offset, x3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
      x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
      x1 = (uint32_t)b;
      x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
      x3 = (uint32_t)a;
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    w[0] = x0;
    w[1] = x1;
    w[2] = x2;
    w[3] = x3;
  }
  __device__ __forceinline__ bool keeps(int i, uint32_t t) const {
    return ((w[i >> 1] >> ((i & 1) * 16)) & 0xffffu) >= t;
  }
};

// Elements in memory order, 16 bytes at a time.  16384 x 2048 bf16 with a residual: 39
// us, 5.1 TB/s; the gradient 23 us, 5.8: the generator's 20 products to 8 elements are
// hidden.
template <int FMT, bool RES>
__global__ __launch_bounds__(kThreads) void k_dropout(Drop a) {
  const uint64_t seed = a.seed_at ? *a.seed_at : a.seed;
  const long long whole = a.count >> 3, step = (long long)gridDim.x * kThreads;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < whole; i += step) {
    float v[8], r[8];
    dense::load_w<8>(a.x, FMT, i * 8, v);
    if constexpr (RES) dense::load_w<8>(a.res, FMT, i * 8, r);
    const Bits bits((uint64_t)i, a.offset, seed);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = bits.keeps(e, a.t) ? v[e] * a.scale : 0.f;
      if constexpr (RES) v[e] += r[e];
    }
    dense::store_w<8>(a.y, FMT, i * 8, v);
  }
  // what is left of a last block
  const int left = (int)(a.count & 7);
  if (blockIdx.x == 0 && (int)threadIdx.x < left) {
    const long long i = whole * 8 + threadIdx.x;
    const Bits bits((uint64_t)whole, a.offset, seed);
    bool keep = false;
#pragma unroll
    for (int e = 0; e < 7; ++e) keep = e == (int)threadIdx.x ? bits.keeps(e, a.t) : keep;
    float v = keep ? dense::load1(a.x, FMT, i) * a.scale : 0.f;
    if constexpr (RES) v += dense::load1(a.res, FMT, i);
    dense::store1(a.y, FMT, i, v);
  }
}

// Rows apart, or elements that begin anywhere: value by value.
__global__ __launch_bounds__(kThreads) void k_dropout_rows(Drop a) {
  const uint64_t seed = a.seed_at ? *a.seed_at : a.seed;
  const long long blocks = (a.count + 7) >> 3, step = (long long)gridDim.x * kThreads;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < blocks; i += step) {
    const Bits bits((uint64_t)i, a.offset, seed);
    long long r = i * 8 / a.cols, c = i * 8 - r * a.cols;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (i * 8 + e >= a.count) break;
      float v = bits.keeps(e, a.t) ? dense::load1(a.x, a.fmt, r * a.ldx + c) * a.scale : 0.f;
      if (a.res) v += dense::load1(a.res, a.fmt, r * a.ldr + c);
      dense::store1(a.y, a.fmt, r * a.ldy + c, v);
      if (++c == a.cols) {
        c = 0;
        ++r;
      }
    }
  }
}

}  // namespace

hipError_t launch_dropout(const Drop &a, hipStream_t st) {
  if (!a.count) return hipSuccess;
  const dim3 grid(workgroups(((a.count + 7) / 8 + kThreads - 1) / kThreads, 1 << 20));
  if (!a.vec) {
    hipLaunchKernelGGL(k_dropout_rows, grid, dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
  Norm n = {};
  n.fmt = a.fmt;
  by_format(n, [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    if (a.res)
      hipLaunchKernelGGL((k_dropout<F, true>), grid, dim3(kThreads), 0, st, a);
    else
      hipLaunchKernelGGL((k_dropout<F, false>), grid, dim3(kThreads), 0, st, a);
  });
  return hipGetLastError();
}

}  // namespace norm
}  // namespace pdr
