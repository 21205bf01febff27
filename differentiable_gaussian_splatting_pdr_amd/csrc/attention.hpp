// attention.hpp -- what the attention kernels share: where a workgroup's rows
// and keys lie, tiles of rows in LDS, and the two kinds of matrix product.
//
// Rows.  A key head is read by G = heads / kv_heads query heads.  Their queries
// are taken together: row r of a sequence and key head is head r % G of token
// r / G.  One pass over the keys then serves the whole group, a single token's
// heads share one tile, and the gradients of shared heads are sums over rows
// like any other.
//
// Products.  Both kinds are 32x32 matrix instructions whose result has 32 tile
// rows in registers and one column per lane (lane % 32): register r of half
// h = lane / 32 holds row 8 (r / 4) + 4 h + r % 4.
//   along()  c[row][col] += sum_d tile[row][d] reg[col][d]: scores, from rows
//            of an LDS tile and rows that the lanes keep in registers;
//   across() c[d][col] += sum_row tile[row][d] p[row][col]: sums over rows,
//            whose weights p are just what along() left in the registers: the
//            sum's order over rows is free, so register r, half h stands for
//            the same row in both operands and nothing moves between lanes.
// A softmax over rows is then a sum over a lane's registers and its other half.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense_epilogue.hpp"
#include "pdr_blocks.h"
#include "pdr_common.hpp"

namespace pdr {
namespace attend {

using dense::bf16_to_f;
using dense::f16_to_f;
using dense::kBf16;
using dense::kF16;
using dense::kF32;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr uint32_t kOutside = 0x80000000u;  // a byte offset beyond every buffer's bound
constexpr long long kMaxRow = 1 << 22, kMaxHead = 1 << 24, kMaxHeads = 1 << 28;  // elements

struct Mat {
  char *p;
  long long row, head, batch;  // elements
};

struct Args {
  Mat q, k, v, o, dy, dq, dk, dv;
  const int *q_offsets, *k_offsets, *key_lengths;
  float *lse;
  float *starts;            // backward: what scores and their gradients' products start from, pairs laid out as lse
  float *part_o, *part_ml;  // few queries: the splits' sums, and their maxima and weights
  float *part_k;            // dk and dv: the parts' sums
  float scale, scale2;      // scale, and scale log2(e)
  int causal, batch, kv_heads, dim, q_rows, k_rows;
  int q_tiles, k_tiles;     // of a sequence; with offsets, of all
  int splits;
  int waves;                // few queries: of a workgroup
  FastDiv group;            // by G
  FastDiv heads;            // by kv_heads
  FastDiv per_tile;         // by the sequences (no offsets)
};

// ------------------------------------------------------------ where things lie

// A workgroup's tile: the sequence, its queries and keys, the tile in it.
struct Place {
  int seq, nq, nk;   // tokens
  int q0, k0;        // first token in the tensor (offsets), or 0
  int stored;        // keys that the tensor has from k0 on and that belong to this sequence
  int tile;          // -1: nothing to do
};

__device__ __forceinline__ int bound_at(const int *off, int n, int total, int i) {
  if (i <= 0) return 0;
  if (i > n + 1) return total;
  const int v = off[i - 1];
  return v < 0 ? 0 : v > total ? total : v;
}

// Tiles of packed sequences.  Bounds 0, off[0], .., off[n], total cut the tokens
// into n + 2 sequences, of which the first and last hold what no sequence has.
// Sequence i's tiles begin at floor(bound_i G / 2^LOG) + i, which leaves room for
// all of them whatever their lengths: no list has to be made first, and at most
// one workgroup a sequence has nothing to do.  The search looks at 64 bounds at
// a time.
template <int LOG>
__device__ __forceinline__ int find_sequence(const int *off, int n, int total, int g, int t) {
  int lo = 0, count = n + 2;
  const int lane = threadIdx.x & 63;
  while (count > 1) {
    const int step = (count + 63) >> 6;
    const int i = lo + lane * step;
    const bool in = lane * step < count &&
                    (int)(((long long)bound_at(off, n, total, i) * g) >> LOG) + i <= t;
    const uint64_t no = ~__ballot(in);
    int k = no ? __ffsll((unsigned long long)no) - 2 : 63;
    k = __builtin_amdgcn_readfirstlane(k < 0 ? 0 : k);
    lo += k * step;
    count = count - k * step < step ? count - k * step : step;
  }
  return lo;
}

// BY_KEYS: t counts tiles of 2^LOG keys; else of 2^LOG rows (g to a token).
template <int LOG, bool BY_KEYS>
__device__ __forceinline__ Place place(const Args &a, int t) {
  Place p;
  const int g = BY_KEYS ? 1 : (int)a.group.d;
  if (!a.q_offsets) {
    // equal tiles of all sequences follow one another, so that where queries see
    // what is before them work is handed out by its length
    p.tile = (int)fdiv((uint32_t)t, a.per_tile);
    p.seq = t - p.tile * a.batch;
    p.nq = a.q_rows;
    p.nk = a.k_rows;
    if (a.key_lengths) {
      const int len = a.key_lengths[p.seq];
      p.nk = len < 0 ? 0 : len > a.k_rows ? a.k_rows : len;
    }
    p.q0 = p.k0 = 0;
    p.stored = a.k_rows;
    return p;
  }
  const int *off = BY_KEYS ? a.k_offsets : a.q_offsets;
  const int total = BY_KEYS ? a.k_rows : a.q_rows;
  const int i = find_sequence<LOG>(off, a.batch, total, g, t);
  const int begin = bound_at(off, a.batch, total, i);
  int end = bound_at(off, a.batch, total, i + 1);
  if (end < begin) end = begin;
  p.seq = 0;
  p.tile = t - ((int)(((long long)begin * g) >> LOG) + i);
  const bool real = i >= 1 && i <= a.batch;
  // the other side's tokens; the first and last sequence have none
  const int *off2 = BY_KEYS ? a.q_offsets : a.k_offsets;
  const int total2 = BY_KEYS ? a.q_rows : a.k_rows;
  const int begin2 = real ? bound_at(off2, a.batch, total2, i) : 0;
  int end2 = real ? bound_at(off2, a.batch, total2, i + 1) : 0;
  if (end2 < begin2) end2 = begin2;
  p.q0 = BY_KEYS ? begin2 : begin;
  p.nq = BY_KEYS ? end2 - begin2 : end - begin;
  p.k0 = BY_KEYS ? begin : begin2;
  p.nk = BY_KEYS ? end - begin : end2 - begin2;
  p.stored = p.nk;
  return p;
}

// First element of a sequence's tokens at a head.
__device__ __forceinline__ long long first_of(const Mat &m, const Place &p, int token0, int head) {
  return p.seq * m.batch + token0 * m.row + head * m.head;
}

// -------------------------------------------------------------- element types

// The same value; what follows from it is not worked out earlier: in a branch that
// few tiles take, or to hold few registers.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The lane's number, worked out anew rather than held in a register.
__device__ __forceinline__ int lane_again() {
  return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, (uint32_t)here(0)));
}

// The order that a stretch of products is to run in: AHEAD reads of LDS first, then
// GROUPS times MFMAS matrix instructions and EACH more reads, until there are READS.
// Left alone, the compiler reads a fragment, waits for it and uses it, one after
// another.
template <int AHEAD, int READS, int EACH, int GROUPS, int MFMAS>
__device__ __forceinline__ void interleave() {
  constexpr int kMfma = 0x8, kRead = 0x100;
  __builtin_amdgcn_sched_group_barrier(kRead, AHEAD, 0);
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMfma, MFMAS, 0);
    if (AHEAD + i * EACH < READS) __builtin_amdgcn_sched_group_barrier(kRead, EACH, 0);
  }
}

// Row of a result's register r in this half.
__device__ __forceinline__ int row_in(int r, int half) { return 8 * (r >> 2) + 4 * half + (r & 3); }

template <int FMT, int DP>  // DP: values a row has in LDS and registers (dim, rounded up)
struct Core {
  static constexpr int kFmt = FMT;
  static constexpr int kSize = FMT == kF32 ? 4 : 2;
  static constexpr int kPer = 16 / kSize;             // values of a 16-byte chunk
  static constexpr int kChunks = DP / kPer;           // of a row
  static constexpr int kSteps = kChunks / 2;          // of along()
  static constexpr int kRowBytes = DP * kSize;
  static constexpr int kBlocks = DP / 32;             // of 32 d

  // LDS: chunk c of row r is stored at chunk c ^ swizzle(r), so that the 256 bytes
  // that are read at a time fall on different banks: equal chunks of sixteen rows
  // (along: whichever rows four groups of four lanes hold, for which bit 4 is
  // folded into bits 2 and 3), and four neighbouring chunks of each of four rows
  // (across, whose transposing read takes 32 bytes of a row to 16 lanes).  It is
  // linear: the swizzle of a sum without carries is that of its parts.
  static __device__ __forceinline__ constexpr int swizzle(int r) {
    const int folded = ((r >> 2) & 3) ^ ((r >> 4) & 1) * 3;
    return (kChunks > 8 ? (r & 3) << 2 : ((r >> 1) & 1) << 2) | folded;
  }

  static __device__ __forceinline__ f32x16 go(i32x4 a, i32x4 b, f32x16 c) {
    if constexpr (FMT == kBf16) {
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                     __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    } else if constexpr (FMT == kF16) {
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                    __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__int_as_float(a[i]), __int_as_float(b[i]), c, 0, 0,
                                                 0);
      return c;
    }
  }

  // A lane's chunks of a row in memory, as along() wants them; zeros past dim.
  static __device__ __forceinline__ void fetch_row(i32x4 (&f)[kSteps], const char *row, int dim,
                                                   int half, bool there) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = 2 * s + half;
      f[s] = i32x4{0, 0, 0, 0};
      if (there && c * kPer < dim) f[s] = *(const i32x4 *)(row + c * 16);
    }
  }

  // The same of rows [first, first + 32) of `rows`, one to a lane and its other half.
  template <class Source>
  static __device__ __forceinline__ void fetch_rows(i32x4 (&f)[kSteps], const Source &from, int first, int rows,
                                                    int dim, int lane) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(from.base + (long long)first * from.row), 0, (int)kOutside, 0x00020000);
    const uint32_t r = lane & 31, half = lane >> 5;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const uint32_t c = 2 * s + half;
      const bool in = first + (int)r < rows && (int)c * kPer < dim;
      f[s] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                           rsrc, (int)(in ? r * from.row + c * 16 : kOutside), 0, 0));
    }
  }

  // Where a lane reads in a tile that begins on 256 bytes.  What the swizzle turns
  // of a chunk's place is turned again for each step or block, by a constant; the
  // rest is the same for all lanes, an offset known when the kernel is compiled.
  // The lane keeps one address of each kind: registers are what these kernels run
  // out of, so the turned ones are made where they are used (here()).
  struct Lane {
    int row, column;
    __device__ __forceinline__ void init(int lane) {
      const int half = lane >> 5, r = lane & 31;
      row = r * kRowBytes + ((half ^ swizzle(r)) << 4);
      if constexpr (FMT != kF32) {
        const int t = lane & 15, k = 4 * half + (t >> 2), c = ((lane >> 4) & 1) * 2 + ((t & 3) >> 1);
        column = k * kRowBytes + ((c ^ swizzle(k)) << 4) + (t & 1) * 8;
      } else {
        column = 4 * half * kRowBytes + (((r >> 2) ^ half) << 4) + (r & 3) * 4;
      }
    }
  };
  // Reads of LDS.  The restrict pointers tell the compiler that they do not wait for
  // loads to LDS in flight.
  template <class T>
  static __device__ __forceinline__ T at_pointer(const __attribute__((address_space(3))) T *__restrict p) {
    return *p;
  }
  template <class T>
  static __device__ __forceinline__ T read(int at) {
    return at_pointer((const __attribute__((address_space(3))) T *)(uintptr_t)(uint32_t)at);
  }

  // Rows 32 u .. 32 u + 31 of the tile.
  static __device__ __forceinline__ void along(f32x16 &c, const lds_char *tile, int u,
                                               const i32x4 (&reg)[kSteps], const Lane &at) {
    const int first = here((int)(uintptr_t)tile + at.row);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      // chunk 2 s + half, of which the swizzle turns the lowest three or four bits
      const int offset = (s >> 3) * 256 + u * 32 * kRowBytes;
      c = go(read<i32x4>((first ^ (s & 7) << 5) + offset), reg[s], c);
    }
  }

  // Eight registers of an along() as the second operand of across().  In 16 bits they are
  // rounded to the operands' type, which the matrix instruction asks for: an error of the
  // size of the result's own rounding (bf16 results are 0.0023 from 64 bits, rounded once
  // they would be 0.0017), where a product of what is lost would be the forward's third
  // beside two.
  struct Weights {
    i32x4 w[FMT == kF32 ? 2 : 1];
  };
  static __device__ __forceinline__ Weights pack(const f32x16 &v, int first) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    Weights o;
    if constexpr (FMT == kF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o.w[i >> 2][i & 3] = __float_as_int(v[first + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 two = {v[first + 2 * i], v[first + 2 * i + 1]};
        o.w[0][i] = FMT == kBf16 ? __builtin_bit_cast(int, __builtin_convertvector(two, b2))
                                 : __builtin_bit_cast(int, __builtin_convertvector(two, h2));
      }
    }
    return o;
  }
  // Rows 16 X .. 16 X + 15 of the tile under these weights.
  static __device__ __forceinline__ void across(f32x16 (&c)[kBlocks], const lds_char *tile, int x,
                                                const Weights &p, const Lane &at) {
    const int first = here((int)(uintptr_t)tile + at.column);
    if constexpr (FMT != kF32) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) c[b] = go(column(first, x, b), p.w[0], c[b]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
          c[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(value(first, x, e, b), __int_as_float(p.w[e >> 2][e & 3]), c[b], 0,
                                                      0, 0);
    }
  }
  // fp32: a value of row 16 x + 8 (e / 4) + e % 4, and 4 half more, of block b.
  static __device__ __forceinline__ float value(int first, int x, int e, int b) {
    const int row = x * 16 + 8 * (e >> 2) + (e & 3), turn = swizzle(row);
    return read<float>((first ^ (turn & 7) << 4) + row * kRowBytes + (b ^ turn >> 3) * 128);
  }
  // Fragment b of those rows (16-bit types).
  static __device__ __forceinline__ i32x4 column(int first, int x, int b) {
    const int lo = (first ^ b << 6 ^ swizzle(x * 16) << 4) + x * 16 * kRowBytes;
    const int hi = (first ^ b << 6 ^ swizzle(x * 16 + 8) << 4) + (x * 16 + 8) * kRowBytes;
    const s16x4 y = transposed((lds_s16x4 *)(uintptr_t)(uint32_t)lo);
    const s16x4 z = transposed((lds_s16x4 *)(uintptr_t)(uint32_t)hi);
    return __builtin_bit_cast(i32x4, __builtin_shufflevector(y, z, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // The order of N calls of along(), after OTHER reads, and of across() over 32 N rows.
  template <int N, int OTHER = 0>
  static __device__ __forceinline__ void pace_along() {
    if constexpr (FMT == kF32)
      interleave<OTHER + 3, OTHER + N * kSteps, 1, N * kSteps, 4>();
    else
      interleave<OTHER + 6, OTHER + N * kSteps, 1, N * kSteps, 1>();
  }
  template <int N>
  static __device__ __forceinline__ void pace_across() {
    if constexpr (FMT == kF32)  // two values of each lane to a read
      interleave<4, N * 8 * kBlocks, 1, N * 8 * kBlocks, 2>();
    else
      interleave<8, N * 4 * kBlocks, 2, N * 2 * kBlocks, 1>();
  }
  // ---- what is not finite where a mask hides it
  //
  // A weight of zero does not hide an infinity or a NaN: their product is NaN.  Where
  // a tile is masked it is looked through, and if there are any, across_careful()
  // sums the finite values and then adds the others where they are seen.
  static __device__ __forceinline__ bool finite(i32x4 v) {
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= not_finite((uint32_t)v[i]);
    return bad == 0;
  }
  // The bits of a word's values that are not finite.
  static __device__ __forceinline__ uint32_t not_finite(uint32_t v) {
    if constexpr (FMT == kF32) return (v & 0x7f800000u) == 0x7f800000u ? ~0u : 0u;
    constexpr uint32_t kExp = FMT == kBf16 ? 0x7f80u : 0x7c00u;
    return ((v & kExp) == kExp ? 0xffffu : 0u) | ((v >> 16 & kExp) == kExp ? 0xffff0000u : 0u);
  }
  // Whether rows 32 u .. 32 u + 31 hold any (the same for all lanes).
  static __device__ __forceinline__ bool any_not_finite(const lds_char *tile, int u, int lane) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 32 * kRowBytes / 1024; ++i)
      bad |= !finite(read<i32x4>((int)(uintptr_t)tile + u * 32 * kRowBytes + i * 1024 + lane * 16));
    return __any(bad);
  }
  // across() of rows 32 u .. 32 u + 31 under weights w; this lane's column sees the
  // first `seen` of them.
  static __device__ __forceinline__ void across_careful(f32x16 (&c)[kBlocks], const lds_char *tile, int u,
                                                        const f32x16 &w, const Lane &at, int half, int seen) {
    const int first = here((int)(uintptr_t)tile + at.column);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const Weights p = pack(w, 8 * x);
      if constexpr (FMT != kF32) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          i32x4 f = column(first, 2 * u + x, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] &= (int)~not_finite((uint32_t)f[i]);
          c[b] = go(f, p.w[0], c[b]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            float f = value(first, 2 * u + x, e, b);
            f = not_finite(__float_as_uint(f)) ? 0.f : f;
            c[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(f, __int_as_float(p.w[e >> 2][e & 3]), c[b], 0, 0, 0);
          }
      }
    }
#pragma unroll 1
    for (int row = 0; row < 32; ++row) {
      const int place = (int)(uintptr_t)tile + (u * 32 + row) * kRowBytes;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int byte = (b * 32 + row_in(r, half)) * kSize;
          const int from = place + ((byte >> 4 ^ swizzle(row)) << 4) + (byte & 15);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v;
            if constexpr (FMT == kF32)
              v = read<float>(from + 4 * i);
            else
              v = dense::to_f<FMT>((uint16_t)read<short>(from + 2 * i));
            if (row < seen && !(fabsf(v) < INFINITY)) c[b][r + i] += v;
          }
        }
    }
  }

  // ds_read_b64_tr_b16: of each 16 lanes' 4 rows of 16 values (a row is four
  // lanes' 8 bytes), lane t receives column t.
  static __device__ __forceinline__ s16x4 transposed(lds_s16x4 *__restrict p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
  }
};

// Copies tiles of ROWS rows to LDS (loads straight to LDS, zeros for rows that
// do not exist and past dim), by NW waves.
struct Source {
  const char *base;    // first token of the sequence, this head
  uint32_t row, head;  // bytes
  __device__ __forceinline__ Source(const Mat &m, long long first, int size)
      : base(scalar(m.p + first * size)), row((uint32_t)(m.row * size)), head((uint32_t)(m.head * size)) {}
  // All lanes have the same place, which the compiler does not see in every kernel:
  // it then puts a loop over lanes around each load.
  static __device__ __forceinline__ const char *scalar(const char *p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const char *)(uintptr_t)((uint64_t)hi << 32 | lo);
  }
};
template <class C, int ROWS, int NW>
struct Loader {
  static constexpr int kBytes = ROWS * C::kRowBytes;
  static constexpr int kIssues = kBytes / (NW * 1024);
  static constexpr int kRowsEach = 1024 / C::kRowBytes;  // rows of one wave's load
  static_assert(kBytes % (NW * 1024) == 0 && kRowsEach * C::kRowBytes == 1024, "whole loads");
  int wave, dim;
  int row0, chunk0;  // this lane's row and chunk in the first load

  __device__ __forceinline__ void init(int dim_, int wave_, int lane) {
    wave = wave_;
    dim = dim_;
    row0 = wave * kRowsEach + lane / C::kChunks;
    chunk0 = (lane % C::kChunks) ^ C::swizzle(row0);
  }
  // The i-th load's row, and its byte in the row or kOutside (whose bit stays when
  // it is added to a place below 2^31).  The rows between
  // two loads are a power of two that row0 stays below, so their swizzles add up.
  __device__ __forceinline__ int row_of(int i) const { return row0 + i * NW * kRowsEach; }
  __device__ __forceinline__ uint32_t byte_of(int i) const {
    const int c = chunk0 ^ C::swizzle(i * NW * kRowsEach);
    return c * C::kPer < dim ? (uint32_t)c * 16u : kOutside;
  }
  static __device__ __forceinline__ uint32_t outside(bool v) { return v ? kOutside : 0u; }
  __device__ __forceinline__ void issue(const char *from, uint32_t off, lds_char *lds, int i) const {
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc((void *)from, 0, (int)kOutside, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(lds + (i * NW + wave) * 1024), 16,
                                             (int)off, 0, 0, 0);
  }
  // Rows [first, first + ROWS) of `rows`.
  __device__ __forceinline__ void tokens(const Source &x, int first, int rows, lds_char *lds) const {
    const char *const from = x.base + (long long)first * x.row;
#pragma unroll
    for (int i = 0; i < kIssues; ++i) {
      const uint32_t r = (uint32_t)row_of(i);
      issue(from, (r * x.row + byte_of(i)) | outside(first + (int)r >= rows), lds, i);
    }
  }
  // The same, of two tensors.
  __device__ __forceinline__ void tokens(const Source &x, const Source &y, int first, int rows, lds_char *lds) const {
    const char *const from_x = x.base + (long long)first * x.row;
    const char *const from_y = y.base + (long long)first * y.row;
#pragma unroll
    for (int i = 0; i < kIssues; ++i) {
      const uint32_t r = (uint32_t)row_of(i), c = byte_of(i), out = outside(first + (int)r >= rows);
      issue(from_x, (r * x.row + c) | out, lds, i);
      issue(from_y, (r * y.row + c) | out, lds + kBytes, i);
    }
  }
  // The same of a group's rows.
  __device__ __forceinline__ void grouped(const Source &x, const Source &y, int first, int rows,
                                          const FastDiv &group, lds_char *lds) const {
    const int token0 = (int)fdiv((uint32_t)first, group);
    const char *const from_x = x.base + (long long)token0 * x.row;
    const char *const from_y = y.base + (long long)token0 * y.row;
#pragma unroll
    for (int i = 0; i < kIssues; ++i) {
      const int r = first + row_of(i);
      const uint32_t c = byte_of(i), token = fdiv((uint32_t)r, group), g = (uint32_t)r - token * group.d;
      const uint32_t out = outside(r >= rows);
      issue(from_x, ((token - token0) * x.row + g * x.head + c) | out, lds, i);
      issue(from_y, ((token - token0) * y.row + g * y.head + c) | out, lds + kBytes, i);
    }
  }
};

// Loads to LDS have landed, but for the wave's last LEFT; its LDS reads are done.
template <int LEFT>
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT) : "memory");
}
// ... and every wave's.
template <int LEFT>
__device__ __forceinline__ void all_landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// The value of the lane 32 further on (or back).
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }

__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }

// Four consecutive values of a row.
template <int FMT>
__device__ __forceinline__ void store4(char *p, const float v[4]) {
  if constexpr (FMT == kF32) {
    *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint16_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = FMT == kBf16 ? dense::f_to_bf16(v[i]) : dense::f_to_f16(v[i]);
    *(uint2 *)p = make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
  }
}

// Columns of across() to memory: this lane's column is the row at `p`.
template <class C, int FMT>
__device__ __forceinline__ void store_columns(const f32x16 (&c)[C::kBlocks], char *p, int dim, int half,
                                              float by) {
#pragma unroll
  for (int b = 0; b < C::kBlocks; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int d = b * 32 + row_in(r, half);
      const float v[4] = {c[b][r] * by, c[b][r + 1] * by, c[b][r + 2] * by, c[b][r + 3] * by};
      if (d < dim) store4<FMT>(p + d * C::kSize, v);
    }
}

__device__ __forceinline__ void fill(f32x16 &c, float v) {
#pragma unroll
  for (int i = 0; i < 16; ++i) c[i] = v;
}
__device__ __forceinline__ void clear(f32x16 &c) { fill(c, 0.f); }

// Launchers (attention_forward.hip, attention_backward.hip).
constexpr int kLogWide = 7;  // 128 rows, or keys, to a workgroup
constexpr int kLogFew = 5;   // 32
hipError_t launch_forward(const Args &a, int fmt, hipStream_t st);
hipError_t launch_forward_few(const Args &a, int fmt, hipStream_t st);
// Without dq they make the rows' starts alone.
hipError_t launch_backward_q(const Args &a, int fmt, hipStream_t st);
hipError_t launch_backward_q_few(const Args &a, int fmt, hipStream_t st);
hipError_t launch_backward_kv(const Args &a, int fmt, hipStream_t st);

}  // namespace attend
}  // namespace pdr
