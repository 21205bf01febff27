// norm.hpp -- launchers of layer norm and dropout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "dense_epilogue.hpp"
#include "pdr_blocks.h"

namespace pdr {
namespace norm {

constexpr long long kMaxCols = 1 << 30;

struct Norm {
  const void *x, *weight, *bias, *dy;
  void *y, *dx, *dweight, *dbias;
  float *stats;
  float *part;  // [2][blocks][cols]: sums of dy xh, then of dy; null: not wanted
  float *offs;  // [norm_offsets]: what the mean's rounding left in xh; null: not wanted
  long long rows, ldx, ldy, lddy, lddx;
  int cols, fmt;
  int vec;      // everything begins on 16 bytes in whole groups of 8
  float eps, by_cols;
};
hipError_t launch_norm(const Norm &a, hipStream_t st);
hipError_t launch_norm_backward(const Norm &a, hipStream_t st);
int norm_blocks(long long rows, long long cols);
long long norm_offsets(long long rows, long long cols);  // a value each, for dweight

struct Drop {
  const void *x, *res;
  void *y;
  const unsigned long long *seed_at;
  unsigned long long seed, offset;
  long long count, cols, ldx, ldr, ldy;
  int fmt, vec;  // vec: one run of elements that begins on 16 bytes
  uint32_t t;
  float scale;
};
hipError_t launch_dropout(const Drop &a, hipStream_t st);

}  // namespace norm
}  // namespace pdr
