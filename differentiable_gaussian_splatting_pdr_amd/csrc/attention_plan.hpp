// attention_plan.hpp -- which of attention's kernels a call takes: host code that
// looks at sizes alone.
#pragma once

#include "pdr_blocks.h"

namespace pdr {
namespace attend {

// Sizes of the average sequence.
struct Sizes {
  long long seqs, rows, keys;  // rows: queries and heads of a key head
  long long wide;              // workgroups of 128 rows
  explicit Sizes(const pdr_attention &p) {
    seqs = p.batch > 0 ? p.batch : 1;
    rows = (p.q_offsets ? (p.q_rows + seqs - 1) / seqs : p.q_rows) * (p.heads / p.kv_heads);
    keys = p.q_offsets ? (p.k_rows + seqs - 1) / seqs : p.k_rows;
    wide = (rows + 127) / 128 * seqs * p.kv_heads;
  }
};

// Whether 32 rows go to a workgroup whose waves share the keys, instead of 128 whose
// waves share tiles of keys: where a sequence has no more, where the larger workgroups
// are fewer than the compute units, and where fp32 workgroups of 64 values a head see
// different numbers of keys, as one to a compute unit waits for the longest.
// Larger against smaller, forward / all gradients, us:
//   bf16 2 x 512, 8 heads of 128      (64 workgroups)   18 /  49     13 /  47
//   bf16 4 x 1024, 4 heads of 128    (128)              27 /  73     24 /  68
//   bf16 8192, 2 heads of 128        (128)             159 / 302    125 / 216
//   fp32 4 x 1024, 8 heads of 64     (256, causal)      84 / 217     63 / 179
//   the same, not causal             (256)              79 / 277     89 / 290
//   fp32 6 x 512, 16 heads of 64     (384, causal)      62 / 184     54 / 185
//   fp32 2 x 2048, 12 heads of 64    (384, causal)     196 / 498    133 / 494
//   fp32 3 x 777, 20 heads of 40     (420, causal)      87 / 241     64 / 230
//   fp32 4096, 15 heads of 32        (480, causal)     399 / 1026   287 / 1041
//   fp32 4 x 1024, 8 heads of 128    (256, causal)     146 / 395    132 / 438
//   fp32 8 x 1024, 8 heads of 64     (512, causal)     110 / 305    102 / 319
inline bool takes_few(const pdr_attention &p) {
  const Sizes n(p);
  const bool uneven = p.fmt == PDR_FMT_F32 && p.causal && p.dim <= 64 && n.wide < 512;
  if (n.rows > 32 && !uneven && n.wide >= 256) return false;
  // a launch has fewer than 2^32 threads
  const long long each = p.heads / p.kv_heads;
  return (p.q_offsets ? (p.q_rows * each >> 5) + n.seqs + 2 : (n.rows + 31) / 32 * n.seqs) * p.kv_heads < 1 << 22;
}

}  // namespace attend
}  // namespace pdr
