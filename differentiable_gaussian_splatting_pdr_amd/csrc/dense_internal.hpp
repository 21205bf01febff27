// dense_internal.hpp -- what the dense operators' translation units share.
#pragma once

#include "dense_gemm.hpp"

namespace pdr {
namespace dense {

// Launch one product (dense_gemm_*.hip: one file per operand format).  g's
// tile counts and splits are chosen here; `ws` is scratch for split sums of
// gemm_scratch_bytes() bytes.
hipError_t launch_gemm_bf16(GemmArgs g, bool a_mc, bool b_mc, EpiKind kind, void *ws, hipStream_t st);
hipError_t launch_gemm_f16(GemmArgs g, bool a_mc, bool b_mc, EpiKind kind, void *ws, hipStream_t st);
size_t gemm_scratch_bytes(const GemmArgs &g, EpiKind kind);

struct TilePlan {
  int tiles_m, tiles_n, tiles, splits;  // tiles: of one batch and part
  bool lower;
  int tile;    // rows and columns: 256, 128 or 64
  int groups;  // of waves that share a tile's contraction: 1, or 2 (128) or 4 (64)
};
TilePlan plan_tiles(const GemmArgs &g, EpiKind kind);

// Products of at most kSkinnyRows rows, read where they lie (dense_skinny.hip):
// x [M][K], w [N][K]; a gated product's up rows begin up_at elements further.
constexpr int kSkinnyRows = 64;
struct SkinnyArgs {
  const void *x, *w;
  long long ldx, ldw, up_at;
  int M, N, K;
  Epi epi;
};
hipError_t launch_skinny(const SkinnyArgs &a, int fmt, bool gated, hipStream_t st);

inline long long round8(long long n) { return (n + 7) & ~7LL; }

}  // namespace dense
}  // namespace pdr
