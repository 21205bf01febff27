// dense_gemm_launch.hpp -- instantiates the products of one operand format.
#pragma once

#include "dense_internal.hpp"

namespace pdr {
namespace dense {

// Sums the parts of one product and applies its epilogue: one thread per W
// columns of a row.
template <int EPI, int W>
__global__ __launch_bounds__(256) void k_join_splits(GemmArgs g, FastDiv groups) {
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  const int batch = blockIdx.z;
  const uint32_t m = fdiv(at, groups);
  if (m >= (uint32_t)g.M) return;
  const int n = (int)(at - m * groups.d) * W;
  const long long each = (long long)g.M * g.N;
  const float *p = g.partial + batch * each + (long long)m * g.N + n;
  const Columns<EPI, W, kAsked> cols(g.epi, batch, n, g.N);
  typename Columns<EPI, W, kAsked>::Row row;
  cols.fetch(g.epi, (int)m, row);
  float v[W];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int s = 0; s < g.splits; ++s) {
    float w[W];
    if constexpr (W == 1)
      w[0] = n < g.N ? p[s * g.batches * each] : 0.f;
    else
      load8(p + s * g.batches * each, kF32, 0, g.N - n, (g.N & 3) == 0, w);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += w[i];
  }
  cols.finish(g.epi, (int)m, v, row);
}

template <int FMT, bool A_MC, bool B_MC, int EPI>
hipError_t launch_one(GemmArgs g, void *ws, hipStream_t st) {
  if (g.M <= 0 || g.epi.store_n <= 0 || g.batches <= 0) return hipSuccess;
  const TilePlan p = plan_tiles(g, (EpiKind)EPI);
  g.tiles_m = p.tiles_m;
  g.tiles_n = p.tiles_n;
  g.splits = p.splits;
  g.lower = p.lower;
  const int steps = (g.K + kBK - 1) / kBK * g.segs;
  g.steps = steps / p.splits;
  g.steps_more = steps % p.splits;
  g.band = make_fastdiv((uint32_t)(kBand * p.tiles_n));
  g.partial = (float *)ws;
  g.epi.vec = g.epi.vec && (g.epi.store_n & 7) == 0;
  const dim3 grid((unsigned)p.tiles, (unsigned)p.splits, (unsigned)g.batches);
  if (p.tile == 256)
    hipLaunchKernelGGL((k_gemm<FMT, 256, 1, A_MC, B_MC, EPI>), grid, dim3(256), 0, st, g);
  else if (p.tile == 128 && p.groups == 1)
    hipLaunchKernelGGL((k_gemm<FMT, 128, 1, A_MC, B_MC, EPI>), grid, dim3(256), 0, st, g);
  else if (p.tile == 128)
    hipLaunchKernelGGL((k_gemm<FMT, 128, 2, A_MC, B_MC, EPI>), grid, dim3(512), 0, st, g);
  else if (p.groups == 1)
    hipLaunchKernelGGL((k_gemm<FMT, 64, 1, A_MC, B_MC, EPI>), grid, dim3(256), 0, st, g);
  else
    hipLaunchKernelGGL((k_gemm<FMT, 64, 4, A_MC, B_MC, EPI>), grid, dim3(1024), 0, st, g);
  if constexpr (EPI != kEpiGated) {
    if (p.splits > 1) {
      const int w = g.epi.vec ? 8 : 1;
      const unsigned groups = (unsigned)((g.epi.store_n + w - 1) / w);
      const dim3 blocks((unsigned)(((long long)groups * g.M + 255) / 256), 1, (unsigned)g.batches);
      if (w == 8)
        hipLaunchKernelGGL((k_join_splits<EPI, 8>), blocks, dim3(256), 0, st, g, make_fastdiv(groups));
      else
        hipLaunchKernelGGL((k_join_splits<EPI, 1>), blocks, dim3(256), 0, st, g, make_fastdiv(groups));
    }
  }
  return hipGetLastError();
}

}  // namespace dense
}  // namespace pdr
