// dense_gemm_launch.hpp -- instantiates the products of one operand format.
#pragma once

#include "dense_internal.hpp"

namespace pdr {
namespace dense {

// Sums the splits of one product and applies its epilogue: one thread per 8
// columns.
template <int EPI>
__global__ __launch_bounds__(256) void k_join_splits(GemmArgs g, int groups) {
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
  const int batch = blockIdx.z;
  const long long m = at / groups;
  if (m >= g.M) return;
  const int n = (int)(at - m * groups) * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < g.splits; ++s) {
    float w[8];
    load8(g.partial + ((long long)s * g.batches + batch) * g.M * g.N, kF32, m * g.N + n, g.N - n,
          (g.N & 3) == 0, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += w[i];
  }
  epi_apply<EPI>(g.epi, batch, (int)m, n, g.N, v);
}

template <int FMT, bool A_MC, bool B_MC, int EPI>
hipError_t launch_one(GemmArgs g, void *ws, hipStream_t st) {
  const TilePlan p = plan_tiles(g, (EpiKind)EPI);
  g.tiles_m = p.tiles_m;
  g.tiles_n = p.tiles_n;
  g.splits = p.splits;
  g.partial = (float *)ws;
  if (g.M <= 0 || g.epi.store_n <= 0 || g.batches <= 0) return hipSuccess;
  const dim3 grid((unsigned)(p.tiles_m * p.tiles_n), (unsigned)p.splits, (unsigned)g.batches);
  hipLaunchKernelGGL((k_gemm<FMT, 128, 128, 2, 2, A_MC, B_MC, EPI>), grid, dim3(256), 0, st, g);
  if (p.splits > 1) {
    if constexpr (EPI != kEpiGated) {
      const int groups = (g.epi.store_n + 7) / 8;
      const long long threads = (long long)groups * g.M;
      hipLaunchKernelGGL((k_join_splits<EPI>),
                         dim3((unsigned)((threads + 255) / 256), 1, (unsigned)g.batches), dim3(256),
                         0, st, g, groups);
    }
  }
  return hipGetLastError();
}

}  // namespace dense
}  // namespace pdr
