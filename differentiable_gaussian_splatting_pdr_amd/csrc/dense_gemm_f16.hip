// dense_gemm_f16.hip -- the products of fp16 operands: fp16 tensors and the
// Newton-Schulz iterates.
#include "dense_gemm_launch.hpp"

namespace pdr {
namespace dense {

hipError_t launch_gemm_f16(GemmArgs g, bool a_mc, bool b_mc, EpiKind kind, void *ws,
                           hipStream_t st) {
  if (kind == kEpiPoly) {
    if (a_mc) return launch_one<kF16, true, true, kEpiPoly>(g, ws, st);
    if (b_mc) return launch_one<kF16, false, true, kEpiPoly>(g, ws, st);
    return launch_one<kF16, false, false, kEpiPoly>(g, ws, st);
  }
  if (kind == kEpiGated) return launch_one<kF16, false, false, kEpiGated>(g, ws, st);
  if (kind == kEpiGatedGrad) return launch_one<kF16, false, true, kEpiGatedGrad>(g, ws, st);
  if (a_mc) return launch_one<kF16, true, true, kEpiLinear>(g, ws, st);
  if (b_mc) return launch_one<kF16, false, true, kEpiLinear>(g, ws, st);
  return launch_one<kF16, false, false, kEpiLinear>(g, ws, st);
}

}  // namespace dense
}  // namespace pdr
