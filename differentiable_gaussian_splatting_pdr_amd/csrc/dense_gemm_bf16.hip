// dense_gemm_bf16.hip -- the products of bf16 operands: bf16 tensors and the
// planes of split fp32 tensors.
#include "dense_gemm_launch.hpp"

namespace pdr {
namespace dense {

hipError_t launch_gemm_bf16(GemmArgs g, bool a_mc, bool b_mc, EpiKind kind, void *ws,
                            hipStream_t st) {
  if (kind == kEpiGated) return launch_one<kBf16, false, false, kEpiGated>(g, ws, st);
  if (kind == kEpiGatedGrad) return launch_one<kBf16, false, true, kEpiGatedGrad>(g, ws, st);
  if (a_mc) return launch_one<kBf16, true, true, kEpiLinear>(g, ws, st);
  if (b_mc) return launch_one<kBf16, false, true, kEpiLinear>(g, ws, st);
  return launch_one<kBf16, false, false, kEpiLinear>(g, ws, st);
}

}  // namespace dense
}  // namespace pdr
