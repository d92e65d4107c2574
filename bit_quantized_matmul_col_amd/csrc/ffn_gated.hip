// H = act(X Wg) * (X Wu): one block computes the same columns of both products,
// so that the activation and the product run on its accumulators.
#include "ffn_gemm.hpp"

namespace llmint8 {

hipError_t launch_ffn_gated(int dtype, const FfnGemm &a, int tile, hipStream_t s) {
  using namespace ffn;
  return dtype == LLMINT8_FP16 ? launch_order<Half, Lay::RowK, Lay::ColK, true>(a, tile, s)
                               : launch_order<Bfloat, Lay::RowK, Lay::ColK, true>(a, tile, s);
}

}  // namespace llmint8
