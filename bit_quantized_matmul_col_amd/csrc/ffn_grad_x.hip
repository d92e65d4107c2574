// dX = dZ W^T, and dG Wg^T + dU Wu^T as one reduction of two segments.
#include "ffn_gemm.hpp"

namespace llmint8 {

hipError_t launch_ffn_grad_x(int dtype, const FfnGemm &a, int tile, hipStream_t s) {
  using namespace ffn;
  return dtype == LLMINT8_FP16 ? launch_order<Half, Lay::RowK, Lay::RowK, false>(a, tile, s)
                               : launch_order<Bfloat, Lay::RowK, Lay::RowK, false>(a, tile, s);
}

}  // namespace llmint8
