// dW = X^T dZ, and X^T dG and X^T dU side by side in one launch.
#include "ffn_gemm.hpp"

namespace llmint8 {

hipError_t launch_ffn_grad_w(int dtype, const FfnGemm &a, int tile, hipStream_t s) {
  using namespace ffn;
  return dtype == LLMINT8_FP16 ? launch_order<Half, Lay::ColK, Lay::ColK, false>(a, tile, s)
                               : launch_order<Bfloat, Lay::ColK, Lay::ColK, false>(a, tile, s);
}

}  // namespace llmint8
