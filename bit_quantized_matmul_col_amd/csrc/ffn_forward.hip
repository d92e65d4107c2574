// Y = act(X W + b) + R: both operands as stored, W's reduction index strided.
#include "ffn_gemm.hpp"

namespace llmint8 {

hipError_t launch_ffn_forward(int dtype, const FfnGemm &a, int tile, hipStream_t s) {
  using namespace ffn;
  return dtype == LLMINT8_FP16 ? launch_order<Half, Lay::RowK, Lay::ColK, false>(a, tile, s)
                               : launch_order<Bfloat, Lay::RowK, Lay::ColK, false>(a, tile, s);
}

}  // namespace llmint8
