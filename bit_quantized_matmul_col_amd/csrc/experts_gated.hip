// H_r = w_r act(x Wg_e) (x Wu_e), x the row of the pair's token.
#include "experts_rows.hpp"

namespace llmint8 {

hipError_t launch_expert_gated(int dtype, const FfnGemm &a, const Pairs &p, int64_t bstride,
                            int tile, hipStream_t s) {
  using namespace ffn;
  return dtype == LLMINT8_FP16
             ? launch_rows_order<Half, Lay::RowKAt, Lay::ColK, true>(a, p, bstride, tile, s)
             : launch_rows_order<Bfloat, Lay::RowKAt, Lay::ColK, true>(a, p, bstride, tile, s);
}

}  // namespace llmint8
