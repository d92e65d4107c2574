// Y rows = H_r Wd_e, rows as they are.
#include "experts_rows.hpp"

namespace llmint8 {

hipError_t launch_expert_forward(int dtype, const FfnGemm &a, const Pairs &p, int64_t bstride,
                            int tile, hipStream_t s) {
  using namespace ffn;
  return dtype == LLMINT8_FP16
             ? launch_rows_order<Half, Lay::RowK, Lay::ColK, false>(a, p, bstride, tile, s)
             : launch_rows_order<Bfloat, Lay::RowK, Lay::ColK, false>(a, p, bstride, tile, s);
}

}  // namespace llmint8
