// The experts' forward products where an expert has few rows (single tokens, decoding
// batches): blocks of ffn_skinny.hpp, a group of up to 16, 32 or 64 rows of one expert by 64
// or 128 columns, which read that expert's weights once. The weights of the experts that
// were chosen bound it.
#include "experts_tile.hpp"
#include "ffn_skinny.hpp"

namespace llmint8 {
namespace ffn {

template <class C>
__global__ __launch_bounds__(64 * kSkWaves, 1) void k_expert_skinny(FfnGemm a,
                                                                   const int32_t *offsets, int E,
                                                                   int64_t bstride, int cols) {
  extern __shared__ u32x4 smem_v[];
  // The launch has blocks for the worst distribution of the rows; those behind the row groups
  // that there are end here. All row groups, column by column: those of one expert share
  // its weights in L2.
  const uint32_t groups = count_tiles<16 * C::MT>(offsets, E, a.all_rows);
  const uint32_t plane = groups * (uint32_t)cols, blocks = plane * (uint32_t)a.ksplit;
  if (blockIdx.x >= blocks) return;
  const uint32_t place = xcd_place(blockIdx.x, blocks);
  ExpertTile t;
  find_rows<16 * C::MT>(offsets, E, a.all_rows, (int)(place % plane % groups), t);
  t.tn = (int)(place % plane / groups), t.part = (int)(place / plane);
  skinny_block<C>(expert_product(a, t, bstride), t.part, 0, (int64_t)t.tn * C::CB,
                  (uint8_t *)smem_v);
}

template <class C>
hipError_t launch_few_cfg(const FfnGemm &a, const Pairs &p, int64_t bstride, hipStream_t s) {
  auto *kern = k_expert_skinny<C>;
  hipError_t e = hipFuncSetAttribute((const void *)kern,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  const int64_t cols = (a.N + C::CB - 1) / C::CB;
  const int64_t blocks = expert_tiles(a.M, p.E, 16 * C::MT) * cols * a.ksplit;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * kSkWaves), C::LDS, s, a, p.offsets,
                     p.E, bstride, (int)cols);
  return hipGetLastError();
}

template <class T, bool GATED, int MT>
hipError_t launch_few_cols(const FfnGemm &a, const Pairs &p, int64_t bstride, int cols,
                           hipStream_t s) {
  if constexpr (!(GATED && MT == 4))
    if (cols == 128) return launch_few_cfg<SkinnyCfg<T, GATED, MT, 128, true>>(a, p, bstride, s);
  return launch_few_cfg<SkinnyCfg<T, GATED, MT, 64, true>>(a, p, bstride, s);
}

template <class T, bool GATED>
hipError_t launch_few(const FfnGemm &a, const Pairs &p, int64_t bstride, const FfnPlan &plan,
                      hipStream_t s) {
  if (plan.rows == 16) return launch_few_cols<T, GATED, 1>(a, p, bstride, plan.tile, s);
  if (plan.rows == 32) return launch_few_cols<T, GATED, 2>(a, p, bstride, plan.tile, s);
  return launch_few_cols<T, GATED, 4>(a, p, bstride, plan.tile, s);
}

}  // namespace ffn

hipError_t launch_expert_skinny(int dtype, bool gated, const FfnGemm &a, const Pairs &p,
                                int64_t bstride, const FfnPlan &plan, hipStream_t s) {
  using namespace ffn;
  if (gated)
    return dtype == LLMINT8_FP16 ? launch_few<Half, true>(a, p, bstride, plan, s)
                                 : launch_few<Bfloat, true>(a, p, bstride, plan, s);
  return dtype == LLMINT8_FP16 ? launch_few<Half, false>(a, p, bstride, plan, s)
                               : launch_few<Bfloat, false>(a, p, bstride, plan, s);
}

}  // namespace llmint8
