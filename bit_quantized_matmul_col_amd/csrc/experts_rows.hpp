// Products over the rows that a router sent to each expert, in square tiles: every tile is one
// of ffn_gemm.hpp, of the rows of one expert. Tiles of 256 rows, whose last of an expert has
// half of them where that is enough, or of 128.
#pragma once

#include "experts_tile.hpp"

namespace llmint8 {
namespace ffn {

template <class C1, class C2>
__global__ __launch_bounds__(C1::THREADS, 2) void k_expert_rows(FfnGemm a, const int32_t *offsets,
                                                               int E, int64_t bstride, int cols) {
  static_assert(C1::THREADS == C2::THREADS && C1::OUTN == C2::OUTN, "one launch");
  extern __shared__ u32x4 smem_v[];
  ExpertTile t;
  if (!expert_tile<C1::BM>(offsets, E, a.all_rows, cols, 1, gemm_detail::kGroupM, blockIdx.x,
                           t))
    return;
  FfnGemm g = expert_product(a, t, bstride);
  // what no such product has, known to the compiler
  g.outs = g.ksplit = 1;
  g.bias = g.residual = nullptr;
  g.zs[0] = g.zs[1] = nullptr;
  if constexpr (C1::GATED)
    g.segs = 1;
  else
    g.act = LLMINT8_ACT_NONE, g.z[0] = nullptr;
  if (C1::BM == C2::BM || t.rows > C2::BM)
    ffn_tile<C1>(g, 0, t.tn, 1, (uint8_t *)smem_v);
  else
    ffn_tile<C2>(g, 0, t.tn, 1, (uint8_t *)smem_v);
}

template <class C1, class C2>
hipError_t launch_rows_cfg(const FfnGemm &a, const Pairs &p, int64_t bstride, hipStream_t s) {
  auto *kern = k_expert_rows<C1, C2>;
  constexpr int LDS = C1::LDS > C2::LDS ? C1::LDS : C2::LDS;
  hipError_t e =
      hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (e != hipSuccess) return e;
  const int64_t cols = (a.N + C1::OUTN - 1) / C1::OUTN;
  const int64_t blocks = expert_tiles(a.M, p.E, C1::BM) * cols;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(C1::THREADS), LDS, s, a, p.offsets, p.E,
                     bstride, (int)cols);
  return hipGetLastError();
}

template <class T, Lay LA, Lay LB, bool GATED>
hipError_t launch_rows_order(const FfnGemm &a, const Pairs &p, int64_t bstride, int tile,
                             hipStream_t s) {
  using Wide = Cfg<T, LA, LB, GATED, 256, 256, 2, 4>;
  using Half_ = Cfg<T, LA, LB, GATED, 128, 256, 2, 4>;
  using Small = Cfg<T, LA, LB, GATED, 128, 128, 2, 2>;
  return tile == 256 ? launch_rows_cfg<Wide, Half_>(a, p, bstride, s)
                     : launch_rows_cfg<Small, Small>(a, p, bstride, s);
}

}  // namespace ffn
}  // namespace llmint8
