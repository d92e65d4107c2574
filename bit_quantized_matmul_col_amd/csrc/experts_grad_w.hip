// dW_e = A_e^T B_e of every expert, A and B its rows: the reduction runs over the rows, as many
// as the router sent, none at all for some (whose gradient is zeros).
#include "experts_tile.hpp"

namespace llmint8 {
namespace ffn {

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_expert_grad_w(FfnGemm a, const int32_t *offsets,
                                                                int64_t rows, int64_t ystride,
                                                                int tiles_m, int cols) {
  extern __shared__ u32x4 smem_v[];
  const uint32_t per = (uint32_t)(tiles_m * cols), place = xcd_place(blockIdx.x, gridDim.x);
  const int e = (int)(place / per);
  // the tiles of one expert in consecutive places, ordered as in tile_at
  constexpr uint32_t GM = gemm_detail::kGroupM;
  const uint32_t v = place % per, first = v / (GM * cols) * GM, in = v % (GM * cols);
  const uint32_t gm = tiles_m - first < GM ? tiles_m - first : GM;
  const int tm = (int)(first + in % gm), tn = (int)(in / gm);
  auto at = [&](int i) {
    const int64_t o = offsets[i];
    return o < 0 ? (int64_t)0 : o < rows ? o : rows;
  };
  const int64_t r0 = at(e), r1 = at(e + 1), m0 = (int64_t)tm * C::BM;
  FfnGemm g = a;
  g.a[0] = (const uint16_t *)a.a[0] + r0 * a.lda + m0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    g.b[i] = (const uint16_t *)a.b[i] + r0 * a.ldb;
    g.y[i] = a.y[i] + e * ystride + m0 * a.ldy;
  }
  g.K = r1 > r0 ? r1 - r0 : 0;
  g.M = a.M - m0 < C::BM ? a.M - m0 : C::BM;
  ffn_tile<C>(g, 0, tn, 1, (uint8_t *)smem_v);
}

template <class C>
hipError_t launch_grad_w_cfg(const FfnGemm &a, const Pairs &p, int64_t ystride, hipStream_t s) {
  auto *kern = k_expert_grad_w<C>;
  hipError_t e = hipFuncSetAttribute((const void *)kern,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  const int64_t tiles_m = (a.M + C::BM - 1) / C::BM, cols = (a.N + C::OUTN - 1) / C::OUTN * a.outs;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles_m * cols * p.E)), dim3(C::THREADS), C::LDS, s, a,
                     p.offsets, p.rows(), ystride, (int)tiles_m, (int)cols);
  return hipGetLastError();
}

template <class T>
hipError_t launch_grad_w(const FfnGemm &a, const Pairs &p, int64_t ystride, hipStream_t s) {
  return launch_grad_w_cfg<Cfg<T, Lay::ColK, Lay::ColK, false, 256, 256, 2, 4>>(a, p, ystride, s);
}

}  // namespace ffn

hipError_t launch_expert_grad_w(int dtype, const FfnGemm &a, const Pairs &p, int64_t ystride,
                                hipStream_t s) {
  return dtype == LLMINT8_FP16 ? ffn::launch_grad_w<Half>(a, p, ystride, s)
                               : ffn::launch_grad_w<Bfloat>(a, p, ystride, s);
}

}  // namespace llmint8
