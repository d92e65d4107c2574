// Both products of a backward pass in one launch, dX = dZ W^T (or dG Wg^T + dU Wu^T)
// and dW = X^T dZ (or X^T dG and X^T dU). They are independent of each other, and
// their tiles differ in length by the ratio of the reductions (N against M), so
// together they fill the chip where either alone leaves a last round half empty or
// needs a split reduction; the epilogues of the short ones run beside the k loops
// of the long ones. The longer tiles come first. The blocks that end the bias gradient
// come last, on CUs that the tiles leave free, rather than in a launch of their own
// (64 x 1024 x 1024 with activation and bias 19.3 -> 17.7 us, 1500 x 2048 x 2048 43.4 ->
// 40.6, and 4 us less of a host's time; 2048 x 4096 x 4096 even).
#include "ffn_gemm.hpp"

namespace llmint8 {
namespace ffn {

template <class CX, class CW>
__global__ __launch_bounds__(CX::THREADS, 2) void k_ffn_back(FfnGemm x, FfnGemm w,
                                                            BiasJoin j, uint32_t blocks_x,
                                                            uint32_t blocks_w, int x_first) {
  static_assert(CX::THREADS == CW::THREADS, "one launch");
  extern __shared__ u32x4 smem_v[];
  if (blockIdx.x >= blocks_x + blocks_w)
    return join_bias<CX::THREADS>(j, blockIdx.x - blocks_x - blocks_w, (float *)smem_v);
  const uint32_t first = x_first ? blocks_x : blocks_w, b = blockIdx.x;
  const bool is_x = (b < first) == (x_first != 0);
  const uint32_t bid = b < first ? b : b - first;
  if (is_x)
    ffn_tile<CX>(x, bid, 0, (int)((x.N + CX::OUTN - 1) / CX::OUTN), (uint8_t *)smem_v);
  else
    ffn_tile<CW>(w, bid, 0, (int)((w.N + CW::OUTN - 1) / CW::OUTN) * w.outs, (uint8_t *)smem_v);
}

template <class C>
uint32_t blocks_of(const FfnGemm &a) {
  return (uint32_t)((a.M + C::BM - 1) / C::BM * ((a.N + C::OUTN - 1) / C::OUTN) * a.outs *
                    a.ksplit);
}

template <class T, int BM, int BN, int NWM, int NWN, int NST>
hipError_t launch_back(const FfnGemm &x, const FfnGemm &w, const BiasJoin &j, hipStream_t s) {
  using CX = Cfg<T, Lay::RowK, Lay::RowK, false, BM, BN, NWM, NWN, NST>;
  using CW = Cfg<T, Lay::ColK, Lay::ColK, false, BM, BN, NWM, NWN, NST>;
  auto *kern = k_ffn_back<CX, CW>;
  constexpr int LDS = CX::LDS > CW::LDS ? CX::LDS : CW::LDS;
  hipError_t e =
      hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (e != hipSuccess) return e;
  const uint32_t bx = blocks_of<CX>(x), bw = blocks_of<CW>(w);
  const int x_first = x.K * x.segs / x.ksplit >= w.K / w.ksplit;
  const uint32_t bj = j.dbias ? (uint32_t)((j.N + 63) / 64) : 0;
  hipLaunchKernelGGL(kern, dim3(bx + bw + bj), dim3(CX::THREADS), LDS, s, x, w, j, bx, bw, x_first);
  return hipGetLastError();
}

template <class T>
hipError_t launch_back_tile(const FfnGemm &x, const FfnGemm &w, const BiasJoin &j, int tile,
                            hipStream_t s) {
  if (tile == 256) return launch_back<T, 256, 256, 2, 4, 2>(x, w, j, s);
  using C = Cfg<T, Lay::RowK, Lay::RowK, false, 128, 128, 2, 2>;
  return deep_ring((int64_t)blocks_of<C>(x) + blocks_of<C>(w))
             ? launch_back<T, 128, 128, 2, 2, 4>(x, w, j, s)
             : launch_back<T, 128, 128, 2, 2, 2>(x, w, j, s);
}

}  // namespace ffn

hipError_t launch_ffn_back(int dtype, const FfnGemm &x, const FfnGemm &w, const BiasJoin &j,
                           int tile, hipStream_t s) {
  return dtype == LLMINT8_FP16 ? ffn::launch_back_tile<Half>(x, w, j, tile, s)
                               : ffn::launch_back_tile<Bfloat>(x, w, j, tile, s);
}

}  // namespace llmint8
