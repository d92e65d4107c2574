// The few-row forward products of one matrix: instances and launches of ffn_skinny.hpp.
#include "ffn_skinny.hpp"

namespace llmint8 {
namespace ffn {

template <class C>
__global__ __launch_bounds__(64 * kSkWaves, 1) void k_ffn_skinny(FfnGemm a) {
  extern __shared__ u32x4 smem_v[];
  // the row groups of a tile, then the tiles, then the parts in consecutive places of
  // an XCD (see tile_at), whose L2 serves what they share
  const uint32_t tiles = (uint32_t)((a.N + C::CB - 1) / C::CB);
  const uint32_t groups = (uint32_t)((a.M + 16 * C::MT - 1) / (16 * C::MT));
  const uint32_t place = xcd_place(blockIdx.x, gridDim.x);
  skinny_block<C>(a, (int)(place / (groups * tiles)), (int64_t)(place % groups) * (16 * C::MT),
                  (int64_t)(place / groups % tiles) * C::CB, (uint8_t *)smem_v);
}

template <class C>
hipError_t launch_skinny_cfg(const FfnGemm &a, hipStream_t s) {
  auto *kern = k_ffn_skinny<C>;
  hipError_t e = hipFuncSetAttribute((const void *)kern,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  const int64_t tiles = (a.N + C::CB - 1) / C::CB, groups = (a.M + 16 * C::MT - 1) / (16 * C::MT);
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * groups * a.ksplit)), dim3(64 * kSkWaves), C::LDS, s, a);
  return hipGetLastError();
}

// All but two shapes: the joined sums of 128 gated columns and 64 rows would not fit
// in LDS, and 32 columns by 64 rows are hardly ever the fastest.
template <class T, bool GATED, int MT>
hipError_t launch_skinny_cols(const FfnGemm &a, int cols, hipStream_t s) {
  if constexpr (!(GATED && MT == 4))
    if (cols == 128) return launch_skinny_cfg<SkinnyCfg<T, GATED, MT, 128>>(a, s);
  if constexpr (MT != 4)
    if (cols == 32) return launch_skinny_cfg<SkinnyCfg<T, GATED, MT, 32>>(a, s);
  return launch_skinny_cfg<SkinnyCfg<T, GATED, MT, 64>>(a, s);
}

template <class T, bool GATED>
hipError_t launch_skinny(const FfnGemm &a, int rows, int cols, hipStream_t s) {
  if (rows == 16) return launch_skinny_cols<T, GATED, 1>(a, cols, s);
  if (rows == 32) return launch_skinny_cols<T, GATED, 2>(a, cols, s);
  return launch_skinny_cols<T, GATED, 4>(a, cols, s);
}

}  // namespace ffn

hipError_t launch_ffn_skinny(int dtype, bool gated, const FfnGemm &a, int rows, int cols,
                             hipStream_t s) {
  using namespace ffn;
  if (gated)
    return dtype == LLMINT8_FP16 ? launch_skinny<Half, true>(a, rows, cols, s)
                                 : launch_skinny<Bfloat, true>(a, rows, cols, s);
  return dtype == LLMINT8_FP16 ? launch_skinny<Half, false>(a, rows, cols, s)
                               : launch_skinny<Bfloat, false>(a, rows, cols, s);
}

}  // namespace llmint8
