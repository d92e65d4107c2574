// dW_e = A_e^T B_e of every expert, A and B its rows: the reduction runs over the rows, as many
// as the router sent, none at all for some (whose gradient is zeros).
#include "experts_core.hpp"

namespace llmint8 {
namespace ffn {

struct ExpertGradArgs {
  FfnGemm a;
  const int32_t *offsets;
  int64_t ystride;
  int E, tiles_m, cols;  // experts, tile rows and tile columns of one
};

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_expert_grad_w(ExpertGradArgs args) {
  extern __shared__ u32x4 smem_v[];
  // an expert's tiles one after the other, ordered as in tile_at
  auto find = [&](const auto *k, uint32_t place, Job &j) {
    constexpr uint32_t GM = gemm_detail::kGroupM;
    const uint32_t cols = (uint32_t)k->cols, tiles_m = (uint32_t)k->tiles_m;
    const uint32_t per = tiles_m * cols, v = place % per;
    const int e = (int)(place / per);
    const uint32_t g0 = v / (GM * cols) * GM, in = v % (GM * cols);
    const uint32_t gm = tiles_m - g0 < GM ? tiles_m - g0 : GM;
    const int64_t m0 = (int64_t)(g0 + in % gm) * C::BM;
    int tn = (int)(in / gm);
    const int tn1 = (int)((k->a.N + C::OUTN - 1) / C::OUTN), out = tn >= tn1;
    if (out) tn -= tn1;
    const int64_t n0 = (int64_t)tn * C::OUTN;
    // by the scalar cache, which holds the offsets after the first tiles
    const int32_t __attribute__((address_space(4))) *const off =
        (const int32_t __attribute__((address_space(4))) *)k->offsets;
    auto at = [&](int o) { return o < 0 ? 0 : o < k->a.all_rows ? o : (int)k->a.all_rows; };
    const int64_t first = at(off[e]);
    const int n = at(off[e + 1]) - (int)first;
    j.a[0] = j.a[1] = (const uint8_t *)((const uint16_t *)k->a.a[0] + first * k->a.lda + m0);
    j.b[0] = j.b[1] = (const uint8_t *)((const uint16_t *)(out ? k->a.b[1] : k->a.b[0]) +
                                        first * k->a.ldb + n0);
    j.K = n > 0 ? n : 0;
    j.pairs = nullptr;
    j.out = Job::Out{(out ? k->a.y[1] : k->a.y[0]) + e * k->ystride + m0 * k->a.ldy + n0, 0, 0,
                     (int)(k->a.M - m0 < C::BM ? k->a.M - m0 : C::BM), (int)(k->a.N - n0)};
  };
  run_tiles<C, ExpertGradArgs>(args.a.lda, args.a.ldb, 1,
                               (uint32_t)(args.E * args.tiles_m * args.cols), find,
                               (uint8_t *)smem_v);
}

template <class C>
hipError_t launch_grad_w_cfg(const FfnGemm &a, const Pairs &p, int64_t ystride, hipStream_t s) {
  auto *kern = k_expert_grad_w<C>;
  constexpr int LDS = tiles_lds<C>();
  hipError_t e =
      hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (e != hipSuccess) return e;
  const int64_t tiles_m = (a.M + C::BM - 1) / C::BM, cols = (a.N + C::OUTN - 1) / C::OUTN * a.outs;
  const int64_t tiles = tiles_m * cols * p.E, room = kFfnCus * (C::BM == 256 ? 1 : 2);
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles < room ? tiles : room)), dim3(C::THREADS), LDS, s,
                     ExpertGradArgs{a, p.offsets, ystride, p.E, (int)tiles_m, (int)cols});
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
