// Products over the rows that a router sent to each expert, in square tiles of 256 or 128 rows of
// one expert.
#pragma once

#include "experts_core.hpp"

namespace llmint8 {
namespace ffn {

struct ExpertRowsArgs {
  FfnGemm a;
  const int32_t *offsets;
  int64_t bstride;
  int E, cols;  // experts, tile columns
};

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_expert_rows(ExpertRowsArgs args) {
  extern __shared__ u32x4 smem_v[];
  ExpertTable table((uint8_t *)smem_v + tiles_lds<C>(), args.E);
  table.fill<C::BM>(args.offsets, args.a.all_rows);
  __syncthreads();
  // (offsets that no plan writes would count rows twice)
  const uint32_t most = (uint32_t)(args.a.all_rows / C::BM + args.E);
  const uint32_t found = table.tiles();
  const uint32_t tiles = (found < most ? found : most) * (uint32_t)args.cols;
  // The tiles of an expert in consecutive places, its tile rows in groups of 8, a group column
  // by column, as in tile_at: neighbours share weights and rows, and the weights, which
  // are most of what is read, leave HBM once.
  auto find = [&](const auto *k, uint32_t place, Job &j) {
    constexpr uint32_t GM = gemm_detail::kGroupM;
    const uint32_t cols = (uint32_t)k->cols;
    const int e = table.expert_of((int)(place / cols));
    const uint32_t rows = (uint32_t)table.tile_rows(e);
    const uint32_t v = place - (uint32_t)table.start(e) * cols;
    const uint32_t g0 = v / (GM * cols) * GM, in = v % (GM * cols);
    const uint32_t gm = rows - g0 < GM ? rows - g0 : GM;
    const int64_t n0 = (int64_t)(in / gm) * C::OUTN;
    ExpertTile t;
    table.rows_of<C::BM>(e, (int)(g0 + in % gm), t);
    const int64_t r = t.row0;
    const int64_t b0 = t.expert * k->bstride + (C::LB == Lay::RowK ? n0 * k->a.ldb : n0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      j.a[q] = (const uint8_t *)((const uint16_t *)k->a.a[q] + (k->a.topk ? 0 : r * k->a.lda));
      j.b[q] = (const uint8_t *)((const uint16_t *)k->a.b[q] + b0);
    }
    j.K = (int)k->a.K;
    j.pairs = k->a.pairs + r;
    j.out = Job::Out{k->a.y[0] + r * k->a.ldy + n0, t.row0, (int)n0, t.rows, (int)(k->a.N - n0)};
  };
  run_tiles<C, ExpertRowsArgs>(args.a.lda, args.a.ldb, args.a.segs, tiles, find,
                               (uint8_t *)smem_v);
}

template <class C>
hipError_t launch_rows_cfg(const FfnGemm &a, const Pairs &p, int64_t bstride, hipStream_t s) {
  auto *kern = k_expert_rows<C>;
  const int lds = tiles_lds<C>() + ExpertTable::bytes(p.E);
  hipError_t e =
      hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  const int64_t cols = (a.N + C::OUTN - 1) / C::OUTN, most = expert_tiles(a.M, p.E, C::BM) * cols;
  const int64_t room = kFfnCus * (C::BM == 256 ? 1 : 2);
  hipLaunchKernelGGL(kern, dim3((unsigned)(most < room ? most : room)), dim3(C::THREADS), lds, s,
                     ExpertRowsArgs{a, p.offsets, bstride, p.E, (int)cols});
  return hipGetLastError();
}

template <class T, Lay LA, Lay LB, bool GATED>
hipError_t launch_rows_order(const FfnGemm &a, const Pairs &p, int64_t bstride, int tile,
                             hipStream_t s) {
  return tile == 256 ? launch_rows_cfg<Cfg<T, LA, LB, GATED, 256, 256, 2, 4>>(a, p, bstride, s)
                     : launch_rows_cfg<Cfg<T, LA, LB, GATED, 128, 128, 2, 2>>(a, p, bstride, s);
}

}  // namespace ffn
}  // namespace llmint8
