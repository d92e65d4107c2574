// Which part of a routed product a block computes.
#pragma once

#include "experts.hpp"
#include "ffn_gemm.hpp"

namespace llmint8 {
namespace ffn {

// Rows row0 .. row0 + rows - 1 of all, all of one expert's; a column tile; a part of the
// reduction.
struct ExpertTile {
  int expert, row0, rows, tn, part;
};

// Block bid's tile of up to BM rows, or false past the last one: the counts of rows are on the
// GPU alone, so that a launch has blocks for the worst distribution, and the ones
// behind the tiles that there are end here. Every wave finds the tile by itself, 64 experts at a
// time: 0.3 us of a block's time for 64 experts, against a launch that would write
// the tiles down.
//
// The tiles go to the XCDs as in tile_at, where `group` neighbouring tile rows take a column
// after the other (0: all of them). The offsets are clamped to the rows that the buffers have.
template <int BM>
__device__ inline bool expert_tile(const int32_t *offsets, int E, int64_t rows, int cols,
                                   int parts, int group, uint32_t bid, ExpertTile &t) {
  const int lane = threadIdx.x & 63;
  auto at = [&](int e) {
    const int o = offsets[e < E ? e : E];
    return o < 0 ? 0 : o < rows ? o : (int)rows;
  };
  auto tiles_of = [&](int e, int &first, int &n) {
    first = at(e), n = at(e + 1) - first;
    n = n > 0 ? n : 0;
    return (n + BM - 1) / BM;
  };
  int total = 0, first, n;
  for (int e = lane; e < E; e += 64) total += tiles_of(e, first, n);
  const uint32_t tiles = (uint32_t)__builtin_amdgcn_readfirstlane(wave_sum(total));
  const uint32_t blocks = tiles * (uint32_t)(cols * parts);
  if (bid >= blocks) return false;
  const uint32_t place = xcd_place(bid, blocks), plane = tiles * (uint32_t)cols;
  t.part = (int)(place / plane);
  const uint32_t v = place % plane, GM = group ? (uint32_t)group : tiles;
  const uint32_t g0 = v / (GM * cols) * GM, in = v % (GM * cols);
  const uint32_t gm = tiles - g0 < GM ? tiles - g0 : GM;
  const int tm = (int)(g0 + in % gm);
  t.tn = (int)(in / gm);
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane, c = tiles_of(e, first, n);
    int upto = c;  // tiles of the experts e0 .. e
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(upto, off, kWave);
      upto += lane >= off ? o : 0;
    }
    const uint64_t hit = __ballot(before + upto > tm);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int r = (tm - before - (__builtin_amdgcn_readlane(upto, l) -
                                    __builtin_amdgcn_readlane(c, l))) * BM;
      t.expert = e0 + l;
      t.row0 = __builtin_amdgcn_readlane(first, l) + r;
      t.rows = __builtin_amdgcn_readlane(n, l) - r;
      t.rows = t.rows < BM ? t.rows : BM;
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// The blocks that a launch needs whatever the distribution: every expert with rows may end
// in a tile that is not full.
inline int64_t expert_tiles(int64_t rows, int64_t E, int BM) {
  return rows / BM + (E < rows ? E : rows);
}

// The product of one tile as one of its own, from the one over all rows.
__device__ inline FfnGemm expert_product(const FfnGemm &a, const ExpertTile &t, int64_t bstride) {
  FfnGemm g = a;
  const int64_t r = t.row0;
  if (!a.topk)
#pragma unroll
    for (int i = 0; i < 2; ++i) g.a[i] = (const uint16_t *)a.a[i] + r * a.lda;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    g.b[i] = (const uint16_t *)a.b[i] + t.expert * bstride;
    g.z[i] = a.z[i] ? (uint16_t *)a.z[i] + r * a.ldz : nullptr;
  }
  g.y[0] = a.y[0] + r * a.ldy;
  g.part = a.part + r * a.N;
  g.pairs = a.pairs + r;
  g.M = t.rows;
  // rows that are read as they are end with the tile's last
  if (!a.topk) g.a_rows = t.rows;
  return g;
}

}  // namespace ffn
}  // namespace llmint8
