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

// The rows of expert e: the first and how many, within the rows that the buffers have.
__device__ inline void expert_rows(const int32_t *offsets, int E, int64_t rows, int e, int &first,
                                   int &n) {
  auto at = [&](int i) {
    const int o = offsets[i < E ? i : E];
    return o < 0 ? 0 : o < rows ? o : (int)rows;
  };
  first = at(e), n = at(e + 1) - first;
  n = n > 0 ? n : 0;
}

// How many tiles of up to BM rows the experts have. The counts of rows are on the GPU alone, so
// every wave adds them up by itself, 64 experts at a time (0.3 us for 64 of them, against a launch
// that would write the tiles down).
template <int BM>
__device__ inline uint32_t count_tiles(const int32_t *offsets, int E, int64_t rows) {
  int total = 0, first, n;
  for (int e = threadIdx.x & 63; e < E; e += 64) {
    expert_rows(offsets, E, rows, e, first, n);
    total += (n + BM - 1) / BM;
  }
  return (uint32_t)__builtin_amdgcn_readfirstlane(wave_sum(total));
}

// Tile row tm of them.
template <int BM>
__device__ inline void find_rows(const int32_t *offsets, int E, int64_t rows, int tm,
                                 ExpertTile &t) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    int first, n;
    expert_rows(offsets, E, rows, e0 + lane, first, n);
    if (e0 + lane >= E) n = 0;
    const int c = (n + BM - 1) / BM;
    int upto = c;  // tiles of the experts e0 .. e0 + lane
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
      return;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  t.expert = t.row0 = t.rows = 0;  // not reached: tm is below their number
}

// Where the experts' rows and tiles begin, in LDS, for blocks that work through many tiles.
// [starts: E + 1][first rows: E][rows: E]
struct ExpertTable {
  int32_t *starts, *first, *rows;
  int E;
  __device__ ExpertTable(void *at, int experts)
      : starts((int32_t *)at), first(starts + experts + 1), rows(first + experts), E(experts) {}
  static int bytes(int64_t E) { return (int)((3 * E + 1) * 4); }

  // Called by the whole block; a barrier is still to come.
  template <int BM>
  __device__ void fill(const int32_t *offsets, int64_t all_rows) {
    if (threadIdx.x >= 64) return;
    const int lane = threadIdx.x;
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      int f, n;
      expert_rows(offsets, E, all_rows, e0 + lane, f, n);
      if (e0 + lane >= E) n = 0;
      int upto = (n + BM - 1) / BM;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(upto, off, kWave);
        upto += lane >= off ? o : 0;
      }
      if (e0 + lane < E) {
        starts[e0 + lane + 1] = before + upto;
        first[e0 + lane] = f, rows[e0 + lane] = n;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (lane == 0) starts[0] = 0;
  }
  __device__ uint32_t tiles() const { return (uint32_t)__builtin_amdgcn_readfirstlane(starts[E]); }

  // The expert of tile row tm, below tiles().
  __device__ int expert_of(int tm) const {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // no register beside a loop's for what follows from it
    for (int e0 = 0; e0 < E; e0 += 64) {
      const uint64_t past = __ballot(e0 + lane < E && starts[e0 + lane + 1] > tm);
      if (past) return e0 + __builtin_ctzll(past);
    }
    return 0;  // not reached
  }
  __device__ int start(int e) const { return __builtin_amdgcn_readfirstlane(starts[e]); }
  __device__ int tile_rows(int e) const { return start(e + 1) - start(e); }

  // Tile row j of expert e.
  template <int BM>
  __device__ void rows_of(int e, int j, ExpertTile &t) const {
    t.expert = e;
    t.row0 = __builtin_amdgcn_readfirstlane(first[e]) + j * BM;
    t.rows = __builtin_amdgcn_readfirstlane(rows[e]) - j * BM;
    t.rows = t.rows < BM ? t.rows : BM;
  }
};

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
