// What the row-streaming passes share: the grid, a thread's 8 columns of a row, and the sum
// of the parts of a split reduction.
#pragma once

#include "ffn_gemm.hpp"

namespace llmint8 {
namespace ffn_rows {

using ffn::load_f8;

constexpr int kThreads = 256;

// A block covers cx chunks of 8 columns (a power of two, 8 to 256, so that the 4
// lanes of a checkpoint block share a wave) and 256 / cx rows at a time; the
// grid's second dimension strides over the rows.
struct RowGrid {
  int cx_log2;
  dim3 grid;
};

inline RowGrid row_grid(int64_t M, int64_t N, int64_t max_rows) {
  const int64_t chunks = (N + 7) / 8;
  int lg = 3;
  while (lg < 8 && ((int64_t)1 << lg) < chunks) ++lg;
  const int64_t gx = (chunks + ((int64_t)1 << lg) - 1) >> lg, ry = kThreads >> lg;
  int64_t gy = (M + ry - 1) / ry;
  if (gy > max_rows) gy = max_rows;
  return RowGrid{lg, dim3((unsigned)gx, (unsigned)gy)};
}

constexpr int64_t kMaxGridY = 65535;

// Calls f(i, n, in) for the rows i and the first column n of this thread's
// chunks; in is false for a chunk past N (its lanes still take part in shuffles).
template <class F>
__device__ inline void for_rows(int cx_log2, int64_t M, int64_t N, F f) {
  const int t = threadIdx.x;
  const int64_t n = (((int64_t)blockIdx.x << cx_log2) + (t & ((1 << cx_log2) - 1))) * 8;
  const int64_t ry = kThreads >> cx_log2;
  for (int64_t i = blockIdx.y * ry + (t >> cx_log2); i < M; i += gridDim.y * ry) f(i, n, n < N);
}

// Sums of the parts s0, s0 + 1, ... of 8 columns, in the order of the parts; the
// loads of four parts are in flight together.
__device__ inline void join_parts(const float *p, int64_t stride, int parts, float *v) {
  for (int s = 0; s < parts; s += 4) {
    float x[4][8];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (s + q < parts) load_f8(p + (s + q) * stride, x[q]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (s + q < parts)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += x[q][e];
  }
}

}  // namespace ffn_rows
}  // namespace llmint8
