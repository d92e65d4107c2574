// Internal launchers of the 16-bit feed-forward kernels: the matrix product
// with its epilogue, the gated block, their backward passes and the 8-bit
// activation checkpoints. Each returns hipSuccess or the error of its launch;
// none synchronizes.
#pragma once

#include "common.hpp"

namespace llmint8 {

// Entries of a row that share one checkpoint scale.
constexpr int kCkptBlock = 32;

// A product of 16-bit matrices, out[i, n] = sum_k A(i, k) B(k, n), in one of
// three operand orders (see ffn_gemm.hpp), and what happens to the sums.
struct FfnGemm {
  const void *a[2];   // A; the second when the reduction has two segments
  int64_t lda;
  const void *b[2];   // B; the second for two segments, two outputs or the gated product
  int64_t ldb;
  int64_t M, N, K;    // rows and columns of one output, length of one segment
  int segs;           // reduction segments (2: A0 B0 + A1 B1)
  int outs;           // outputs side by side (2: A B0 and A B1)
  uint16_t *y[2];
  int64_t ldy;
  int act;
  const uint16_t *bias;      // [N]
  const uint16_t *residual;  // [M x ldr]
  int64_t ldr;
  void *z[2];     // pre-activations out: 16 bits, or 8-bit codes where zs is set
  int64_t ldz;
  uint8_t *zs[2];
  int64_t ldzs;
  float *part;    // split reduction: partial sums [ksplit][outs or 2][M][N]
  int ksplit;
  // products over the rows that a router sent to an expert (see experts.hpp): row i of
  // the product is that of the pair pairs[i], and A's row is
  //   pairs[i] / topk of a matrix of a_rows rows, or i where topk is 0.
  const int32_t *pairs;
  int topk;
  int64_t a_rows;
  const float *w;  // [pairs] what a gated row is multiplied by (null: nothing)
  int64_t all_rows;  // rows of all experts, and of a plane of partial sums
  int to_parts;      // the sums go to `part`, split or not
};

// Which kernel a product takes: square tiles of `tile` rows and columns (256 or
// 128), or the kernel for few rows with blocks of `tile` columns (32, 64 or 128) and
// `rows` rows (16, 32 or 64); and in how many parts the reduction is split.
struct FfnPlan {
  bool few;
  int tile;
  int ksplit;
  int rows;
};

// 256-tiles run in rounds of one block per CU. Where the last round of a launch
// would be less than half full, the tile columns from tail_cut() on take tiles of
// half the rows instead, twice as many blocks that finish in about half the time
// (the first tile column of the tail; `cols` where there is none).
constexpr int64_t kFfnCus = 256;
inline int64_t tail_cut(int64_t rows, int64_t cols, int64_t parts) {
  const int64_t full = rows * cols / kFfnCus;
  if (parts > 1 || full == 0 || rows * cols % kFfnCus == 0) return cols;
  const int64_t cut = full * kFfnCus / rows;
  return 2 * rows * (cols - cut) <= kFfnCus ? cut : cols;
}

// A launch of at most one 128-tile per CU runs with a ring of four stages, which covers the
// latency that the second block of a CU covers otherwise (see launch_order).
inline bool deep_ring(int64_t blocks128) { return blocks128 <= kFfnCus; }

enum class FfnKind { Forward, Gated, GradX, GradW };

FfnPlan ffn_plan(FfnKind kind, int64_t M, int64_t N, int64_t K, int segs, int outs);
// bytes of the partial sums of a plan
size_t ffn_part_bytes(const FfnPlan &p, int64_t M, int64_t N, int outs);

// How a backward pass runs its products: where only one is asked for, by its own
// plan; both in one launch of square tiles, with the parts of each.
struct FfnBackPlan {
  FfnPlan x, w;
  int tile, xsplit, wsplit;
};
// dZ is [M x N], X [M x K]; grads: gradients of one (1) or two (2) products.
FfnBackPlan ffn_back_plan(int64_t M, int64_t K, int64_t N, int grads);
// The bias gradient's last step, dbias[n] = the sum of `rows` partial sums part[r][n]
// (dbias null: none).
struct BiasJoin {
  const float *part;
  int64_t rows, N;
  float *dbias;
};
hipError_t launch_ffn_together(int dtype, const FfnGemm &x, const FfnGemm &w, const BiasJoin &j,
                               const FfnBackPlan &p, hipStream_t s);
hipError_t launch_ffn_back(int dtype, const FfnGemm &x, const FfnGemm &w, const BiasJoin &j,
                           int tile, hipStream_t s);
hipError_t launch_bias_join(const BiasJoin &j, hipStream_t s);

// The plan's kernel and, for a split reduction, the pass that joins the parts.
// dtype: 0 fp16, 1 bf16.
hipError_t launch_ffn(FfnKind kind, int dtype, const FfnGemm &a, const FfnPlan &p, hipStream_t s);

hipError_t launch_ffn_forward(int dtype, const FfnGemm &a, int tile, hipStream_t s);
hipError_t launch_ffn_gated(int dtype, const FfnGemm &a, int tile, hipStream_t s);
hipError_t launch_ffn_grad_x(int dtype, const FfnGemm &a, int tile, hipStream_t s);
hipError_t launch_ffn_grad_w(int dtype, const FfnGemm &a, int tile, hipStream_t s);
hipError_t launch_ffn_skinny(int dtype, bool gated, const FfnGemm &a, int rows, int cols,
                             hipStream_t s);
hipError_t launch_ffn_finish(int dtype, bool gated, const FfnGemm &a, hipStream_t s);

// dZ = dY act'(Z) (dz null: not written; act none: dZ = dY) and, with part, partial
// column sums of dZ: bias_rows(M, N) x N floats, for a BiasJoin.
int64_t bias_rows(int64_t M, int64_t N);
hipError_t launch_act_grad(int dtype, int act, const uint16_t *dy, int64_t lddy, const uint16_t *z,
                           int64_t ldz, int64_t M, int64_t N, uint16_t *dz, int64_t lddz,
                           float *part, hipStream_t s);

// A saved matrix: 16 bits (scales null) or 8-bit codes.
struct Saved {
  void *data;
  int64_t ld;
  uint8_t *scales;
  int64_t lds;
};

// dG = dH U act'(G), dU = dH act(G).
hipError_t launch_gated_grad(int dtype, int act, const uint16_t *dh, int64_t lddh, const Saved &g,
                             const Saved &u, int64_t M, int64_t N, uint16_t *dg, uint16_t *du,
                             int64_t ldd, hipStream_t s);

hipError_t launch_ckpt_pack(int dtype, const uint16_t *x, int64_t M, int64_t K, int64_t ldx,
                            const Saved &out, hipStream_t s);
hipError_t launch_ckpt_unpack(int dtype, const Saved &in, int64_t M, int64_t K, uint16_t *x,
                              int64_t ldx, hipStream_t s);

}  // namespace llmint8
