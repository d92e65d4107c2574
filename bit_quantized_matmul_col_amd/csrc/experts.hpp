// Internal launchers of the routed feed-forward kernels: the router, the order of the
// (token, expert) pairs, and the experts' products over it. Each returns hipSuccess or the
// error of its launch; none synchronizes.
#pragma once

#include "ffn.hpp"

namespace llmint8 {

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopk = 64;
constexpr int64_t kMaxGroups = 64;
// Rows of an expert, on the mean, up to which the few-row kernel is considered.
constexpr int64_t kFewRows = 200;
// Pairs of a token and an expert: passes with a wave for each have fewer than 2^32 threads.
constexpr int64_t kMaxPairs = (int64_t)1 << 25;

struct Route {
  const void *logits;  // [M x ld], dtype 0 fp16, 1 bf16, 2 fp32
  int64_t M, ld;
  int E, k, dtype;
  int sigmoid, renorm;
  float scale;
  const float *bias;  // [E] or null
  int groups, top_groups, group_best;
};

hipError_t launch_route(const Route &r, int32_t *ids, float *weights, hipStream_t s);
hipError_t launch_route_backward(const Route &r, const int32_t *ids, const float *dweights,
                                 void *dlogits, int64_t ldd, hipStream_t s);

// The pairs i k + j by expert: expert e has the rows offsets[e] .. offsets[e + 1] - 1, row r
// is the pair order[r], and pair p is row places[p] (-1: no expert).
struct Pairs {
  const int32_t *offsets, *order, *places;
  int64_t tokens;
  int E, k;
  __host__ __device__ int64_t rows() const { return tokens * k; }
};

// Bytes of its scratch: 0 for few pairs.
size_t expert_plan_scratch(int64_t pairs, int E);
hipError_t launch_expert_plan(const int32_t *ids, int64_t pairs, int E, int32_t *offsets,
                              int32_t *order, int32_t *places, int32_t *scratch, hipStream_t s);

// How a product over the experts' rows runs: square tiles of 256 or 128 rows, or the
// few-row kernel with `tile` columns by `rows` rows; in how many parts the reduction is split.
FfnPlan experts_plan(FfnKind kind, int64_t pairs, int E, int64_t N, int64_t K);

// Products over the rows of each expert: `a` for all rows (a.M = the number of pairs, a.b and
// a.pairs those of expert 0 and row 0); expert e's B is bstride elements after the last's.
// Forward: rows as they are, sums to a.part in fp32. GradX: the same, or to a.y in 16 bits. Gated: rows
// of the tokens, or as they are.
hipError_t launch_expert_rows(FfnKind kind, int dtype, const FfnGemm &a, const Pairs &p,
                              int64_t bstride, const FfnPlan &plan, hipStream_t s);
hipError_t launch_expert_skinny(int dtype, bool gated, const FfnGemm &a, const Pairs &p,
                                int64_t bstride, const FfnPlan &plan, hipStream_t s);
// dW_e = A_e^T B_e for every expert, `outs` of them; A and B by row. ystride: elements from one
// expert's gradient to the next's.
hipError_t launch_expert_grad_w(int dtype, const FfnGemm &a, const Pairs &p, int64_t ystride,
                                hipStream_t s);

// out[r] = x[token of row r]
hipError_t launch_take_rows(int dtype, const uint16_t *x, int64_t ldx, int64_t cols,
                            const Pairs &p, uint16_t *out, hipStream_t s);
// y[i] = residual[i] + the sum over token i's pairs of their rows, `parts` planes of fp32
// [rows x N].
struct Combine {
  const float *part;
  int parts;
  int64_t N;
  const uint16_t *residual;
  int64_t ldr;
  uint16_t *y;
  int64_t ldy;
};
hipError_t launch_combine(int dtype, const Combine &c, const Pairs &p, hipStream_t s);
// With d' = w d: dG = d' U act'(G), dU = d' act(G) (16 bits), dw = sum of d act(G) U.
hipError_t launch_expert_gated_grad(int dtype, int act, const uint16_t *dh, int64_t lddh,
                                    const uint16_t *g, const uint16_t *u, int64_t ldz, int64_t N,
                                    const Pairs &p, const float *w, uint16_t *dg, uint16_t *du,
                                    float *dw, hipStream_t s);
// The epilogue of a gated product split into parts.
hipError_t launch_expert_gated_finish(int dtype, const FfnGemm &a, const Pairs &p, hipStream_t s);

}  // namespace llmint8
