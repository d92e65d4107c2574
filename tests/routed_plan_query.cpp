// The plans of the experts' products and of the block-scaled FP8 product for a host without a GPU
// (built with the plans' own sources): one query per kind of call that names the kernel
// variant a call of a shape runs.
#include "blockwise.hpp"
#include "experts.hpp"

using namespace llmint8;

extern "C" {

// kind: 0 second product, 1 gated, 2 gradient of the rows. out: few, tile, split, rows
void query_experts(int kind, int64_t pairs, int E, int64_t N, int64_t K, int *out) {
  const FfnKind kinds[] = {FfnKind::Forward, FfnKind::Gated, FfnKind::GradX};
  const FfnPlan p = experts_plan(kinds[kind], pairs, E, N, K);
  out[0] = p.few, out[1] = p.tile, out[2] = p.ksplit > 1, out[3] = p.rows;
}

// out: few, fused, tile or columns, split, half tiles at the end, ring of four stages
void query_fp8(int64_t M, int64_t K, int64_t N, int *out) {
  const Fp8Plan p = fp8_plan(M, K, N);
  const int64_t rows = (M + 255) / 256, cols = (N + 255) / 256;
  out[0] = p.few, out[1] = p.fused, out[2] = p.few ? p.cols : p.tile, out[3] = p.ksplit > 1;
  out[4] = !p.few && p.tile == 256 && tail_cut(rows, cols, p.ksplit) < cols;
  out[5] = !p.few && p.tile == 128 &&
           deep_ring((M + 127) / 128 * ((N + 127) / 128) * p.ksplit);
}

}
