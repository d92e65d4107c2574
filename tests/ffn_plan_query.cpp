// The plan of the 16-bit feed-forward products for a host without a GPU: the plan's
// source itself, the launches it calls left out, and one query per kind of call that
// names the kernel variants a call of a shape runs.
#include "ffn_plan.hip"

namespace llmint8 {

hipError_t launch_ffn_forward(int, const FfnGemm &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_gated(int, const FfnGemm &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_grad_x(int, const FfnGemm &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_grad_w(int, const FfnGemm &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_skinny(int, bool, const FfnGemm &, int, int, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_ffn_finish(int, bool, const FfnGemm &, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_back(int, const FfnGemm &, const FfnGemm &, const BiasJoin &, int,
                           hipStream_t) {
  return hipSuccess;
}

}  // namespace llmint8

using namespace llmint8;

namespace {

enum { kFew = 1, kTail = 2, kDeep = 4, kSplit = 8, kSplitW = 16, kXFirst = 32 };

int flags_of(const FfnPlan &p, FfnKind kind, int64_t M, int64_t N, int outs) {
  int f = (p.few ? kFew : 0) | (p.ksplit > 1 ? kSplit : 0);
  const Shape s{kind, M, N, 0, outs};
  if (!p.few && p.tile == 128 && deep_ring(tile_blocks(s, 128, p.ksplit))) f |= kDeep;
  if (!p.few && p.tile == 256) {
    const int64_t rows = cdiv(M, 256), cols = tile_blocks(s, 256, 1) / rows;
    if (tail_cut(rows, cols, p.ksplit) < cols) f |= kTail;
  }
  return f;
}

}  // namespace

// Every out is three numbers: tile (or columns), rows of a few-row block, flags.
extern "C" void query_forward(int gated, int64_t M, int64_t K, int64_t N, int *out) {
  const FfnKind kind = gated ? FfnKind::Gated : FfnKind::Forward;
  const FfnPlan p = ffn_plan(kind, M, N, K, 1, 1);
  out[0] = p.tile, out[1] = p.few ? p.rows : 0, out[2] = flags_of(p, kind, M, N, 1);
}

// dX alone, dW alone and both together.
extern "C" void query_backward(int grads, int64_t M, int64_t K, int64_t N, int *out) {
  const FfnBackPlan p = ffn_back_plan(M, K, N, grads);
  out[0] = p.x.tile, out[1] = 0, out[2] = flags_of(p.x, FfnKind::GradX, M, K, 1);
  out[3] = p.w.tile, out[4] = 0, out[5] = flags_of(p.w, FfnKind::GradW, K, N, grads);
  const Shape x{FfnKind::GradX, M, K, N * grads, 1}, w{FfnKind::GradW, K, N, M, grads};
  const int64_t blocks = tile_blocks(x, p.tile, p.xsplit) + tile_blocks(w, p.tile, p.wsplit);
  out[6] = p.tile, out[7] = 0;
  out[8] = (p.tile == 128 && deep_ring(blocks) ? kDeep : 0) | (p.xsplit > 1 ? kSplit : 0) |
           (p.wsplit > 1 ? kSplitW : 0) | (N * grads / p.xsplit >= M / p.wsplit ? kXFirst : 0);
}
