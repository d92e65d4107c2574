// Which kernel a 16-bit product takes.
#include "ffn.hpp"
#include "llmint8.h"

namespace llmint8 {

namespace {

// The plan is a function of the shape alone (the MI355X's 256 CUs, not a device
// query), so that the workspace queries and the launches agree.
constexpr int64_t kCus = 256;

int64_t tiles_of(int tile, bool gated, int64_t M, int64_t N, int outs) {
  const int64_t bn = gated ? tile / 2 : tile;
  return ((M + tile - 1) / tile) * ((N + bn - 1) / bn) * outs;
}

}  // namespace

FfnPlan ffn_plan(FfnKind kind, int64_t M, int64_t N, int64_t K, int segs, int outs) {
  const bool gated = kind == FfnKind::Gated;
  if (M <= 64 && (gated || kind == FfnKind::Forward)) {
    const int64_t blocks = (N + 63) / 64, stages = (K + 127) / 128;
    int64_t s = (kCus + blocks / 2) / blocks;
    while (s > 1 && stages < 4 * s) --s;
    return FfnPlan{0, (int)(s < 1 ? 1 : s)};
  }
  if (tiles_of(256, gated, M, N, outs) >= kCus / 2) return FfnPlan{256, 1};
  return FfnPlan{128, 1};
}

size_t ffn_part_bytes(const FfnPlan &p, int64_t M, int64_t N, int outs) {
  return p.ksplit > 1 ? (size_t)p.ksplit * outs * M * N * 4 : 0;
}

hipError_t launch_ffn(FfnKind kind, int dtype, const FfnGemm &args, const FfnPlan &p,
                      hipStream_t s) {
  FfnGemm a = args;
  a.ksplit = p.ksplit;
  hipError_t e = hipSuccess;
  if (p.tile == 0)
    e = launch_ffn_skinny(dtype, kind == FfnKind::Gated, a, s);
  else switch (kind) {
    case FfnKind::Forward: e = launch_ffn_forward(dtype, a, p.tile, s); break;
    case FfnKind::Gated: e = launch_ffn_gated(dtype, a, p.tile, s); break;
    case FfnKind::GradX: e = launch_ffn_grad_x(dtype, a, p.tile, s); break;
    case FfnKind::GradW: e = launch_ffn_grad_w(dtype, a, p.tile, s); break;
  }
  if (e == hipSuccess && p.ksplit > 1)
    e = launch_ffn_finish(dtype, kind == FfnKind::Gated, a, s);
  return e;
}

}  // namespace llmint8
