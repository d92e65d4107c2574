// C ABI of the block-scaled FP8 product: argument checks, workspace layout, the choice of
// kernels and the launch sequence. Every check runs before the first HIP call.
#include "blockwise.hpp"
#include "ffn_check.hpp"

using namespace llmint8;

namespace {

void check_sizes(Check &c, int64_t M, int64_t K, int64_t N) {
  c.dims(M, K, N);
  c.need(K <= kFp8MaxK);
  c.want(K % 16 == 0);
  c.want(((M + 15) / 16) * ((N + 15) / 16) < kMaxDim);
}

bool fp8_sizes_ok(int64_t M, int64_t K, int64_t N) {
  Check c;
  check_sizes(c, M, K, N);
  return c.status() == LLMINT8_OK;
}

int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

struct Layout {
  size_t codes, scales, part, total;
  Fp8Plan plan;
};
Layout layout(int64_t M, int64_t K, int64_t N) {
  Layout L{};
  L.plan = fp8_plan(M, K, N);
  size_t o = 0;
  L.codes = o;
  if (!L.plan.fused) o += up((size_t)M * K);
  L.scales = o;
  if (!L.plan.fused) o += up((size_t)M * fp8_scale_pitch(K));
  L.part = o;
  if (L.plan.ksplit > 1) o += up((size_t)L.plan.ksplit * M * N * 4);
  L.total = o;
  return L;
}

}  // namespace

LLMINT8_EXPORT int llmint8_quantize_blockwise_fp8(const uint16_t *W, int64_t K, int64_t N,
                                                  int64_t ldw, int dtype, uint8_t *Wq8,
                                                  uint8_t *scales, void *stream) {
  Check c;
  check_sizes(c, 1, K, N);
  c.type(dtype, LLMINT8_ACT_NONE);
  c.matrix(W, N, ldw);
  c.need(Wq8 && scales);
  c.want(aligned16(Wq8));
  if (const int st = c.status()) return st;
  return hip_status(
      launch_quant_weights_fp8(dtype, W, K, N, ldw, Wq8, scales, (hipStream_t)stream));
}

LLMINT8_EXPORT int llmint8_quantize_rowblock_fp8(const uint16_t *X, int64_t M, int64_t K,
                                                 int64_t ldx, int dtype, uint8_t *Xq8,
                                                 uint8_t *scales, int64_t ld_scales,
                                                 void *stream) {
  Check c;
  check_sizes(c, M, K, 8);
  c.type(dtype, LLMINT8_ACT_NONE);
  c.matrix(X, K, ldx);
  c.need(Xq8 && scales && ld_scales >= fp8_scale_pitch(K) && ld_scales < kMaxLd);
  c.want(aligned16(Xq8));
  if (const int st = c.status()) return st;
  return hip_status(launch_quant_rows_fp8(dtype, X, M, K, ldx, Xq8, scales, ld_scales,
                                          (hipStream_t)stream));
}

LLMINT8_EXPORT size_t llmint8_linear_blockwise_fp8_workspace_size(int64_t M, int64_t K,
                                                                  int64_t N) {
  return fp8_sizes_ok(M, K, N) ? layout(M, K, N).total : 0;
}

LLMINT8_EXPORT int llmint8_linear_blockwise_fp8(const uint16_t *X, int64_t M, int64_t K,
                                                int64_t ldx, const uint8_t *Wq8,
                                                const uint8_t *scales, int64_t ld_scales,
                                                int64_t N, int dtype, const uint16_t *bias,
                                                uint16_t *Y, int64_t ldy, void *workspace,
                                                size_t workspace_bytes, void *stream) {
  Check c;
  check_sizes(c, M, K, N);
  c.type(dtype, LLMINT8_ACT_NONE);
  c.matrix(X, K, ldx);
  c.need(Wq8 && scales && ld_scales >= blocks_of(K) && ld_scales < kMaxLd);
  c.want(aligned16(Wq8));
  c.vec(bias);
  c.matrix(Y, N, ldy);
  if (const int st = c.status()) return st;
  const Layout L = layout(M, K, N);
  if (const int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t *ws = (uint8_t *)workspace;
  Fp8Gemm a{};
  a.w = Fp8Codes{Wq8, scales, ld_scales};
  a.K = K;
  a.out.M = M, a.out.N = N;
  a.out.outs = 1;
  a.out.y[0] = Y, a.out.ldy = ldy;
  a.out.bias = bias;
  a.out.ksplit = L.plan.ksplit;
  a.out.part = (float *)(ws + L.part);
  hipError_t e = hipSuccess;
  if (L.plan.fused) {
    a.x16 = X, a.ldx = ldx;
  } else {
    const int64_t pitch = fp8_scale_pitch(K);
    e = launch_quant_rows_fp8(dtype, X, M, K, ldx, ws + L.codes, ws + L.scales, pitch, s);
    a.x = Fp8Codes{ws + L.codes, ws + L.scales, pitch};
  }
  if (e == hipSuccess)
    e = L.plan.few ? launch_fp8_few(dtype, a, L.plan, s)
                   : launch_fp8_tiles(dtype, a, L.plan.tile, s);
  if (e == hipSuccess && a.out.ksplit > 1) e = launch_ffn_finish(dtype, false, a.out, s);
  return hip_status(e);
}
