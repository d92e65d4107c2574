// C ABI of the 16-bit feed-forward operators: argument checks, workspace layout
// and the launch sequences. Every check runs before the first HIP call.
#include "ffn_check.hpp"

using namespace llmint8;

namespace {

Saved saved_of(const llmint8_saved *s) { return Saved{s->data, s->ld, s->scales, s->ld_scales}; }

// Workspace of a backward pass: the 16-bit operands of its products (`grads` of
// them), a checkpointed X expanded to 16 bits, the bias gradient's partial sums,
// and the partial sums of the split products, dX's and dW's.
struct BackLayout {
  size_t dz, x, bias, part_x, part_w, total;
  FfnBackPlan plan;
};

BackLayout back_layout(int64_t M, int64_t K, int64_t N, int grads) {
  BackLayout L{};
  L.plan = ffn_back_plan(M, K, N, grads);
  size_t o = 0;
  L.dz = o;
  o += up((size_t)grads * M * N * 2);
  L.x = o;
  o += up((size_t)M * K * 2);
  L.bias = o;
  if (grads == 1) o += up((size_t)bias_rows(M, N) * N * 4);
  const FfnPlan tx{false, L.plan.tile, L.plan.xsplit, 0},
      tw{false, L.plan.tile, L.plan.wsplit, 0};
  auto room = [](size_t x, size_t y) { return up(x > y ? x : y); };
  L.part_x = o;
  o += room(ffn_part_bytes(L.plan.x, M, K, 1), ffn_part_bytes(tx, M, K, 1));
  L.part_w = o;
  o += room(ffn_part_bytes(L.plan.w, K, N, grads), ffn_part_bytes(tw, K, N, grads));
  L.total = o;
  return L;
}

// The products of a backward pass: dX = sum of dZ_i W_i^T and dW_i = X^T dZ_i for
// `grads` products, either of them only where its outputs are given. A
// checkpointed X is expanded into the workspace first, exactly: a pass of 3 bytes
// an entry against a product of 2 N or 4 N operations an entry. Expanding the
// codes inside the product's tiles instead (8-bit loads to registers, 16-bit
// stores to LDS) cost more than the pass at 2048 x 4096 x 11008: 438 against
// 412 + 6 us.
struct Grads {
  int count;
  const uint16_t *dz[2];
  int64_t lddz;
  const llmint8_saved *X;
  const uint16_t *w[2];
  int64_t ldw;
  uint16_t *dX;
  int64_t lddx;
  uint16_t *dW[2];
  int64_t lddw;
  BiasJoin bias;
};

hipError_t run_grads(int dtype, const Grads &g, int64_t M, int64_t K, int64_t N, uint8_t *ws,
                     const BackLayout &L, hipStream_t s) {
  FfnGemm x{}, w{};
  if (g.dX) {
    for (int i = 0; i < g.count; ++i) x.a[i] = g.dz[i], x.b[i] = g.w[i];
    x.lda = g.lddz, x.ldb = g.ldw;
    x.M = M, x.N = K, x.K = N;
    x.segs = g.count, x.outs = 1;
    x.y[0] = g.dX, x.ldy = g.lddx;
    x.part = (float *)(ws + L.part_x);
  }
  if (g.dW[0]) {
    w.a[0] = g.X->data, w.lda = g.X->ld;
    if (g.X->scales) {
      uint16_t *room = (uint16_t *)(ws + L.x);
      const hipError_t e = launch_ckpt_unpack(dtype, saved_of(g.X), M, K, room, K, s);
      if (e != hipSuccess) return e;
      w.a[0] = room, w.lda = K;
    }
    for (int i = 0; i < g.count; ++i) w.b[i] = g.dz[i], w.y[i] = g.dW[i];
    w.ldb = g.lddz;
    w.M = K, w.N = N, w.K = M;
    w.segs = 1, w.outs = g.count;
    w.ldy = g.lddw;
    w.part = (float *)(ws + L.part_w);
  }
  if (g.dX && g.dW[0]) return launch_ffn_together(dtype, x, w, g.bias, L.plan, s);
  hipError_t e = g.bias.dbias ? launch_bias_join(g.bias, s) : hipSuccess;
  if (e != hipSuccess) return e;
  e = g.dX ? launch_ffn(FfnKind::GradX, dtype, x, L.plan.x, s) : hipSuccess;
  if (e == hipSuccess && g.dW[0]) e = launch_ffn(FfnKind::GradW, dtype, w, L.plan.w, s);
  return e;
}

}  // namespace

LLMINT8_EXPORT int llmint8_checkpoint_pack(const uint16_t *X, int64_t M, int64_t K, int64_t ldx,
                                           int dtype, const llmint8_saved *out, void *stream) {
  Check c;
  c.dims(M, K, 8);
  c.type(dtype, 0);
  c.matrix(X, K, ldx);
  c.need(out && out->scales);
  c.saved(out, K);
  if (const int st = c.status()) return st;
  return hip_status(launch_ckpt_pack(dtype, X, M, K, ldx, saved_of(out), (hipStream_t)stream));
}

LLMINT8_EXPORT int llmint8_checkpoint_unpack(const llmint8_saved *in, int64_t M, int64_t K,
                                             int dtype, uint16_t *X, int64_t ldx, void *stream) {
  Check c;
  c.dims(M, K, 8);
  c.type(dtype, 0);
  c.matrix(X, K, ldx);
  c.need(in && in->scales);
  c.saved(in, K);
  if (const int st = c.status()) return st;
  return hip_status(launch_ckpt_unpack(dtype, saved_of(in), M, K, X, ldx, (hipStream_t)stream));
}

LLMINT8_EXPORT size_t llmint8_matmul_workspace_size(int64_t M, int64_t K, int64_t N) {
  if (!sizes_ok(M, K, N)) return 0;
  return ffn_part_bytes(ffn_plan(FfnKind::Forward, M, N, K, 1, 1), M, N, 1);
}

LLMINT8_EXPORT int llmint8_matmul(const uint16_t *X, int64_t M, int64_t K, int64_t ldx,
                                  const uint16_t *W, int64_t ldw, int64_t N, int dtype,
                                  uint16_t *Y, int64_t ldy, const llmint8_matmul_opts *opts,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  llmint8_matmul_opts o{};
  if (opts) {
    if (opts->struct_size != sizeof(o)) return LLMINT8_ERR_INVALID_ARG;
    o = *opts;
  }
  Check c;
  c.dims(M, K, N);
  c.type(dtype, o.activation);
  c.matrix(X, K, ldx);
  c.matrix(W, N, ldw);
  c.matrix(Y, N, ldy);
  c.vec(o.bias);
  if (o.residual) c.matrix(o.residual, N, o.ldr);
  if (o.Z) c.matrix(o.Z, N, o.ldz);
  if (const int st = c.status()) return st;
  const FfnPlan p = ffn_plan(FfnKind::Forward, M, N, K, 1, 1);
  if (const int st = check_workspace(workspace, workspace_bytes, ffn_part_bytes(p, M, N, 1)))
    return st;
  FfnGemm a{};
  a.a[0] = X, a.lda = ldx;
  a.b[0] = W, a.ldb = ldw;
  a.M = M, a.N = N, a.K = K;
  a.segs = a.outs = 1;
  a.y[0] = Y, a.ldy = ldy;
  a.act = o.activation, a.bias = o.bias, a.residual = o.residual, a.ldr = o.ldr;
  a.z[0] = o.Z, a.ldz = o.ldz;
  a.part = (float *)workspace;
  return hip_status(launch_ffn(FfnKind::Forward, dtype, a, p, (hipStream_t)stream));
}

LLMINT8_EXPORT size_t llmint8_matmul_backward_workspace_size(int64_t M, int64_t K, int64_t N) {
  return sizes_ok(M, K, N) ? back_layout(M, K, N, 1).total : 0;
}

LLMINT8_EXPORT int llmint8_matmul_backward(const uint16_t *dY, int64_t M, int64_t N, int64_t lddy,
                                           const llmint8_saved *X, int64_t K, const uint16_t *W,
                                           int64_t ldw, const uint16_t *Z, int64_t ldz,
                                           int activation, int dtype, uint16_t *dX, int64_t lddx,
                                           uint16_t *dW, int64_t lddw, float *dbias,
                                           void *workspace, size_t workspace_bytes,
                                           void *stream) {
  Check c;
  c.dims(M, K, N);
  c.type(dtype, activation);
  c.matrix(dY, N, lddy);
  c.need(dX || dW || dbias);
  if (activation != LLMINT8_ACT_NONE) c.matrix(Z, N, ldz);
  if (dX) c.matrix(W, N, ldw), c.matrix(dX, K, lddx);
  if (dW) c.saved(X, K), c.matrix(dW, N, lddw);
  c.vec(dbias);
  if (const int st = c.status()) return st;
  const BackLayout L = back_layout(M, K, N, 1);
  if (const int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t *ws = (uint8_t *)workspace;
  const bool act = activation != LLMINT8_ACT_NONE, products = dX || dW;
  uint16_t *own = (uint16_t *)(ws + L.dz);
  float *part = (float *)(ws + L.bias);
  const uint16_t *dz = act ? own : dY;
  const int64_t lddz = act ? N : lddy;
  hipError_t e = hipSuccess;
  if (act || dbias)
    e = launch_act_grad(dtype, activation, dY, lddy, Z, ldz, M, N, act && products ? own : nullptr,
                        lddz, dbias ? part : nullptr, s);
  if (e == hipSuccess)
    e = run_grads(dtype, Grads{1, {dz, nullptr}, lddz, X, {W, nullptr}, ldw, dX, lddx,
                               {dW, nullptr}, lddw, {part, bias_rows(M, N), N, dbias}},
                  M, K, N, ws, L, s);
  return hip_status(e);
}

LLMINT8_EXPORT size_t llmint8_gated_workspace_size(int64_t M, int64_t K, int64_t N) {
  if (!sizes_ok(M, K, N)) return 0;
  return ffn_part_bytes(ffn_plan(FfnKind::Gated, M, N, K, 1, 1), M, N, 2);
}

LLMINT8_EXPORT int llmint8_gated(const uint16_t *X, int64_t M, int64_t K, int64_t ldx,
                                 const uint16_t *Wg, const uint16_t *Wu, int64_t ldw, int64_t N,
                                 int activation, int dtype, uint16_t *H, int64_t ldh,
                                 const llmint8_saved *G, const llmint8_saved *U, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  Check c;
  c.dims(M, K, N);
  c.type(dtype, activation);
  c.matrix(X, K, ldx);
  c.matrix(Wg, N, ldw);
  c.matrix(Wu, N, ldw);
  c.matrix(H, N, ldh);
  c.need(!G == !U);
  if (G && U) {
    c.saved(G, N);
    c.saved(U, N);
    c.need(!G->scales == !U->scales && G->ld == U->ld);
    c.need(!G->scales || G->ld_scales == U->ld_scales);
  }
  if (const int st = c.status()) return st;
  const FfnPlan p = ffn_plan(FfnKind::Gated, M, N, K, 1, 1);
  if (const int st = check_workspace(workspace, workspace_bytes, ffn_part_bytes(p, M, N, 2)))
    return st;
  FfnGemm a{};
  a.a[0] = X, a.lda = ldx;
  a.b[0] = Wg, a.b[1] = Wu, a.ldb = ldw;
  a.M = M, a.N = N, a.K = K;
  a.segs = a.outs = 1;
  a.y[0] = H, a.ldy = ldh;
  a.act = activation;
  if (G) {
    a.z[0] = G->data, a.z[1] = U->data, a.ldz = G->ld;
    a.zs[0] = G->scales, a.zs[1] = U->scales, a.ldzs = G->ld_scales;
  }
  a.part = (float *)workspace;
  return hip_status(launch_ffn(FfnKind::Gated, dtype, a, p, (hipStream_t)stream));
}

LLMINT8_EXPORT size_t llmint8_gated_backward_workspace_size(int64_t M, int64_t K, int64_t N) {
  return sizes_ok(M, K, N) ? back_layout(M, K, N, 2).total : 0;
}

LLMINT8_EXPORT int llmint8_gated_backward(const uint16_t *dH, int64_t M, int64_t N, int64_t lddh,
                                          const llmint8_saved *X, int64_t K, const uint16_t *Wg,
                                          const uint16_t *Wu, int64_t ldw, const llmint8_saved *G,
                                          const llmint8_saved *U, int activation, int dtype,
                                          uint16_t *dX, int64_t lddx, uint16_t *dWg,
                                          uint16_t *dWu, int64_t lddw, void *workspace,
                                          size_t workspace_bytes, void *stream) {
  Check c;
  c.dims(M, K, N);
  c.type(dtype, activation);
  c.matrix(dH, N, lddh);
  c.saved(G, N);
  c.saved(U, N);
  c.need(G && U && !G->scales == !U->scales);
  c.need(!dWg == !dWu && (dX || dWg));
  if (dX) c.matrix(Wg, N, ldw), c.matrix(Wu, N, ldw), c.matrix(dX, K, lddx);
  if (dWg && dWu) c.saved(X, K), c.matrix(dWg, N, lddw), c.matrix(dWu, N, lddw);
  if (const int st = c.status()) return st;
  const BackLayout L = back_layout(M, K, N, 2);
  if (const int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t *ws = (uint8_t *)workspace;
  uint16_t *dg = (uint16_t *)(ws + L.dz), *du = dg + M * N;
  hipError_t e = launch_gated_grad(dtype, activation, dH, lddh, saved_of(G), saved_of(U), M, N, dg,
                                   du, N, s);
  if (e == hipSuccess)
    e = run_grads(dtype, Grads{2, {dg, du}, N, X, {Wg, Wu}, ldw, dX, lddx, {dWg, dWu}, lddw, {}},
                  M, K, N, ws, L, s);
  return hip_status(e);
}
