// C ABI of the router and of the experts' products: argument checks, workspace layout, the
// choice of kernels and the launch sequences. Every check runs before the first HIP call.
#include "experts.hpp"
#include "ffn_check.hpp"

using namespace llmint8;

namespace llmint8 {

hipError_t launch_expert_forward(int dtype, const FfnGemm &a, const Pairs &p, int64_t bstride,
                                 int tile, hipStream_t s);
hipError_t launch_expert_gated(int dtype, const FfnGemm &a, const Pairs &p, int64_t bstride,
                               int tile, hipStream_t s);
hipError_t launch_expert_grad_x(int dtype, const FfnGemm &a, const Pairs &p, int64_t bstride,
                                int tile, hipStream_t s);

hipError_t launch_expert_rows(FfnKind kind, int dtype, const FfnGemm &a, const Pairs &p,
                              int64_t bstride, const FfnPlan &plan, hipStream_t s) {
  if (plan.few) return launch_expert_skinny(dtype, kind == FfnKind::Gated, a, p, bstride, plan, s);
  if (kind == FfnKind::Gated) return launch_expert_gated(dtype, a, p, bstride, plan.tile, s);
  if (kind == FfnKind::Forward) return launch_expert_forward(dtype, a, p, bstride, plan.tile, s);
  return launch_expert_grad_x(dtype, a, p, bstride, plan.tile, s);
}

}  // namespace llmint8

namespace {

constexpr int64_t kSpan = (int64_t)1 << 31;  // bytes that a routed operand's offsets reach

// Sizes of a call over the experts' rows.
void check_rows(Check &c, int64_t M, int64_t K, int64_t N, int64_t E, int64_t k) {
  c.dims(M, K, N);
  c.need(E > 0 && k > 0);
  c.need(E <= kMaxExperts && k <= kMaxTopk && k <= E);
  c.need(k > 0 && M <= (kMaxPairs - 1) / k);
  if (c.arg) return;
  // Tiles are counted in 32 bits. Few-row blocks (16 by 64 columns; in parts only where they are
  // few) have fewer than 2^32 threads.
  const int64_t rows = M * k, wide = K > N ? K : N, most = (kFewRows + 1) * E;
  const int64_t few = rows < most ? rows : most;
  c.want((rows / 128 + E) * (wide / 128 + 1) < kMaxDim);
  c.want(E * (K / 128 + 1) * (N / 128 + 1) < kMaxDim);
  c.want((few / 16 + E) * (wide / 64 + 1) < (int64_t)1 << 24);
}

bool rows_ok(int64_t M, int64_t K, int64_t N, int64_t E, int64_t k) {
  Check c;
  check_rows(c, M, K, N, E, k);
  return c.status() == LLMINT8_OK;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

void check_plan(Check &c, const llmint8_expert_rows *r) {
  c.need(r && r->offsets && r->order && r->places);
  if (r) c.want(aligned4(r->offsets) && aligned4(r->order) && aligned4(r->places));
}

// Weights of all experts, [E][rows x cols].
void check_experts(Check &c, const void *p, int64_t cols, int64_t ld, int64_t stride) {
  c.matrix(p, cols, ld);
  c.need(stride >= 0 && stride < (int64_t)1 << 40);
  c.want(stride % 8 == 0);
}
// The same as an output: no expert's part overlaps another's.
void check_experts_out(Check &c, const void *p, int64_t rows, int64_t cols, int64_t ld,
                       int64_t stride, int64_t E) {
  check_experts(c, p, cols, ld, stride);
  c.need(E == 1 || stride >= (rows - 1) * ld + cols);
}

Pairs pairs_of(const llmint8_expert_rows *r, int64_t M) {
  return Pairs{r->offsets, r->order, r->places, M, (int)r->E, (int)r->k};
}

// A product over the experts' rows, in one segment.
FfnGemm rows_gemm(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t N, int64_t K,
                  const Pairs &p, uint16_t *y, int64_t ldy) {
  FfnGemm a{};
  a.a[0] = A, a.lda = lda;
  a.b[0] = B, a.ldb = ldb;
  a.M = p.rows(), a.N = N, a.K = K;
  a.segs = a.outs = 1, a.ksplit = 1;
  a.y[0] = y, a.ldy = ldy;
  a.all_rows = p.rows();
  a.pairs = p.order;
  return a;
}

// X of more than 2 GiB is copied into the experts' order first.
bool spans(int64_t M, int64_t K, int64_t ldx) { return ((M - 1) * ldx + K) * 2 >= kSpan; }

size_t part_bytes(const FfnPlan &p, int64_t rows, int64_t N, int sums) {
  return (size_t)p.ksplit * sums * rows * N * 4;
}

struct GatedLayout {
  size_t x, part, total;
  FfnPlan plan;
};
GatedLayout gated_layout(int64_t M, int64_t K, int64_t N, int64_t E, int64_t k) {
  GatedLayout L{};
  L.plan = experts_plan(FfnKind::Gated, M * k, (int)E, N, K);
  size_t o = 0;
  L.x = o;
  if (spans(M, K, K)) o += up((size_t)M * k * K * 2);
  L.part = o;
  if (L.plan.ksplit > 1) o += up(part_bytes(L.plan, M * k, N, 2));
  L.total = o;
  return L;
}

// The second product's rows before they are summed, in fp32, in the plan's parts.
struct MatmulLayout {
  size_t total;
  FfnPlan plan;
};
MatmulLayout matmul_layout(int64_t M, int64_t K, int64_t N, int64_t E, int64_t k) {
  MatmulLayout L{};
  L.plan = experts_plan(FfnKind::Forward, M * k, (int)E, K, N);
  L.total = up(part_bytes(L.plan, M * k, K, 1));
  return L;
}

struct GatedBackLayout {
  size_t dg, du, x, rows, total;
};
GatedBackLayout gated_back_layout(int64_t M, int64_t K, int64_t N, int64_t k) {
  const size_t R = (size_t)M * k, z = up(R * N * 2), x = up(R * K * 2);
  return GatedBackLayout{0, z, 2 * z, 2 * z + x, 2 * z + x + up(R * K * 4)};
}

bool route_ok(Check &c, const void *logits, int64_t M, int64_t E, int64_t ld, int dtype, int64_t k,
              const llmint8_route_opts *opts, Route &r) {
  llmint8_route_opts o{};
  o.scale = 1.f, o.groups = o.top_groups = o.group_best = 1;
  if (opts) {
    c.need(opts->struct_size == sizeof(o));
    if (c.arg) return false;
    o = *opts;
  }
  c.need(M > 0 && E > 0 && k > 0 && E <= kMaxExperts && k <= E && k <= kMaxTopk);
  c.need(k > 0 && M <= (kMaxPairs - 1) / k);
  c.need(logits && ld >= E && ld < kMaxLd);
  c.need(dtype == LLMINT8_FP16 || dtype == LLMINT8_BF16 || dtype == LLMINT8_FP32);
  c.need(o.scores == LLMINT8_SCORE_SOFTMAX || o.scores == LLMINT8_SCORE_SIGMOID);
  c.need(o.renormalize == 0 || o.renormalize == 1);
  c.need(o.groups > 0 && o.groups <= kMaxGroups && (o.groups <= 0 || E % o.groups == 0));
  c.need(o.top_groups > 0 && o.top_groups <= o.groups);
  c.need(o.group_best == 1 || o.group_best == 2);
  c.want(((uintptr_t)logits & (dtype == LLMINT8_FP32 ? 3u : 1u)) == 0 && aligned4(o.bias));
  r = Route{logits,  M,      ld,       (int)E,       (int)k,      dtype,
            o.scores, o.renormalize, o.scale, o.bias, o.groups, o.top_groups,
            // one group's value decides nothing
            o.groups > 1 ? o.group_best : 1};
  return c.status() == LLMINT8_OK;
}

}  // namespace

LLMINT8_EXPORT int llmint8_route(const void *logits, int64_t M, int64_t E, int64_t ld, int dtype,
                                 int64_t k, const llmint8_route_opts *opts, int32_t *ids,
                                 float *weights, void *stream) {
  Check c;
  Route r;
  c.need(ids && weights);
  c.want(aligned4(ids) && aligned4(weights));
  if (!route_ok(c, logits, M, E, ld, dtype, k, opts, r)) return c.status();
  return hip_status(launch_route(r, ids, weights, (hipStream_t)stream));
}

LLMINT8_EXPORT int llmint8_route_backward(const float *dweights, const void *logits, int64_t M,
                                          int64_t E, int64_t ld, int dtype, int64_t k,
                                          const int32_t *ids, const llmint8_route_opts *opts,
                                          void *dlogits, int64_t ldd, void *stream) {
  Check c;
  Route r;
  c.need(dweights && ids && dlogits && ldd >= E && ldd < kMaxLd);
  c.want(aligned4(ids) && aligned4(dweights));
  c.want(((uintptr_t)dlogits & (dtype == LLMINT8_FP32 ? 3u : 1u)) == 0);
  if (!route_ok(c, logits, M, E, ld, dtype, k, opts, r)) return c.status();
  return hip_status(launch_route_backward(r, ids, dweights, dlogits, ldd, (hipStream_t)stream));
}

LLMINT8_EXPORT size_t llmint8_expert_plan_workspace_size(int64_t M, int64_t k, int64_t E) {
  return rows_ok(M, 8, 8, E, k) ? expert_plan_scratch(M * k, (int)E) : 0;
}

LLMINT8_EXPORT int llmint8_expert_plan(const int32_t *ids, int64_t M, int64_t k, int64_t E,
                                       int32_t *offsets, int32_t *order, int32_t *places,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  Check c;
  check_rows(c, M, 8, 8, E, k);
  c.need(ids && offsets && order && places);
  c.want(aligned4(ids) && aligned4(offsets) && aligned4(order) && aligned4(places));
  if (const int st = c.status()) return st;
  const size_t need = expert_plan_scratch(M * k, (int)E);
  if (const int st = check_workspace(workspace, workspace_bytes, need)) return st;
  return hip_status(launch_expert_plan(ids, M * k, (int)E, offsets, order, places,
                                       (int32_t *)workspace, (hipStream_t)stream));
}

LLMINT8_EXPORT size_t llmint8_experts_gated_workspace_size(int64_t M, int64_t K, int64_t N,
                                                           int64_t E, int64_t k) {
  return rows_ok(M, K, N, E, k) ? gated_layout(M, K, N, E, k).total : 0;
}

LLMINT8_EXPORT int llmint8_experts_gated(const uint16_t *X, int64_t M, int64_t K, int64_t ldx,
                                         const uint16_t *Wg, const uint16_t *Wu, int64_t ldw,
                                         int64_t stride_w, int64_t N,
                                         const llmint8_expert_rows *rows, const float *weights,
                                         int activation, int dtype, uint16_t *H, int64_t ldh,
                                         uint16_t *G, uint16_t *U, int64_t ldz, void *workspace,
                                         size_t workspace_bytes, void *stream) {
  Check c;
  check_plan(c, rows);
  if (c.arg) return c.arg;
  check_rows(c, M, K, N, rows->E, rows->k);
  c.type(dtype, activation);
  c.matrix(X, K, ldx);
  check_experts(c, Wg, N, ldw, stride_w);
  check_experts(c, Wu, N, ldw, stride_w);
  c.matrix(H, N, ldh);
  c.need(!G == !U);
  if (G && U) c.matrix(G, N, ldz), c.matrix(U, N, ldz);
  c.want(aligned4(weights));
  if (const int st = c.status()) return st;
  const bool copy = spans(M, K, ldx);
  if (copy && !spans(M, K, K)) return LLMINT8_ERR_UNSUPPORTED;
  const GatedLayout L = gated_layout(M, K, N, rows->E, rows->k);
  if (const int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t *ws = (uint8_t *)workspace;
  const Pairs p = pairs_of(rows, M);
  FfnGemm a = rows_gemm(X, ldx, Wg, ldw, N, K, p, H, ldh);
  a.b[1] = Wu;
  a.act = activation;
  a.z[0] = G, a.z[1] = U, a.ldz = ldz;
  a.w = weights;
  a.topk = p.k, a.a_rows = M;
  hipError_t e = hipSuccess;
  if (copy) {
    uint16_t *xs = (uint16_t *)(ws + L.x);
    e = launch_take_rows(dtype, X, ldx, K, p, xs, s);
    a.a[0] = xs, a.lda = K, a.topk = 0;
  }
  a.part = (float *)(ws + L.part);
  a.ksplit = L.plan.ksplit, a.to_parts = a.ksplit > 1;
  if (e == hipSuccess) e = launch_expert_rows(FfnKind::Gated, dtype, a, p, stride_w, L.plan, s);
  if (e == hipSuccess && a.to_parts) e = launch_expert_gated_finish(dtype, a, p, s);
  return hip_status(e);
}

LLMINT8_EXPORT size_t llmint8_experts_gated_backward_workspace_size(int64_t M, int64_t K,
                                                                    int64_t N, int64_t E,
                                                                    int64_t k) {
  return rows_ok(M, K, N, E, k) ? gated_back_layout(M, K, N, k).total : 0;
}

LLMINT8_EXPORT int llmint8_experts_gated_backward(
    const uint16_t *dH, int64_t M, int64_t N, int64_t lddh, const uint16_t *X, int64_t K,
    int64_t ldx, const uint16_t *Wg, const uint16_t *Wu, int64_t ldw, int64_t stride_w,
    const uint16_t *G, const uint16_t *U, int64_t ldz, const llmint8_expert_rows *rows,
    const float *weights, int activation, int dtype, uint16_t *dX, int64_t lddx, uint16_t *dWg,
    uint16_t *dWu, int64_t lddw, int64_t stride_dw, float *dweights, void *workspace,
    size_t workspace_bytes, void *stream) {
  Check c;
  check_plan(c, rows);
  if (c.arg) return c.arg;
  check_rows(c, M, K, N, rows->E, rows->k);
  c.type(dtype, activation);
  c.matrix(dH, N, lddh);
  c.matrix(G, N, ldz);
  c.matrix(U, N, ldz);
  c.need(!dWg == !dWu && (dX || dWg || dweights));
  if (dX) {
    check_experts(c, Wg, N, ldw, stride_w);
    check_experts(c, Wu, N, ldw, stride_w);
    c.matrix(dX, K, lddx);
  }
  if (dWg && dWu) {
    c.matrix(X, K, ldx);
    check_experts_out(c, dWg, K, N, lddw, stride_dw, rows->E);
    check_experts_out(c, dWu, K, N, lddw, stride_dw, rows->E);
  }
  c.want(aligned4(weights) && aligned4(dweights));
  if (const int st = c.status()) return st;
  const GatedBackLayout L = gated_back_layout(M, K, N, rows->k);
  if (const int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  hipStream_t s = (hipStream_t)stream;
  uint8_t *ws = (uint8_t *)workspace;
  const Pairs p = pairs_of(rows, M);
  uint16_t *dg = (uint16_t *)(ws + L.dg), *du = (uint16_t *)(ws + L.du);
  uint16_t *xs = (uint16_t *)(ws + L.x);
  float *xrows = (float *)(ws + L.rows);
  hipError_t e = launch_expert_gated_grad(dtype, activation, dH, lddh, G, U, ldz, N, p, weights,
                                          dg, du, dweights, s);
  if (e == hipSuccess && dX) {
    // The rows stay in fp32: dG and dU were rounded already, and with a second rounding of
    // one size dX would be off by 1.7 times what one rounded once is, not 1.4 (50 us of 1450 at
    // 4096 tokens x 4 of 32 experts, 4096 x 2048).
    FfnGemm a = rows_gemm(dg, N, Wg, ldw, K, N, p, nullptr, 0);
    a.a[1] = du, a.b[1] = Wu, a.segs = 2;
    a.part = xrows, a.to_parts = 1;
    const FfnPlan plan = experts_plan(FfnKind::GradX, p.rows(), p.E, K, 2 * N);
    e = launch_expert_rows(FfnKind::GradX, dtype, a, p, stride_w, plan, s);
    if (e == hipSuccess)
      e = launch_combine(dtype, Combine{xrows, 1, K, nullptr, 0, dX, lddx}, p, s);
  }
  if (e == hipSuccess && dWg) {
    e = launch_take_rows(dtype, X, ldx, K, p, xs, s);
    FfnGemm a = rows_gemm(xs, K, dg, N, N, 0, p, dWg, lddw);
    a.M = K, a.b[1] = du, a.y[1] = dWu, a.outs = 2;
    if (e == hipSuccess) e = launch_expert_grad_w(dtype, a, p, stride_dw, s);
  }
  return hip_status(e);
}

LLMINT8_EXPORT size_t llmint8_experts_matmul_workspace_size(int64_t M, int64_t K, int64_t N,
                                                            int64_t E, int64_t k) {
  return rows_ok(M, K, N, E, k) ? matmul_layout(M, K, N, E, k).total : 0;
}

LLMINT8_EXPORT int llmint8_experts_matmul(const uint16_t *H, int64_t M, int64_t N, int64_t ldh,
                                          const uint16_t *Wd, int64_t ldw, int64_t stride_w,
                                          int64_t K, const llmint8_expert_rows *rows,
                                          const uint16_t *residual, int64_t ldr, int dtype,
                                          uint16_t *Y, int64_t ldy, void *workspace,
                                          size_t workspace_bytes, void *stream) {
  Check c;
  check_plan(c, rows);
  if (c.arg) return c.arg;
  check_rows(c, M, K, N, rows->E, rows->k);
  c.type(dtype, LLMINT8_ACT_NONE);
  c.matrix(H, N, ldh);
  check_experts(c, Wd, K, ldw, stride_w);
  if (residual) c.matrix(residual, K, ldr);
  c.matrix(Y, K, ldy);
  if (const int st = c.status()) return st;
  const MatmulLayout L = matmul_layout(M, K, N, rows->E, rows->k);
  if (const int st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  hipStream_t s = (hipStream_t)stream;
  const Pairs p = pairs_of(rows, M);
  FfnGemm a = rows_gemm(H, ldh, Wd, ldw, K, N, p, nullptr, 0);
  a.part = (float *)workspace, a.ksplit = L.plan.ksplit, a.to_parts = 1;
  hipError_t e = launch_expert_rows(FfnKind::Forward, dtype, a, p, stride_w, L.plan, s);
  if (e == hipSuccess)
    e = launch_combine(dtype, Combine{a.part, a.ksplit, K, residual, ldr, Y, ldy}, p, s);
  return hip_status(e);
}

LLMINT8_EXPORT size_t llmint8_experts_matmul_backward_workspace_size(int64_t M, int64_t K,
                                                                     int64_t N, int64_t E,
                                                                     int64_t k) {
  return rows_ok(M, K, N, E, k) ? up((size_t)M * k * K * 2) : 0;
}

LLMINT8_EXPORT int llmint8_experts_matmul_backward(
    const uint16_t *dY, int64_t M, int64_t K, int64_t lddy, const uint16_t *H, int64_t N,
    int64_t ldh, const uint16_t *Wd, int64_t ldw, int64_t stride_w,
    const llmint8_expert_rows *rows, int dtype, uint16_t *dH, int64_t lddh, uint16_t *dWd,
    int64_t lddw, int64_t stride_dw, void *workspace, size_t workspace_bytes, void *stream) {
  Check c;
  check_plan(c, rows);
  if (c.arg) return c.arg;
  check_rows(c, M, K, N, rows->E, rows->k);
  c.type(dtype, LLMINT8_ACT_NONE);
  c.matrix(dY, K, lddy);
  c.need(dH || dWd);
  if (dH) check_experts(c, Wd, K, ldw, stride_w), c.matrix(dH, N, lddh);
  if (dWd) c.matrix(H, N, ldh), check_experts_out(c, dWd, N, K, lddw, stride_dw, rows->E);
  if (const int st = c.status()) return st;
  const size_t need = up((size_t)M * rows->k * K * 2);
  if (const int st = check_workspace(workspace, workspace_bytes, need)) return st;
  hipStream_t s = (hipStream_t)stream;
  const Pairs p = pairs_of(rows, M);
  uint16_t *dys = (uint16_t *)workspace;
  hipError_t e = launch_take_rows(dtype, dY, lddy, K, p, dys, s);
  if (e == hipSuccess && dH) {
    const FfnGemm a = rows_gemm(dys, K, Wd, ldw, N, K, p, dH, lddh);
    const FfnPlan plan = experts_plan(FfnKind::GradX, p.rows(), p.E, N, K);
    e = launch_expert_rows(FfnKind::GradX, dtype, a, p, stride_w, plan, s);
  }
  if (e == hipSuccess && dWd) {
    FfnGemm a = rows_gemm(H, ldh, dys, K, K, 0, p, dWd, lddw);
    a.M = N;
    e = launch_expert_grad_w(dtype, a, p, stride_dw, s);
  }
  return hip_status(e);
}
