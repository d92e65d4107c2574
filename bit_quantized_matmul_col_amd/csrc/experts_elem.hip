// Row-streaming passes of the experts' products: rows taken in the experts' order, the gradient
// of the gate with that of the weights, and the sums over a token's experts. All are bound by
// HBM; see ffn_elem.hip for the grid.
#include "experts.hpp"
#include "ffn_rows.hpp"

namespace llmint8 {

namespace {

using namespace ffn_rows;

__device__ inline int64_t last_row(const Pairs &p) {
  const int64_t n = p.offsets[p.E];
  return n < p.rows() ? n : p.rows();
}

__global__ __launch_bounds__(kThreads) void k_take_rows(const uint16_t *x, int64_t ldx, int64_t N,
                                                        Pairs p, uint16_t *out, int cx_log2) {
  for_rows(cx_log2, last_row(p), N, [&](int64_t r, int64_t n, bool in) {
    const uint32_t token = (uint32_t)p.order[r] / (uint32_t)p.k;
    if (in && (int64_t)token < p.tokens)
      *(u32x4 *)(out + r * N + n) = *(const u32x4 *)(x + token * ldx + n);
  });
}

// The rows of a token's pairs come in fp32, the second product's and dX's alike, and are summed in the
// order of its choices; the sum is rounded once. Rows in 16 bits would be half the bytes (the second
// product of 4096 tokens x 4 of 32 experts, 2048 x 4096: 339 us instead of 397), but they may cancel,
// or lie beyond fp16's range, where their sum does not.
template <class T>
__global__ __launch_bounds__(kThreads) void k_combine(Combine c, Pairs p, int cx_log2) {
  const int64_t rows = p.rows();
  for_rows(cx_log2, p.tokens, c.N, [&](int64_t i, int64_t n, bool in) {
    if (!in) return;
    float v[8] = {0.f};
    if (c.residual) load8<T>(c.residual + i * c.ldr + n, v);
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      float x[4][8];
      bool has[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t r = j0 + q < p.k ? p.places[i * p.k + j0 + q] : -1;
        has[q] = r >= 0 && r < rows;
        if (!has[q]) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[q][e] = 0.f;
        join_parts(c.part + r * c.N + n, rows * c.N, c.parts, x[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (has[q])
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += x[q][e];
    }
    store8<T>(c.y + i * c.ldy + n, v);
  });
}

// A wave has a pair: its row's dw is a sum over the row, which stays within the wave. Pairs in
// their own order, so that those without an expert are seen too (dw = 0). dG and dU are
// rounded to 16 bits as operands of the products (see k_gated_grad); dw sums the unrounded.
template <class T>
__global__ __launch_bounds__(kThreads) void k_expert_gated_grad(
    int act, const uint16_t *dh, int64_t lddh, const uint16_t *g, const uint16_t *u, int64_t ldz,
    int64_t N, Pairs p, const float *w, uint16_t *dg, uint16_t *du, float *dw) {
  const int lane = threadIdx.x & 63;
  const int64_t pair = (int64_t)blockIdx.x * (kThreads / kWave) + ffn::wave_id();
  if (pair >= p.rows()) return;
  const int64_t r = p.places[pair];
  if (r < 0 || r >= p.rows()) {
    if (dw && lane == 0) dw[pair] = 0.f;
    return;
  }
  const float wr = w ? w[pair] : 1.f;
  float sum = 0.f;
  for (int64_t n = 8 * lane; n < N; n += 8 * kWave) {
    float h[8], gv[8], uv[8];
    load8<T>(dh + r * lddh + n, h);
    load8<T>(g + r * ldz + n, gv);
    load8<T>(u + r * ldz + n, uv);
    with_act(act, [&](auto tag) {
      constexpr int A = decltype(tag)::value;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = gv[e], a = act_of<A>(z), d = wr * h[e];
        sum += h[e] * a * uv[e];
        gv[e] = d * uv[e] * act_grad<A>(z);
        uv[e] = d * a;
      }
    });
    store8<T>(dg + r * N + n, gv);
    store8<T>(du + r * N + n, uv);
  }
  if (!dw) return;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if (lane == 0) dw[pair] = sum;
}

// Joins the parts of a gated product and runs its epilogue, on the rows that there are.
template <class T>
__global__ __launch_bounds__(kThreads) void k_expert_gated_finish(FfnGemm a, Pairs p, int cx_log2) {
  const int64_t plane = a.all_rows * a.N;
  for_rows(cx_log2, last_row(p), a.N, [&](int64_t i, int64_t n, bool in) {
    float v[8] = {0.f}, u[8] = {0.f};
    if (in) {
      const float *part = a.part + i * a.N + n;
      join_parts(part, 2 * plane, a.ksplit, v);
      join_parts(part + plane, 2 * plane, a.ksplit, u);
    }
    ffn::finish_gated<T, true>(a, i, n, in, v, u);
  });
}

}  // namespace

hipError_t launch_take_rows(int, const uint16_t *x, int64_t ldx, int64_t cols, const Pairs &p,
                            uint16_t *out, hipStream_t s) {
  const RowGrid g = row_grid(p.rows(), cols, kMaxGridY);
  hipLaunchKernelGGL(k_take_rows, g.grid, dim3(kThreads), 0, s, x, ldx, cols, p, out, g.cx_log2);
  return hipGetLastError();
}

hipError_t launch_combine(int dtype, const Combine &c, const Pairs &p, hipStream_t s) {
  const RowGrid g = row_grid(p.tokens, c.N, kMaxGridY);
  auto *kern = dtype == LLMINT8_FP16 ? k_combine<Half> : k_combine<Bfloat>;
  hipLaunchKernelGGL(kern, g.grid, dim3(kThreads), 0, s, c, p, g.cx_log2);
  return hipGetLastError();
}

hipError_t launch_expert_gated_grad(int dtype, int act, const uint16_t *dh, int64_t lddh,
                                    const uint16_t *g, const uint16_t *u, int64_t ldz, int64_t N,
                                    const Pairs &p, const float *w, uint16_t *dg, uint16_t *du,
                                    float *dw, hipStream_t s) {
  constexpr int64_t per = kThreads / kWave;
  auto *kern = dtype == LLMINT8_FP16 ? k_expert_gated_grad<Half> : k_expert_gated_grad<Bfloat>;
  hipLaunchKernelGGL(kern, dim3((unsigned)((p.rows() + per - 1) / per)), dim3(kThreads), 0, s, act,
                     dh, lddh, g, u, ldz, N, p, w, dg, du, dw);
  return hipGetLastError();
}

hipError_t launch_expert_gated_finish(int dtype, const FfnGemm &a, const Pairs &p, hipStream_t s) {
  const RowGrid g = row_grid(a.M, a.N, kMaxGridY);
  auto *kern =
      dtype == LLMINT8_FP16 ? k_expert_gated_finish<Half> : k_expert_gated_finish<Bfloat>;
  hipLaunchKernelGGL(kern, g.grid, dim3(kThreads), 0, s, a, p, g.cx_log2);
  return hipGetLastError();
}

}  // namespace llmint8
