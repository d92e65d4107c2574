// Row-streaming kernels of the 16-bit feed-forward operators: checkpoint pack
// and unpack, the gradient of the activation (with the bias gradient), the
// gradient of the gate, and the pass that joins a split reduction. All are
// bound by HBM; a thread owns 8 consecutive columns (16 bytes) of a row, and the
// grid holds a block per 256 chunks, so that the chip's memory system is kept full
// by many short blocks rather than by loops. Measured (MI355X):
//   pack, unpack        4096 x 13824 bf16     36, 31 us (4.7, 5.5 TB/s; with 2 or 4
//                       rows a thread in flight 35 to 36 and 32 to 33)
//   gated gradients     2048 x 11008 fp16     38 us (225 MB, 5.9 TB/s)
//   activation's        2048 x 4096 bf16, with the bias gradient 14.8 us (50 MB),
//                       4096 x 11008 50 us (5.4 TB/s)
//   join                2 parts of 2048 x 4096, residual 16 us (101 MB, 6.3 TB/s)
#include "ffn_rows.hpp"

namespace llmint8 {

namespace {

using namespace ffn_rows;

// 8 entries of a saved matrix. The scale byte is shared by 4 lanes.
template <class T, bool Q8>
__device__ inline void load_saved(const Saved &s, int64_t i, int64_t n, float *v) {
  if constexpr (Q8) {
    const u32x2 w = *(const u32x2 *)((const uint8_t *)s.data + i * s.ld + n);
    const float scale = ckpt_scale(s.scales[i * s.lds + n / kCkptBlock]);
    ckpt_value4(w[0], scale, v);
    ckpt_value4(w[1], scale, v + 4);
  } else {
    load8<T>((const uint16_t *)s.data + i * s.ld + n, v);
  }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_ckpt_pack(const uint16_t *x, int64_t M, int64_t K,
                                                        int64_t ldx, Saved out, int cx_log2) {
  for_rows(cx_log2, M, K, [&](int64_t i, int64_t n, bool in) {
    float v[8] = {0.f};
    if (in) load8<T>(x + i * ldx + n, v);
    ffn::save8<T>(out.data, out.ld, out.scales, out.lds, i, n, in, v);
  });
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_ckpt_unpack(Saved in8, int64_t M, int64_t K,
                                                          uint16_t *x, int64_t ldx, int cx_log2) {
  for_rows(cx_log2, M, K, [&](int64_t i, int64_t n, bool in) {
    if (!in) return;
    float v[8];
    load_saved<T, true>(in8, i, n, v);
    store8<T>(x + i * ldx + n, v);
  });
}

// dG = dH U act'(G), dU = dH act(G), computed in fp32 and rounded to 16 bits: they are
// operands of 16-bit MFMAs, as dZ below is. Against 64 bits the gradients then are off by
// 1.4 times what a gradient rounded once is (0.0023 to 0.0024 against 0.0017 of their norm
// in bf16, 0.00029 against 0.00021 in fp16: two independent roundings of one size);
// products of two 16-bit halves of each would take twice the MFMAs to avoid it.
template <class T, bool Q8>
__global__ __launch_bounds__(kThreads) void k_gated_grad(int act, const uint16_t *dh, int64_t lddh,
                                                         Saved g, Saved u, int64_t M, int64_t N,
                                                         uint16_t *dg, uint16_t *du, int64_t ldd,
                                                         int cx_log2) {
  for_rows(cx_log2, M, N, [&](int64_t i, int64_t n, bool in) {
    if (!in) return;
    float h[8], gv[8], uv[8];
    load8<T>(dh + i * lddh + n, h);
    load_saved<T, Q8>(g, i, n, gv);
    load_saved<T, Q8>(u, i, n, uv);
    with_act(act, [&](auto tag) {
      constexpr int A = decltype(tag)::value;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = gv[e];
        gv[e] = h[e] * uv[e] * act_grad<A>(z);
        uv[e] = h[e] * act_of<A>(z);
      }
    });
    store8<T>(dg + i * ldd + n, gv);
    store8<T>(du + i * ldd + n, uv);
  });
}

// dz = dy act'(z), rounded to 16 bits for the products (see k_gated_grad), and, with
// part, the column sums of the unrounded dz over this block's rows in fp32: each thread sums its own rows, LDS joins the block's, join_bias the blocks'.
// Always in the same order, so the result does not vary. A thread's rows go four
// at a time, with their loads in flight together, so a grid of one row a thread, which
// suits the passes above, would waste the other three (4096 x 64 x 11008 without the
// bias gradient: 167 us for the whole call against 100).
template <class T>
__global__ __launch_bounds__(kThreads) void k_act_grad(int act, const uint16_t *dy, int64_t lddy,
                                                       const uint16_t *z, int64_t ldz, int64_t M,
                                                       int64_t N, uint16_t *dz, int64_t lddz,
                                                       float *part, int cx_log2) {
  constexpr int R = 4;
  const int t = threadIdx.x, cx = 1 << cx_log2;
  const int64_t n = (((int64_t)blockIdx.x << cx_log2) + (t & (cx - 1))) * 8;
  const int64_t ry = kThreads >> cx_log2, step = gridDim.y * ry;
  float sum[8] = {0.f};
  for (int64_t i0 = blockIdx.y * ry + (t >> cx_log2); i0 < M; i0 += R * step) {
    float d[R][8], zv[R][8];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t i = i0 + q * step;
      if (i < M && n < N) {
        load8<T>(dy + i * lddy + n, d[q]);
        if (act != LLMINT8_ACT_NONE) load8<T>(z + i * ldz + n, zv[q]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[q][e] = zv[q][e] = 0.f;
      }
    }
    if (act != LLMINT8_ACT_NONE)
      with_act(act, [&](auto tag) {
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) d[q][e] *= act_grad<decltype(tag)::value>(zv[q][e]);
      });
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t i = i0 + q * step;
      if (dz && i < M && n < N) store8<T>(dz + i * lddz + n, d[q]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += d[q][e];
    }
  }
  if (!part) return;
  __shared__ float s[kThreads][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[t][e] = sum[e];
  __syncthreads();
  if (t < cx && n < N) {
    for (int r = t + cx; r < kThreads; r += cx)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += s[r][e];
    ffn::store_f8(part + (int64_t)blockIdx.y * N + n, sum);
  }
}

constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void k_bias_join(BiasJoin j) {
  __shared__ float s[64 * 64];
  ffn::join_bias<kJoinThreads>(j, blockIdx.x, s);
}

// Joins the partial sums of a split reduction and runs the epilogue.
template <class T, bool GATED>
__global__ __launch_bounds__(kThreads) void k_ffn_finish(FfnGemm a, int cx_log2) {
  const int64_t plane = a.M * a.N;
  const int out = blockIdx.z;
  for_rows(cx_log2, a.M, a.N, [&](int64_t i, int64_t n, bool in) {
    float v[8] = {0.f}, u[8] = {0.f};
    if (in) {
      const int64_t per = (GATED ? 2 : a.outs) * plane;
      const float *p = a.part + (GATED ? 0 : out) * plane + i * a.N + n;
      join_parts(p, per, a.ksplit, v);
      if constexpr (GATED) join_parts(p + plane, per, a.ksplit, u);
    }
    if constexpr (GATED)
      ffn::finish_gated<T>(a, i, n, in, v, u);
    else if (in) {
      float b[8];
      ffn::load_bias<T>(a, n, b);
      ffn::finish_forward<T>(a, out, i, n, v, b, ffn::load_residual(a, i, n));
    }
  });
}

}  // namespace

hipError_t launch_ckpt_pack(int dtype, const uint16_t *x, int64_t M, int64_t K, int64_t ldx,
                            const Saved &out, hipStream_t s) {
  const RowGrid g = row_grid(M, K, kMaxGridY);
  auto *kern = dtype == LLMINT8_FP16 ? k_ckpt_pack<Half> : k_ckpt_pack<Bfloat>;
  hipLaunchKernelGGL(kern, g.grid, dim3(kThreads), 0, s, x, M, K, ldx, out, g.cx_log2);
  return hipGetLastError();
}

hipError_t launch_ckpt_unpack(int dtype, const Saved &in, int64_t M, int64_t K, uint16_t *x,
                              int64_t ldx, hipStream_t s) {
  const RowGrid g = row_grid(M, K, kMaxGridY);
  auto *kern = dtype == LLMINT8_FP16 ? k_ckpt_unpack<Half> : k_ckpt_unpack<Bfloat>;
  hipLaunchKernelGGL(kern, g.grid, dim3(kThreads), 0, s, in, M, K, x, ldx, g.cx_log2);
  return hipGetLastError();
}

hipError_t launch_gated_grad(int dtype, int act, const uint16_t *dh, int64_t lddh, const Saved &g,
                             const Saved &u, int64_t M, int64_t N, uint16_t *dg, uint16_t *du,
                             int64_t ldd, hipStream_t s) {
  const RowGrid r = row_grid(M, N, kMaxGridY);
  auto *kern = dtype == LLMINT8_FP16
                   ? (g.scales ? k_gated_grad<Half, true> : k_gated_grad<Half, false>)
                   : (g.scales ? k_gated_grad<Bfloat, true> : k_gated_grad<Bfloat, false>);
  hipLaunchKernelGGL(kern, r.grid, dim3(kThreads), 0, s, act, dh, lddh, g, u, M, N, dg, du, ldd,
                     r.cx_log2);
  return hipGetLastError();
}

// Row blocks of the activation's gradient: a thread's rows in fours (see k_act_grad),
// as few as leave no more than 256 row blocks for join_bias, or 512 blocks in all
// where the columns are few. 2048 x 4096 with the bias gradient, 8 rows a thread 14.8 us,
// 4 (512 row blocks) 16.6, 16 18.2; 4096 x 11008 16 rows 50.0, 48 69.0.
int64_t bias_rows(int64_t M, int64_t N) {
  const RowGrid g = row_grid(M, N, kMaxGridY);
  const int64_t ry = kThreads >> g.cx_log2, all = 512 / (int64_t)g.grid.x;
  const int64_t most = all > 256 ? all : 256;
  const int64_t per = 4 * ((M + 4 * ry * most - 1) / (4 * ry * most));  // rows a thread
  return (M + ry * per - 1) / (ry * per);
}

hipError_t launch_act_grad(int dtype, int act, const uint16_t *dy, int64_t lddy, const uint16_t *z,
                           int64_t ldz, int64_t M, int64_t N, uint16_t *dz, int64_t lddz,
                           float *part, hipStream_t s) {
  const RowGrid g = row_grid(M, N, bias_rows(M, N));
  auto *kern = dtype == LLMINT8_FP16 ? k_act_grad<Half> : k_act_grad<Bfloat>;
  hipLaunchKernelGGL(kern, g.grid, dim3(kThreads), 0, s, act, dy, lddy, z, ldz, M, N, dz, lddz,
                     part, g.cx_log2);
  return hipGetLastError();
}

hipError_t launch_bias_join(const BiasJoin &j, hipStream_t s) {
  hipLaunchKernelGGL(k_bias_join, dim3((unsigned)((j.N + 63) / 64)), dim3(kJoinThreads), 0, s, j);
  return hipGetLastError();
}

hipError_t launch_ffn_finish(int dtype, bool gated, const FfnGemm &a, hipStream_t s) {
  RowGrid g = row_grid(a.M, a.N, kMaxGridY);
  if (!gated) g.grid.z = a.outs;
  auto *kern = dtype == LLMINT8_FP16
                   ? (gated ? k_ffn_finish<Half, true> : k_ffn_finish<Half, false>)
                   : (gated ? k_ffn_finish<Bfloat, true> : k_ffn_finish<Bfloat, false>);
  hipLaunchKernelGGL(kern, g.grid, dim3(kThreads), 0, s, a, g.cx_log2);
  return hipGetLastError();
}

}  // namespace llmint8
