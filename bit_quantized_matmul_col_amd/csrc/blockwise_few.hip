// The block-scaled FP8 product for few rows (single tokens, decoding batches): W's codes are read
// once and bound everything.
//
// A wave reads W from memory straight into the MFMA's registers: both codes and
// MFMA run along the reduction, a load of 16 bytes a lane covers 64 bytes of each of 16 columns,
// and nothing is shared that LDS would save. It keeps D blocks of the reduction in flight
// in registers; the waves of a block take the blocks of the reduction in turn, and their
// sums meet in LDS in a fixed order. For the fewest rows X comes in 16 bits and every wave codes
// what it needs itself, which its loads of W leave time for, so that a token is one launch;
// for more rows a pass has coded X before.
#include "blockwise_math.hpp"

namespace llmint8 {
namespace fp8 {

template <class T_, int MT_, int NB_, int WAVES_, bool FUSED_>
struct FewCfg {
  using T = T_;
  static constexpr int MT = MT_, NB = NB_, WAVES = WAVES_;  // row tiles, column tiles, waves
  static constexpr bool FUSED = FUSED_;
  static constexpr int D = NB * MT >= 8 || (FUSED && NB == 4) ? 2 : 4;  // blocks in flight
  static constexpr int CB = 16 * NB, THREADS = 64 * WAVES;
  static constexpr int REDP = CB + 4;  // fp32 pitch of the joined sums
  static constexpr int LDS = WAVES * 16 * MT * REDP * 4;
  static_assert(!FUSED || MT == 1, "one tile of rows is coded in place");
};

__device__ inline i32x4 load16(rsrc_t rs, int off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

template <class C>
__global__ __launch_bounds__(C::THREADS, 1) void k_fp8_few(Fp8Gemm a) {
  using T = typename C::T;
  constexpr int MT = C::MT, NB = C::NB, D = C::D;
  extern __shared__ u32x4 smem_v[];
  const int t = threadIdx.x, lane = t & 63, wv = wave_id(), i = lane & 15, g = lane >> 4;
  const FfnGemm &o = a.out;
  const uint32_t groups = (uint32_t)((o.M + 16 * MT - 1) / (16 * MT));
  const uint32_t place = xcd_place(blockIdx.x, gridDim.x);
  const int64_t n0 = (int64_t)(place / groups) * C::CB, m0 = (int64_t)(place % groups) * 16 * MT;
  const int64_t rows = o.M - m0 < 16 * MT ? o.M - m0 : 16 * MT;
  const int64_t cols = o.N - n0 < C::CB ? o.N - n0 : C::CB;
  const int K = (int)a.K, nb = (K + kFp8Block - 1) / kFp8Block;

  const rsrc_t rw = make_rsrc(a.w.codes + n0 * K, cols * K);
  const uint8_t *const sw = a.w.scales + n0 / kFp8Block * a.w.lds;
  const rsrc_t rsw = make_rsrc(sw, nb);
  const rsrc_t rx = C::FUSED ? make_rsrc(a.x16 + m0 * a.ldx, ((rows - 1) * a.ldx + K) * 2)
                             : make_rsrc(a.x.codes + m0 * K, rows * K);
  const rsrc_t rsx = make_rsrc(C::FUSED ? sw : a.x.scales + m0 * a.x.lds,
                               C::FUSED ? 0 : rows * a.x.lds);

  // What a block of the reduction needs: chunks g and g + 4 (16 codes each) of every
  // column's and row's 128.
  struct Stage {
    i32x4 w[NB][2];
    i32x4 x[C::FUSED ? 4 : 2 * MT];
    int sw, sx[MT];
  };
  auto load = [&](Stage &st, int b) {
    const int k = b * kFp8Block + 16 * g;
    const bool in0 = b < nb && k < K, in1 = b < nb && k + 64 < K;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int off = (16 * n + i) * K + k;
      st.w[n][0] = load16(rw, in0 ? off : kOob);
      st.w[n][1] = load16(rw, in1 ? off + 64 : kOob);
    }
    if constexpr (C::FUSED) {
      const int off = (i * (int)a.ldx + k) * 2;
      const bool row = i < rows;
      st.x[0] = load16(rx, row && in0 ? off : kOob);
      st.x[1] = load16(rx, row && in0 ? off + 16 : kOob);
      st.x[2] = load16(rx, row && in1 ? off + 128 : kOob);
      st.x[3] = load16(rx, row && in1 ? off + 144 : kOob);
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = 16 * m + i, off = r * K + k;
        st.x[2 * m] = load16(rx, in0 ? off : kOob);
        st.x[2 * m + 1] = load16(rx, in1 ? off + 64 : kOob);
        const int at = b < nb ? r * (int)a.x.lds + b : kOob;
        st.sx[m] = __builtin_amdgcn_raw_buffer_load_b8(rsx, at, 0, 0);
      }
    }
    st.sw = __builtin_amdgcn_raw_buffer_load_b8(rsw, b < nb ? b : kOob, 0, 0);
  };

  f32x4 acc[NB][MT];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = (f32x4){};
  auto compute = [&](const Stage &st) {
    i32x8 x[MT];
    int sx[MT];
    if constexpr (C::FUSED) {
      float v[32];
      uint32_t top = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u16x8 h = __builtin_bit_cast(u16x8, st.x[q]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * q + e] = T::to_f(h[e]);
        const uint32_t m = top8(v + 8 * q);
        top = m > top ? m : top;
      }
#pragma unroll
      for (int off = 16; off < 64; off <<= 1) {
        const uint32_t u = __shfl_xor(top, off, kWave);
        top = u > top ? u : top;
      }
      const uint32_t byte = scale_byte(top);
      sx[0] = (int)byte;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[0][q] = (int)codes4(v + 4 * q, byte);
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        x[m] = pair(st.x[2 * m], st.x[2 * m + 1]);
        sx[m] = st.sx[m] & 0xff;
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        acc[n][m] = mfma_block(pair(st.w[n][0], st.w[n][1]), x[m], acc[n][m], st.sw & 0xff, sx[m]);
  };

  Stage st[D];
#pragma unroll
  for (int q = 0; q < D; ++q) load(st[q], wv + q * C::WAVES);
  // past the last block the loads give zeros, codes and scales, which add nothing
  for (int b = wv; b < nb; b += D * C::WAVES)
#pragma unroll
    for (int q = 0; q < D; ++q) {
      compute(st[q]);
      load(st[q], b + (D + q) * C::WAVES);
    }

  // Lane l of an accumulator holds row l % 16, columns 4 (l / 16) .. + 3.
  float *red = (float *)smem_v;
  constexpr int PLANE = 16 * MT * C::REDP;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      *(f32x4 *)(red + wv * PLANE + (m * 16 + i) * C::REDP + n * 16 + 4 * g) = acc[n][m];
  __syncthreads();
  constexpr int CPR = C::CB / 8;
  for (int x = t; x < (int)rows * CPR; x += C::THREADS) {
    const int m = x / CPR, c8 = (x % CPR) * 8;
    if (c8 >= cols) continue;
    float v[8], u[8];
    load_f8(red + m * C::REDP + c8, v);
#pragma unroll
    for (int w = 1; w < C::WAVES; ++w) {
      load_f8(red + w * PLANE + m * C::REDP + c8, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += u[e];
    }
    load_bias<T>(o, n0 + c8, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += u[e];
    store8<T>(o.y[0] + (m0 + m) * o.ldy + n0 + c8, v);
  }
}

template <class C>
hipError_t launch_few_cfg(const Fp8Gemm &a, hipStream_t s) {
  auto *kern = k_fp8_few<C>;
  hipError_t e = hipFuncSetAttribute((const void *)kern,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  const int64_t groups = (a.out.M + 16 * C::MT - 1) / (16 * C::MT);
  const int64_t blocks = (a.out.N + C::CB - 1) / C::CB * groups;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(C::THREADS), C::LDS, s, a);
  return hipGetLastError();
}

template <class T, int MT, bool FUSED>
hipError_t launch_few_cols(const Fp8Gemm &a, int cols, hipStream_t s) {
  if (cols == 16) return launch_few_cfg<FewCfg<T, MT, 1, 8, FUSED>>(a, s);
  if (cols == 32) return launch_few_cfg<FewCfg<T, MT, 2, 4, FUSED>>(a, s);
  return launch_few_cfg<FewCfg<T, MT, 4, 4, FUSED>>(a, s);
}

template <class T>
hipError_t launch_few_type(const Fp8Gemm &a, const Fp8Plan &p, hipStream_t s) {
  return p.fused ? launch_few_cols<T, 1, true>(a, p.cols, s)
                 : launch_few_cols<T, 2, false>(a, p.cols, s);
}

}  // namespace fp8

hipError_t launch_fp8_few(int dtype, const Fp8Gemm &a, const Fp8Plan &p, hipStream_t s) {
  return dtype == 0 ? fp8::launch_few_type<Half>(a, p, s) : fp8::launch_few_type<Bfloat>(a, p, s);
}

}  // namespace llmint8
