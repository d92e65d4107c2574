// 16-bit matrices to block-scaled E4M3: X by rows, W by 128 x 128 blocks and transposed. Each entry
// is read once. X is bound by memory: 8192 x 8192 bf16 36.5 us, 5.5 TB/s of reads and writes
// together. W is bound by LDS: 8192 x 28672 221 us, 3.2 TB/s; LDS is busy for 0.88 of the time, 0.81
// with bank conflicts, as the bytes that a transposed entry is written in fall in two banks for the 16
// lanes of a row.
#include "blockwise_math.hpp"

namespace llmint8 {
namespace fp8 {

constexpr int kThreads = 256;

// 16 lanes have a block of a row, 8 entries each. The scales' rows are padded to a multiple of
// 4 bytes, which are written too.
template <class T>
__global__ __launch_bounds__(kThreads) void k_quant_rows(const uint16_t *x, int64_t M, int64_t K,
                                                         int64_t ldx, uint8_t *codes,
                                                         uint8_t *scales, int64_t lds,
                                                         int64_t pad) {
  const int t = threadIdx.x, l = t % 16;
  const int64_t blocks = M * pad;
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 16) + t / 16; i < blocks;
       i += (int64_t)gridDim.x * (kThreads / 16)) {
    const int64_t row = i / pad, b = i % pad, k = b * kFp8Block + 8 * l;
    const bool in = k < K;
    float v[8] = {0.f};
    if (in) load8<T>(x + row * ldx + k, v);
    uint32_t top = top8(v);
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      const uint32_t o = __shfl_xor(top, off, kWave);
      top = o > top ? o : top;
    }
    const uint32_t byte = scale_byte(top);
    if (in) *(u32x2 *)(codes + row * K + k) = u32x2{codes4(v, byte), codes4(v + 4, byte)};
    if (l == 0) scales[row * lds + b] = (uint8_t)byte;
  }
}

// A block of the grid has one 128 x 128 block of W: thread t the rows t / 16 + 16 j, columns
// 8 (t % 16) .. + 7. The codes meet in LDS, transposed, and go out in rows of 128 bytes.
template <class T>
__global__ __launch_bounds__(kThreads) void k_quant_weights(const uint16_t *w, int64_t K, int64_t N,
                                                            int64_t ldw, uint8_t *codes,
                                                            uint8_t *scales, int64_t lds) {
  constexpr int PITCH = kFp8Block + 16;
  __shared__ u32x4 out_v[kFp8Block * PITCH / 16];
  __shared__ uint32_t tops[kThreads / kWave];
  uint8_t *const out = (uint8_t *)out_v;
  const int t = threadIdx.x, c8 = t % 16 * 8, r = t / 16;
  const int64_t k0 = (int64_t)blockIdx.x * kFp8Block, n0 = (int64_t)blockIdx.y * kFp8Block;
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t k = k0 + r + 16 * j, n = n0 + c8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = 0.f;
    if (k < K && n < N) load8<T>(w + k * ldw + n, v[j]);
    const uint32_t m = top8(v[j]);
    top = m > top ? m : top;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = __shfl_xor(top, off, kWave);
    top = o > top ? o : top;
  }
  if (t % kWave == 0) tops[t / kWave] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / kWave; ++i) top = tops[i] > top ? tops[i] : top;
  const uint32_t byte = scale_byte(top);
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t c = codes4(v[j] + 4 * q, byte);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[(c8 + 4 * q + e) * PITCH + r + 16 * j] = (uint8_t)(c >> (8 * e));
    }
  __syncthreads();
  for (int i = t; i < kFp8Block * 8; i += kThreads) {
    const int n = i / 8, c = i % 8 * 16;
    if (n0 + n < N && k0 + c < K)  // K is a multiple of 16
      *(u32x4 *)(codes + (n0 + n) * K + k0 + c) = *(const u32x4 *)(out + n * PITCH + c);
  }
  if (t == 0) scales[blockIdx.y * lds + blockIdx.x] = (uint8_t)byte;
}

}  // namespace fp8

hipError_t launch_quant_rows_fp8(int dtype, const uint16_t *x, int64_t M, int64_t K, int64_t ldx,
                                 uint8_t *codes, uint8_t *scales, int64_t lds, hipStream_t s) {
  using namespace fp8;
  const int64_t pad = fp8_scale_pitch(K), per = kThreads / 16;
  int64_t grid = (M * pad + per - 1) / per;
  if (grid > 1 << 20) grid = 1 << 20;
  auto *kern = dtype == 0 ? k_quant_rows<Half> : k_quant_rows<Bfloat>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kThreads), 0, s, x, M, K, ldx, codes, scales,
                     lds, pad);
  return hipGetLastError();
}

hipError_t launch_quant_weights_fp8(int dtype, const uint16_t *w, int64_t K, int64_t N,
                                    int64_t ldw, uint8_t *codes, uint8_t *scales, hipStream_t s) {
  using namespace fp8;
  const int64_t kb = (K + kFp8Block - 1) / kFp8Block, nb = (N + kFp8Block - 1) / kFp8Block;
  auto *kern = dtype == 0 ? k_quant_weights<Half> : k_quant_weights<Bfloat>;
  hipLaunchKernelGGL(kern, dim3((unsigned)kb, (unsigned)nb), dim3(kThreads), 0, s, w, K, N, ldw,
                     codes, scales, kb);
  return hipGetLastError();
}

}  // namespace llmint8
