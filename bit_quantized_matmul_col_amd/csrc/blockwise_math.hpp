// Device arithmetic of the block-scaled FP8 kernels.
#pragma once

#include "blockwise.hpp"
#include "ffn_gemm.hpp"

namespace llmint8 {
namespace fp8 {

using namespace ffn;

constexpr uint32_t kNanByte = 255;

// The scale byte of a block whose largest magnitude has these fp32 bits: 448 = 1.75 x 2^8.
__device__ inline uint32_t scale_byte(uint32_t top) {
  const int e = (int)(top >> 23);
  if (e == 255) return kNanByte;
  const int b = e - 8 + ((top & 0x7fffffu) > 0x600000u);
  return (uint32_t)(b > 0 ? b : 0);
}

// 2^-(byte - 127): exact for every byte that scale_byte gives but 255, whose codes are NaN.
__device__ inline float scale_inverse(uint32_t byte) {
  return __builtin_bit_cast(float, (254u - byte) << 23);
}

// Codes of 4 entries of a block.
__device__ inline uint32_t codes4(const float *v, uint32_t byte) {
  if (byte == kNanByte) return 0x7f7f7f7fu;
  const float s = scale_inverse(byte);
  const float t[4] = {v[0] * s, v[1] * s, v[2] * s, v[3] * s};
  return CodecE4M3::code4(t);
}

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 columns of W by 16 rows of X over a block of 128: lane l gives 32 codes of column (row)
// l % 16, the same places of the block for both, and the scale byte of it; it receives row
// l % 16, columns 4 (l / 16) .. + 3.
__device__ inline f32x4 mfma_block(i32x8 w, i32x8 x, f32x4 c, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, sw, 0, sx);
}

__device__ inline i32x8 pair(i32x4 a, i32x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

}  // namespace fp8
}  // namespace llmint8
