// Block-scaled FP8: E4M3 codes in blocks of 128 along the reduction that share a power-of-two
// scale (of a row of X; of 128 columns of W), and the product of two such matrices.
//
// The scale 2^e of a block is the smallest with max |x| <= 448 2^e, held as the byte e + 127 (E8M0,
// at least 0). Dividing by it is exact, so a code is the one rounding of its entry, whatever
// order or precision anything is computed in; and the scaled MFMA of gfx950 takes such bytes
// next to its operands, so that the scales cost the product no instruction: its sums stay in the
// fp32 accumulators from the first block to the last. A block with an infinity or a NaN takes
// the byte 255 and NaN codes throughout.
#pragma once

#include "ffn.hpp"

namespace llmint8 {

constexpr int kFp8Block = 128;
constexpr int64_t kFp8MaxK = 131072;  // W's scales of a tile's columns are kept in LDS

// Codes [rows x K] without gaps, scale bytes [.. x lds].
struct Fp8Codes {
  const uint8_t *codes;
  const uint8_t *scales;
  int64_t lds;
};

// Y = X W + bias. For few rows X may be the 16-bit matrix itself (x.codes null).
struct Fp8Gemm {
  Fp8Codes x, w;  // x.lds a multiple of 4, its scales 4-byte aligned
  const uint16_t *x16;
  int64_t ldx;
  int64_t K;
  FfnGemm out;  // M, N, y, ldy, bias, part, ksplit
};

// The few-row kernel with `cols` columns a block, X coded in it or not; or tiles of `tile` rows
// and columns.
struct Fp8Plan {
  bool few, fused;
  int tile, ksplit, cols;
};
Fp8Plan fp8_plan(int64_t M, int64_t K, int64_t N);

// Row pitch of X's scales: a tile reads four blocks' bytes at a time.
inline int64_t fp8_scale_pitch(int64_t K) { return (K + 4 * kFp8Block - 1) / (4 * kFp8Block) * 4; }

hipError_t launch_quant_rows_fp8(int dtype, const uint16_t *x, int64_t M, int64_t K, int64_t ldx,
                                 uint8_t *codes, uint8_t *scales, int64_t lds, hipStream_t s);
hipError_t launch_quant_weights_fp8(int dtype, const uint16_t *w, int64_t K, int64_t N,
                                    int64_t ldw, uint8_t *codes, uint8_t *scales, hipStream_t s);
hipError_t launch_fp8_tiles(int dtype, const Fp8Gemm &a, int tile, hipStream_t s);
hipError_t launch_fp8_few(int dtype, const Fp8Gemm &a, const Fp8Plan &p, hipStream_t s);

}  // namespace llmint8
