// Device arithmetic of the 16-bit feed-forward kernels: the two 16-bit types,
// the activations with their derivatives, and the 8-bit checkpoint blocks.
#pragma once

#include "ffn.hpp"
#include "llmint8.h"

namespace llmint8 {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct Half {
  __device__ static float to_f(uint16_t u) { return (float)__builtin_bit_cast(_Float16, u); }
  __device__ static uint16_t from_f(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
  __device__ static f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};

struct Bfloat {
  __device__ static float to_f(uint16_t u) { return __builtin_bit_cast(float, (uint32_t)u << 16); }
  __device__ static uint16_t from_f(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
  __device__ static f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};

template <class T>
__device__ inline void load8(const uint16_t *p, float *v) {
  const u16x8 h = __builtin_bit_cast(u16x8, *(const u32x4 *)p);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = T::to_f(h[e]);
}

template <class T>
__device__ inline void store8(uint16_t *p, const float *v) {
  u16x8 h;
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = T::from_f(v[e]);
  *(u32x4 *)p = __builtin_bit_cast(u32x4, h);
}

// 1 / (1 + e^-z). e^-z overflows to infinity for z below -88.7, whose reciprocal
// is 0 for a value below 3e-39. The hardware exponential and reciprocal are good to
// about 1 ulp of fp32 each, far below the 16-bit rounding of every result.
__device__ inline float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

constexpr float kTanhA = 1.5957691216f;   // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// e^(-z^2 / 2), which the normal density and distribution share. Zero from |z| = 13.2 on,
// where the hardware exponential's result would be subnormal.
__device__ inline float normal_exp(float z) {
  return __builtin_amdgcn_exp2f(-0.72134752f * z * z);
}

// Phi(z) = erfc(-z / sqrt 2) / 2 with e = normal_exp(z). The tail Phi(-|z|) is e t P(t),
// t = 1 / (1 + 0.305 |z|): P has the smallest largest relative error of its degree over
// |z| up to 14.5 (a least-squares fit of the scaled tail, reweighted until the ripples
// were level), 1.0e-7, 4.2e-7 with its roundings in fp32. From the tail itself rather than
// from 1 + erf(z / sqrt 2), which cancels below -3 (4 % off at -5, nothing left from -5.8
// on), and without the branches of the library's functions. A NaN stays NaN.
__device__ inline float normal_cdf(float z, float e) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.305f * __builtin_fabsf(z));
  const float p = 0.121640244f + t * (0.122458658f + t * (0.103473846f + t * (0.120839870f +
                  t * (-0.0376196416f + t * (0.185313750f + t * (-0.152745381f + t * 0.0366386891f))))));
  const float q = e * t * p;
  return z < 0.f ? q : 1.0f - q;
}

// act(z) and act'(z). gelu_tanh: (1 + tanh v) / 2 is the logistic of 2v. A NaN
// stays NaN (relu' is z > 0, 0 at a NaN); where a formula is 0 * infinity (silu and
// gelu at -infinity), so is the result NaN.
template <int ACT>
__device__ inline float act_of(float z) {
  if constexpr (ACT == LLMINT8_ACT_RELU) return z > 0.f ? z : (z == z ? 0.f : z);
  if constexpr (ACT == LLMINT8_ACT_GELU) return z * normal_cdf(z, normal_exp(z));
  if constexpr (ACT == LLMINT8_ACT_GELU_TANH)
    return z * logistic(kTanhA * (z + kTanhB * z * z * z));
  if constexpr (ACT == LLMINT8_ACT_SILU) return z * logistic(z);
  return z;
}

template <int ACT>
__device__ inline float act_grad(float z) {
  if constexpr (ACT == LLMINT8_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == LLMINT8_ACT_GELU) {
    const float e = normal_exp(z);
    return normal_cdf(z, e) + z * 0.39894228f * e;
  }
  if constexpr (ACT == LLMINT8_ACT_GELU_TANH) {
    // p is exactly 0 or 1 beyond 20, where z * z could overflow against 1 - p = 0
    const float c = z < -20.f ? -20.f : z > 20.f ? 20.f : z;
    const float p = logistic(kTanhA * (c + kTanhB * c * c * c));
    return p + c * p * (1.f - p) * kTanhA * (1.f + 3.f * kTanhB * c * c);
  }
  if constexpr (ACT == LLMINT8_ACT_SILU) {
    const float p = logistic(z);
    return p * (1.f + z * (1.f - p));
  }
  return 1.f;
}

// f(ActTag<ACT>) for the run-time activation, which is uniform over the launch.
template <int V>
struct ActTag {
  static constexpr int value = V;
};
template <class F>
__device__ inline void with_act(int act, F f) {
  switch (act) {
    case LLMINT8_ACT_RELU: f(ActTag<LLMINT8_ACT_RELU>()); break;
    case LLMINT8_ACT_GELU: f(ActTag<LLMINT8_ACT_GELU>()); break;
    case LLMINT8_ACT_GELU_TANH: f(ActTag<LLMINT8_ACT_GELU_TANH>()); break;
    case LLMINT8_ACT_SILU: f(ActTag<LLMINT8_ACT_SILU>()); break;
    default: f(ActTag<LLMINT8_ACT_NONE>()); break;
  }
}

// ---- 8-bit checkpoint blocks ---------------------------------------------------------
// 32 entries of a row share the scale 2^e, e = floor(log2 max|x|) - 6 (at least
// -127), held as the byte e + 127; code = clamp(rint(x 2^-e), -127, 127) and the
// entry stands for code 2^e: seven significant bits, exact in bf16, and in fp16 where
// the entries were fp16 themselves, so a product takes a checkpointed X without a second
// rounding. (Sums below 2^-18 or above 65504, as G and U may hold in an fp16 block, are
// not exact in fp16; their gradients read them in fp32.) A block with an infinity or a
// NaN takes the byte 255 and zero codes and stands for NaN throughout.

__device__ inline float ckpt_scale(uint32_t byte) {
  // 255 gives infinity, and 0 * infinity the NaN the block stands for
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

// The scale byte for a block whose largest magnitude has these fp32 bits.
__device__ inline uint32_t ckpt_byte(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23);  // biased exponent; 0 for subnormals
  return e == 255 ? 255u : (uint32_t)(e > 6 ? e - 6 : 0);
}

// 2^-(byte - 127) for a byte from ckpt_byte below 255 (at most 248).
__device__ inline float ckpt_inv(uint32_t byte) {
  return __builtin_bit_cast(float, (254u - byte) << 23);
}

// Codes of 8 entries, little-endian in two words.
__device__ inline u32x2 ckpt_codes8(const float *v, uint32_t byte) {
  u32x2 w = {0u, 0u};
  if (byte == 255u) return w;
  const float inv = ckpt_inv(byte);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float r = __builtin_rintf(v[e] * inv);
    r = __builtin_fminf(__builtin_fmaxf(r, -127.0f), 127.0f);
    w[e >> 2] |= ((uint32_t)(int)r & 0xffu) << (8 * (e & 3));
  }
  return w;
}

// Largest |v| of 8 entries as fp32 bits: as integers, a NaN counts as the largest.
__device__ inline uint32_t top8(const float *v) {
  uint32_t t = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
    t = b > t ? b : t;
  }
  return t;
}

// The same over the 4 lanes of a block of 32 (lanes 4q .. 4q + 3).
__device__ inline uint32_t block_top(uint32_t t) {
  uint32_t o = __shfl_xor(t, 1, kWave);
  t = o > t ? o : t;
  o = __shfl_xor(t, 2, kWave);
  return o > t ? o : t;
}

// The 4 entries of one word of codes.
__device__ inline void ckpt_value4(uint32_t w, float scale, float *v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)((int)(w << (24 - 8 * e)) >> 24) * scale;
}

}  // namespace llmint8
