// Argument checks that the C entry points of the 16-bit operators share.
#pragma once

#include <cstdint>

#include "ffn.hpp"
#include "llmint8.h"

#define LLMINT8_EXPORT extern "C" __attribute__((visibility("default")))

namespace llmint8 {

constexpr int64_t kMaxDim = (int64_t)1 << 30;  // stage offsets are 32-bit
constexpr int64_t kMaxLd = (int64_t)1 << 21;  // 256 rows x 2 bytes x 2^21 = 2^30

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? LLMINT8_OK : LLMINT8_ERR_HIP; }

// The first failed check of a call; alignment faults rank below argument faults.
struct Check {
  int arg = LLMINT8_OK, sup = LLMINT8_OK;
  void need(bool ok) {
    if (!ok) arg = LLMINT8_ERR_INVALID_ARG;
  }
  void want(bool ok) {
    if (!ok) sup = LLMINT8_ERR_UNSUPPORTED;
  }
  void dims(int64_t M, int64_t K, int64_t N) {
    for (const int64_t d : {M, K, N}) need(d > 0 && d < kMaxDim);
    want(K % 8 == 0 && N % 8 == 0);
  }
  void matrix(const void *p, int64_t cols, int64_t ld) {
    need(p && ld >= cols && ld < kMaxLd);
    want(aligned16(p) && ld % 8 == 0);
  }
  void vec(const void *p) { want(aligned16(p)); }  // NULL passes
  void saved(const llmint8_saved *s, int64_t cols) {
    if (!s) return need(false);
    if (!s->scales) return matrix(s->data, cols, s->ld);
    need(s->data && s->ld >= cols && s->ld < kMaxLd);
    need(s->ld_scales >= (cols + kCkptBlock - 1) / kCkptBlock && s->ld_scales < kMaxLd);
    want(aligned16(s->data) && s->ld % 16 == 0);
  }
  void type(int dtype, int act) {
    need(dtype == LLMINT8_FP16 || dtype == LLMINT8_BF16);
    need(act >= LLMINT8_ACT_NONE && act <= LLMINT8_ACT_SILU);
  }
  int status() const { return arg ? arg : sup; }
};

inline bool sizes_ok(int64_t M, int64_t K, int64_t N) {
  Check c;
  c.dims(M, K, N);
  return c.status() == LLMINT8_OK;
}

inline int check_workspace(const void *ws, size_t bytes, size_t need) {
  if (need == 0) return LLMINT8_OK;
  if (!ws || bytes < need) return LLMINT8_ERR_WORKSPACE;
  return aligned16(ws) ? LLMINT8_OK : LLMINT8_ERR_UNSUPPORTED;
}

}  // namespace llmint8
