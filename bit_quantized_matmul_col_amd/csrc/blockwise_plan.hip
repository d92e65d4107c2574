// Which kernel a block-scaled FP8 product takes.
//
// The candidates are square tiles of 256 or 128 rows and columns, whole or with the reduction split
// in up to 8 parts (X is coded by a pass before), and for few rows the kernel that reads W
// straight into registers, with 16, 32 or 64 columns a block and 32 rows (X coded before) or 16
// (coded in it: one launch). The plan is the one with the smallest estimated time, the coding
// pass and the join of the parts included. The estimates' constants were fitted to 4330
// timed calls on MI355X (bf16, graph replay, M 1 to 4500, K 256 to 11008, N 256 to 14336; root
// mean square 8 % off); the plans chosen by them cost 0.6 % more than the best candidate (geometric
// mean over 400 shapes, at worst 17 %). The timings are not kept here. Some of the choices, in
// microseconds:
//   1 x 8192 x 28672       few rows, coded in place, 64 columns 44, 32 columns 52
//   64 x 2048 x 2048       few rows 10.8, 128-tiles in 4 parts 12.9
//   128 x 11008 x 4096     128-tiles in 8 parts 28, whole 60; few rows 36
//   1024 x 4096 x 11008    256-tiles 67, 128-tiles 91
//   2048 x 11008 x 4096    256-tiles in 2 parts 119, whole 162; 128-tiles 125
// The plan is a function of the shape alone, so that the workspace query and the call agree.
#include "blockwise.hpp"

namespace llmint8 {

namespace {

constexpr int64_t kCus = kFfnCus;
constexpr int64_t kFusedMaxM = 48, kFewMaxM = 512;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
double mix(double a, double b, double f) { return a + (b - a) * f; }

// The larger of two times, a little more where they are close.
double larger(double a, double b) {
  const double hi = a > b ? a : b, r = (a > b ? b : a) / hi, r2 = r * r;
  return hi * (1.0 + 0.1225 * r2 * r2 * r2);
}

struct Size {
  double M, K, N;
  int64_t m, k, n;
  double mb() const { return 1e-6 * K * (M + N); }
  double part_mb(int parts) const { return 4e-6 * parts * M * N; }
  double coding(double per_mb) const { return 2.0 + per_mb * 1e-6 * M * K; }
};

// Rounds of one 256-tile a CU, or of up to two 128-tiles, as in the 16-bit plan.
double tile256_us(const Size &s, int parts) {
  const int64_t rows = cdiv(s.m, 256), cols = cdiv(s.n, 256), blocks = rows * cols * parts;
  const double st = (double)cdiv(cdiv(s.k, kFp8Block), parts), f = (double)(blocks % kCus) / kCus;
  double t = 0.14 + (double)(blocks / kCus) * (st * 1.98 + 7.99);
  if (f > 0)
    t += (tail_cut(rows, cols, parts) < cols ? 0.811 : 1.0) *
         (st * mix(1.26, 1.98, f) + mix(6.46, 7.99, f));
  if (parts > 1) t += 2.31 + 0.376 * s.part_mb(parts);
  return larger(t, 0.14 + s.mb() / 2.89) + s.coding(0.744);
}
double tile128_us(const Size &s, int parts) {
  const int64_t blocks = cdiv(s.m, 128) * cdiv(s.n, 128) * parts;
  const double st = (double)cdiv(cdiv(s.k, kFp8Block), parts);
  double t = 1.96;
  if (blocks <= kCus) {
    const double f = (double)blocks / kCus;
    t += st * mix(0.502, 0.733, f) + mix(2.85, 4.77, f);
  } else {
    const double f = (double)(blocks % (2 * kCus)) / kCus;  // blocks per CU of the last round
    t += (double)(blocks / (2 * kCus)) * (st * 1.34 + 3.33);
    if (f > 1)
      t += st * mix(1.14, 1.34, f - 1) + mix(4.67, 3.33, f - 1);
    else if (f > 0)
      t += st * mix(0.508, 1.14, f) + mix(5.14, 4.67, f);
  }
  if (parts > 1) t += 2.32 + 0.475 * s.part_mb(parts);
  return larger(t, 1.96 + s.mb() / 3.25) + s.coding(0.626);
}

// The few-row kernel: a wave's blocks of the reduction one after the other, a CU's bytes, and W
// from memory (again, from the caches, for further groups of rows).
double few_us(const Size &s, bool fused, int cols) {
  const int c = cols == 16 ? 0 : cols == 32 ? 1 : 2, waves = cols == 16 ? 8 : 4;
  const int rows = fused ? 16 : 32;
  const double groups = (double)cdiv(s.m, rows), w = 1e-6 * s.K * s.N;
  const double st = (double)cdiv(cdiv(s.k, kFp8Block), waves);
  const double rounds = (double)cdiv(cdiv(s.n, cols) * cdiv(s.m, rows), kCus);
  if (fused) {
    const double start[3] = {1.84, 1.28, 0.10}, step[3] = {0.0, 0.455, 0.887};
    const double rate[3] = {21.3, 107.0, 1e9};  // KB a microsecond and CU
    const double kb = st * waves * 0.128 * (cols + 0.19 * rows);
    return 0.2 + start[c] + st * step[c] + rounds * (kb / rate[c] + 2.87) +
           w * (1 + 1.27 * (groups - 1)) / 11.8;
  }
  const double start[3] = {1.36, 0.97, 0.2}, step[3] = {0.0, 0.1, 0.47};
  const double rate[3] = {35.5, 55.9, 107.0};
  const double kb = st * waves * 0.128 * (cols + 0.49 * rows);
  return 1.58 + start[c] + st * step[c] + rounds * (kb / rate[c] + 1.2) +
         w * (1 + 0.58 * (groups - 1)) / 8.9 + s.coding(2.2);
}

Fp8Plan best_plan(int64_t M, int64_t K, int64_t N) {
  const Size s{(double)M, (double)K, (double)N, M, K, N};
  Fp8Plan best{};
  double best_us = 1e300;
  auto consider = [&](const Fp8Plan &p, double us) {
    // what a host takes for a call of one, two or three launches
    const double host = p.fused ? 8.0 : p.ksplit == 1 ? 10.5 : 13.0;
    us = (us > host ? us : host) + 1e-3 * us;
    if (us < best_us) best = p, best_us = us;
  };
  for (const int cols : {16, 32, 64}) {
    if (M <= kFusedMaxM) consider(Fp8Plan{true, true, 0, 1, cols}, few_us(s, true, cols));
    if (M <= kFewMaxM) consider(Fp8Plan{true, false, 0, 1, cols}, few_us(s, false, cols));
  }
  const int64_t stages = cdiv(K, kFp8Block);
  for (const int parts : {1, 2, 3, 4, 6, 8}) {
    if (parts > 1 && stages < 2 * parts) break;
    // more parts than fill the chip once only add partial sums
    if (parts == 1 || cdiv(M, 256) * cdiv(N, 256) * parts <= kCus)
      consider(Fp8Plan{false, false, 256, parts, 0}, tile256_us(s, parts));
    if (parts == 1 || cdiv(M, 128) * cdiv(N, 128) * parts <= 2 * kCus)
      consider(Fp8Plan{false, false, 128, parts, 0}, tile128_us(s, parts));
  }
  return best;
}

}  // namespace

// A call and its workspace query ask for the same plan one after the other: each thread keeps
// the last one with its shape.
Fp8Plan fp8_plan(int64_t M, int64_t K, int64_t N) {
  thread_local struct {
    int64_t M, K, N;
    Fp8Plan plan;
  } last{};  // M = 0: none yet
  if (M != last.M || K != last.K || N != last.N) last = {M, K, N, best_plan(M, K, N)};
  return last.plan;
}

}  // namespace llmint8
