// Which kernel a product over the experts' rows takes.
//
// The candidates are square tiles of 256 or 128 rows of an expert, and for the forward products
// the few-row kernel with 16, 32 or 64 rows by 64 or 128 columns a block, whole or with the
// reduction in 2 or 4 parts. The plan is the one with the smallest estimated time. How many rows
// each expert has is known on the GPU alone, so the estimates take the mean and add a part of a
// group for what each expert's last one lacks. Their constants were fitted to 3160 timed calls on
// MI355X (bf16, graph replay; 8 to 128 experts, 512 x 512 to 4096 x 11008, 1 to 400 rows an
// expert, unevenly spread): the plans chosen by them cost 3.7 % more than the best candidate
// (geometric mean over 224 products, at worst 48 %, where the spread makes one more round of
// 256-tiles than the mean does; on 84 products not fitted to, whose weights came from HBM, 2.1 %).
// Some of the choices, in microseconds:
//   2 of 16, 1 token, 4096 x 2048, gated             16 rows by 64 columns in 4 parts 20, whole 22
//   8 of 128, 8 tokens, 768 x 2048, second product   16 rows by 64 columns 25.4, by 128 26.1
//   8 of 128, 192 tokens, the same                   128-tiles 46, few rows 53
//   2 of 8, 160 tokens, 11008 x 4096, the same       64 rows by 128 in 2 parts 153, whole 180
//   4 of 32, 720 tokens, 2048 x 1024, gated          256-tiles 63, 128-tiles 75, few rows 84
//   8 of 32, 1600 tokens, 7168 x 2048, gated         256-tiles 872, 128-tiles 985
// Pairs without an expert (padding, experts of other ranks) are known on the GPU alone too and count
// as rows, so such a call is planned for more rows than there are.
// The timings are not kept here. The second product's tiles were timed with rows in 16 bits then;
// with rows in fp32 (88 products timed again) the same constants choose within 3.1 % of the best,
// refitted ones within 3.9 %.
// The plan is a function of the shape alone, so that the workspace query and the call agree.
#include "experts.hpp"

namespace llmint8 {

namespace {

struct Size {
  double pairs, used, N, K;
  bool gated;
  double weights_mb() const { return used * K * N * (gated ? 4e-6 : 2e-6); }
  // Groups of T rows, `last` of one an expert beyond the mean.
  double groups(int T, double last) const {
    const double g = pairs / used / T + last;
    return used * (g > 1 ? g : 1);
  }
};

double larger(double a, double b) {
  const double hi = a > b ? a : b, r = (a > b ? b : a) / hi, r2 = r * r;
  return hi * (1.0 + 0.1225 * r2 * r2 * r2);
}
double up_to(double n, int to) { return (double)(((int64_t)n + to - 1) / to); }

// A CU's blocks one after the other, their bytes at the rate a CU reads (KB a microsecond); all
// weights from memory, again, from the caches, for further groups of an expert.
double few_us(const Size &s, int rows, int cols, int parts) {
  const double rate = rows == 16   ? (cols == 64 ? 103.7 : 88.6)
                      : rows == 32 ? (cols == 64 ? 78.5 : 74.7)
                                   : (cols == 64 ? 62.1 : 69.7);
  const double groups = s.groups(rows, 0.625), blocks = groups * up_to(s.N, cols) * parts;
  const double kb = s.K / parts * 2e-3 * (cols * (s.gated ? 2 : 1) + rows);
  const double rounds = blocks > kFfnCus ? blocks / kFfnCus + 0.99 : 1.0;
  const double us = 4.42 + larger(rounds * (kb / rate + 1.06),
                                  s.weights_mb() * (1 + 0.362 * (groups / s.used - 1)) / 6.5);
  const double part_mb = 4e-6 * parts * s.pairs * s.N;
  if (!s.gated) return us + 2.13 + 0.578 * part_mb;
  return parts == 1 ? us : us + 2.13 + 1.16 * part_mb;
}

double tile_us(const Size &s, int tile) {
  const bool big = tile == 256;
  const double groups = s.groups(tile, 0.755), stages = up_to(s.K, 64);
  const double f = groups * up_to(s.N * (s.gated ? 2 : 1), tile) / (big ? 1.0 : 2.0) / kFfnCus;
  // of a stage where few CUs and where all work; of a tile beside its stages; of a round begun
  const double s1 = big ? 1.387 : 0.791, s2 = big ? 1.416 : 1.056;
  const double step = big ? 0.263 : 0.481, again = big ? 1.385 : 0.005;
  double us = f <= 1 ? stages * (s1 + (s2 - s1) * f)
                     : stages * s2 * f + stages * s1 * step * (f < 1.25 ? 4 * (f - 1) : 1.0);
  us = larger(us, s.weights_mb() * (1 + again * (groups / s.used - 1)) / 6.5);
  return us + (big ? 8.0 : 5.85) + (s.gated ? 0 : 0.906 + 0.276 * 2e-6 * s.pairs * s.N);
}

}  // namespace

FfnPlan experts_plan(FfnKind kind, int64_t pairs, int E, int64_t N, int64_t K) {
  const Size s{(double)pairs, (double)(E < pairs ? E : pairs), (double)N, (double)K,
               kind == FfnKind::Gated};
  FfnPlan best{};
  double best_us = 1e300;
  auto consider = [&](const FfnPlan &p, double us) {
    if (us < best_us) best = p, best_us = us;
  };
  for (const int tile : {128, 256}) consider(FfnPlan{false, tile, 1, 0}, tile_us(s, tile));
  if (kind == FfnKind::GradX || pairs > kFewRows * s.used) return best;
  for (const int rows : {16, 32, 64})
    for (const int cols : {64, 128}) {
      if (rows == 64 && cols == 128 && s.gated) continue;  // its sums take too many registers
      for (const int parts : {1, 2, 4}) {
        // a part has a few steps for each of the four waves; past some blocks a CU, parts only
        // add sums
        const double blocks = s.groups(rows, 0.625) * up_to(s.N, cols) * parts;
        if (parts > 1 && (K < 512 * parts || blocks > 4 * kFfnCus)) break;
        consider(FfnPlan{true, cols, parts, rows}, few_us(s, rows, cols, parts));
      }
    }
  return best;
}

}  // namespace llmint8
