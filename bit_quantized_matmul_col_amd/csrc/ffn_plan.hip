// Which kernel a 16-bit product takes.
//
// The candidates are square tiles of 256 or 128 rows and columns and, for the
// forward products of up to kFewMaxM rows, the few-row kernel with blocks of 32, 64
// or 128 columns and 16, 32 or 64 rows, each with the reduction whole or split into
// up to 8 parts. The plan is the candidate with the smallest estimated time. The
// estimates are sums of a few terms whose constants were fitted to 3900 timed
// launches of square tiles (M 1 to 4096, all four products) and 6500 of the few-row
// kernel (M 1 to 512) on MI355X (bf16; K and N 256 to 28672, every candidate): they
// are within 7 % (256-tiles), 8 % (128-tiles) and 6 % (few rows) of the measured
// times (root mean square). The plans chosen by them cost 1 % more than the best
// candidate (geometric mean over the shapes; at worst 33 % with the square tiles,
// 19 % over 289 forward shapes of up to 512 rows). The best candidate itself is far
// from the bytes' and operations' floor between about 64 and 1000 rows (1.3 to 2.9
// times it): groups of rows read W again from the caches, 128-tiles are too few for
// the chip or, as tiles of dW over few rows, mostly fill and epilogue.
// Some of the choices, in microseconds:
//   1 x 4096 x 4096       few rows: 32 columns 12.5, 64 13.0, in 4 parts 11.8 (one by one
//                         from a host 12.0 against 14.8)
//   1 x 8192 x 28672      few rows: 128 columns 89.9, 64 columns 106.4
//   64 x 2048 x 2048      few rows: 32 columns by 16 rows 7.4, 64 by 64 11.8
//   300 x 1040 x 520      few rows 5.9, 128-tiles in 4 parts 11.2
//   256 x 4096 x 4096     few rows, 64 by 64 21.7, 32 by 16 53.9; 128-tiles in 4 parts
//                         23.3, whole 37.7
//   2048 x 4096 x 4096    dX: 128-tiles 62.6, 256-tiles in 2 parts 75.5
//   2048 x 11008 x 4096   256-tiles in 2 parts 158, whole 212; 128-tiles 164
//   2048 x 4096 x 11008   gated: 256-tiles 293, 128-tiles 410
// The plan is a function of the shape alone (the MI355X's 256 CUs, not a device
// query), so that the workspace queries and the launches agree.
#include <cmath>

#include "ffn.hpp"
#include "llmint8.h"

namespace llmint8 {

namespace {

constexpr int64_t kCus = kFfnCus;
constexpr int64_t kFewMaxM = 512;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

double mix(double a, double b, double f) { return a + (b - a) * f; }

// Shape of a product: rows and columns of the output(s), reduction length.
struct Shape {
  FfnKind kind;
  int64_t M, N, red;
  int outs;  // outputs side by side; the gated product has two sums per output
  bool gated() const { return kind == FfnKind::Gated; }
  double part_mb(int parts) const {
    return parts > 1 ? 4e-6 * parts * (gated() ? 2 : outs) * (double)M * (double)N : 0.0;
  }
};

int64_t tile_blocks(const Shape &s, int tile, int parts) {
  return cdiv(s.M, tile) * cdiv(s.N, s.gated() ? tile / 2 : tile) * s.outs * parts;
}

// The larger of two times, a little more where they are close: within 0.9 % of
// (a^6 + b^6)^(1/6), without the powers (a plan is made on every call).
double larger(double a, double b) {
  const double hi = a > b ? a : b, r = (a > b ? b : a) / hi, r2 = r * r;
  return hi * (1.0 + 0.1225 * r2 * r2 * r2);
}

// Microseconds of a launch of square tiles: rounds of as many blocks as the chip
// holds (one 256-tile or two 128-tiles per CU; up to one 128-tile per CU runs with
// a deeper ring), each a number of 64-step stages and an epilogue, and not less
// than reading the operands takes.
double tile_us(const Shape &s, int tile, int parts) {
  const int64_t blocks = tile_blocks(s, tile, parts);
  const double mb = 2e-6 * (double)s.red * ((double)s.M + (double)s.N * (s.gated() ? 2 : s.outs));
  double st = (double)cdiv(cdiv(s.red, 64), parts), t, floor;
  if (tile == 256) {
    st *= s.kind == FfnKind::GradX ? 0.911 : s.kind == FfnKind::GradW ? 1.046 : 1.0;
    const double f = (double)(blocks % kCus) / kCus;
    const int64_t rows = cdiv(s.M, 256), cols = blocks / (rows * parts);
    const double half = tail_cut(rows, cols, parts) < cols ? 0.68 : 1.0;
    t = 2.59 + (double)(blocks / kCus) * (st * 1.371 + 9.31);
    if (f > 0) t += half * (st * mix(1.139, 1.371, f) + mix(6.7, 9.31, f));
    if (parts > 1) t += 1.21 + 0.302 * s.part_mb(parts);
    floor = 2.59 + mb / 4.02;
  } else {
    st *= s.kind == FfnKind::GradX ? 0.88 : s.kind == FfnKind::GradW ? 1.042 : 1.0;
    t = 2.06;
    if (blocks <= kCus) {
      const double f = (double)blocks / kCus;
      t += st * mix(0.465, 0.51, f) + mix(3.51, 5.55, f);
    } else {
      const double f = (double)(blocks % (2 * kCus)) / kCus;  // blocks per CU of the last round
      t += (double)(blocks / (2 * kCus)) * (st * 0.863 + 4.43);
      if (f > 1)
        t += st * mix(0.739, 0.863, f - 1) + mix(5.55, 4.43, f - 1);
      else if (f > 0)
        t += st * mix(0.55, 0.739, f) + mix(3.51, 5.55, f);
    }
    if (parts > 1) t += 1.63 + 0.436 * s.part_mb(parts);
    floor = 2.06 + mb / 4.29;
  }
  return larger(t, floor);
}

int64_t few_blocks(const Shape &s, int cols, int rows, int parts) {
  return cdiv(s.N, cols) * cdiv(s.M, rows) * parts;
}

// Microseconds of the few-row kernel: what a CU takes for its blocks' bytes (it has
// about 256 lines of 128 bytes on their way at a time, so that blocks of 32 columns
// take as long for a row as those of 64), what the chip takes for the weights (and
// for reading them again, from the caches, for further groups of rows), and the join.
double few_us(const Shape &s, int cols, int rows, int parts) {
  const int c = cols == 32 ? 0 : cols == 64 ? 1 : 2, p = s.gated() ? 2 : 1, mt = rows / 16;
  const double cu_rate[3] = {63.4, 85.9, 96.7}, chip_rate[3] = {5.21, 6.47, 7.39};
  const int64_t groups = cdiv(s.M, rows), tiles = cdiv(s.N, cols);
  const int step = cols == 32 ? 64 : 32;
  const double st = (double)cdiv(cdiv(cdiv(s.red, step), parts), 4);  // stages of a wave
  const double kb = st * 4e-3 * step * (p * cols * 2 + 0.706 * mt * 32);  // per block
  const double wmb = 2e-6 * (double)s.red * (double)s.N * p;
  const double xmb = 2e-6 * (double)(tiles * groups * s.red) * rows + (double)(groups - 1) * wmb;
  const double rounds = (double)cdiv(few_blocks(s, cols, rows, parts), kCus);
  double t = 2.3 + rounds * (0.31 + 0.33 * mt * p * cols / 64 + kb / cu_rate[c]) +
             wmb / chip_rate[c] + xmb / 300.0;
  if (parts > 1) t += 2.5 + 0.435 * s.part_mb(parts);
  return t;
}

}  // namespace

namespace {

FfnPlan best_plan(FfnKind kind, int64_t M, int64_t N, int64_t K, int segs, int outs) {
  const Shape s{kind, M, N, K * segs, outs};
  FfnPlan best{false, 256, 1, 0};
  double best_us = 1e300;
  auto consider = [&](bool few, int tile, int parts, int rows, double us) {
    // A host takes 12 to 15 us for a call of two launches with a workspace, 8 to 10 for
    // one launch, and gains nothing from a split that the GPU ends before. (Under graph
    // replay it would: 1 x 4096 x 4096 11.8 us in 4 parts against 12.5 whole.)
    if (parts > 1) us = us + 1.0 < 15.0 ? 15.0 : us + 1.0;
    if (us < best_us) best = FfnPlan{few, tile, parts, rows}, best_us = us;
  };
  const int64_t stages = cdiv(s.red, 64);
  for (const int parts : {1, 2, 3, 4, 6, 8}) {
    if (parts > 1 && stages < 3 * parts) break;
    // more parts than fill the chip once only add partial sums
    if (parts == 1 || tile_blocks(s, 256, parts) <= kCus)
      consider(false, 256, parts, 0, tile_us(s, 256, parts));
    if (parts == 1 || tile_blocks(s, 128, parts) <= 2 * kCus)
      consider(false, 128, parts, 0, tile_us(s, 128, parts));
    if ((s.gated() || kind == FfnKind::Forward) && M <= kFewMaxM)
      for (const int rows : {16, 32, 64})
        for (const int cols : {32, 64, 128}) {
          if (rows > 16 && rows / 2 >= M) continue;
          if (rows == 64 && (cols == 32 || (cols == 128 && s.gated()))) continue;
          if (parts == 1 || few_blocks(s, cols, rows, parts) <= kCus)
            consider(true, cols, parts, rows, few_us(s, cols, rows, parts));
        }
  }
  return best;
}

}  // namespace

// A call and its workspace query ask for the same plan one after the other, which
// takes up to 0.6 us to find: each thread keeps the last one with its shape.
FfnPlan ffn_plan(FfnKind kind, int64_t M, int64_t N, int64_t K, int segs, int outs) {
  thread_local struct {
    FfnKind kind;
    int64_t M, N, K;
    int segs, outs;
    FfnPlan plan;
  } last{};  // M = 0: none yet
  if (M != last.M || N != last.N || K != last.K || kind != last.kind || segs != last.segs ||
      outs != last.outs)
    last = {kind, M, N, K, segs, outs, best_plan(kind, M, N, K, segs, outs)};
  return last.plan;
}

namespace {

// Microseconds of both products of a backward pass in one launch of tiles: the
// CUs' shares of all blocks' times, and at least the longest block.
double together_us(const Shape &x, int xparts, const Shape &w, int wparts, int tile) {
  const int64_t nx = tile_blocks(x, tile, xparts), nw = tile_blocks(w, tile, wparts);
  const double slots = (double)(tile == 256 ? kCus : 2 * kCus);
  const double sx = (double)cdiv(cdiv(x.red, 64), xparts), sw = (double)cdiv(cdiv(w.red, 64), wparts);
  const double fill = (double)(nx + nw) / slots < 1.0 ? (double)(nx + nw) / slots : 1.0;
  double dx, dw, tail;
  if (tile == 256) {
    const double st = mix(1.104, 1.305, fill), e = mix(12.3, 15.4, fill);
    dx = sx * st * 0.897 + e, dw = sw * st * 1.012 + e, tail = 0.175;
  } else {
    const double st = fill <= 0.5 ? mix(0.408, 0.667, 2 * fill) : mix(0.613, 0.849, 2 * fill - 1);
    dx = sx * st * 0.784 + 6.71, dw = sw * st * 0.991 + 6.71, tail = 0.267;
  }
  const double longest = dx > dw ? dx : dw, shortest = dx > dw ? dw : dx;
  const double share = ((double)nx * dx + (double)nw * dw) / slots;
  double t = fill < 1.0 ? longest : larger(longest, share + tail * shortest);
  for (const double mb : {x.part_mb(xparts), w.part_mb(wparts)})
    if (mb > 0) t += 1.5 + (tile == 256 ? 2.44 + 0.136 * mb : 2.8 + 0.23 * mb);
  return t;
}

}  // namespace

// Together in one launch the two products took 24 % less time than one after the
// other (geometric mean over 144 shapes, M 16 to 4096, K and N 512 to 13824; 1 %
// more at worst): 512 x 4096 x 4096 59 -> 49 us, 1024 x 1024 x 1024 31 -> 16,
// gated 2048 x 4096 x 11008 694 -> 671, gated 4096 x 5120 x 13824 2165 -> 1890. The
// tile and the parts chosen by the estimates cost 1.5 % more than the best ones.
FfnBackPlan ffn_back_plan(int64_t M, int64_t K, int64_t N, int grads) {
  FfnBackPlan p{best_plan(FfnKind::GradX, M, K, N, grads, 1),
                best_plan(FfnKind::GradW, K, N, M, 1, grads), 256, 1, 1};
  const Shape x{FfnKind::GradX, M, K, N * grads, 1}, w{FfnKind::GradW, K, N, M, grads};
  double best = 1e300;
  const int64_t stx = cdiv(x.red, 64), stw = cdiv(w.red, 64);
  for (const int tile : {256, 128})
    for (const int xs : {1, 2, 4, 8})
      for (const int ws : {1, 2, 4}) {
        if ((xs > 1 && stx < 3 * xs) || (ws > 1 && stw < 3 * ws)) continue;
        const int64_t room = tile == 256 ? kCus : 2 * kCus;
        if ((xs > 1 && tile_blocks(x, tile, xs) > room) ||
            (ws > 1 && tile_blocks(w, tile, ws) > room))
          continue;
        const double us = together_us(x, xs, w, ws, tile);
        if (us < best) best = us, p.tile = tile, p.xsplit = xs, p.wsplit = ws;
      }
  return p;
}

size_t ffn_part_bytes(const FfnPlan &p, int64_t M, int64_t N, int outs) {
  return p.ksplit > 1 ? (size_t)p.ksplit * outs * M * N * 4 : 0;
}

hipError_t launch_ffn_together(int dtype, const FfnGemm &x, const FfnGemm &w, const BiasJoin &j,
                               const FfnBackPlan &p, hipStream_t s) {
  FfnGemm gx = x, gw = w;
  gx.ksplit = p.xsplit, gw.ksplit = p.wsplit;
  hipError_t e = launch_ffn_back(dtype, gx, gw, j, p.tile, s);
  if (e == hipSuccess && p.xsplit > 1) e = launch_ffn_finish(dtype, false, gx, s);
  if (e == hipSuccess && p.wsplit > 1) e = launch_ffn_finish(dtype, false, gw, s);
  return e;
}

hipError_t launch_ffn(FfnKind kind, int dtype, const FfnGemm &args, const FfnPlan &p,
                      hipStream_t s) {
  FfnGemm a = args;
  a.ksplit = p.ksplit;
  hipError_t e = hipSuccess;
  if (p.few)
    e = launch_ffn_skinny(dtype, kind == FfnKind::Gated, a, p.rows, p.tile, s);
  else if (kind == FfnKind::Forward)
    e = launch_ffn_forward(dtype, a, p.tile, s);
  else if (kind == FfnKind::Gated)
    e = launch_ffn_gated(dtype, a, p.tile, s);
  else if (kind == FfnKind::GradX)
    e = launch_ffn_grad_x(dtype, a, p.tile, s);
  else
    e = launch_ffn_grad_w(dtype, a, p.tile, s);
  if (e == hipSuccess && p.ksplit > 1)
    e = launch_ffn_finish(dtype, kind == FfnKind::Gated, a, s);
  return e;
}

}  // namespace llmint8
