// Tiled 16-bit matrix product on gfx950 MFMA for the feed-forward operators
// (kernel templates; each operand order is instantiated in its own translation
// unit).
//
//   forward   Y  = act(X W + b) + R        A = X  [M x K]   B = W  [K x N]
//   gated     H  = act(X Wg) * (X Wu)      A = X            B = Wg and Wu
//   grad X    dX = dZ W^T (+ dZ' W'^T)     A = dZ [M x N]   B = W  [K x N]
//   grad W    dW = X^T dZ                  A = X  [M x K]   B = dZ [M x N]
//
// All four sum over a "reduction" index that is either contiguous in memory
// (RowK: X and dZ in the first three, W in grad X) or strided (ColK: W in the
// forward products, both operands of grad W). Neither order is copied or
// transposed beforehand:
//  * a stage is 64 reduction steps of both operands, brought to LDS by 16-byte
//    direct-to-LDS loads; a RowK tile keeps rows of 64 steps (128 bytes), a ColK
//    tile the 64 rows of the matrix (2 bytes a column of the tile).
//  * MFMA fragments (8 consecutive reduction steps of one row per lane) are one
//    16-byte LDS read from a RowK tile and two transposed 8-byte reads from a
//    ColK tile: a group of 16 lanes addresses a 4 x 16 block of 16-bit values
//    row by row and each lane receives one column of it.
//  * 16-byte chunks are permuted within each stored row (chunk c of row r sits at
//    c ^ key(r)), so that the lanes of one LDS access fall in different bank
//    groups: conflicts cost under 1 % of the LDS cycles.
//  * Reduction steps past the end read as zero in both operands, so no infinity
//    or NaN of a neighbouring row is multiplied by a zero: every load goes through
//    a buffer resource that ends with the last element of the stage's last row,
//    and a RowK lane whose chunk lies past the reduction length takes an offset
//    outside it. Rows of a RowK tile past the matrix read as zero too. Columns of a
//    ColK tile past the matrix read what lies behind them in memory (the gap
//    between rows, the next row, zeros after the last): a column meets only its own
//    outputs, and those past the matrix are not stored.
//
// A block computes BM x BN outputs with NWM x NWN waves. The MFMAs take the
// operands in the order (B, A), so a lane's accumulators hold 4 consecutive
// columns of one row; the epilogue passes 32 rows at a time through LDS in fp32,
// after which a lane owns 8 consecutive columns and every load and store of the
// epilogue is 16 bytes.
//
// What bounds it: at 8192 x 8192 x 28672 (gated) the card's power. It runs at 1240
// to 1345 TFLOP/s, by card and by what ran before, with the MFMA units busy 71 % of
// the time at 1.65 to 1.73 GHz; the library's product of the same sizes reaches 1273.
// The LDS is active 28 % of the time. Smaller products lose to partial rounds and to
// the epilogue, 7 to 9 us a round of 256-tiles (33 MB written at once): 1020 to 1250
// TFLOP/s at 4096 x 5120 x 13824 with 8-bit G and U.
//
// Measured against it at 8192 x 8192 x 28672: 32x32x16 MFMAs 6.12 against 5.72 ms (the
// clock falls further for the same work), stages of 32 steps in rings of 4 or 5 10 %
// slower, 4 waves of 128 x 128 instead of 8 of 128 x 64 7.0 against 5.9 ms, a stage's
// loads issued together after the barrier instead of between the MFMAs 10 % slower.
#pragma once

#include "ffn_math.hpp"
#include "gemm_core.hpp"

namespace llmint8 {
namespace ffn {

using gemm_detail::lptr_t;
using gemm_detail::make_rsrc;
using gemm_detail::rsrc_t;
using gemm_detail::wait_vm;

constexpr int kStep = 64;  // reduction steps per stage
constexpr int kOob = (int)0x80000000;  // an offset past the end of every resource

// The wave's number in its block, known to be the same for all its lanes.
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// First of n stages that part `split` of `parts` takes.
__device__ inline int part_begin(int n, int split, int parts) {
  return (int)((uint64_t)n * split / (uint32_t)parts);
}

// The blocks of one XCD (they are dealt out round robin) take consecutive places.
__device__ inline uint32_t xcd_place(uint32_t bid, uint32_t blocks) {
  constexpr uint32_t X = gemm_detail::kXcds;
  const uint32_t x = bid % X, rem = blocks % X;
  return x * (blocks / X) + (x < rem ? x : rem) + bid / X;
}

// Tile and part of block bid. The places of xcd_place are in the order parts, groups of up to 8 tile rows,
// columns, rows of the group, so that an XCD works on few parts and neighbouring
// tiles and its L2 serves the operands that they share.
__device__ inline void tile_at(uint32_t bid, uint32_t tiles_m, uint32_t tiles_n, uint32_t parts,
                               int &tm, int &tn, int &part) {
  constexpr uint32_t GM = gemm_detail::kGroupM;
  const uint32_t tiles = tiles_m * tiles_n, place = xcd_place(bid, tiles * parts);
  part = (int)(place / tiles);
  const uint32_t v = place % tiles;
  const uint32_t first = v / (GM * tiles_n) * GM, in = v % (GM * tiles_n);
  const uint32_t gm = tiles_m - first < GM ? tiles_m - first : GM;
  tm = (int)(first + in % gm);
  tn = (int)(in / gm);
}

template <int N>
struct Count {
  static constexpr int value = N;
};

enum class Lay { RowK, ColK };

__device__ inline int clip31(int64_t bytes) {
  return (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff);
}

// ROWS output rows (or columns) x kStep reduction steps, reduction contiguous.
template <int ROWS, int NW>
struct RowKTile {
  static constexpr int PITCH = kStep * 2;    // bytes of a stored row
  static constexpr int BYTES = ROWS * PITCH;
  static constexpr int CH = PITCH / 16;      // chunks per stored row, 8
  static constexpr int RPI = 64 / CH;        // rows per 1 KB load
  static constexpr int G = ROWS / (RPI * NW);  // loads per wave per stage
  int bytes;  // of the tile's rows, from the first element to the last
  int voff[G];
  int chunk;      // first reduction step of this lane's chunk within a stage

  __device__ static int key(int r) { return (r >> 1) & 7; }

  // rows: rows of the matrix from the tile's first on; len: the reduction length.
  __device__ void init(int64_t ld, int64_t rows, int64_t len) {
    rows = rows < ROWS ? rows : ROWS;
    bytes = (int)((rows - 1) * ld + len) * 2;
    const int lane = threadIdx.x & 63, wv = wave_id();
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int r = (wv + NW * j) * RPI + lane / CH;
      const int c = (lane % CH) ^ key(r);
      voff[j] = r * (int)ld * 2 + 16 * c;
      chunk = 8 * c;  // the same for every j: the key repeats every 16 rows
    }
  }
  static_assert((RPI * NW) % 16 == 0, "the chunk key must not depend on j");

  // What the loads of one stage share: the resource from reduction step k on
  // (mat: the tile's first row), and whether this lane's chunk is within the
  // reduction length.
  struct Stage {
    rsrc_t rs;
    bool in;
  };
  __device__ Stage stage(const uint8_t *mat, int64_t, int k, int len) const {
    const int left = bytes - 2 * k;  // empty past the end
    return Stage{make_rsrc(mat + 2 * (int64_t)k, left > 0 ? left : 0), k + chunk < len};
  }
  // the j-th load of the stage, to LDS at `to`
  __device__ void load(const Stage &st, uint8_t *to, int j) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rs, (lptr_t)(to + (wave_id() + NW * j) * 1024), 16,
                                             st.in ? voff[j] : kOob, 0, 0, 0);
  }

  // Fragment of 16 rows from row0 for reduction steps 32 ks .. 32 ks + 31.
  __device__ static s16x8 frag(const uint8_t *tile, int row0, int ks, int lane) {
    const int r = row0 + (lane & 15);
    return *(const s16x8 *)(tile + r * PITCH + 16 * ((4 * ks + (lane >> 4)) ^ key(r)));
  }
};

// Transposed LDS read: the 16 lanes of a group address a 4 x 16 block of 16-bit
// values, lane i the entries 4 (i % 4) .. + 3 of row i / 4, and lane i receives
// column i. The restrict parameter only gives the access alias information:
// without any, the compiler takes it to depend on the direct-to-LDS loads in
// flight and waits for all of them first (the ring's own waits and barriers
// order the two).
typedef __attribute__((address_space(3))) s16x4 *tr_ptr_t;
__device__ inline s16x4 read_tr16(tr_ptr_t __restrict p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// kStep reduction steps x COLS output rows (or columns), reduction strided.
template <int COLS, int NW>
struct ColKTile {
  static constexpr int PITCH = COLS * 2;     // bytes of a stored row
  static constexpr int BYTES = kStep * PITCH;
  static constexpr int CH = COLS / 8;      // chunks per stored row
  static constexpr int RPI = 64 / CH;      // stored rows per 1 KB load
  static constexpr int G = kStep / (RPI * NW);
  int voff[G];
  int cols;  // columns of the matrix from the tile's first on

  // Half a wave reads 8 rows (r % 16 in 0 .. 3 and 8 .. 11, or 4 more) x 2 chunks;
  // rows of 8 chunks lie in opposite halves of the banks by twos already, rows of 4
  // in four quarters.
  __device__ static int key(int r) {
    return CH >= 16  ? 2 * ((r & 3) | (r >> 1 & 4))
           : CH == 8 ? 2 * ((r >> 1 & 1) | (r >> 2 & 2))
                     : 2 * (r >> 3 & 1);
  }

  __device__ void init(int64_t ld, int64_t ncols, int64_t) {
    cols = (int)ncols;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int r = (wv + NW * j) * RPI + lane / CH;
      voff[j] = r * (int)ld * 2 + 16 * ((lane % CH) ^ key(r));
    }
  }

  // mat: element (0, first column of the tile). The resource ends with the last
  // column of the stage's last row of the matrix (it is empty past the length).
  struct Stage {
    rsrc_t rs;
  };
  __device__ Stage stage(const uint8_t *mat, int64_t ld, int k, int len) const {
    // len >= k: 0 rows at least (and n at most 0 then, as cols <= ld), so that nothing wraps
    const int left = len - k, rows = left < kStep ? left : kStep;
    const int n = ((rows - 1) * (int)ld + cols) * 2;
    return Stage{make_rsrc(mat + 2 * (int64_t)k * ld, n > 0 ? n : 0)};
  }
  __device__ void load(const Stage &st, uint8_t *to, int j) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rs, (lptr_t)(to + (wave_id() + NW * j) * 1024), 16,
                                             voff[j], 0, 0, 0);
  }

  // Fragment of 16 columns from col0 for reduction steps 32 ks .. 32 ks + 31.
  __device__ static s16x8 frag(const uint8_t *tile, int col0, int ks, int lane) {
    const int i = lane & 15, r = (lane >> 4) * 8 + (i >> 2);
    const int c = (col0 >> 3) + ((i & 3) >> 1);
    const uint8_t *p = tile + (ks * 32 + r) * PITCH + 16 * (c ^ key(r)) + 8 * (i & 1);
    const s16x4 lo = read_tr16((tr_ptr_t)p), hi = read_tr16((tr_ptr_t)(p + 4 * PITCH));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// ---- epilogue -------------------------------------------------------------------------

// 8 consecutive columns of one row: act(v + b) + r; the sums v + b go to z on the
// way. b: the bias of the columns (zeros without one); r: the residual's 16 bytes.
template <class T>
__device__ inline void finish_forward(const FfnGemm &a, int out, int64_t i, int64_t n, float *v,
                                      const float *b, const u32x4 &r) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += b[e];
  if (a.z[0]) store8<T>((uint16_t *)a.z[0] + i * a.ldz + n, v);
  if (a.act != LLMINT8_ACT_NONE)
    with_act(a.act, [&](auto tag) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = act_of<decltype(tag)::value>(v[e]);
    });
  if (a.residual) {
    const u16x8 h = __builtin_bit_cast(u16x8, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += T::to_f(h[e]);
  }
  store8<T>((out ? a.y[1] : a.y[0]) + i * a.ldy + n, v);
}

template <class T>
__device__ inline void load_bias(const FfnGemm &a, int64_t n, float *b) {
  if (a.bias) return load8<T>(a.bias + n, b);
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = 0.f;
}

__device__ inline u32x4 load_residual(const FfnGemm &a, int64_t i, int64_t n) {
  return a.residual ? *(const u32x4 *)(a.residual + i * a.ldr + n) : u32x4{0, 0, 0, 0};
}

// Saves 8 pre-activations in 16 or 8 bits. The 4 lanes of a block of 32 columns
// call it together; `in` is false for columns past N, which hold zeros.
template <class T>
__device__ inline void save8(void *z, int64_t ldz, uint8_t *zs, int64_t ldzs, int64_t i, int64_t n,
                             bool in, const float *v) {
  if (!zs) {
    if (in) store8<T>((uint16_t *)z + i * ldz + n, v);
    return;
  }
  const uint32_t byte = ckpt_byte(block_top(in ? top8(v) : 0u));
  if (!in) return;
  *(u32x2 *)((uint8_t *)z + i * ldz + n) = ckpt_codes8(v, byte);
  if (n % kCkptBlock == 0) zs[i * ldzs + n / kCkptBlock] = (uint8_t)byte;
}

// act(g) * u of 8 columns of one row, and g and u to their places.
template <class T>
__device__ inline void finish_gated(const FfnGemm &a, int64_t i, int64_t n, bool in, float *g,
                                    float *u) {
  if (a.z[0]) {
    save8<T>(a.z[0], a.ldz, a.zs[0], a.ldzs, i, n, in, g);
    save8<T>(a.z[1], a.ldz, a.zs[1], a.ldzs, i, n, in, u);
  }
  if (!in) return;
  with_act(a.act, [&](auto tag) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = act_of<decltype(tag)::value>(g[e]) * u[e];
  });
  store8<T>(a.y[0] + i * a.ldy + n, g);
}

__device__ inline void store_f8(float *p, const float *v) {
  *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4 *)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ inline void load_f8(const float *p, float *v) {
  const f32x4 x = *(const f32x4 *)p, y = *(const f32x4 *)(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = x[e], v[4 + e] = y[e];
}

// Columns 64 block .. + 63 of a BiasJoin, the same sums in the same order for every
// number of THREADS: 64 streams take every 64th partial sum, a thread 4 columns of
// 1024 / THREADS streams with 4 loads of each in flight; they meet in s, 64 x 64 floats.
template <int THREADS>
__device__ inline void join_bias(const BiasJoin &j, int64_t block, float *s) {
  constexpr int V = 1024 / THREADS, STEP = THREADS / 16;
  const int t = threadIdx.x, q4 = t % 16 * 4, r = t / 16;
  const int64_t n0 = block * 64;
  f32x4 sum[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = f32x4{};
  if (n0 + q4 < j.N)  // N is a multiple of 8
    for (int64_t r0 = r; r0 < j.rows; r0 += 4 * 64) {
      f32x4 v[V][4];
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t i = r0 + k * STEP + q * 64;
          v[k][q] = i < j.rows ? *(const f32x4 *)(j.part + i * j.N + n0 + q4) : f32x4{};
        }
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[k][e] += v[k][q][e];
    }
#pragma unroll
  for (int k = 0; k < V; ++k) *(f32x4 *)(s + (r + k * STEP) * 64 + q4) = sum[k];
  __syncthreads();
  if (t < 64 && n0 + t < j.N) {
    float d = 0.f;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) d += s[i * 64 + t];
    j.dbias[n0 + t] = d;
  }
}

// ---- kernel ---------------------------------------------------------------------------

template <Lay L, int N, int NW>
struct TileOf {
  using type = RowKTile<N, NW>;
};
template <int N, int NW>
struct TileOf<Lay::ColK, N, NW> {
  using type = ColKTile<N, NW>;
};

// One launch shape: operand orders, block tile, waves.
template <class T_, Lay LA_, Lay LB_, bool GATED_, int BM_, int BN_, int NWM_, int NWN_, int NST_ = 2>
struct Cfg {
  using T = T_;
  static constexpr Lay LA = LA_, LB = LB_;
  static constexpr bool GATED = GATED_;
  static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, NW = NWM * NWN;
  static constexpr int THREADS = 64 * NW;
  static constexpr int WM = BM / NWM, WN = BN / NWN, MI = WM / 16, NI = WN / 16;
  // columns of one output that a block covers, and of its B tile
  static constexpr int OUTN = GATED ? BN / 2 : BN, BCOLS = OUTN;
  static constexpr int NST = NST_;  // stages in the LDS ring
  static constexpr int STAGE = (BM + BN) * kStep * 2;
  static constexpr int SLABP = WN + 4;  // fp32 pitch of the epilogue's rows
  static constexpr int SLABS = NW * 32 * SLABP * 4;
  static constexpr int LDS = NST * STAGE > SLABS ? NST * STAGE : SLABS;
  static constexpr int WO = GATED ? WN / 2 : WN;  // output columns of a wave
  static_assert(WO % 32 == 0, "a wave holds whole checkpoint blocks");
};

// Block bid of the tiles in tile columns col0 .. col0 + cols - 1 (counted over the
// outputs side by side).
template <class C>
__device__ __forceinline__ void ffn_tile(const FfnGemm &a, uint32_t bid, int col0, int cols,
                                         uint8_t *smem) {
  using T = typename C::T;
  constexpr int BM = C::BM, MI = C::MI, NI = C::NI, NW = C::NW;
  using TA = typename TileOf<C::LA, BM, NW>::type;
  using TB = typename TileOf<C::LB, C::BCOLS, NW>::type;
  constexpr int BOFF = TA::BYTES;          // B's place in a stage
  constexpr int UOFF = BOFF + TB::BYTES;   // the second product's B (gated)
  constexpr int LPS = TA::G + TB::G * (C::GATED ? 2 : 1);  // loads per wave per stage
  const int t = threadIdx.x, lane = t & 63, wv = wave_id();
  const int wm = wv / C::NWN, wn = wv % C::NWN;

  const int tiles_m = (int)((a.M + BM - 1) / BM);
  const int tn1 = (int)((a.N + C::OUTN - 1) / C::OUTN);
  int tm, tn, split;
  tile_at(bid, tiles_m, cols, a.ksplit, tm, tn, split);
  tn += col0;
  const int out = tn >= tn1;
  if (out) tn -= tn1;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * C::OUTN;

  // first element of the tile in each operand (of each segment or product)
  const uint8_t *pa[2], *pb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    pa[i] = (const uint8_t *)a.a[i] + (C::LA == Lay::RowK ? m0 * a.lda : m0) * 2;
    const void *b = a.outs == 2 ? (out ? a.b[1] : a.b[0]) : a.b[i];
    pb[i] = (const uint8_t *)b + (C::LB == Lay::RowK ? n0 * a.ldb : n0) * 2;
  }

  TA A;
  TB B;
  A.init(a.lda, a.M - m0, a.K);
  B.init(a.ldb, a.N - n0, a.K);

  f32x4 acc[MI * NI];
#pragma unroll
  for (int i = 0; i < MI * NI; ++i) acc[i] = (f32x4){};

  const int n1 = (int)((a.K + kStep - 1) / kStep), nst = n1 * a.segs;
  const int s0 = part_begin(nst, split, a.ksplit), s1 = part_begin(nst, split + 1, a.ksplit);

  // The loads of one stage: set up once, then issued one at a time. Past the last
  // stage every address is out of range, and the loads only write zeros to a
  // slot that nothing reads: the loop needs no branch for its end.
  struct Loads {
    typename TA::Stage a;
    typename TB::Stage b, u;
  };
  auto loads_of = [&](int s) {
    const int seg = s >= n1 && a.segs > 1;
    // (clamping len - k instead makes the compiler build the resources in vector
    // registers, with a loop around every load: 6 % slower)
    const int k = (s - (seg ? n1 : 0)) * kStep, len = s < s1 ? (int)a.K : k;
    const uint8_t *b0 = seg ? pb[1] : pb[0];
    return Loads{A.stage(seg ? pa[1] : pa[0], a.lda, k, len), B.stage(b0, a.ldb, k, len),
                 C::GATED ? B.stage(pb[1], a.ldb, k, len) : B.stage(b0, a.ldb, k, len)};
  };
  auto load = [&](const Loads &l, uint8_t *buf, int j) {
    if (j < TA::G)
      A.load(l.a, buf, j);
    else if (C::GATED && j >= TA::G + TB::G)
      B.load(l.u, buf + UOFF, j - TA::G - TB::G);
    else
      B.load(l.b, buf + BOFF, j - TA::G);
  };
  // the f-th fragment of step ks: B's first, then A's, in the order of the MFMAs
  s16x8 av[2][MI], bv[2][NI];
  constexpr int FR = MI + NI;
  auto frag = [&](const uint8_t *cur, int ks, int f) {
    const int b = ks & 1;
    if (f < NI)
      bv[b][f] = C::GATED ? TB::frag(cur + (f >= NI / 2 ? UOFF : BOFF),
                                     wn * C::WO + (f % (NI / 2)) * 16, ks, lane)
                          : TB::frag(cur + BOFF, wn * C::WN + f * 16, ks, lane);
    else
      av[b][f - NI] = TA::frag(cur, wm * C::WM + (f - NI) * 16, ks, lane);
  };
  // MFMAs i0 .. i1 - 1 of step ks, hook(i) after the i-th: a wave's LDS reads and
  // loads go out one at a time between its MFMAs.
  constexpr int MM = MI * NI;
  auto step = [&](int ks, int i0, int i1, auto hook) {
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < MM; ++i)
      if (i >= i0 && i < i1) {
        acc[i] = T::mfma16(bv[ks & 1][i % NI], av[ks & 1][i / NI], acc[i]);
        hook(i);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  // This wave's loads but for the last `younger` have landed and its LDS reads are
  // done, then those of the others. Loads are counted, so every stage issues all
  // of its loads, also past the end.
  auto ring_sync = [&](auto younger) {
    __builtin_amdgcn_s_setprio(0);
    wait_vm<decltype(younger)::value>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };

  // The k loop. The fragments of a step of 32 are read while the MFMAs before run,
  // also across stages: once a wave holds the last fragments of stage s it meets
  // the others, which frees the stage's slot for stage s + NST and shows stage
  // s + 1, and runs the last quarter of the MFMAs with the first fragments of
  // s + 1 and half of the loads of s + NST between them; the other half goes out
  // during the next quarter.
  if (s0 < s1) {
    static_assert(FR <= MM / 2 && LPS % 2 == 0 && LPS <= MM, "they fit between the MFMAs");
    constexpr int NST = C::NST, H = LPS / 2, Q = MM / 2;  // loads and MFMAs of a quarter stage
    auto slot = [&](int i) { return smem + i * C::STAGE; };
    Loads l = loads_of(s0);
#pragma unroll
    for (int q = 0; q < NST; ++q) {
      if (q) l = loads_of(s0 + q);
#pragma unroll
      for (int j = 0; j < (q + 1 < NST ? LPS : H); ++j) load(l, slot(q), j);
    }
    ring_sync(Count<(NST - 2) * LPS + H>());
#pragma unroll
    for (int f = 0; f < FR; ++f) frag(smem, 0, f);
    int at = 0;  // the slot of stage s
    for (int s = s0; s < s1; ++s) {
      uint8_t *const cur = slot(at), *const last = slot(at == 0 ? NST - 1 : at - 1);
      at = at + 1 == NST ? 0 : at + 1;
      const uint8_t *const next = slot(at);
      step(0, 0, MM, [&](int i) {
        if (i < FR) frag(cur, 1, i);
        if (i % (Q / H) == 0 && i / (Q / H) < H) load(l, last, H + i / (Q / H));
      });
      step(1, 0, Q, [](int) {});
      ring_sync(Count<(NST - 2) * LPS>());
      l = loads_of(s + NST);
      step(1, Q, MM, [&](int i) {
        i -= Q;
        if (i < FR) frag(next, 0, i);
        if (i % (Q / H) == 0 && i / (Q / H) < H) load(l, cur, i / (Q / H));
      });
    }
  }
  wait_vm<0>();     // this wave's loads past the end
  __syncthreads();  // the ring is free for the epilogue

  // Lane l of accumulator (mi, ni) holds row l % 16, columns 4 (l / 16) .. + 3 of
  // its 16 x 16 block.
  float *slab = (float *)smem + wv * 32 * C::SLABP;
  constexpr int CPR = C::WO / 8;          // 8-column chunks per row
  constexpr int PASSES = 32 * CPR / 64;   // rows of a slab go in so many passes
  const int64_t n = n0 + wn * C::WO + (lane % CPR) * 8;  // this lane's columns
  auto row_of = [&](int mi, int p) {
    return m0 + wm * C::WM + mi * 32 + p * (64 / CPR) + lane / CPR;
  };
  // the residual of a slab is loaded while the slab before is finished
  u32x4 res[2][PASSES];
  auto prefetch = [&](int mi) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int64_t i = row_of(mi, p);
      if (i < a.M && n < a.N) res[mi & 1][p] = load_residual(a, i, n);
    }
  };
  float bias[8];
  if constexpr (!C::GATED) {
    if (n < a.N) load_bias<T>(a, n, bias);
    if (a.ksplit == 1) prefetch(0);
  }
#pragma unroll
  for (int mi = 0; mi < MI / 2; ++mi) {
    if constexpr (!C::GATED)
      if (a.ksplit == 1 && mi + 1 < MI / 2) prefetch(mi + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        *(f32x4 *)(slab + (h * 16 + (lane & 15)) * C::SLABP + ni * 16 + 4 * (lane >> 4)) =
            acc[(2 * mi + h) * NI + ni];
    // the slab is this wave's own: its LDS operations complete in order
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * (64 / CPR) + lane / CPR, c8 = (lane % CPR) * 8;
      const int64_t i = row_of(mi, p);
      const bool in = i < a.M && n < a.N;
      float v[8], u[8];
      load_f8(slab + r * C::SLABP + c8, v);
      if constexpr (C::GATED) load_f8(slab + r * C::SLABP + C::WO + c8, u);
      if (a.ksplit > 1) {
        if (in) {
          float *part = a.part + (((int64_t)split * (C::GATED ? 2 : a.outs) + out) * a.M + i) * a.N + n;
          store_f8(part, v);
          if constexpr (C::GATED) store_f8(part + a.M * a.N, u);
        }
      } else if constexpr (C::GATED) {
        if (i < a.M) finish_gated<T>(a, i, n, in, v, u);  // the 4 lanes of a block together
      } else if (in) {
        finish_forward<T>(a, out, i, n, v, bias, res[mi & 1][p]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// The last `blocks1` blocks take the C1 tiles of the tile columns before `cut`, the
// first ones the C2 tiles of the rest (see tail_cut): with the halves first, the
// CUs stand at different places of their tiles from then on and their epilogues
// write at different times (1 to 2 % faster than with the halves last).
template <class C1, class C2>
__global__ __launch_bounds__(C1::THREADS, 2) void k_ffn_gemm(FfnGemm a, int cut, int cols,
                                                            uint32_t blocks1) {
  static_assert(C1::THREADS == C2::THREADS && C1::OUTN == C2::OUTN, "one launch");
  extern __shared__ u32x4 smem_v[];
  const uint32_t blocks2 = gridDim.x - blocks1;
  if (blockIdx.x >= blocks2)
    ffn_tile<C1>(a, blockIdx.x - blocks2, 0, cut, (uint8_t *)smem_v);
  else
    ffn_tile<C2>(a, blockIdx.x, cut, cols - cut, (uint8_t *)smem_v);
}

template <class C1, class C2>
hipError_t launch_tiles(const FfnGemm &a, hipStream_t stream) {
  auto *kern = k_ffn_gemm<C1, C2>;
  constexpr int LDS = C1::LDS > C2::LDS ? C1::LDS : C2::LDS;
  hipError_t e =
      hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
  if (e != hipSuccess) return e;
  const int64_t rows = (a.M + C1::BM - 1) / C1::BM;
  const int64_t cols = (a.N + C1::OUTN - 1) / C1::OUTN * a.outs;
  const int64_t cut = C1::BM == C2::BM ? cols : tail_cut(rows, cols, a.ksplit);
  const int64_t blocks1 = rows * cut * a.ksplit;
  const int64_t blocks2 = (a.M + C2::BM - 1) / C2::BM * (cols - cut) * a.ksplit;
  hipLaunchKernelGGL(kern, dim3((unsigned)(blocks1 + blocks2)), dim3(C1::THREADS), LDS, stream, a,
                     (int)cut, (int)cols, (uint32_t)blocks1);
  return hipGetLastError();
}

// The tile shapes of one operand order. With at most one 128-tile per CU a ring of
// four stages covers the latency that the second block of the CU covers otherwise
// (256 x 4096 x 4096 in 4 parts 27.3 -> 23.3 us, whole 49 -> 38; gated
// 192 x 4096 x 4096 39.9 -> 33.0).
template <class T, Lay LA, Lay LB, bool GATED>
hipError_t launch_order(const FfnGemm &a, int tile, hipStream_t stream) {
  using Wide = Cfg<T, LA, LB, GATED, 256, 256, 2, 4>;
  using Tail = Cfg<T, LA, LB, GATED, 128, 256, 2, 4>;
  using Small = Cfg<T, LA, LB, GATED, 128, 128, 2, 2>;
  using Deep = Cfg<T, LA, LB, GATED, 128, 128, 2, 2, 4>;
  if (tile == 256) return launch_tiles<Wide, Tail>(a, stream);
  const int64_t blocks = (a.M + 127) / 128 * ((a.N + Small::OUTN - 1) / Small::OUTN) * a.outs *
                         a.ksplit;
  return deep_ring(blocks) ? launch_tiles<Deep, Deep>(a, stream)
                           : launch_tiles<Small, Small>(a, stream);
}

}  // namespace ffn
}  // namespace llmint8
