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
//  * a stage is 64 reduction steps of both operands, 128 bytes per output row or
//    column, brought to LDS by 16-byte direct-to-LDS loads; a RowK tile keeps
//    its rows of 128 bytes, a ColK tile its 64 rows of the matrix.
//  * MFMA fragments (8 consecutive reduction steps of one row per lane) are one
//    16-byte LDS read from a RowK tile and two transposed 8-byte reads from a
//    ColK tile: a group of 16 lanes addresses a 4 x 16 block of 16-bit values
//    row by row and each lane receives one column of it.
//  * 16-byte chunks are permuted within each stored row, so that the lanes of
//    one LDS access fall in different bank groups: chunk c of row r sits at
//    c ^ ((r >> 1) & 7) in a RowK tile (rows of 8 chunks) and at c ^ 4 (r & 3)
//    in a ColK tile (the 4 rows of a transposed block, 4 chunks each).
//  * Operands past the end of the matrix (rows, columns, reduction) read as
//    zero: every load goes through a buffer resource that ends with the last
//    element, and a RowK lane whose chunk lies past the reduction length takes
//    an offset outside it. Both operands are zero there, so no infinity or NaN
//    of a neighbouring row is multiplied by a zero.
//  * The checkpointed X of grad W (ColK8) is read as 8-bit codes, expanded to
//    16 bits in registers (exactly, see ffn_math.hpp) and written to LDS in the
//    ColK order.
//
// A block computes BM x BN outputs with NWM x NWN waves. The MFMAs take the
// operands in the order (B, A), so a lane's accumulators hold 4 consecutive
// columns of one row; the epilogue passes 32 rows at a time through LDS in fp32,
// after which a lane owns 8 consecutive columns and every load and store of the
// epilogue is 16 bytes.
#pragma once

#include "ffn_math.hpp"
#include "gemm_core.hpp"

namespace llmint8 {
namespace ffn {

using gemm_detail::lptr_t;
using gemm_detail::make_rsrc;
using gemm_detail::rsrc_t;
using gemm_detail::tile_of_block;
using gemm_detail::wait_vm;

constexpr int kStep = 64;  // reduction steps per stage
constexpr int kOob = (int)0x80000000;  // an offset past the end of every resource

enum class Lay { RowK, ColK, ColK8 };

__device__ inline int clip31(int64_t bytes) {
  return (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff);
}

// ROWS output rows (or columns) x 64 reduction steps, reduction contiguous.
template <int ROWS, int NW>
struct RowKTile {
  static constexpr int BYTES = ROWS * 128;
  static constexpr int G = ROWS / (8 * NW);  // 1 KB loads per wave per stage
  static constexpr int REGS = 1;             // LDS address registers per fragment row block
  int64_t bytes;  // of the tile's rows, from the first element to the last
  int voff[G];
  int chunk;      // first reduction step of this lane's chunk within a stage

  // mat: the first row of the tile; rows: rows of the matrix from there on.
  __device__ void init(int64_t ld, int64_t rows, int64_t len) {
    rows = rows < ROWS ? rows : ROWS;
    bytes = ((rows - 1) * ld + len) * 2;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    chunk = 0;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int r = (wv + NW * j) * 8 + lane / 8;
      const int c = (lane % 8) ^ ((r >> 1) & 7);
      voff[j] = r * (int)ld * 2 + 16 * c;
      chunk = 8 * c;  // the same for every j: the key repeats every 16 rows
    }
  }
  static_assert(NW % 2 == 0, "the chunk key must not depend on j");

  // Groups j0 .. j1 - 1 of the stage starting at reduction step k.
  __device__ void load(const void *mat, int64_t len, int64_t, uint8_t *stage, int64_t k, int j0,
                       int j1) const {
    const int wv = threadIdx.x >> 6;
    const rsrc_t rs = make_rsrc((const uint8_t *)mat + 2 * k, clip31(bytes - 2 * k));
    const bool in = k + chunk < len;
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (j >= j0 && j < j1)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lptr_t)(stage + (wv + NW * j) * 1024), 16,
                                                 in ? voff[j] : kOob, 0, 0, 0);
  }

  // Fragment of 32 rows from row0 for reduction steps 16 ks .. 16 ks + 15.
  __device__ static s16x8 frag(const uint8_t *tile, int row0, int ks, int lane) {
    const int r = row0 + (lane & 31);
    return *(const s16x8 *)(tile + r * 128 + 16 * ((2 * ks + (lane >> 5)) ^ ((r >> 1) & 7)));
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

// 64 reduction steps x COLS output rows (or columns), reduction strided.
template <int COLS, int NW>
struct ColKTile {
  static constexpr int BYTES = COLS * 128;
  static constexpr int PITCH = COLS * 2;
  static constexpr int CH = COLS / 8;      // chunks per stored row
  static constexpr int RPI = 64 / CH;      // stored rows per 1 KB load
  static constexpr int G = kStep / (RPI * NW);
  int voff[G];
  int64_t cols;  // columns of the matrix from the tile's first on

  // Rows of 8 chunks: rows r and r + 1 lie in opposite halves of the banks already.
  __device__ static int key(int r) { return CH >= 16 ? 4 * (r & 3) : 4 * ((r >> 1) & 1); }

  __device__ void init(int64_t ld, int64_t ncols, int64_t) {
    cols = ncols;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int r = (wv + NW * j) * RPI + lane / CH;
      voff[j] = r * (int)ld * 2 + 16 * ((lane % CH) ^ key(r));
    }
  }

  // mat: element (0, first column of the tile). The resource ends with the last
  // column of the stage's last row of the matrix.
  __device__ void load(const void *mat, int64_t len, int64_t ld, uint8_t *stage, int64_t k, int j0,
                       int j1) const {
    const int wv = threadIdx.x >> 6;
    const int64_t rows = len - k < kStep ? len - k : kStep;
    const rsrc_t rs = make_rsrc((const uint8_t *)mat + 2 * k * ld,
                                clip31(((rows - 1) * ld + cols) * 2));
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (j >= j0 && j < j1)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lptr_t)(stage + (wv + NW * j) * 1024), 16,
                                                 voff[j], 0, 0, 0);
  }

  __device__ static s16x8 frag(const uint8_t *tile, int col0, int ks, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const int c = (col0 >> 3) + (g & 1) * 2 + ((i & 3) >> 1);
    const uint8_t *p = tile + (ks * 16 + (g >> 1) * 8 + (i >> 2)) * PITCH +
                       16 * (c ^ key(i >> 2)) + 8 * (i & 1);
    const s16x4 lo = read_tr16((tr_ptr_t)p), hi = read_tr16((tr_ptr_t)(p + 4 * PITCH));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// ColKTile filled from 8-bit codes through registers: fetch() starts the loads
// of a stage, commit() expands them into LDS. Rows of codes are read to the next
// multiple of 16 entries (their pitch is one); what lies there past the last
// column only reaches outputs that are not stored.
template <class T, int COLS, int NW>
struct ColK8Tile : ColKTile<COLS, NW> {
  using Base = ColKTile<COLS, NW>;
  static constexpr int CPR = COLS / 16;               // 16-code chunks per row
  static constexpr int J = kStep * CPR / (64 * NW);   // chunks per thread
  static constexpr int RPJ = 64 * NW / CPR;           // rows between a thread's chunks
  u32x4 q[J];
  uint32_t sc[J];

  __device__ void fetch(const void *mat, int64_t ld, const uint8_t *scales, int64_t lds,
                        int64_t len, int64_t k) {
    const int t = threadIdx.x, r0 = t / CPR, c = t % CPR;
    const int64_t rows = len - k < kStep ? len - k : kStep;
    const rsrc_t rs = make_rsrc((const uint8_t *)mat + k * ld,
                                clip31((rows - 1) * ld + (Base::cols + 15) / 16 * 16));
    const rsrc_t rc = make_rsrc(scales + k * lds,
                                clip31((rows - 1) * lds + (Base::cols + kCkptBlock - 1) / kCkptBlock));
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int r = r0 + RPJ * j;
      q[j] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, r * (int)ld + 16 * c, 0, 0));
      sc[j] = __builtin_amdgcn_raw_buffer_load_b8(rc, r * (int)lds + c / 2, 0, 0);
    }
  }

  __device__ void commit(uint8_t *stage) const {
    const int t = threadIdx.x, r0 = t / CPR, c = t % CPR;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int r = r0 + RPJ * j;
      const float scale = ckpt_scale(sc[j] & 0xffu);
      float v[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) ckpt_value4(q[j][e], scale, v + 4 * e);
      uint8_t *row = stage + r * Base::PITCH;
      const int key = Base::key(r);
      store8<T>((uint16_t *)(row + 16 * ((2 * c) ^ key)), v);
      store8<T>((uint16_t *)(row + 16 * ((2 * c + 1) ^ key)), v + 8);
    }
  }
};

// ---- epilogue -------------------------------------------------------------------------

// 8 consecutive columns of one row: act(v + bias) + residual; the sums v + bias
// go to z on the way.
template <class T>
__device__ inline void finish_forward(const FfnGemm &a, int out, int64_t i, int64_t n, float *v) {
  if (a.bias) {
    float b[8];
    load8<T>(a.bias + n, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += b[e];
  }
  if (a.z[0]) store8<T>((uint16_t *)a.z[0] + i * a.ldz + n, v);
  if (a.act != LLMINT8_ACT_NONE)
    with_act(a.act, [&](auto tag) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = act_of<decltype(tag)::value>(v[e]);
    });
  if (a.residual) {
    float r[8];
    load8<T>(a.residual + i * a.ldr + n, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  store8<T>((out ? a.y[1] : a.y[0]) + i * a.ldy + n, v);
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

// ---- kernel ---------------------------------------------------------------------------

template <class T, Lay L, int N, int NW>
struct TileOf {
  using type = RowKTile<N, NW>;
};
template <class T, int N, int NW>
struct TileOf<T, Lay::ColK, N, NW> {
  using type = ColKTile<N, NW>;
};
template <class T, int N, int NW>
struct TileOf<T, Lay::ColK8, N, NW> {
  using type = ColK8Tile<T, N, NW>;
};

// One launch shape: operand orders, block tile, waves.
template <class T_, Lay LA_, Lay LB_, bool GATED_, int BM_, int BN_, int NWM_, int NWN_>
struct Cfg {
  using T = T_;
  static constexpr Lay LA = LA_, LB = LB_;
  static constexpr bool GATED = GATED_;
  static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, NW = NWM * NWN;
  static constexpr int THREADS = 64 * NW;
  static constexpr int WM = BM / NWM, WN = BN / NWN, MI = WM / 32, NI = WN / 32;
  // columns of one output that a block covers, and of its B tile
  static constexpr int OUTN = GATED ? BN / 2 : BN, BCOLS = OUTN;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int SLABP = WN + 4;  // fp32 pitch of the epilogue's rows
  static constexpr int SLABS = NW * 32 * SLABP * 4;
  static constexpr int LDS = 2 * STAGE > SLABS ? 2 * STAGE : SLABS;
  static_assert(!GATED || NI == 2, "a gated wave holds 32 columns of each product");
};

template <class C>
__device__ __forceinline__ void ffn_tile(const FfnGemm &a, int64_t bid, uint8_t *smem) {
  using T = typename C::T;
  constexpr int BM = C::BM, MI = C::MI, NI = C::NI, NW = C::NW;
  constexpr bool A8 = C::LA == Lay::ColK8;
  constexpr int BOFF = BM * 128;           // B's place in a stage
  constexpr int UOFF = BOFF + C::BCOLS * 128;  // the second product's B (gated)
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  const int wm = wv / C::NWN, wn = wv % C::NWN;

  const int64_t tiles_m = (a.M + BM - 1) / BM;
  const int64_t tn1 = (a.N + C::OUTN - 1) / C::OUTN, tiles_n = tn1 * a.outs;
  const int64_t tiles = tiles_m * tiles_n;
  const int split = (int)(bid / tiles);
  int64_t tm, tn;
  tile_of_block(bid % tiles, tiles_m, tiles_n, tm, tn);
  const int out = tn >= tn1;
  if (out) tn -= tn1;
  const int64_t m0 = tm * BM, n0 = tn * C::OUTN;

  // first element of the tile in each operand (of each segment or product)
  const uint8_t *pa[2], *pb[2];
  constexpr int ea = A8 ? 1 : 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    pa[i] = (const uint8_t *)a.a[i] + (C::LA == Lay::RowK ? m0 * a.lda : m0) * ea;
    const void *b = a.outs == 2 ? (out ? a.b[1] : a.b[0]) : a.b[i];
    pb[i] = (const uint8_t *)b + (C::LB == Lay::RowK ? n0 * a.ldb : n0) * 2;
  }

  typename TileOf<T, C::LA, BM, NW>::type A;
  typename TileOf<T, C::LB, C::BCOLS, NW>::type B;
  A.init(a.lda, a.M - m0, a.K);
  B.init(a.ldb, a.N - n0, a.K);

  f32x16 acc[MI * NI];
#pragma unroll
  for (int i = 0; i < MI * NI; ++i) acc[i] = (f32x16){};

  const int64_t n1 = (a.K + kStep - 1) / kStep, nst = n1 * a.segs;
  const int64_t s0 = nst * split / a.ksplit, s1 = nst * (split + 1) / a.ksplit;

  // direct-to-LDS loads of stage s, half h of them (0, 1; 2: both)
  auto load = [&](int64_t s, int h) {
    const int seg = s >= n1;
    const int64_t k = (s - (seg ? n1 : 0)) * kStep;
    uint8_t *buf = smem + ((s - s0) & 1) * C::STAGE;
    if constexpr (!A8) {
      constexpr int G = decltype(A)::G;
      A.load(seg ? pa[1] : pa[0], a.K, a.lda, buf, k, h == 1 ? G / 2 : 0, h == 0 ? G / 2 : G);
    }
    constexpr int G = decltype(B)::G;
    const int j0 = h == 1 ? G / 2 : 0, j1 = h == 0 ? G / 2 : G;
    if constexpr (C::GATED) {
      B.load(pb[0], a.K, a.ldb, buf + BOFF, k, j0, j1);
      B.load(pb[1], a.K, a.ldb, buf + UOFF, k, j0, j1);
    } else {
      B.load(seg ? pb[1] : pb[0], a.K, a.ldb, buf + BOFF, k, j0, j1);
    }
  };
  auto fetch = [&](int64_t s) {
    if constexpr (A8)
      A.fetch(pa[0], a.lda, a.as + m0 / kCkptBlock, a.ldas, a.K, s * kStep);
  };
  auto commit = [&](int64_t s) {
    if constexpr (A8) A.commit(smem + ((s - s0) & 1) * C::STAGE);
  };

  if (s0 < s1) {
    fetch(s0);
    load(s0, 2);
    commit(s0);
  }
  for (int64_t s = s0; s < s1; ++s) {
    // Stage s has landed for this wave, then for all; that also means that
    // every wave has read the other buffer to the end. The LDS waits cover a
    // checkpointed A, written by this wave's own stores.
    wait_vm<0>();
    if constexpr (A8) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    asm volatile("s_barrier" ::: "memory");
    const bool more = s + 1 < s1;
    if (more) {
      fetch(s + 1);
      load(s + 1, 0);
    }
    const uint8_t *cur = smem + ((s - s0) & 1) * C::STAGE;
    s16x8 av[2][MI], bv[2][NI];
    auto frags = [&](int ks, int b) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        av[b][mi] = decltype(A)::frag(cur, wm * C::WM + mi * 32, ks, lane);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        bv[b][ni] = C::GATED
                        ? decltype(B)::frag(cur + (ni ? UOFF : BOFF), wn * 32, ks, lane)
                        : decltype(B)::frag(cur + BOFF, wn * C::WN + ni * 32, ks, lane);
    };
    frags(0, 0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) frags(ks + 1, (ks + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi * NI + ni] = T::mfma32(bv[ks & 1][ni], av[ks & 1][mi], acc[mi * NI + ni]);
      if (ks == 0 && more) load(s + 1, 1);
      if (ks == 2 && more) commit(s + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();  // the ring is free for the epilogue

  // Lane l of accumulator (mi, ni) holds row l % 32, columns
  // 8 (r / 4) + 4 (l / 32) + r % 4 of its 32 x 32 block.
  float *slab = (float *)smem + wv * 32 * C::SLABP;
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16 &c = acc[mi * NI + ni];
        *(f32x4 *)(slab + (lane & 31) * C::SLABP + ni * 32 + 8 * q + 4 * (lane >> 5)) =
            f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
    // the slab is this wave's own: its LDS operations complete in order
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if constexpr (C::GATED) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int r = p * 16 + lane / 4, c8 = (lane % 4) * 8;
        const int64_t i = m0 + wm * C::WM + mi * 32 + r, n = n0 + wn * 32 + c8;
        float g[8], u[8];
        load_f8(slab + r * C::SLABP + c8, g);
        load_f8(slab + r * C::SLABP + 32 + c8, u);
        if (a.ksplit > 1) {
          if (i < a.M && n < a.N) {
            float *part = a.part + ((int64_t)split * 2 * a.M + i) * a.N + n;
            store_f8(part, g);
            store_f8(part + a.M * a.N, u);
          }
        } else if (i < a.M) {  // uniform over the 4 lanes of a row's block
          finish_gated<T>(a, i, n, n < a.N, g, u);
        }
      }
    } else {
      constexpr int CPR = C::WN / 8;  // 8-column chunks per row
#pragma unroll
      for (int p = 0; p < 32 * CPR / 64; ++p) {
        const int r = p * (64 / CPR) + lane / CPR, c8 = (lane % CPR) * 8;
        const int64_t i = m0 + wm * C::WM + mi * 32 + r, n = n0 + wn * C::WN + c8;
        if (i < a.M && n < a.N) {
          float v[8];
          load_f8(slab + r * C::SLABP + c8, v);
          if (a.ksplit > 1)
            store_f8(a.part + (((int64_t)split * a.outs + out) * a.M + i) * a.N + n, v);
          else
            finish_forward<T>(a, out, i, n, v);
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_ffn_gemm(FfnGemm a) {
  extern __shared__ u32x4 smem_v[];
  ffn_tile<C>(a, blockIdx.x, (uint8_t *)smem_v);
}

template <class C>
hipError_t launch_tile(const FfnGemm &a, hipStream_t stream) {
  auto *kern = k_ffn_gemm<C>;
  hipError_t e = hipFuncSetAttribute((const void *)kern,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  const int64_t blocks = ((a.M + C::BM - 1) / C::BM) * ((a.N + C::OUTN - 1) / C::OUTN) * a.outs *
                         a.ksplit;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(C::THREADS), C::LDS, stream, a);
  return hipGetLastError();
}

// The two tile shapes of one operand order.
template <class T, Lay LA, Lay LB, bool GATED>
hipError_t launch_order(const FfnGemm &a, int tile, hipStream_t stream) {
  if (tile == 256) return launch_tile<Cfg<T, LA, LB, GATED, 256, 256, 2, 4>>(a, stream);
  return launch_tile<Cfg<T, LA, LB, GATED, 128, 128, 2, 2>>(a, stream);
}

}  // namespace ffn
}  // namespace llmint8
