// Tiles of the experts' products, one after the other without a gap.
//
// The experts' tiles are many and often short: a weight gradient's reduction is as long as the
// expert has rows, 8 stages of 64 for 512 of them, beside which filling the ring and storing the
// result (two thirds of the time of ffn_gemm.hpp's tiles there) count. So a block stays on its CU
// and works through tiles with one ring that does not stop between them:
//  * the loads run two stages ahead of the MFMAs, past the end of a tile into the next one;
//  * the fragments of a next tile's first stage are read under the last MFMAs of this one;
//  * the epilogue takes no LDS: lanes 16 apart swap registers (v_permlane16_swap), after which a
//    lane has 8 consecutive columns of a row, and stores 16 bytes of it, 64 contiguous bytes
//    a row and instruction. All of the next loads are issued before the stores, so
//    that the next stage's wait counts the stores instead of waiting for them (buffer stores,
//    which are issued also where every lane is out of range: the count is exact).
// Waves whose part of a tile lies past its rows or columns load and wait with the others but
// compute nothing.
//
// The stage, its operands in LDS and the order of loads, LDS reads and MFMAs are those of
// ffn_gemm.hpp. Where a tile begins, nothing waits for memory: the experts' places are in LDS or
// in the scalar cache, and the pairs of a tile's rows have been brought to LDS while the tile
// before was loaded; their weights follow, long before the epilogue takes them.
//
// Measured, 4096 tokens x 4 of 32 experts, 4096 x 2048, bf16: gated 600 us (0.92 PFLOP/s; with one
// tile a block 633), dX 616, the pair of weight gradients 750 (the whole backward call 1465; with dX's
// rows in 16 bits 1390, and 1870 with one tile a block); the MFMAs are busy for 0.52, 0.49 and 0.38
// of the time, at a clock of 1.95 GHz, since 2.4 GHz would take more power than the card has. What
// remains is
// tiles that are not full where the router is uneven (80 tile rows for 64 tiles' worth of rows;
// 485 us with even experts), the weights' way from HBM (454 where all experts share one's) and, for
// weight gradients, their stores (1.07 GB; 610 without them). Stages of 32 in a ring of four were
// slower (545 against 485 even), prefetches into L2 (by 5 %), experts sorted by their rows (515),
// 128-tiles for weight gradients (964). Non-temporal stores and whole lines made the 16-bit dWd of
// 12004 rows 308 us from 405.
#pragma once

#include "experts_tile.hpp"

namespace llmint8 {
namespace ffn {

// A RowKTile whose rows are anywhere in a matrix of less than 2^31 bytes: row r of the tile
// is row at(r) of it, or zeros where that is negative.
template <int ROWS, int NW>
struct RowKAtTile : RowKTile<ROWS, NW> {
  using Base = RowKTile<ROWS, NW>;
  template <class At>
  __device__ void init_at(int64_t ld, int64_t mat_rows, int64_t len, int lane, At at) {
    this->bytes = (int)((mat_rows - 1) * ld + len) * 2;
    const int wv = wave_id();
#pragma unroll
    for (int j = 0; j < Base::G; ++j) {
      const int r = (wv + NW * j) * Base::RPI + lane / Base::CH;
      const int c = (lane % Base::CH) ^ Base::key(r);
      const int64_t row = at(r);
      this->voff[j] = row < 0 ? kOob : (int)row * (int)ld * 2 + 16 * c;
      this->chunk = 8 * c;
    }
  }
};

template <int N, int NW>
struct TileOf<Lay::RowKAt, N, NW> {
  using type = RowKAtTile<N, NW>;
};

// One tile: operands at its first row and column (of both segments, or of the gated product's
// two), what it writes, and how much of each there is.
struct Job {
  const uint8_t *a[2], *b[2];
  int K;                 // length of the reduction
  const int32_t *pairs;  // of the tile's rows
  struct Out {
    uint16_t *y;         // the tile's place in the result
    int row0, n0;        // its first row and column (where they lead to further results)
    int rows, cols;      // rows and columns from there on
  } out;
};

// The arguments of a kernel that has them all in one struct, read again from where the launch
// put them. What a tile begins and ends with needs many of them, and kept in scalar registers
// beside the loop's own they would not fit.
template <class K>
__device__ inline const K __attribute__((address_space(4))) * kernel_args() {
  auto p = (const K __attribute__((address_space(4))) *)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// Cache policy of stores whose lines are not read soon.
constexpr int kNonTemporal = 2;

// acc: two 16 x 16 blocks side by side, lane l with row l % 16 and columns 4 (l / 16) .. + 3 of
// each. v: 8 columns of the row, from 16 (g % 2) + 8 (g / 2) on, g = l / 16.
__device__ inline void join_blocks(const f32x4 &c0, const f32x4 &c1, float *v) {
  // (casts of whole vectors: those of their elements were compiled to the first one's)
  const u32x4 x = __builtin_bit_cast(u32x4, c0), y = __builtin_bit_cast(u32x4, c1);
  u32x4 lo, hi;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto s = __builtin_amdgcn_permlane16_swap(x[e], y[e], false, false);
    lo[e] = s[0], hi[e] = s[1];
  }
  const f32x4 l = __builtin_bit_cast(f32x4, lo), h = __builtin_bit_cast(f32x4, hi);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = l[e], v[4 + e] = h[e];
}

template <class T>
__device__ inline u32x4 pack8(const float *v) {
  u16x8 h;
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = T::from_f(v[e]);
  return __builtin_bit_cast(u32x4, h);
}

// LDS behind the ring: for routed rows the pairs and the weights of two tiles.
template <class C>
constexpr int tiles_lds() {
  return 2 * C::STAGE + (C::ROUTED ? 4 * C::BM * 4 : 0);
}

// The tiles place, place + step, ... below `tiles` of find(args, tile, job). K: the kernel's
// arguments, with the product as K::a.
template <class C, class K, class Find>
__device__ __forceinline__ void run_tiles(int64_t lda, int64_t ldb, int nsegs, uint32_t tiles,
                                          Find find, uint8_t *smem) {
  using T = typename C::T;
  static_assert(C::NST == 2, "two stages");
  constexpr int BM = C::BM, MI = C::MI, NI = C::NI, NW = C::NW;
  using TA = typename TileOf<C::LA, BM, NW>::type;
  using TB = typename TileOf<C::LB, C::BCOLS, NW>::type;
  constexpr int BOFF = TA::BYTES, UOFF = BOFF + TB::BYTES;
  constexpr int LPS = TA::G + TB::G * (C::GATED ? 2 : 1);
  constexpr int STORES = C::GATED ? MI : MI * NI / 2;  // of one result, per tile and wave
  const int t = threadIdx.x, lane = t & 63, wv = wave_id();
  const int wm = wv / C::NWN, wn = wv % C::NWN;
  // of two tiles' rows, by the tile's parity
  int32_t *const prow = (int32_t *)(smem + 2 * C::STAGE);
  float *const wrow = (float *)(smem + 2 * C::STAGE + 2 * BM * 4);
  const int row64 = wv % (BM / 64) * 64;  // the rows that this wave brings

  const int segs = C::GATED ? 1 : nsegs;
  const uint32_t step = gridDim.x;
  uint32_t tile = xcd_place(blockIdx.x, step);  // the tile that is loaded
  if (tile >= tiles) return;
  Job ld;
  TA A;
  TB B;
  int n1, nst, ls, lpar = 0;  // its stages a segment and in all, the next to load, its parity
  bool more = true;
  // the pairs of a tile's rows to LDS; past them 0, which is not used
  auto bring_pairs = [&](const Job &j, int par, int lane) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(j.pairs, j.out.rows * 4),
                                             (lptr_t)(prow + par * BM + row64), 4,
                                             (row64 + lane) * 4, 0, 0, 0);
  };
  auto begin = [&]() {
    const auto *k = kernel_args<K>();
    find(k, tile, ld);
    if constexpr (C::ROUTED) {
      int lane = threadIdx.x & 63;  // computed here (see store_tile)
      asm volatile("" : "+v"(lane));
      const int32_t *const pr = prow + lpar * BM;
      const int rows = ld.out.rows;
      const uint32_t topk = (uint32_t)k->a.topk;
      const int64_t a_rows = topk ? k->a.a_rows : rows;
      A.init_at(lda, a_rows, ld.K, lane, [&](int r) {
        const int64_t row = topk ? (uint32_t)pr[r] / topk : r;
        return r < rows && row < a_rows ? row : -1;
      });
      // a weight of a pair that no plan can hold is 0, by the buffer's end
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          make_rsrc(k->a.w, k->a.w ? k->a.all_rows * 4 : 0),
          (lptr_t)(wrow + lpar * BM + row64), 4,
          row64 + lane < rows ? (int)((uint32_t)pr[row64 + lane] < 0x20000000u
                                          ? pr[row64 + lane] * 4 : kOob) : kOob, 0, 0, 0);
      if (tile + step < tiles) {
        Job j;
        find(k, tile + step, j);
        bring_pairs(j, lpar ^ 1, lane);
      }
    } else {
      A.init(lda, ld.out.rows, ld.K);
    }
    B.init(ldb, ld.out.cols, ld.K);
    n1 = (ld.K + kStep - 1) / kStep;
    // two at least: the loads are never more than one tile ahead
    nst = n1 * segs > 2 ? n1 * segs : 2;
    ls = 0;
  };
  struct Loads {
    typename TA::Stage a;
    typename TB::Stage b, u;
  };
  // The next stage; behind the last tile, and behind a short one's stages, everything is out of
  // range and the loads only write zeros.
  auto next = [&]() {
    if (ls == nst && more) {
      tile += step, lpar ^= 1;
      more = tile < tiles;
      if (more) begin();
    }
    const bool in = more && ls < n1 * segs;
    const bool seg = !C::GATED && in && ls >= n1;
    const int k = in ? (ls - (seg ? n1 : 0)) * kStep : 0, len = in ? ld.K : 0;
    ++ls;
    const uint8_t *const b0 = seg ? ld.b[1] : ld.b[0];
    return Loads{A.stage(seg ? ld.a[1] : ld.a[0], lda, k, len), B.stage(b0, ldb, k, len),
                 C::GATED ? B.stage(ld.b[1], ldb, k, len) : B.stage(b0, ldb, k, len)};
  };
  auto load = [&](const Loads &l, uint8_t *buf, int j) {
    if (j < TA::G)
      A.load(l.a, buf, j);
    else if (C::GATED && j >= TA::G + TB::G)
      B.load(l.u, buf + UOFF, j - TA::G - TB::G);
    else
      B.load(l.b, buf + BOFF, j - TA::G);
  };
  // A stage is S steps of NI MFMAs, a row block of 32 reduction steps each. A's fragments go
  // through a ring of eight, AHEAD steps ahead of their use; B's for 32 reduction steps are
  // kept and the next 32's read beside them.
  constexpr int S = 2 * MI, AHEAD = MI == 8 ? 6 : 4, MEET = S - S / 4, HOOKS = (S - MEET) * NI;
  s16x8 av[8], bv[2][NI];
  auto read_a = [&](const uint8_t *buf, int n) {
    av[n % 8] = TA::frag(buf, wm * C::WM + n % MI * 16, n / MI, lane);
  };
  auto read_b = [&](const uint8_t *buf, int ks, int f) {
    bv[ks][f] = C::GATED ? TB::frag(buf + (f >= NI / 2 ? UOFF : BOFF),
                                    wn * C::WO + (f % (NI / 2)) * 16, ks, lane)
                         : TB::frag(buf + BOFF, wn * C::WN + f * 16, ks, lane);
  };
  constexpr int MM = MI * NI;
  f32x4 acc[MM];
  // Steps n0 .. n1 - 1, hook(i) after the i-th of their MFMAs.
  auto steps = [&](int n0, int n1, auto hook) {
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < S; ++n)
      if (n >= n0 && n < n1)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const int c = n % MI * NI + ni;
          acc[c] = T::mfma16(bv[n / MI][ni], av[n % 8], acc[c]);
          hook((n - n0) * NI + ni);
          __builtin_amdgcn_sched_barrier(0);
        }
  };
  auto sync = [&](auto younger) {
    __builtin_amdgcn_s_setprio(0);
    wait_vm<decltype(younger)::value>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MM; ++i) acc[i] = (f32x4){};
  };

  // The tile that is computed.
  Job::Out cur;
  bool active;  // this wave's part of it has rows and columns
  int left, cpar = 0;
  auto take = [&]() {
    cur = ld.out, left = nst;
    active = wm * C::WM < cur.rows && wn * C::WO < cur.cols;
  };
  // whether the rows go to `part` in fp32: the second product's always (a token's are still to be
  // summed, and rounded then), of the gradients by rows dX's
  const bool wide =
      C::LA == Lay::RowK && (C::LB == Lay::ColK || kernel_args<K>()->a.to_parts);
  auto store_tile = [&]() {
    // computed here, not kept in registers beside the loop's
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const auto *k = kernel_args<K>();
    const int64_t cols = cur.cols < C::OUTN ? cur.cols : C::OUTN;
    const int ldy = (int)k->a.ldy;
    const rsrc_t ry = make_rsrc(cur.y, ((int64_t)(cur.rows - 1) * ldy + cols) * 2);
    const int r0 = wm * C::WM + (lane & 15), g = lane >> 4;
    const int c0 = wn * C::WO + 16 * (g & 1) + 8 * (g >> 1);
    if constexpr (C::GATED) {
      const int ldz = (int)k->a.ldz, act = k->a.act;
      const int64_t zb = ((int64_t)(cur.rows - 1) * ldz + cols) * 2;
      const int64_t z0 = (int64_t)cur.row0 * ldz + cur.n0;
      const bool save = k->a.z[0] != nullptr, weighted = k->a.w != nullptr;
      const rsrc_t rg = make_rsrc((uint16_t *)k->a.z[0] + z0, zb);
      const rsrc_t ru = make_rsrc((uint16_t *)k->a.z[1] + z0, zb);
      const bool in = c0 < cur.cols;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        const int r = r0 + mi * 16;
        float gv[8], uv[8];
        join_blocks(acc[mi * NI], acc[mi * NI + 1], gv);
        join_blocks(acc[mi * NI + 2], acc[mi * NI + 3], uv);
        if (save) {
          const int off = in ? r * ldz * 2 + c0 * 2 : kOob;
          __builtin_amdgcn_raw_buffer_store_b128(pack8<T>(gv), rg, off, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(pack8<T>(uv), ru, off, 0, 0);
        }
        const float w = weighted ? wrow[cpar * BM + r] : 1.f;
        with_act(act, [&](auto tag) {
#pragma unroll
          for (int e = 0; e < 8; ++e) gv[e] = act_of<decltype(tag)::value>(gv[e]) * uv[e] * w;
        });
        __builtin_amdgcn_raw_buffer_store_b128(pack8<T>(gv), ry,
                                               in ? r * ldy * 2 + c0 * 2 : kOob, 0, 0);
      }
    } else if (wide) {
      const int ldp = (int)k->a.N;
      float *const part = k->a.part + (int64_t)cur.row0 * ldp + cur.n0;
      const rsrc_t rp = make_rsrc(part, ((int64_t)(cur.rows - 1) * ldp + cols) * 4);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int q = 0; q < NI / 2; ++q) {
          float v[8];
          join_blocks(acc[mi * NI + 2 * q], acc[mi * NI + 2 * q + 1], v);
          const int c = c0 + 32 * q, off = ((r0 + mi * 16) * ldp + c) * 4;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const u32x4 w = __builtin_bit_cast(
                u32x4, f32x4{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]});
            __builtin_amdgcn_raw_buffer_store_b128(w, rp, c < cur.cols ? off + 16 * e : kOob, 0, 0);
          }
        }
    } else {
      // Two instructions a row block, of 8 rows and 128 bytes of each: lanes 8 apart swap
      // halves, so that whole lines are written.
      static_assert(NI == 4, "64 columns a wave");
      const int hi = lane >> 3 & 1, c = c0 + 32 * hi;
      const int r = wm * C::WM + (lane & 7);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        float v[2][8];
        join_blocks(acc[mi * NI], acc[mi * NI + 1], v[0]);
        join_blocks(acc[mi * NI + 2], acc[mi * NI + 3], v[1]);
        const u32x4 x = pack8<T>(v[0]), y = pack8<T>(v[1]);
        u32x4 lo, up;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // row_ror:8 into lanes 8 .. 15, 0 .. 7 of each 16
          const int a = (int)x[e], b = (int)y[e];
          lo[e] = (uint32_t)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xf, 0xc, false);
          up[e] = (uint32_t)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xf, 0x3, false);
        }
        // weight gradients are not read soon, rows by the next launch
        constexpr int policy = C::LA == Lay::ColK ? kNonTemporal : 0;
        const int off = (r + mi * 16) * ldy * 2 + c * 2;
        __builtin_amdgcn_raw_buffer_store_b128(lo, ry, c < cur.cols ? off : kOob, 0, policy);
        __builtin_amdgcn_raw_buffer_store_b128(up, ry, c < cur.cols ? off + 16 * ldy : kOob, 0,
                                               policy);
      }
    }
  };

  static_assert(AHEAD + NI <= HOOKS && LPS <= HOOKS && S - AHEAD <= MEET && S - AHEAD >= 0,
                "the reads and the loads fit between the MFMAs");
  auto slot = [&](int i) { return smem + i * C::STAGE; };
  if constexpr (C::ROUTED) {
    find(kernel_args<K>(), tile, ld);
    bring_pairs(ld, 0, lane);
    wait_vm<0>();  // the other waves read them behind the barrier
    __syncthreads();
  }
  begin();
  Loads l = next();
#pragma unroll
  for (int j = 0; j < LPS; ++j) load(l, slot(0), j);
  l = next();
#pragma unroll
  for (int j = 0; j < LPS; ++j) load(l, slot(1), j);
  sync(Count<LPS>());
#pragma unroll
  for (int f = 0; f < NI; ++f) read_b(smem, 0, f);
#pragma unroll
  for (int n = 0; n < AHEAD; ++n) read_a(smem, n);
  take();
  clear();
  const bool saves = C::GATED && kernel_args<K>()->a.z[0] != nullptr;
  int at = 0;
  bool fresh = false;  // a tile has just been stored: its stores are younger than all loads
  for (;;) {
    uint8_t *const buf = slot(at);
    const uint8_t *const other = slot(at ^ 1);
    at ^= 1;
    if (active)
      steps(0, MEET, [&](int i) {
        if (i % NI == 0 && i / NI + AHEAD < S) read_a(buf, i / NI + AHEAD);
        if (i % NI == 1 && i / NI < NI) read_b(buf, 1, i / NI);
      });
    __builtin_amdgcn_s_setprio(0);
    if (!fresh)
      wait_vm<0>();
    else if (C::GATED && saves)
      wait_vm<3 * STORES>();
    else if (!C::GATED && wide)
      wait_vm<2 * STORES>();
    else
      wait_vm<STORES>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    l = next();
    if (active) {
      steps(MEET, S, [&](int i) {
        // B's and A's first; those of A whose place in the ring is still in use come behind it
        if (i < NI) read_b(other, 0, i);
        if (i >= NI && i < NI + AHEAD) read_a(other, i - NI);
        if (i % (HOOKS / LPS) == 0 && i / (HOOKS / LPS) < LPS) load(l, buf, i / (HOOKS / LPS));
      });
    } else {
#pragma unroll
      for (int j = 0; j < LPS; ++j) load(l, buf, j);
#pragma unroll
      for (int f = 0; f < NI; ++f) read_b(other, 0, f);
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) read_a(other, n);
    }
    fresh = --left == 0;
    if (fresh) {
      store_tile();
      if (!more) break;
      take();
      cpar ^= 1;
      clear();
    }
  }
  wait_vm<0>();  // the loads past the end write to this block's LDS
}

}  // namespace ffn
}  // namespace llmint8
