// Tiles of the block-scaled FP8 product, for all but few rows.
//
// The operands are both contiguous along the reduction. Two codes of a row take the place of
// a 16-bit value in the tiles of ffn_gemm.hpp: a stage is one block of 128 codes (128
// bytes a row), brought to LDS by the same loads into the same permuted chunks. A lane's 32
// codes of a row are chunks g and g + 4 of its 8 (g = lane / 16): which places of the block
// they are does not matter as long as both operands take the same ones, since a block has one
// scale. X's scale bytes of the stage come along with it, four blocks' at a time (4 bytes
// a row, by a load of their own); W's, one byte a block for 128 columns, wait in LDS from
// the start.
//
// The MFMA has 32 codes a lane and operand, 8 registers, twice those of a 16-bit one, for
// twice the reduction. So A's fragments go through a ring of four registers sets, read
// two steps ahead, and B's (all columns of the wave) are replaced one by one by the next
// stage's behind their last use.
//
// What bounds it: power. 8192 x 8192 x 28672 runs at 2.3 PFLOP/s, 1.69 ms, at a clock of 1.87 GHz
// with the MFMAs busy for 0.55 of the time; a pass that codes X before it takes 44 us of that.
// 1777 x 5120 x 13824 takes 119 us at 2.12 GHz and 8 us of coding: 378 tiles on 256 CUs, the last
// 122 of them in halves (the call 144 us, with whole tiles 155).
#include "blockwise_math.hpp"

namespace llmint8 {
namespace fp8 {

template <class T_, int BM_, int BN_, int NWM_, int NWN_, int NST_>
struct Fp8Cfg {
  using T = T_;
  static constexpr int BM = BM_, BN = BN_, NWM = NWM_, NWN = NWN_, NW = NWM * NWN, NST = NST_;
  static constexpr int THREADS = 64 * NW;
  static constexpr int WM = BM / NWM, WN = BN / NWN, MI = WM / 16, NI = WN / 16;
  using TA = RowKTile<BM, NW>;
  using TB = RowKTile<BN, NW>;
  static constexpr int SX = TA::BYTES + TB::BYTES;  // place of X's scales in a stage
  static constexpr int STAGE = SX + BM * 4;
  static constexpr int LPS = TA::G + TB::G + 1;     // loads per wave per stage
  static constexpr int CB = BN / kFp8Block;         // blocks of columns
  static constexpr int SLABP = WN + 4;
  static constexpr int SLABS = NW * 32 * SLABP * 4;
  static constexpr int RING = NST * STAGE > SLABS ? NST * STAGE : SLABS;
  static constexpr int64_t lds(int64_t K) {
    return RING + CB * ((K + kFp8Block - 1) / kFp8Block + 15) / 16 * 16;
  }
  static_assert(MI % 4 == 0 && WN <= kFp8Block, "a ring of four fragments; one scale a wave");
};

// Block bid of the tiles in tile columns col0 .. col0 + cols - 1.
template <class C>
__device__ __forceinline__ void fp8_tile(const Fp8Gemm &a, uint32_t bid, int col0, int cols,
                                         uint8_t *const smem) {
  using T = typename C::T;
  constexpr int MI = C::MI, NI = C::NI, LPS = C::LPS, NST = C::NST;
  const int t = threadIdx.x, lane = t & 63, wv = wave_id();
  const int wm = wv / C::NWN, wn = wv % C::NWN;
  const FfnGemm &o = a.out;

  int tm, tn, split;
  tile_at(bid, (uint32_t)((o.M + C::BM - 1) / C::BM), (uint32_t)cols, o.ksplit, tm, tn, split);
  tn += col0;
  const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN;
  const int64_t half = a.K / 2;  // pairs of codes in a row
  const int nst = (int)((a.K + kFp8Block - 1) / kFp8Block);
  const int s0 = part_begin(nst, split, o.ksplit), s1 = part_begin(nst, split + 1, o.ksplit);

  typename C::TA A;
  typename C::TB B;
  A.init(half, o.M - m0, half);
  B.init(half, o.N - n0, half);
  const uint8_t *const pa = a.x.codes + m0 * a.K, *const pb = a.w.codes + n0 * a.K;
  // X's scales: wave wv brings the four bytes of row srow + lane
  const int srow = (wv % (C::BM / 64)) * 64;
  const uint8_t *const psx = a.x.scales + m0 * a.x.lds;
  const int svoff = (srow + lane) * (int)a.x.lds;
  const int sbytes = (int)((o.M - m0 < C::BM ? o.M - m0 : C::BM) * a.x.lds);

  // W's scales of the tile's columns; a block of columns past N has none
  uint8_t *const swl = smem + C::RING;
  for (int i = t; i < C::CB * nst; i += C::THREADS) {
    const int cb = i / nst, b = i % nst;
    const int64_t nb = n0 / kFp8Block + cb;
    swl[i] = nb * kFp8Block < o.N ? a.w.scales[nb * a.w.lds + b] : 0;
  }
  const uint8_t *const sww = swl + wn * C::WN / kFp8Block * nst;
  __syncthreads();

  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = (f32x4){};

  struct Loads {
    typename C::TA::Stage a;
    typename C::TB::Stage b;
    rsrc_t s;
  };
  // past the last stage every address is out of range (see ffn_gemm.hpp)
  auto loads_of = [&](int s) {
    const int k = s * (kFp8Block / 2), len = s < s1 ? (int)half : k;
    const int so = s / 4 * 4, left = s < s1 ? sbytes - so : 0;
    return Loads{A.stage(pa, half, k, len), B.stage(pb, half, k, len), make_rsrc(psx + so, left)};
  };
  auto load = [&](const Loads &l, uint8_t *buf, int j) {
    if (j < C::TA::G)
      A.load(l.a, buf, j);
    else if (j < C::TA::G + C::TB::G)
      B.load(l.b, buf + C::TA::BYTES, j - C::TA::G);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(l.s, (lptr_t)(buf + C::SX + srow * 4), 4, svoff, 0,
                                               0, 0);
  };
  i32x8 av[4], bv[NI];
  int sx[MI], sw[2];
  auto frag = [&](const uint8_t *tile, int row0) {
    using TA = typename C::TA;
    return pair(__builtin_bit_cast(i32x4, TA::frag(tile, row0, 0, lane)),
                __builtin_bit_cast(i32x4, TA::frag(tile, row0, 1, lane)));
  };
  auto read_a = [&](const uint8_t *buf, int mi) {
    av[mi % 4] = frag(buf, wm * C::WM + mi * 16);
  };
  auto read_b = [&](const uint8_t *buf, int ni) {
    bv[ni] = frag(buf + C::TA::BYTES, wn * C::WN + ni * 16);
  };
  auto read_sx = [&](const uint8_t *buf, int s, int mi) {
    sx[mi] = buf[C::SX + (wm * C::WM + mi * 16 + (lane & 15)) * 4 + (s & 3)];
  };
  auto ring_sync = [&](auto younger) {
    __builtin_amdgcn_s_setprio(0);
    wait_vm<decltype(younger)::value>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };

  // A stage's MFMAs go row block by row block. Behind the last but two, all of the stage's A
  // is in registers: the waves meet, which frees its slot for stage s + NST and shows stage
  // s + 1, whose first fragments are read under the last two row blocks' MFMAs. Half of the
  // loads go out there, the other half at the beginning of the next stage.
  if (s0 < s1) {
    constexpr int H = (LPS + 1) / 2;
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
    for (int ni = 0; ni < NI; ++ni) read_b(smem, ni);
    read_a(smem, 0), read_a(smem, 1);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) read_sx(smem, s0, mi);
    sw[0] = sww[s0];
    int at = 0;
    for (int s = s0; s < s1; ++s) {
      uint8_t *const cur = slot(at), *const last = slot(at == 0 ? NST - 1 : at - 1);
      at = at + 1 == NST ? 0 : at + 1;
      const uint8_t *const next = slot(at);
      sw[1] = sww[s + 1 < s1 ? s + 1 : s];
      __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        if (mi == MI - 2) {
          ring_sync(Count<(NST - 2) * LPS>());
          l = loads_of(s + NST);
          __builtin_amdgcn_s_setprio(1);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const int i = mi * NI + ni;
          acc[mi][ni] = mfma_block(bv[ni], av[mi % 4], acc[mi][ni], sw[0], sx[mi]);
          if (ni == 0) {
            if (mi + 2 < MI)
              read_a(cur, mi + 2);
            else
              read_a(next, mi + 2 - MI);
          }
          if (mi == MI - 1) read_b(next, ni);
          // the scales of the next stage, behind their last use
          if (ni == 1 && mi >= MI - 2)
#pragma unroll
            for (int q = 0; q < (MI - 2) / 2; ++q)
              read_sx(next, s + 1, (mi - MI + 2) * (MI - 2) / 2 + q);
          if (mi == MI - 1 && ni == NI - 1)
            read_sx(next, s + 1, MI - 2), read_sx(next, s + 1, MI - 1);
          if (i % 2 == 1 && i / 2 < LPS - H) load(l, last, H + i / 2);
          const int r = i - (MI - 2) * NI;  // MFMAs since the waves met
          if (r >= 0) {
            // H loads over 2 NI MFMAs
#pragma unroll
            for (int j = 0; j < H; ++j)
              if (j * 2 * NI / H == r) load(l, cur, j);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      sw[0] = sw[1];
    }
  }
  wait_vm<0>();
  __syncthreads();

  // Lane l of acc[mi][ni] has row l % 16, columns 4 (l / 16) .. + 3 of its 16 x 16 block: through
  // LDS in fp32, as in ffn_gemm.hpp.
  float *slab = (float *)smem + wv * 32 * C::SLABP;
  constexpr int CPR = C::WN / 8, PASSES = 32 * CPR / 64;
  const int64_t n = n0 + wn * C::WN + (lane % CPR) * 8;
  float bias[8];
  if (n < o.N) load_bias<T>(o, n, bias);
#pragma unroll
  for (int mi = 0; mi < MI / 2; ++mi) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        *(f32x4 *)(slab + (h * 16 + (lane & 15)) * C::SLABP + ni * 16 + 4 * (lane >> 4)) =
            acc[2 * mi + h][ni];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * (64 / CPR) + lane / CPR;
      const int64_t i = m0 + wm * C::WM + mi * 32 + r;
      if (i >= o.M || n >= o.N) continue;
      float v[8];
      load_f8(slab + r * C::SLABP + (lane % CPR) * 8, v);
      if (o.ksplit > 1) {
        store_f8(o.part + ((int64_t)split * o.M + i) * o.N + n, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += bias[e];
        store8<T>(o.y[0] + i * o.ldy + n, v);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// The last blocks take the C1 tiles of the tile columns before `cut`, the first ones the C2
// tiles of the rest: half tiles where the last round would be nearly empty (see tail_cut).
template <class C1, class C2>
__global__ __launch_bounds__(C1::THREADS, 2) void k_fp8_tiles(Fp8Gemm a, int cut, int cols,
                                                             uint32_t blocks1) {
  static_assert(C1::THREADS == C2::THREADS && C1::BN == C2::BN, "one launch");
  extern __shared__ u32x4 smem_v[];
  const uint32_t blocks2 = gridDim.x - blocks1;
  if (blockIdx.x >= blocks2)
    fp8_tile<C1>(a, blockIdx.x - blocks2, 0, cut, (uint8_t *)smem_v);
  else
    fp8_tile<C2>(a, blockIdx.x, cut, cols - cut, (uint8_t *)smem_v);
}

template <class C1, class C2>
hipError_t launch_cfg(const Fp8Gemm &a, hipStream_t s) {
  auto *kern = k_fp8_tiles<C1, C2>;
  const int64_t lds = C1::lds(a.K) > C2::lds(a.K) ? C1::lds(a.K) : C2::lds(a.K);
  hipError_t e = hipFuncSetAttribute((const void *)kern,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const int64_t rows = (a.out.M + C1::BM - 1) / C1::BM, cols = (a.out.N + C1::BN - 1) / C1::BN;
  const int64_t cut = C1::BM == C2::BM ? cols : tail_cut(rows, cols, a.out.ksplit);
  const int64_t blocks1 = rows * cut * a.out.ksplit;
  const int64_t blocks2 = (a.out.M + C2::BM - 1) / C2::BM * (cols - cut) * a.out.ksplit;
  hipLaunchKernelGGL(kern, dim3((unsigned)(blocks1 + blocks2)), dim3(C1::THREADS), (unsigned)lds, s,
                     a, (int)cut, (int)cols, (uint32_t)blocks1);
  return hipGetLastError();
}

template <class T>
hipError_t launch_type(const Fp8Gemm &a, int tile, hipStream_t s) {
  using Wide = Fp8Cfg<T, 256, 256, 2, 4, 2>;
  using Tail = Fp8Cfg<T, 128, 256, 2, 4, 2>;
  using Small = Fp8Cfg<T, 128, 128, 2, 2, 2>;
  using Deep = Fp8Cfg<T, 128, 128, 2, 2, 4>;
  if (tile == 256) return launch_cfg<Wide, Tail>(a, s);
  const int64_t blocks = (a.out.M + 127) / 128 * ((a.out.N + 127) / 128) * a.out.ksplit;
  return deep_ring(blocks) ? launch_cfg<Deep, Deep>(a, s) : launch_cfg<Small, Small>(a, s);
}

}  // namespace fp8

hipError_t launch_fp8_tiles(int dtype, const Fp8Gemm &a, int tile, hipStream_t s) {
  return dtype == 0 ? fp8::launch_type<Half>(a, tile, s) : fp8::launch_type<Bfloat>(a, tile, s);
}

}  // namespace llmint8
