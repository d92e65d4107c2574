// The forward products for few rows (single tokens, decoding batches): the
// weights are read once and bound everything, so the kernel is built around
// keeping HBM busy.
//
// A block owns 32, 64 or 128 output columns and 16, 32 or 64 rows of X (groups of
// rows are blocks of their own, next to each other on an XCD, whose L2 gives them the
// same W). Its waves take stages of the reduction in turn (32 steps; 64 with 32
// columns), each through a ring of its own in LDS that only this wave writes
// (direct-to-LDS loads) and reads, so the loop has no barrier: a wave waits for its
// own oldest stage and keeps the others in flight. W is read from LDS transposed, as
// in ffn_gemm.hpp, into v_mfma_f32_16x16x32 (16 columns by 16 rows a time). The
// waves' sums meet in LDS in a fixed order, where the epilogue runs on 8 columns of a
// row per thread; when the blocks are still few, the reduction is split over blocks
// as well and launch_ffn_finish joins the parts.
//
// What bounds it: HBM where the weights are large (gated 1 x 4096 x 11008 reads its
// 180 MB at 5.9 TB/s, 20 x 5120 x 13824 its 283 MB at 5.7); before that a CU's lines
// in flight, about 256 of 128 bytes (33 to 40 GB/s a CU), whatever the ring's depth
// and the number of waves, so the way to more bandwidth is more blocks:
//   64 x 2048 x 2048    64 columns by 64 rows 11.8 us, 32 by 16 7.4
//   301 x 1040 x 520    64 by 64 7.6, 64 by 16 5.8
//   1 x 1024 x 1024     64 columns 4.9, 32 columns 4.0
//   1 x 8192 x 28672    64 columns 105.4, 128 columns (two lines a row) 87.7
#include "ffn_gemm.hpp"

namespace llmint8 {
namespace ffn {

constexpr int kSkStep = 32;   // reduction steps per stage
constexpr int kSkWaves = 4;

template <class T_, bool GATED_, int MT_, int CB_>
struct SkinnyCfg {
  static constexpr int SUB = CB_ == 32 ? 2 : 1;  // 32-step parts of a stage
  using T = T_;
  static constexpr bool GATED = GATED_;
  static constexpr int MT = MT_;  // 16-row tiles
  static constexpr int CB = CB_;  // output columns per block
  static constexpr int P = GATED ? 2 : 1;
  static constexpr int WBYTES = SUB * kSkStep * CB * 2;  // one product's W in a stage
  static constexpr int STAGE = P * WBYTES + SUB * MT * 1024;
  static constexpr int LOADS = STAGE / 1024;
  static constexpr int REDP = CB + 4;  // fp32 pitch of the joined sums
  static constexpr int RED = kSkWaves * P * 16 * MT * REDP * 4;
  // three stages, two where three would not fit in LDS; deeper rings (up to 8
  // stages) measured the same within 3 %
  static constexpr int FIT = 160 * 1024 / (kSkWaves * STAGE), D = FIT < 3 ? FIT : 3;
  static constexpr int RING = kSkWaves * D * STAGE;
  static constexpr int LDS = RING > RED ? RING : RED;
};

// 16-byte chunk c of row r of an X stage (64-byte rows) sits at c ^ xkey(r)
__device__ inline int xkey(int r) { return (r >> 2) & 3; }

template <class C>
__device__ __forceinline__ void skinny_block(const FfnGemm &a, uint8_t *smem) {
  using T = typename C::T;
  constexpr int MT = C::MT, P = C::P, D = C::D;
  const int t = threadIdx.x, lane = t & 63, wv = wave_id();
  uint8_t *ring = smem + wv * D * C::STAGE;

  constexpr int SUB = C::SUB, STEP = SUB * kSkStep;
  // the row groups of a tile, then the tiles, then the parts in consecutive places of
  // an XCD (see tile_at), whose L2 serves what they share
  const uint32_t tiles = (uint32_t)((a.N + C::CB - 1) / C::CB);
  const uint32_t groups = (uint32_t)((a.M + 16 * MT - 1) / (16 * MT));
  const uint32_t place = xcd_place(blockIdx.x, gridDim.x);
  const int split = (int)(place / (groups * tiles));
  const int64_t n0 = (int64_t)(place / groups % tiles) * C::CB;
  const int64_t m0 = (int64_t)(place % groups) * (16 * MT);
  const int nst = (int)((a.K + STEP - 1) / STEP);
  const int s0 = part_begin(nst, split, a.ksplit) + wv;
  const int s1 = part_begin(nst, split + 1, a.ksplit);

  const int64_t rows = a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT;
  const uint8_t *px = (const uint8_t *)a.a[0] + m0 * a.lda * 2;
  const int64_t xbytes = ((rows - 1) * a.lda + a.K) * 2;
  const uint8_t *pw[2] = {(const uint8_t *)a.b[0] + n0 * 2, (const uint8_t *)a.b[1] + n0 * 2};

  // W stages in the order of a ColKTile
  using TW = ColKTile<C::CB, 1>;
  constexpr int WL = C::WBYTES / 1024, CH = TW::CH, RPI = TW::RPI;
  int wvoff[WL], xvoff[SUB * MT];
#pragma unroll
  for (int j = 0; j < WL; ++j) {
    const int r = RPI * j + lane / CH;
    wvoff[j] = r * (int)a.ldb * 2 + 16 * ((lane % CH) ^ TW::key(r));
  }
  const int xc = (lane % 4) ^ xkey(lane / 4);  // the same chunk in every 16-row tile
#pragma unroll
  for (int j = 0; j < SUB * MT; ++j)
    xvoff[j] = (16 * (j % MT) + lane / 4) * (int)a.lda * 2 + 16 * xc + 64 * (j / MT);

  auto load = [&](int s, uint8_t *buf) {
    const int64_t k = (int64_t)s * STEP;
    const int64_t left = a.K - k < STEP ? a.K - k : STEP;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const rsrc_t rw = make_rsrc(pw[p] + 2 * k * a.ldb, clip31(((left - 1) * a.ldb + a.N - n0) * 2));
#pragma unroll
      for (int j = 0; j < WL; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lptr_t)(buf + p * C::WBYTES + j * 1024), 16,
                                                 wvoff[j], 0, 0, 0);
    }
    const rsrc_t rx = make_rsrc(px + 2 * k, clip31(xbytes - 2 * k));
#pragma unroll
    for (int j = 0; j < SUB * MT; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lptr_t)(buf + P * C::WBYTES + j * 1024), 16,
                                               8 * xc + 32 * (j / MT) < left ? xvoff[j] : kOob, 0,
                                               0, 0);
  };

  constexpr int NB = C::CB / 16;
  f32x4 acc[P][NB][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[p][nb][mt] = (f32x4){};

  const int i = lane & 15, g = lane >> 4;
  // this wave's stages: s0, s0 + 4, ... below s1
  const int n = s1 > s0 ? (s1 - s0 + kSkWaves - 1) / kSkWaves : 0;
#pragma unroll
  for (int q = 0; q < D - 1; ++q)
    if (q < n) load(s0 + q * kSkWaves, ring + q * C::STAGE);
  for (int it = 0, slot = 0; it < n; ++it) {
    const int nx = it + D - 1;
    int free_slot = slot + D - 1;
    if (free_slot >= D) free_slot -= D;
    // the reads of the slot about to be refilled have been consumed
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (nx < n) {
      load(s0 + nx * kSkWaves, ring + free_slot * C::STAGE);
      wait_vm<(D - 1) * C::LOADS>();
    } else {
      // the tail: wait for everything; the remaining stages have been in flight
      // together and land together
      wait_vm<0>();
    }
    const uint8_t *buf = ring + slot * C::STAGE;
#pragma unroll
    for (int ks = 0; ks < SUB; ++ks) {
      s16x8 xv[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        xv[mt] = *(const s16x8 *)(buf + P * C::WBYTES + (ks * MT + mt) * 1024 + i * 64 +
                                  16 * (g ^ xkey(i)));
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const s16x8 wf = TW::frag(buf + p * C::WBYTES, nb * 16, ks, lane);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc[p][nb][mt] = T::mfma16(wf, xv[mt], acc[p][nb][mt]);
        }
    }
    if (++slot == D) slot = 0;
  }

  // Lane l of an accumulator holds row l % 16, columns 4 (l / 16) .. + 3.
  __syncthreads();
  float *red = (float *)smem;
  constexpr int PLANE = 16 * MT * C::REDP;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        *(f32x4 *)(red + (wv * P + p) * PLANE + (mt * 16 + i) * C::REDP + nb * 16 + 4 * g) =
            acc[p][nb][mt];
  __syncthreads();
  constexpr int CPR = C::CB / 8;  // 8-column chunks per row
  for (int x = t; x < (int)rows * CPR; x += 64 * kSkWaves) {
    const int m = x / CPR, c8 = (x % CPR) * 8;
    const int64_t row = m0 + m, col = n0 + c8;
    float v[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      load_f8(red + p * PLANE + m * C::REDP + c8, v[p]);
#pragma unroll
      for (int w = 1; w < kSkWaves; ++w) {
        float o[8];
        load_f8(red + (w * P + p) * PLANE + m * C::REDP + c8, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[p][e] += o[e];
      }
    }
    const bool in = col < a.N;
    if (a.ksplit > 1) {
      if (in)
#pragma unroll
        for (int p = 0; p < P; ++p)
          store_f8(a.part + (((int64_t)split * P + p) * a.M + row) * a.N + col, v[p]);
    } else if constexpr (C::GATED) {
      finish_gated<T>(a, row, col, in, v[0], v[P - 1]);
    } else if (in) {
      float b[8];
      load_bias<T>(a, col, b);
      finish_forward<T>(a, 0, row, col, v[0], b, load_residual(a, row, col));
    }
  }
}

template <class C>
__global__ __launch_bounds__(64 * kSkWaves, 1) void k_ffn_skinny(FfnGemm a) {
  extern __shared__ u32x4 smem_v[];
  skinny_block<C>(a, (uint8_t *)smem_v);
}

template <class C>
hipError_t launch_skinny_cfg(const FfnGemm &a, hipStream_t s) {
  auto *kern = k_ffn_skinny<C>;
  hipError_t e = hipFuncSetAttribute((const void *)kern,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  const int64_t tiles = (a.N + C::CB - 1) / C::CB, groups = (a.M + 16 * C::MT - 1) / (16 * C::MT);
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * groups * a.ksplit)), dim3(64 * kSkWaves), C::LDS, s, a);
  return hipGetLastError();
}

// All but two shapes: the joined sums of 128 gated columns and 64 rows would not fit
// in LDS, and 32 columns by 64 rows are hardly ever the fastest.
template <class T, bool GATED, int MT>
hipError_t launch_skinny_cols(const FfnGemm &a, int cols, hipStream_t s) {
  if constexpr (!(GATED && MT == 4))
    if (cols == 128) return launch_skinny_cfg<SkinnyCfg<T, GATED, MT, 128>>(a, s);
  if constexpr (MT != 4)
    if (cols == 32) return launch_skinny_cfg<SkinnyCfg<T, GATED, MT, 32>>(a, s);
  return launch_skinny_cfg<SkinnyCfg<T, GATED, MT, 64>>(a, s);
}

template <class T, bool GATED>
hipError_t launch_skinny(const FfnGemm &a, int rows, int cols, hipStream_t s) {
  if (rows == 16) return launch_skinny_cols<T, GATED, 1>(a, cols, s);
  if (rows == 32) return launch_skinny_cols<T, GATED, 2>(a, cols, s);
  return launch_skinny_cols<T, GATED, 4>(a, cols, s);
}

}  // namespace ffn

hipError_t launch_ffn_skinny(int dtype, bool gated, const FfnGemm &a, int rows, int cols,
                             hipStream_t s) {
  using namespace ffn;
  if (gated)
    return dtype == LLMINT8_FP16 ? launch_skinny<Half, true>(a, rows, cols, s)
                                 : launch_skinny<Bfloat, true>(a, rows, cols, s);
  return dtype == LLMINT8_FP16 ? launch_skinny<Half, false>(a, rows, cols, s)
                               : launch_skinny<Bfloat, false>(a, rows, cols, s);
}

}  // namespace llmint8
