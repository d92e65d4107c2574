// The router: which experts a token's row of logits chooses and with what weights, the
// gradient of the logits, and the order of the (token, expert) pairs by expert.
//
// A wave has one row, lane l its experts l, l + 64, ... in registers.
//
// Selection. An expert whose logit is -infinity or NaN is out; +infinity counts as the largest
// fp32 value. The value that experts are chosen by is the score (softmax or logistic) plus the
// bias, in 64 bits: two scores close to each other fall the same way in any careful
// implementation, where fp32 would leave their order to the rounding of an exponential. Without a
// bias, and without sums of two scores for a group, the logits have the scores' order and no
// exponential is needed. Values are turned into 64-bit integers of the same order; a step of
// the top-k is a wave-wide maximum of the upper words (DPP moves, no LDS), a ballot of
// who holds it, and the lower words or the indexes only where several lanes do.
//
// Weights and gradients in fp32; a renormalized weight is a softmax over the chosen logits (or
// over the logarithms of their logistic scores), which has no 0 / 0 however small the scores.
//
// What bounds it: for few rows the launch and the k dependent steps (about 0.2 us each); for
// many the instructions of the selection, not the 4 bytes a logit.
#include <type_traits>

#include "experts.hpp"
#include "llmint8.h"

namespace llmint8 {

namespace {

constexpr int kRows = 4;  // waves, and rows, of a block
constexpr float kTop = 3.4028234663852886e38f;
constexpr float kInf = __builtin_inff();

template <int CTRL, int ROWS>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest of the wave's values, known to be uniform.
__device__ inline uint32_t wave_umax(uint32_t v) {
  v = umax(v, dpp<0x111, 0xf>(v));  // row_shr:1, 2, 4, 8
  v = umax(v, dpp<0x112, 0xf>(v));
  v = umax(v, dpp<0x114, 0xf>(v));
  v = umax(v, dpp<0x118, 0xf>(v));
  v = umax(v, dpp<0x142, 0xa>(v));  // row_bcast:15, 31
  v = umax(v, dpp<0x143, 0xc>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

template <class F>
__device__ inline F wave_add(F v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// Order-preserving integers; 0 is below every number.
__device__ inline uint64_t ordered(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 to 0
  return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ inline uint32_t ordered(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);
  return b >> 31 ? ~b : b | 1u << 31;
}

__device__ inline float load_logit(const void *p, int64_t i, int dtype) {
  if (dtype == 2) return ((const float *)p)[i];
  const uint16_t h = ((const uint16_t *)p)[i];
  return dtype == LLMINT8_FP16 ? h2f(h) : __builtin_bit_cast(float, (uint32_t)h << 16);
}

__device__ inline float log_logistic(float x) {
  return __builtin_fminf(x, 0.f) - log1pf(expf(-__builtin_fabsf(x)));
}

// A row's logits: x[v] of expert lane + 64 v, -infinity where it is out or past the last.
template <int V>
__device__ inline void load_row(const Route &r, int64_t row, int lane, float *x) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    const float l = e < r.E ? load_logit(r.logits, row * r.ld + e, r.dtype) : -kInf;
    x[v] = l > -kInf ? __builtin_fminf(l, kTop) : -kInf;  // a NaN compares false
  }
}

// The chosen experts' weights before the scale: lane j has the logit c of slot j, or -infinity;
// x the row.
template <int V>
__device__ inline float mix(const Route &r, const float *x, float c) {
  const bool has = c > -kInf;
  if (r.sigmoid && !r.renorm) return has ? 1.f / (1.f + expf(-c)) : 0.f;
  if (r.renorm) {
    const float z = !has ? -kInf : r.sigmoid ? log_logistic(c) : c;
    const float top = wave_max(z);
    const float p = has ? expf(z - top) : 0.f;
    const float sum = wave_add(p);
    return has ? p / sum : 0.f;
  }
  float top = -kInf;
#pragma unroll
  for (int v = 0; v < V; ++v) top = __builtin_fmaxf(top, x[v]);
  top = wave_max(top);
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += x[v] > -kInf ? expf(x[v] - top) : 0.f;
  sum = wave_add(sum);
  return has ? expf(c - top) / sum : 0.f;
}

// LOGITS: the logits themselves have the order, and 32-bit keys.
template <int V, bool LOGITS>
__global__ __launch_bounds__(64 * kRows) void k_route(Route r, int32_t *ids, float *weights) {
  using Key = std::conditional_t<LOGITS, uint32_t, uint64_t>;
  using Value = std::conditional_t<LOGITS, float, double>;
  constexpr Value kNone = -__builtin_inf();
  extern __shared__ double values_v[];
  Value *const values = (Value *)values_v;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * kRows + wv;
  if (row >= r.M) return;  // no barrier below: a wave uses its own part of `values`
  float x[V];
  load_row<V>(r, row, lane, x);

  // the values that experts are chosen by
  Value val[V];
  if constexpr (LOGITS) {
#pragma unroll
    for (int v = 0; v < V; ++v) val[v] = x[v];
  } else {
    if (r.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) val[v] = 1.0 / (1.0 + exp(-(double)x[v]));
    } else {
      float top = -kInf;
#pragma unroll
      for (int v = 0; v < V; ++v) top = __builtin_fmaxf(top, x[v]);
      top = wave_max(top);
      double sum = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        val[v] = x[v] > -kInf ? exp((double)x[v] - (double)top) : 0.0;
        sum += val[v];
      }
      sum = wave_add(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) val[v] = sum > 0.0 ? val[v] / sum : 0.0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      if (r.bias && e < r.E) val[v] += (double)r.bias[e];
    }
  }
  Key key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = x[v] > -kInf && val[v] > kNone ? ordered(val[v]) : 0;

  if (r.groups > 1) {
    // `per` lanes (a power of two) have a group: its best values, then how many groups come
    // before it
    Value *const mine = values + (size_t)wv * r.E;
    const int each = r.E / r.groups;
    int per = 1;
    while (2 * per * r.groups <= kWave) per *= 2;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 64 * v < r.E) mine[lane + 64 * v] = key[v] ? val[v] : kNone;
    // the lanes read what others wrote: no instruction, since a wave's LDS accesses are in order,
    // but the compiler has to keep them so
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    Value best = kNone, second = kNone;
    const int group = lane / per;
    if (group < r.groups)
      for (int i = lane % per; i < each; i += per) {
        const Value d = mine[group * each + i];
        second = d > best ? best : d > second ? d : second;
        best = d > best ? d : best;
      }
    for (int off = 1; off < per; off <<= 1) {
      const Value b = __shfl_xor(best, off, kWave), s = __shfl_xor(second, off, kWave);
      const Value low = b < best ? b : best, high = s > second ? s : second;
      second = low > high ? low : high;
      best = b > best ? b : best;
    }
    if (r.group_best == 2 && second > kNone) best += second;
    int before = 0;
    for (int g = 0; g < r.groups; ++g) {
      const Value o = __shfl(best, g * per, kWave);
      before += o > best || (o == best && g < group);
    }
    const uint64_t keep = __ballot(group < r.groups && before < r.top_groups);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      if (e < r.E && !(keep >> (e / each * per) & 1)) key[v] = 0;
    }
  }

  int id = -1;        // of slot `lane`
  float c = -kInf;    // its logit
  for (int j = 0; j < r.k; ++j) {
    Key best = key[0];
    int bv = 0;
    float bx = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) best = key[v], bv = v, bx = x[v];  // the lower index of equals
    const uint32_t hi = (uint32_t)(LOGITS ? best : best >> (LOGITS ? 0 : 32)), lo = (uint32_t)best;
    const uint32_t top = wave_umax(hi);
    if (top == 0) break;  // every number's upper word is positive: none is left
    uint64_t who = __ballot(hi == top);
    if (who & (who - 1)) {
      if constexpr (!LOGITS) {
        const uint32_t low = wave_umax(hi == top ? lo : 0);
        who = __ballot(hi == top && lo == low);
      }
      if (who & (who - 1)) {
        const bool in = who >> lane & 1;
        const uint32_t first = wave_umax(in ? ~(uint32_t)(lane + 64 * bv) : 0);
        who = __ballot(in && ~(uint32_t)(lane + 64 * bv) == first);
      }
    }
    const int win = __builtin_ctzll(who);
    const int wb = __builtin_amdgcn_readlane(bv, win);
    const float wx = __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, bx), win));
    if (lane == j) id = win + 64 * wb, c = wx;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane == win && v == wb) key[v] = 0;
  }
  const float w = mix<V>(r, x, c) * r.scale;
  if (lane < r.k) {
    ids[row * r.k + lane] = id;
    weights[row * r.k + lane] = id < 0 ? 0.f : w;
  }
}

// With weights w (before the scale), d = scale dweights and s = logistic:
//   softmax                 dx_e = p_e (d_e - sum_j p_j d_j), d_e = 0 where e is not chosen
//   softmax, renormalized   dx_j = w_j (d_j - sum_i w_i d_i), of chosen experts alone
//   sigmoid                 dx_j = d_j s(x_j) s(-x_j)
//   sigmoid, renormalized   dx_j = w_j s(-x_j) (d_j - sum_i w_i d_i)
// An expert named twice gets both slots' gradients, in the slots' order.
template <int V>
__global__ __launch_bounds__(64 * kRows) void k_route_backward(Route r, const int32_t *ids,
                                                               const float *dweights, void *dl,
                                                               int64_t ldd) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * kRows + wv;
  if (row >= r.M) return;
  float x[V];
  load_row<V>(r, row, lane, x);
  int id = -1;
  float c = -kInf, d = 0.f;
  if (lane < r.k) {
    id = ids[row * r.k + lane];
    if (id < 0 || id >= r.E) {
      id = -1;
    } else {
      const float l = load_logit(r.logits, row * r.ld + id, r.dtype);
      if (l > -kInf) c = __builtin_fminf(l, kTop), d = dweights[row * r.k + lane] * r.scale;
    }
  }
  const float w = mix<V>(r, x, c);
  const float mean = r.sigmoid && !r.renorm ? 0.f : wave_add(w * d);
  float g;
  if (r.sigmoid)
    g = w * (d - mean) / (1.f + expf(c > -kInf ? c : 0.f));
  else
    g = r.renorm ? w * (d - mean) : w * d;
  if (!(c > -kInf)) g = 0.f;
  float out[V];
  if (r.sigmoid || r.renorm) {
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.f;
  } else {
    float top = -kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) top = __builtin_fmaxf(top, x[v]);
    top = wave_max(top);
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      out[v] = x[v] > -kInf ? expf(x[v] - top) : 0.f;
      sum += out[v];
    }
    sum = wave_add(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = sum > 0.f ? -mean * (out[v] / sum) : 0.f;
  }
  for (int j = 0; j < r.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float gj =
        __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, g), j));
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 64 * v == e) out[v] += gj;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    if (e >= r.E) continue;
    if (r.dtype == 2)
      ((float *)dl)[row * ldd + e] = out[v];
    else
      ((uint16_t *)dl)[row * ldd + e] = r.dtype == LLMINT8_FP16
                                            ? f2h(out[v])
                                            : __builtin_bit_cast(uint16_t, (__bf16)out[v]);
  }
}

// Block e of 0 .. E writes expert e's part of the order: it counts the pairs of the experts
// before e, which is where e's rows begin, and e's own in each wave's stretch of the pairs,
// then goes through them once more and puts each at its place. So one launch does it, pairs
// of an expert keep their order and no atomic decides anything; block E has the pairs without an
// expert. Every block reads all ids twice, from L2, at what one CU takes in.
constexpr int64_t kPlanOnce = 24576;  // pairs up to which this one launch is quicker
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;

__global__ __launch_bounds__(kPlanThreads) void k_expert_plan(const int32_t *ids, int64_t pairs,
                                                              int E, int32_t *offsets,
                                                              int32_t *order, int32_t *places) {
  __shared__ int before[kPlanWaves], own[kPlanWaves];
  const int e = blockIdx.x, lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // wave wv has the pairs p0 .. p1 - 1, in steps of 256: 4 of a lane
  const int64_t step = (pairs + 256 * kPlanWaves - 1) / (256 * kPlanWaves) * 256;
  const int64_t p0 = wv * step, p1 = p0 + step < pairs ? p0 + step : pairs;
  const bool whole = ((uintptr_t)ids & 15u) == 0;  // four ids a load
  auto load = [&](int64_t p, int *id) {
    if (whole && p + 4 <= p1) {
      const i32x4 v = *(const i32x4 *)(ids + p);
#pragma unroll
      for (int q = 0; q < 4; ++q) id[q] = (uint32_t)v[q] < (uint32_t)E ? v[q] : E;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int v = p + q < p1 ? ids[p + q] : -2;
        id[q] = p + q >= p1 ? E + 1 : (uint32_t)v < (uint32_t)E ? v : E;
      }
    }
  };
  int less = 0, same = 0;
  for (int64_t p = p0 + 4 * lane; p < p1; p += 256) {
    int id[4];
    load(p, id);
#pragma unroll
    for (int q = 0; q < 4; ++q) less += id[q] < e, same += id[q] == e;
  }
  less = wave_sum(less), same = wave_sum(same);
  if (lane == 0) before[wv] = less, own[wv] = same;
  __syncthreads();
  int begin = 0, at = 0, count = 0;
#pragma unroll
  for (int i = 0; i < kPlanWaves; ++i) {
    begin += before[i], count += own[i];
    at += i < wv ? own[i] : 0;
  }
  if (threadIdx.x == 0) offsets[e] = begin;
  if (count == 0) return;
  at += begin;
  const uint64_t lower = ((uint64_t)1 << lane) - 1;
  for (int64_t q0 = p0; q0 < p1; q0 += 256) {
    int id[4] = {E + 1, E + 1, E + 1, E + 1};
    const int64_t p = q0 + 4 * lane;
    if (p < p1) load(p, id);
    int ahead = 0, all = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t m = __ballot(id[q] == e);
      ahead += __popcll(m & lower), all += __popcll(m);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (id[q] == e) {
        const int r = at + ahead++;
        places[p + q] = e < E ? r : -1;
        order[r] = e < E ? (int32_t)(p + q) : -1;
      }
    at += all;
  }
}

// More pairs: in chunks, so that a CU reads its own part of the ids alone. First each chunk's
// pairs of every expert are counted; then a chunk's block adds up what the chunks before it have,
// which is where its pairs of each expert go, and puts them there in their order: lanes with
// the same expert find each other by a ballot for each bit of its number. A CU keeps about 256
// lines in flight, 37 KB a microsecond, which is what bounds the one launch above: 131072 pairs
// of 256 experts 26.5 us, in chunks 11.7; 65536 pairs 14.9 and 9.6; 16384 pairs 6.1 and 7.5.
constexpr int kChunkThreads = 1024, kChunkWaves = kChunkThreads / 64;

// The expert of pair p of a chunk that ends at p1; E: none; -1: no pair.
__device__ inline int pair_expert(const int32_t *ids, int64_t p, int64_t p1, int E) {
  if (p >= p1) return -1;
  const int id = ids[p];
  return (uint32_t)id < (uint32_t)E ? id : E;
}

__global__ __launch_bounds__(kChunkThreads) void k_plan_count(const int32_t *ids, int64_t pairs,
                                                             int E, int64_t chunk,
                                                             int32_t *counts) {
  extern __shared__ int32_t hist[];  // [E + 1]
  for (int e = threadIdx.x; e <= E; e += kChunkThreads) hist[e] = 0;
  __syncthreads();
  const int64_t p0 = blockIdx.x * chunk, p1 = p0 + chunk < pairs ? p0 + chunk : pairs;
  for (int64_t p = p0 + threadIdx.x; p < p1; p += kChunkThreads)
    atomicAdd(hist + pair_expert(ids, p, p1, E), 1);  // sums of ones: in any order the same
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kChunkThreads)
    counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

__global__ __launch_bounds__(kChunkThreads) void k_plan_place(const int32_t *ids, int64_t pairs,
                                                             int E, int64_t chunk,
                                                             const int32_t *counts,
                                                             int32_t *offsets, int32_t *order,
                                                             int32_t *places) {
  extern __shared__ int32_t smem[];
  const int n = E + 1;
  int32_t *const base = smem, *const mine = smem + n;  // [n], [waves][n]
  __shared__ int sums[kChunkWaves];
  const int t = threadIdx.x, lane = t & 63;
  const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
  const int chunks = gridDim.x, me = blockIdx.x;
  // the chunks before this one and all of them, several threads an expert
  for (int e = t; e < n; e += kChunkThreads) base[e] = 0, mine[e] = 0;
  __syncthreads();
  const int parts = n < kChunkThreads ? kChunkThreads / n : 1;
  for (int i = t; i < n * parts; i += kChunkThreads) {
    const int e = i % n;
    int prior = 0, all = 0;
#pragma unroll 16
    for (int c = i / n; c < chunks; c += parts) {
      const int v = counts[(int64_t)c * n + e];
      prior += c < me ? v : 0, all += v;
    }
    atomicAdd(base + e, prior), atomicAdd(mine + e, all);
  }
  __syncthreads();
  constexpr int PER = (int)(kMaxExperts + 1 + kChunkThreads - 1) / kChunkThreads;
  const int per = (n + kChunkThreads - 1) / kChunkThreads;
  int all[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * per + i;
    all[i] = i < per && e < n ? mine[e] : 0;
    sum += all[i];
  }
  int upto = sum;  // of the threads up to this one
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(upto, off, kWave);
    upto += lane >= off ? o : 0;
  }
  if (lane == 63) sums[wv] = upto;
  __syncthreads();
  int first = upto - sum;
  for (int i = 0; i < wv; ++i) first += sums[i];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * per + i;
    if (i >= per || e >= n) break;
    base[e] += first;
    if (me == 0) offsets[e] = first;
    first += all[i];
  }
  __syncthreads();

  const int64_t p0 = me * chunk, p1 = p0 + chunk < pairs ? p0 + chunk : pairs;
  const int bits = 32 - __builtin_clz(n);
  int32_t *const own = mine + wv * n;
  for (int64_t s0 = p0; s0 < p1; s0 += kChunkThreads) {
    for (int i = t; i < kChunkWaves * n; i += kChunkThreads) mine[i] = 0;
    __syncthreads();
    const int64_t p = s0 + t;
    const int id = pair_expert(ids, p, p1, E);
    uint64_t same = __ballot(id >= 0);  // the lanes with the same expert
    for (int b = 0; b < bits; ++b) {
      const bool bit = id >> b & 1;
      const uint64_t m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
    if (id >= 0 && same >> lane == 1) own[id] = rank + 1;  // the last of them
    __syncthreads();
    if (id >= 0) {
      int r = base[id] + rank;
      for (int w = 0; w < wv; ++w) r += mine[w * n + id];
      places[p] = id < E ? r : -1;
      order[r] = id < E ? (int32_t)p : -1;
    }
    if (s0 + kChunkThreads >= p1) return;
    __syncthreads();
    for (int e = t; e < n; e += kChunkThreads)
      for (int w = 0; w < kChunkWaves; ++w) base[e] += mine[w * n + e];
    __syncthreads();
  }
}

// At most 256 chunks, of whole blocks' threads.
int64_t plan_chunk(int64_t pairs) {
  const int64_t subs = (pairs + kChunkThreads - 1) / kChunkThreads;
  return (subs + 255) / 256 * kChunkThreads;
}

template <int V>
struct Width {
  static constexpr int value = V;  // logits a lane
};
template <class F>
hipError_t with_width(int E, F f) {
  if (E <= 64) return f(Width<1>());
  if (E <= 128) return f(Width<2>());
  if (E <= 256) return f(Width<4>());
  if (E <= 512) return f(Width<8>());
  return f(Width<16>());
}

}  // namespace

hipError_t launch_route(const Route &r, int32_t *ids, float *weights, hipStream_t s) {
  const bool logits = !r.bias && r.group_best == 1;
  const size_t value = logits ? sizeof(float) : sizeof(double);
  const size_t lds = r.groups > 1 ? (size_t)kRows * r.E * value : 0;
  return with_width(r.E, [&](auto w) {
    auto *kern = logits ? k_route<decltype(w)::value, true> : k_route<decltype(w)::value, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)((r.M + kRows - 1) / kRows)), dim3(64 * kRows), lds, s,
                       r, ids, weights);
    return hipGetLastError();
  });
}

hipError_t launch_route_backward(const Route &r, const int32_t *ids, const float *dweights,
                                 void *dlogits, int64_t ldd, hipStream_t s) {
  return with_width(r.E, [&](auto w) {
    hipLaunchKernelGGL((k_route_backward<decltype(w)::value>),
                       dim3((unsigned)((r.M + kRows - 1) / kRows)), dim3(64 * kRows), 0, s, r, ids,
                       dweights, dlogits, ldd);
    return hipGetLastError();
  });
}

size_t expert_plan_scratch(int64_t pairs, int E) {
  if (pairs <= kPlanOnce) return 0;
  const int64_t chunk = plan_chunk(pairs);
  return (size_t)((pairs + chunk - 1) / chunk * (E + 1)) * sizeof(int32_t);
}

hipError_t launch_expert_plan(const int32_t *ids, int64_t pairs, int E, int32_t *offsets,
                              int32_t *order, int32_t *places, int32_t *scratch, hipStream_t s) {
  if (pairs <= kPlanOnce) {
    hipLaunchKernelGGL(k_expert_plan, dim3((unsigned)(E + 1)), dim3(kPlanThreads), 0, s, ids,
                       pairs, E, offsets, order, places);
    return hipGetLastError();
  }
  const int64_t chunk = plan_chunk(pairs);
  const dim3 grid((unsigned)((pairs + chunk - 1) / chunk));
  const unsigned row = (unsigned)(E + 1) * sizeof(int32_t);
  hipLaunchKernelGGL(k_plan_count, grid, dim3(kChunkThreads), row, s, ids, pairs, E, chunk,
                     scratch);
  const unsigned lds = (1 + kChunkWaves) * row;
  const hipError_t e = hipFuncSetAttribute((const void *)k_plan_place,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_plan_place, grid, dim3(kChunkThreads), lds, s, ids, pairs, E, chunk, scratch,
                     offsets, order, places);
  return hipGetLastError();
}

}  // namespace llmint8
