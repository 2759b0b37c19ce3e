// Routing by scores: softmax or sigmoid scores, a bias for balance, groups of
// experts, top-k and renormalised weights (build log "Two 96 GB Ascend cards
// run Qwen3.8 Flash-Next", section "Keep low-bit weights packed, do the work
// on the NPU": tokens are scored and routed on the device).
//
// Scores and choice values are 64-bit numbers.  Which experts are chosen hangs
// on their order, which 32 bits lose: sigmoids of logits above 17 are all 1
// there, and a bias added to scores of 1e-3 drops a third of their bits.
//
// A wave routes one token.  Its lanes are dealt to the groups, LG lanes each
// (the largest power of two with LG * n_group <= 64), so that a group's best
// two values are a butterfly over its own lanes, and no step needs LDS: lane l
// holds the experts i = l % LG, + LG, ... of group l / LG.
#include <algorithm>

#include "route_common.h"

namespace moe {

namespace {

constexpr int kScoredWaves = 4;   // tokens per workgroup

template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp_d(double old, double v) {
  const long long o = __double_as_longlong(old), x = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)dpp_i<CTRL, ROW_MASK>((int)o, (int)x);
  const uint32_t hi = (uint32_t)dpp_i<CTRL, ROW_MASK>((int)(o >> 32), (int)(x >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double lane_d(double v, int lane) {
  const long long x = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// Sum over the wave in a fixed order, the same in every lane.
__device__ __forceinline__ double wave_sum_d(double v) {
  v += dpp_d<kDppXor1>(v, v);
  v += dpp_d<kDppXor2>(v, v);
  v += dpp_d<kDppRowHalfMirror>(v, v);
  v += dpp_d<kDppRowMirror>(v, v);
  v += dpp_d<kDppRowBcast15, 0xA>(0.0, v);
  v += dpp_d<kDppRowBcast31, 0xC>(0.0, v);
  return lane_d(v, 63);
}

__device__ __forceinline__ float wave_max_f(float v) {
  v = fmaxf(v, dpp_f<kDppXor1>(v, v));
  v = fmaxf(v, dpp_f<kDppXor2>(v, v));
  v = fmaxf(v, dpp_f<kDppRowHalfMirror>(v, v));
  v = fmaxf(v, dpp_f<kDppRowMirror>(v, v));
  v = fmaxf(v, dpp_f<kDppRowBcast15, 0xA>(v, v));
  v = fmaxf(v, dpp_f<kDppRowBcast31, 0xC>(v, v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
#define MOE_STEP(CTRL, MASK)                                     \
  {                                                              \
    const uint32_t o = (uint32_t)dpp_i<CTRL, MASK>((int)v, (int)v); \
    v = o > v ? o : v;                                           \
  }
  MOE_STEP(kDppXor1, 0xF)
  MOE_STEP(kDppXor2, 0xF)
  MOE_STEP(kDppRowHalfMirror, 0xF)
  MOE_STEP(kDppRowMirror, 0xF)
  MOE_STEP(kDppRowBcast15, 0xA)
  MOE_STEP(kDppRowBcast31, 0xC)
#undef MOE_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The order of choice values as that of unsigned numbers above 0, which stands
// for "not to be chosen"; NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint64_t choice_key(double c) {
  const uint64_t u = (uint64_t)__double_as_longlong(c + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Joins a lane's two largest values with those of another.
__device__ __forceinline__ void join2(double& a, double& b, double oa, double ob) {
  const double hi = fmax(a, oa), lo = fmin(a, oa);
  b = fmax(lo, a >= oa ? b : ob);
  a = hi;
}

// NV: experts per lane, lg: LG's logarithm.
template <int NV>
__global__ __launch_bounds__(64 * kScoredWaves) void route_scored_kernel(ScoredArgs a, int lg) {
  const int lane = threadIdx.x & 63;
  const int t = (blockIdx.y * gridDim.x + blockIdx.x) * kScoredWaves + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int size = a.E / a.n_group, LG = 1 << lg;
  const int g = lane >> lg, i0 = lane & (LG - 1);
  const float* row = a.logits + (size_t)t * a.E + g * size;
  const bool mine = g < a.n_group;

  float l[NV], bias[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = i0 + (j << lg);
    const bool in = mine && i < size;
    l[j] = in ? row[i] : -INFINITY;
    bias[j] = in && a.bias ? a.bias[g * size + i] : 0.0f;
  }
  // ---- scores
  double s[NV];
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, l[j]);
    m = wave_max_f(m);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // a row without a logit above -inf has scores of 0
      s[j] = l[j] == -INFINITY ? 0.0 : exp((double)l[j] - (double)m);
      sum += s[j];
    }
    sum = wave_sum_d(sum);
    if (sum == 0.0) sum = 1.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) s[j] /= sum;
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) s[j] = 1.0 / (1.0 + exp(-(double)l[j]));
  }
  double c[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    c[j] = s[j] + (double)bias[j];
    if (c[j] != c[j] || !(mine && i0 + (j << lg) < size)) c[j] = -INFINITY;
  }
  // ---- groups
  bool stays = mine;
  if (a.topk_group < a.n_group) {
    double v = -INFINITY, v2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) join2(v, v2, c[j], -INFINITY);
    if (lg > 0) join2(v, v2, dpp_d<kDppXor1>(v, v), dpp_d<kDppXor1>(v2, v2));
    if (lg > 1) join2(v, v2, dpp_d<kDppXor2>(v, v), dpp_d<kDppXor2>(v2, v2));
    if (lg > 2) join2(v, v2, dpp_d<kDppRowHalfMirror>(v, v), dpp_d<kDppRowHalfMirror>(v2, v2));
    if (lg > 3) join2(v, v2, dpp_d<kDppRowMirror>(v, v), dpp_d<kDppRowMirror>(v2, v2));
    if (lg > 4) join2(v, v2, __shfl_xor(v, 16), __shfl_xor(v2, 16));
    if (a.group_best == 2 && size > 1) v += v2;
    // a group stays if fewer than topk_group come before it
    int before = 0;
    for (int o = 0; o < a.n_group; ++o) {
      const double ov = lane_d(v, o << lg);
      before += ov > v || (ov == v && o < g);
    }
    stays = mine && before < a.topk_group;
  }
  // ---- the k best, one a round
  uint64_t key[NV];
  int sel_id = 0;
  double sel_s = 0.0, total = 0.0;
  // k above a wave's lanes: once for the sum of the chosen scores, once to write
  const int passes = a.renorm && a.k > 64 ? 2 : 1;
  for (int pass = 0; pass < passes; ++pass) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      key[j] = stays && i0 + (j << lg) < size ? choice_key(c[j]) : 0ull;
    double sum = 0.0;
    for (int r = 0; r < a.k; ++r) {
      uint64_t best = key[0];
      int bj = 0;
      double bs = s[0];
#pragma unroll
      for (int j = 1; j < NV; ++j)
        if (key[j] > best) {
          best = key[j];
          bj = j;
          bs = s[j];
        }
      const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
      const int e = g * size + i0 + (bj << lg);
      const uint32_t top = wave_max_u(hi);
      uint64_t at = __ballot(hi == top);
      int w = __builtin_ctzll(at);
      if (at & (at - 1)) {
        // several lanes: the low words, then the lowest index
        uint32_t wl = (uint32_t)__builtin_amdgcn_readlane((int)lo, w);
        int we = __builtin_amdgcn_readlane(e, w);
        for (at &= at - 1; at; at &= at - 1) {
          const int o = __builtin_ctzll(at);
          const uint32_t ol = (uint32_t)__builtin_amdgcn_readlane((int)lo, o);
          const int oe = __builtin_amdgcn_readlane(e, o);
          if (ol > wl || (ol == wl && oe < we)) {
            wl = ol;
            we = oe;
            w = o;
          }
        }
      }
      const int we = __builtin_amdgcn_readlane(e, w);
      const double ws = lane_d(bs, w);
      sum += ws;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (lane == w && j == bj) key[j] = 0ull;
      if (lane == (r & 63)) {
        sel_id = we;
        sel_s = ws;
      }
      // a full set of 64, or the last ones
      if (a.k > 64 && pass == passes - 1 && ((r & 63) == 63 || r == a.k - 1)) {
        const int at_r = (r & ~63) + lane;
        if (at_r <= r) {
          const double wn = a.renorm ? (total > 0.0 || total != total ? sel_s / total : 0.0) : sel_s;
          a.ids[(size_t)t * a.k + at_r] = sel_id;
          a.w[(size_t)t * a.k + at_r] = (float)(wn * (double)a.scale);
        }
      }
    }
    total = sum;
  }
  if (a.k <= 64 && lane < a.k) {
    const double wn = a.renorm ? (total > 0.0 || total != total ? sel_s / total : 0.0) : sel_s;
    a.ids[(size_t)t * a.k + lane] = sel_id;
    a.w[(size_t)t * a.k + lane] = (float)(wn * (double)a.scale);
  }
}

}  // namespace

hipError_t launch_route_scored(const ScoredArgs& a, hipStream_t st) {
  int lg = 6;
  while (lg > 0 && (a.n_group << lg) > 64) --lg;
  const int size = a.E / a.n_group, nv = (size + (1 << lg) - 1) >> lg;
  const int wgs = (a.T + kScoredWaves - 1) / kScoredWaves, block = 64 * kScoredWaves;
  // a launch has fewer than 2^32 lanes along x
  const dim3 grid(std::min(wgs, 1 << 20), (wgs + (1 << 20) - 1) >> 20);
  if (nv <= 1) route_scored_kernel<1><<<grid, block, 0, st>>>(a, lg);
  else if (nv <= 2) route_scored_kernel<2><<<grid, block, 0, st>>>(a, lg);
  else if (nv <= 4) route_scored_kernel<4><<<grid, block, 0, st>>>(a, lg);
  else if (nv <= 8) route_scored_kernel<8><<<grid, block, 0, st>>>(a, lg);
  else if (nv <= 16) route_scored_kernel<16><<<grid, block, 0, st>>>(a, lg);
  else route_scored_kernel<32><<<grid, block, 0, st>>>(a, lg);
  return hipGetLastError();
}

}  // namespace moe
