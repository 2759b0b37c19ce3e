// Grouped MXFP4 projections on tiles of at most 16 activation rows.
//
//   gate/up: h[r][i] = SiLU(g) * u, g = x_r . W[i], u = x_r . W[I + i]
//   down:    y[r][n] = h_r . W[n]
//
// Few rows per expert: bound by streaming the packed weights (0.53 bytes per
// weight, read once) and, for a handful of tokens, by the latency of that one
// pass: a turn's weights, scales and activations are loaded at once.  Both operands go
// from memory straight into the matrix instruction's registers, the weights as
// tiled pieces (a contiguous kilobyte per load), the activations as the same
// blocks of their rows.  A16 expands a block of weights to bf16 by the
// conversion instruction that takes the scale (exact) and runs four 16x16x32
// bf16 steps; A4 quantises the block of activations, which one lane holds
// whole, in registers and feeds codes and scale bytes of both sides to the
// scaled 16x16x128 instruction.
//
// A workgroup owns 16 units (a gate and an up row each, or 2 x 16 down rows) of
// one tile; its waves split K and meet in LDS.  With ROUTE (a few tokens) every
// workgroup routes and sorts the batch itself: that costs less than the launch
// and the round trip of a routing kernel.
//
// Measured (H 2048, I 768, 128 experts, k 8; kernel trace, median and fastest of 30
// calls on three sets of weights): A4 gate/up of 64 tokens 35.0 / 33.9 us = 6.1
// TB/s of codes and scales (a plain read reaches 6.3); A16 of one token with a
// shared expert 6.4 / 5.2 us, of 15 MB; routed inside 7.6 / 7.2; down of one token
// 5.1 / 3.9, of 12 tokens 11.3 / 10.2, of 64 29.6 / 28.9.  What a short gate/up
// pass waits for is trips to memory one behind the other: the offsets, the row's
// pair (the loop's first loads, weights too, stand behind it and behind the
// division that makes a token of it, though the weights need the tile alone),
// then rows and weights, then the reduction; a second turn's loads (K above 2048)
// start when the first turn's products are done.  A16 gate/up of 8 tokens 22.6 us
// against 13.7 for its bytes, of 16 33.4 against 22: every weight is converted for
// 16 columns of which one or two are used.
// Four waves: with eight, each with half the K, gate/up of one token took 0.7 us
// longer, of 8 tokens 27.4 against 22.6 - more waves to start and to join for the
// same loads in flight.  A kernel that joined down and the weighted sum (a
// workgroup per 16 columns, all experts) was no faster for one token (8.2
// against 8.0 us) and slower for more (3 tokens 15.7 against 11.5).
#include "mx_common.h"
#include "route_common.h"

namespace moe {

namespace {

constexpr int kTM = 16;        // rows per tile
constexpr int kWaves = 4;      // share K
constexpr int kThreads = 64 * kWaves;
constexpr int kPitch = 20;     // LDS words per 16 (4 rows of 20 words: 16 banks apart)

// The scale bytes of NB pieces from piece s on (s % NB == 0): bytes of the
// lane's word of four pieces.
template <int NB>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* __restrict__ word, int s) {
  const uint8_t* p = word + (s & 3);
  if (NB == 4) return *reinterpret_cast<const uint32_t*>(p);
  if (NB == 2) return *reinterpret_cast<const uint16_t*>(p);
  return *p;
}

// 32 bf16 values of one block to codes and scale byte (the rule of
// mx_quant_kernel, the same instructions).
__device__ __forceinline__ mx_u32x4 quantise_block(const mx_u32x4 (&x)[4], uint32_t& sb) {
  uint32_t m = 0;   // two magnitudes per word, compared as 16-bit integers
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = x[t][i];
      m = max(m, max(v & 0x7FFFu, (v >> 16) & 0x7FFFu));
    }
  sb = mx_scale_byte(m << 16);
  const float sc = mx_scale_f32(sb);
  mx_u32x4 q;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    uint32_t w = 0;
    const uint32_t v0 = x[t].x, v1 = x[t].y, v2 = x[t].z, v3 = x[t].w;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, v0), sc, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, v1), sc, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, v2), sc, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, v3), sc, 3);
    q[t] = w;
  }
  return q;
}

// The lane's block of one piece: 16 rows of weights (codes w, scale byte in
// byte J of sw) times its activation block x, into acc.
template <bool ACT4, int J>
__device__ __forceinline__ mx_f32x4 piece_product(mx_u32x4 w, uint32_t sw, const mx_u32x4 (&x)[4],
                                                  mx_u32x4 xq, uint32_t sx, mx_f32x4 acc) {
  if constexpr (ACT4) {
    const mx_i32x8 av = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    const mx_i32x8 bv = {(int)xq.x, (int)xq.y, (int)xq.z, (int)xq.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 4, J, (int)sw, 0,
                                                            (int)sx);
  } else {
    const float f = mx_scale_f32((sw >> (8 * J)) & 255u);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_word_to_bf16(w[t], f),
                                                    __builtin_bit_cast(mx_bf16x8, x[t]), acc, 0, 0, 0);
    return acc;
  }
}

// NB pieces of F row blocks against the same activation blocks.
template <bool ACT4, int NB, int F, int J = 0>
__device__ __forceinline__ void products(const mx_u32x4 (&w)[F][NB], const uint32_t (&sw)[F],
                                         const mx_u32x4 (&x)[NB][4], mx_f32x4 (&acc)[F]) {
  if constexpr (J < NB) {
    mx_u32x4 xq = {0, 0, 0, 0};
    uint32_t sx = 0;
    if (ACT4) xq = quantise_block(x[J], sx);
#pragma unroll
    for (int f = 0; f < F; ++f)
      acc[f] = piece_product<ACT4, J>(w[f][J], sw[f], x[J], xq, sx, acc[f]);
    products<ACT4, NB, F, J + 1>(w, sw, x, acc);
  }
}

// The same with the activations' codes x and scale word sx from memory.
template <int NB, int J = 0>
__device__ __forceinline__ void code_products(const mx_u32x4 (&w)[2][NB], const uint32_t (&sw)[2],
                                              const mx_u32x4 (&x)[NB], uint32_t sx,
                                              mx_f32x4 (&acc)[2]) {
  if constexpr (J < NB) {
#pragma unroll
    for (int f = 0; f < 2; ++f) acc[f] = mx_mfma_fp4<J>(w[f][J], sw[f], x[J], sx, acc[f]);
    code_products<NB, J + 1>(w, sw, x, sx, acc);
  }
}

// Routing outputs of the fused launch (written by workgroup 0 alone).
struct MxRoute {
  const float* logits;
  int renorm;
  int32_t* ids;
  float* w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* sorted_pair;
  int32_t* pair_pos;
};

// Up to this many tokens and pairs route inside the gate/up launch.  (Fewer
// than kRouteRowMinT tokens: their gate weights are summed over 64 lanes, as
// the routing kernels do for them.)  At three tokens of 8 pairs it gains 2.9
// us of 29.6; a fourth would leave no wave to bring the rows.
constexpr int kRouteT = 3;
constexpr int kRouteP = 64;
static_assert(kRouteT < kRouteRowMinT, "the order of the gate weights' sum");
static_assert(kRouteT < kWaves, "a wave is left to stage the rows");

// LDS of the routed launch (dynamic): masks of the chosen experts [T][W], then
// (workgroup 0) the chosen ids and their order keys [P], and the tokens' rows,
// 16 bytes apart beyond their length.
struct RouteLds {
  uint64_t* mask;
  int* ids;
  uint32_t* key;
  unsigned char* x;
  int W, pitch;
  static __host__ __device__ size_t head(int T, int E) {
    return ((size_t)T * ((E + 63) / 64) * 8 + kRouteP * 8 + 15) / 16 * 16;
  }
  static __host__ __device__ size_t bytes(int T, int E, int H) {
    return head(T, E) + (size_t)T * (H * 2 + 16);
  }
  __device__ RouteLds(unsigned char* p, int T, int E, int H) : W((E + 63) / 64), pitch(H * 2 + 16) {
    mask = reinterpret_cast<uint64_t*>(p);
    ids = reinterpret_cast<int*>(mask + T * W);
    key = reinterpret_cast<uint32_t*>(ids + kRouteP);
    x = p + head(T, E);
  }
};

// One wave, one token: the mask of the k experts with the largest order keys
// (of equal keys the smaller index).  The k-th largest key is found from the top
// two bits at a time, counting the keys not below a candidate by ballots; that
// takes half the time of k arg-max rounds, whose order only workgroup 0 needs.
template <int NV>
__device__ __forceinline__ void select_topk(const float* __restrict__ logits, int E, int k,
                                            uint64_t* mask) {
  const int lane = threadIdx.x & 63;
  uint32_t key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) key[j] = __float_as_uint(logits[min(lane + 64 * j, E - 1)]);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    key[j] = lane + 64 * j < E ? route_ord(__uint_as_float(key[j])) : 0u;
  uint32_t thr = 0;
  for (int b = 30; b >= 0; b -= 2) {
    int n[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 1; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < NV; ++j) n[q] += __popcll(__ballot(key[j] >= (thr | ((uint32_t)q << b))));
    thr |= (n[3] >= k ? 3u : n[2] >= k ? 2u : n[1] >= k ? 1u : 0u) << b;
  }
  int need = k;
#pragma unroll
  for (int j = 0; j < NV; ++j) need -= __popcll(__ballot(key[j] > thr));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    uint64_t m = __ballot(key[j] > thr), eq = __ballot(key[j] == thr);
    for (; need > 0 && eq; --need) {
      m |= eq & (0 - eq);
      eq &= eq - 1;
    }
    if (lane == 0 && 64 * j < E) mask[j] = m;
  }
}

// Waves 0 .. T-1 of the workgroup route a token each, the others bring the
// tokens' rows into LDS.
__device__ __forceinline__ void route_and_stage(const MxProj& a, const float* __restrict__ logits,
                                                bool route, const RouteLds& L) {
  const int wave = threadIdx.x >> 6;
  const int first = route ? a.T : 0;
  if (wave < first) {
    uint64_t* m = L.mask + wave * L.W;
    const float* row = logits + wave * a.E;
    if (a.E <= 128) select_topk<2>(row, a.E, a.k, m);
    else select_topk<8>(row, a.E, a.k, m);
  } else {
    const int n = a.ld_in / 8;   // 16-byte chunks per row
    for (int t = 0; t < a.T; ++t)
      for (int i = threadIdx.x - 64 * first; i < n; i += 64 * (kWaves - first))
        *reinterpret_cast<mx_u32x4*>(L.x + t * L.pitch + i * 16) =
            *reinterpret_cast<const mx_u32x4*>(a.x + (size_t)t * a.ld_in + i * 8);
  }
  __syncthreads();
}

// The workgroup that writes the tables of moe_route_topk and moe_permute.
__device__ __forceinline__ void write_routing(const MxProj& a, const MxRoute& ro,
                                              const RouteLds& L) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E, k = a.k, W = L.W;
  auto chosen = [&](int t, int e) { return (int)(L.mask[t * W + e / 64] >> (e & 63)) & 1; };
  // token t's chosen experts below e
  auto below = [&](int t, int e) {
    int o = __popcll(L.mask[t * W + e / 64] & ((1ull << (e & 63)) - 1));
    for (int w = 0; w < e / 64; ++w) o += __popcll(L.mask[t * W + w]);
    return o;
  };
  for (int i = tid; i < a.T * E; i += kThreads) {
    const int t = i / E, e = i - t * E;
    if (chosen(t, e)) {
      const int p = t * k + below(t, e);
      L.ids[p] = e;
      L.key[p] = route_ord(ro.logits[i]);
    }
  }
  for (int e = tid; e < E; e += kThreads) {
    int c = 0, o = 0;
    for (int t = 0; t < a.T; ++t) {
      c += chosen(t, e);
      o += below(t, e);
    }
    ro.counts[e] = c;
    ro.offsets[e] = o;
  }
  if (tid == 0) ro.offsets[E] = a.P;
  __syncthreads();
  // pair tid: the rank of its expert among the token's chosen ones, its place in
  // the stable sort (smaller experts of every token, the same one of earlier
  // tokens), and its gate weight
  const int t = tid / k, i0 = t * k;
  int e = 0, rank = 0;
  uint32_t key = 0;
  if (tid < a.P) {
    e = L.ids[tid];
    key = L.key[tid];
    for (int q = i0; q < i0 + k; ++q) rank += L.key[q] > key || (L.key[q] == key && q < tid);
    int pos = 0;
    for (int u = 0; u < a.T; ++u) pos += below(u, e) + (u < t ? chosen(u, e) : 0);
    const int p = i0 + rank;
    ro.ids[p] = e;
    ro.pair_pos[p] = pos;
    ro.sorted_pair[pos] = p;
  }
  __syncthreads();
  if (tid < a.P) L.key[i0 + rank] = key;   // in order of rank from here on
  __syncthreads();
  // one wave per token, choice r in lane r, the sums of route_group_vals
  for (int u = wave; u < a.T; u += kThreads / 64) {
    const float v = lane < k ? route_unord(L.key[u * k + lane]) : 0.0f;
    const float top = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
    const float ex = lane < k ? expf(v - top) : 0.0f;
    float sum = ex;
    if (!ro.renorm) {
      sum = 0.0f;
      for (int x = lane; x < E; x += 64) sum += expf(ro.logits[u * E + x] - top);
    }
    const float denom = wave_sum(sum);
    if (lane < k) ro.w[u * k + lane] = ex / denom;
  }
}

// Tile j of the routed experts (each has at most T <= 16 rows: one tile): its
// expert, rows, and the token of this lane's row (-1: none).
__device__ __forceinline__ bool find_masked(const MxProj& a, const RouteLds& L, int j, int& e,
                                            int& r0, int& r1, int& token) {
  const int c = threadIdx.x & 15;
  r0 = 0;
  for (int w = 0; w < L.W; ++w) {
    uint64_t any = 0;
    for (int t = 0; t < a.T; ++t) any |= L.mask[t * L.W + w];
    const int n = __popcll(any);
    if (j < n) {
      for (; j > 0; --j) any &= any - 1;
      const int b = __builtin_ctzll(any);
      e = 64 * w + b;
      int rows = 0;
      token = -1;
      for (int t = 0; t < a.T; ++t) {
        const uint64_t m = L.mask[t * L.W + w];
        r0 += __popcll(m & ((1ull << b) - 1));
        if ((m >> b) & 1) {
          if (rows == c) token = t;
          ++rows;
        }
      }
      r1 = r0 + rows;
      return true;
    }
    j -= n;
    for (int t = 0; t < a.T; ++t) r0 += __popcll(L.mask[t * L.W + w]);
  }
  return false;
}

// XQ (A4): the activations' codes and scales come from memory; else they are
// quantised here.  ROUTE: the workgroup routes the tokens itself, and workgroup
// 0 writes the tables; else the tables come from memory.
template <int MODE, bool ACT4, bool XQ, int NB, bool ROUTE>
__global__ __launch_bounds__(kThreads) void mx_rows16_kernel(MxProj a, MxRoute ro, int n_sh_tiles,
                                                            int n_ub) {
  __shared__ float red[kWaves][2][kTM * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int blk = ROUTE ? (int)blockIdx.x - 1 : (int)blockIdx.x;
  const int c = lane & 15, g = lane >> 4;

  // ---- the tile: shared experts' first
  bool is_sh = false;
  int e = 0, r0 = 0, r1 = 0;
  int token = -1;   // routed launch: the token of this lane's column
  const int slot = blk / n_ub, ub = blk - slot * n_ub;
  extern __shared__ __align__(16) unsigned char route_smem[];
  const RouteLds L(route_smem, ROUTE ? a.T : 0, a.E, ROUTE ? a.ld_in : 0);
  if constexpr (ROUTE) route_and_stage(a, ro.logits, blk < 0 || slot >= n_sh_tiles, L);
  if (blk >= 0 && slot < n_sh_tiles) {
    const int per = (a.T + kTM - 1) / kTM;
    is_sh = true;
    e = slot / per;
    r0 = (slot - e * per) * kTM;
    r1 = min(a.T, r0 + kTM);
  } else if constexpr (ROUTE) {
    if (blk < 0) {
      write_routing(a, ro, L);
      return;
    }
    if (!find_masked(a, L, slot - n_sh_tiles, e, r0, r1, token)) return;
  } else {
    // E <= 512: two or eight experts per lane
    const int j = slot - n_sh_tiles;
    bool ok;
    if (a.E <= 128) {
      MxTiles<kTM, 2> t;
      t.load(a.offsets, a.E, a.P);
      ok = t.find(j, e, r0, r1);
    } else {
      MxTiles<kTM, 8> t;
      t.load(a.offsets, a.E, a.P);
      ok = t.find(j, e, r0, r1);
    }
    if (!ok) return;
  }
  const int U = is_sh ? a.U_sh : a.U, K = is_sh ? a.K_sh : a.K;
  const int u0 = ub * (MODE == 0 ? 16 : 32);   // first unit (gate/up) or row (down)
  if (u0 >= U) return;
  const int N = MODE == 0 ? 2 * U : U;
  const int nblk = K / kMxBlock, pieces = mx_pieces(K), words = (pieces + 3) / 4;
  const uint8_t* wq = (is_sh ? a.w_sh : a.w) + e * mx_code_bytes(N, K);
  const uint8_t* wsc = (is_sh ? a.ws_sh : a.ws) + e * mx_scale_bytes(N, K);
  // the two 16-row blocks of this workgroup
  const size_t rb0 = u0 / 16, rb1 = MODE == 0 ? (U + u0) / 16 : u0 / 16 + 1;
  const mx_u32x4* q0 = reinterpret_cast<const mx_u32x4*>(wq) + rb0 * pieces * 64 + lane;
  const mx_u32x4* q1 = reinterpret_cast<const mx_u32x4*>(wq) + rb1 * pieces * 64 + lane;
  const uint8_t* sw0 = wsc + (rb0 * words * 64 + lane) * 4;
  const uint8_t* sw1 = wsc + (rb1 * words * 64 + lane) * 4;

  // ---- the activation row of this lane's column
  const int orow = is_sh ? a.P + e * a.T + r0 : r0;   // first row of h / y
  bool have = r0 + c < r1;
  long long xrow = 0;
  if (have) {
    if (MODE == 1) {
      xrow = orow + c;
    } else if (is_sh) {
      xrow = r0 + c;
    } else if (ROUTE) {
      xrow = token;
    } else {
      const int p = a.sorted_pair[r0 + c];
      have = (unsigned)p < (unsigned)a.P;
      xrow = have ? p / a.k : 0;
    }
  }

  mx_f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  const mx_u32x4 zero = {0, 0, 0, 0};
  for (int s = wave * NB; s < pieces; s += kWaves * NB) {
    mx_u32x4 w[2][NB];
    uint32_t sw[2];
#pragma unroll
    for (int j = 0; j < NB; ++j)
      w[0][j] = s + j < pieces ? __builtin_nontemporal_load(q0 + (s + j) * 64) : zero;
#pragma unroll
    for (int j = 0; j < NB; ++j)
      w[1][j] = s + j < pieces ? __builtin_nontemporal_load(q1 + (s + j) * 64) : zero;
    sw[0] = load_scales<NB>(sw0 + (s >> 2) * 256, s);
    sw[1] = load_scales<NB>(sw1 + (s >> 2) * 256, s);
    if constexpr (XQ) {
      // rows of whole words, zeros behind K
      const int KP = mx_pad_k(a.ld_in);
      mx_u32x4 x[NB];
      const mx_u32x4* px = reinterpret_cast<const mx_u32x4*>(a.q + xrow * (KP / 2)) + 4 * s + g;
#pragma unroll
      for (int j = 0; j < NB; ++j) x[j] = have && s + j < pieces ? px[4 * j] : zero;
      const uint32_t sx =
          have ? load_scales<NB>(a.s + xrow * (KP / kMxBlock) + (s >> 2) * 16 + 4 * g, s) : 0u;
      code_products<NB>(w, sw, x, sx, acc);
    } else {
      mx_u32x4 x[NB][4];
      const mx_u32x4* px = ROUTE ? reinterpret_cast<const mx_u32x4*>(L.x + xrow * L.pitch)
                                 : reinterpret_cast<const mx_u32x4*>(a.x + xrow * a.ld_in);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int b = 4 * (s + j) + g;
#pragma unroll
        for (int t = 0; t < 4; ++t) x[j][t] = have && b < nblk ? px[b * 4 + t] : zero;
      }
      products<ACT4, NB, 2>(w, sw, x, acc);
    }
  }

  mx_keep(acc[0]);
  mx_keep(acc[1]);
  // ---- the waves' parts of K meet: word [unit][row]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    red[wave][0][(4 * g + i) * kPitch + c] = acc[0][i];
    red[wave][1][(4 * g + i) * kPitch + c] = acc[1][i];
  }
  __syncthreads();
  const int u = tid & 15, m = tid >> 4;   // unit, row
  if (r0 + m >= r1) return;
  float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    v0 += red[w][0][u * kPitch + m];
    v1 += red[w][1][u * kPitch + m];
  }
  const size_t o = (size_t)(orow + m) * a.ld_out + u0 + u;
  if (MODE == 0) {
    const float gv[1] = {v0}, uv[1] = {v1};
    float hv[1];
    mx_silu_mul(gv, uv, hv);
    if (u0 + u < U) static_cast<uint16_t*>(a.out)[o] = (uint16_t)mx_bf16(hv[0]);
  } else {
    if (u0 + u < U) static_cast<float*>(a.out)[o] = v0;
    if (u0 + 16 + u < U) static_cast<float*>(a.out)[o + 16] = v1;
  }
}

// Blocks of columns: of 16 units, or of 32 down rows.
int col_blocks(const MxProj& a, int mode) {
  const int step = mode == 0 ? 16 : 32;
  const int U = a.n_shared > 0 && a.U_sh > a.U ? a.U_sh : a.U;
  return (U + step - 1) / step;
}

template <int MODE, bool ACT4, bool XQ, bool ROUTE>
hipError_t launch(const MxProj& a, const MxRoute& ro, hipStream_t st) {
  const int n_sh_tiles = a.n_shared * ((a.T + kTM - 1) / kTM);
  const int n_ub = col_blocks(a, MODE);
  const long long grid = mx_rows16_grid(a, MODE) + (ROUTE ? 1 : 0);
  if (grid > kMxMaxGrid) return hipErrorInvalidValue;
  const int K = a.n_shared > 0 && a.K_sh > a.K ? a.K_sh : a.K;
  const int pieces = mx_pieces(K);
  const size_t lds = ROUTE ? RouteLds::bytes(a.T, a.E, a.ld_in) : 0;
  // Pieces per wave and turn, so that the four waves pass K in few turns: each
  // turn is a trip to memory (down of one token, K 768, NB 1 7.6 us, 2 7.3; A4
  // of 64 tokens 31.3, 29.4).  At K between 1024 and 2048 NB 4 would leave waves
  // idle (K 1408, 12 tokens: 14.3 us, NB 2 12.8).  NB 2 leaves one of the four idle
  // at K 640 and 768 (five and six pieces), NB 1 at K 352, and K 1408 and 1536 (11
  // and 12) go 2, 2, 1, 1: K of 768 in down costs its workgroup a turn for 13 KB.
#define MX_GO(NB) \
  mx_rows16_kernel<MODE, ACT4, XQ, NB, ROUTE><<<(int)grid, kThreads, lds, st>>>(a, ro, n_sh_tiles, n_ub)
  if (pieces >= 16) MX_GO(4);
  else if (pieces > 4) MX_GO(2);
  else MX_GO(1);
#undef MX_GO
  return hipGetLastError();
}

}  // namespace

long long mx_rows16_grid(const MxProj& a, int mode) {
  const long long slots =
      a.n_shared * ((a.T + kTM - 1LL) / kTM) + moe_permute_max_tiles(a.T, a.k, a.E, kTM);
  return slots * col_blocks(a, mode);
}

hipError_t launch_mx_rows16(const MxProj& a, int mode, int act4, hipStream_t st) {
  const MxRoute none = {};
  const bool xq = act4 && a.q != nullptr;
#define MX_L(MODE)                                              \
  (xq     ? launch<MODE, true, true, false>(a, none, st)        \
   : act4 ? launch<MODE, true, false, false>(a, none, st)       \
          : launch<MODE, false, false, false>(a, none, st))
  return mode == 0 ? MX_L(0) : MX_L(1);
#undef MX_L
}

bool mx_route_gateup_ok(int T, int k, int E, int H) {
  return T <= kRouteT && T * k <= kRouteP && E <= kPermMaxE &&
         RouteLds::bytes(T, E, H) <= 40 * 1024;
}

hipError_t launch_mx_route_gateup(const MxProj& a, int act4, const float* logits, int renorm,
                                  int32_t* ids, float* w, int32_t* counts, int32_t* offsets,
                                  int32_t* sorted_pair, int32_t* pair_pos, hipStream_t st) {
  const MxRoute ro = {logits, renorm, ids, w, counts, offsets, sorted_pair, pair_pos};
  return act4 ? launch<0, true, false, true>(a, ro, st) : launch<0, false, false, true>(a, ro, st);
}

}  // namespace moe
