// Grouped MXFP4 projections on tiles of at most 16 activation rows.
//
//   gate/up: h[r][i] = SiLU(g) * u, g = x_r . W[i], u = x_r . W[I + i]
//   down:    y[r][n] = h_r . W[n]
//
// Few rows per expert: bound by streaming the packed weights (0.53 bytes per
// weight, read once) and, for a handful of tokens, by the latency of that one
// pass, so everything a workgroup needs is loaded at once.  Both operands go
// from memory straight into the matrix instruction's registers, the weights as
// tiled pieces (a contiguous kilobyte per load), the activations as the same
// blocks of their rows.  A16 expands a block of weights to bf16 by the
// conversion instruction that takes the scale (exact) and runs four 16x16x32
// bf16 steps; A4 quantises the block of activations, which one lane holds
// whole, in registers and feeds codes and scale bytes of both sides to the
// scaled 16x16x128 instruction.
//
//  * mx_rows16_kernel: a workgroup owns 16 units (a gate and an up row each, or
//    2 x 16 down rows) of one tile; its waves split K and meet in LDS.  With
//    NV > 0 (a few tokens) every workgroup routes and sorts the batch itself:
//    that costs less than the launch and the round trip of a routing kernel.
//  * mx_down_combine_kernel (a few tokens): a workgroup owns 16 output columns
//    of every token; its waves share the (tile, part of K) products, which meet
//    in LDS, where the weighted sum of each token is formed: no fp32 rows
//    through memory and no combine launch.
#include "mx_common.h"
#include "route_common.h"

namespace moe {

namespace {

constexpr int kTM = 16;        // rows per tile
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
// the routing kernels do for them.)
constexpr int kRouteT = 4;
constexpr int kRouteP = 64;
static_assert(kRouteT < kRouteRowMinT, "the order of the gate weights' sum");

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
template <int WV>
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
      for (int i = threadIdx.x - 64 * first; i < n; i += 64 * (WV - first))
        *reinterpret_cast<mx_u32x4*>(L.x + t * L.pitch + i * 16) =
            *reinterpret_cast<const mx_u32x4*>(a.x + (size_t)t * a.ld_in + i * 8);
  }
  __syncthreads();
}

// The workgroup that writes the tables of moe_route_topk and moe_permute.
template <int THREADS>
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
  for (int i = tid; i < a.T * E; i += THREADS) {
    const int t = i / E, e = i - t * E;
    if (chosen(t, e)) {
      const int p = t * k + below(t, e);
      L.ids[p] = e;
      L.key[p] = route_ord(ro.logits[i]);
    }
  }
  for (int e = tid; e < E; e += THREADS) {
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
  for (int u = wave; u < a.T; u += THREADS / 64) {
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
// 0 writes the tables; else the tables come from memory.  WV waves.
template <int MODE, bool ACT4, bool XQ, int NB, bool ROUTE, int WV>
__global__ __launch_bounds__(64 * WV) void mx_rows16_kernel(MxProj a, MxRoute ro, int n_sh_tiles,
                                                            int n_ub) {
  __shared__ float red[WV][2][kTM * kPitch];
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
  if constexpr (ROUTE) route_and_stage<WV>(a, ro.logits, blk < 0 || slot >= n_sh_tiles, L);
  if (blk >= 0 && slot < n_sh_tiles) {
    const int per = (a.T + kTM - 1) / kTM;
    is_sh = true;
    e = slot / per;
    r0 = (slot - e * per) * kTM;
    r1 = min(a.T, r0 + kTM);
  } else if constexpr (ROUTE) {
    if (blk < 0) {
      write_routing<64 * WV>(a, ro, L);
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
  for (int s = wave * NB; s < pieces; s += WV * NB) {
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
  if (m >= kTM || r0 + m >= r1) return;
  float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
  for (int w = 0; w < WV; ++w) {
    v0 += red[w][0][u * kPitch + m];
    v1 += red[w][1][u * kPitch + m];
  }
  const size_t o = (size_t)(orow + m) * a.ld_out + u0 + u;
  if (MODE == 0) {
    if (u0 + u < U) static_cast<uint16_t*>(a.out)[o] = (uint16_t)mx_bf16(mx_silu_mul(v0, v1));
  } else {
    if (u0 + u < U) static_cast<float*>(a.out)[o] = v0;
    if (u0 + 16 + u < U) static_cast<float*>(a.out)[o + 16] = v1;
  }
}

int max_slots(const MxProj& a) {
  return a.n_shared * ((a.T + kTM - 1) / kTM) + moe_permute_max_tiles(a.T, a.k, a.E, kTM);
}

template <int MODE, bool ACT4, bool XQ, bool ROUTE>
hipError_t launch(const MxProj& a, const MxRoute& ro, hipStream_t st) {
  const int n_sh_tiles = a.n_shared * ((a.T + kTM - 1) / kTM);
  const int step = MODE == 0 ? 16 : 32;
  const int U = a.n_shared > 0 && a.U_sh > a.U ? a.U_sh : a.U;
  const int n_ub = (U + step - 1) / step;
  const long long grid = (long long)max_slots(a) * n_ub + (ROUTE ? 1 : 0);
  if (grid >= (1LL << 31)) return hipErrorInvalidValue;
  const int K = a.n_shared > 0 && a.K_sh > a.K ? a.K_sh : a.K;
  const int pieces = mx_pieces(K);
  const size_t lds = ROUTE ? RouteLds::bytes(a.T, a.E, a.ld_in) : 0;
  // Up to 64 pairs (a few tokens) eight waves split K, so that each has little
  // to do behind its loads; else four, with longer runs.  The same rule with
  // and without the routing: both sum in the same order.
#define MX_GO(NB, WV)                                                                         \
  mx_rows16_kernel<MODE, ACT4, XQ, NB, ROUTE, WV><<<(int)grid, 64 * WV, lds, st>>>(a, ro, n_sh_tiles, \
                                                                                   n_ub)
  if (ROUTE || a.P <= kRouteP) {
    if (pieces >= 16) MX_GO(2, 8);
    else MX_GO(1, 8);
  } else if constexpr (!ROUTE) {
    if (pieces >= 16) MX_GO(4, 4);
    else if (pieces >= 8) MX_GO(2, 4);
    else MX_GO(1, 4);
  }
#undef MX_GO
  return hipGetLastError();
}

// ---------------------------------------------------------------------
constexpr int kDnWaves = 8;
constexpr int kDnThreads = 64 * kDnWaves;
constexpr int kDnNB = 2;      // pieces per item
constexpr int kDnItems = 4;   // items of a wave whose loads are in flight together

struct MxCombine {
  const float* topk_w;
  const int32_t* pair_pos;
  const float* sh_gate;   // or null
  void* out;
  int out_f32;
  int max_tiles;   // routed
  int n_ch;        // parts of K: items per tile
};

// COLS: 16 output columns per workgroup, or 8 (half the rows of a piece: 128-byte
// runs of it) where 16 would leave compute units without a workgroup - one of
// them draws about 23 GB/s, so a token's 7 MB want all 256.
template <bool ACT4, int COLS>
__global__ __launch_bounds__(kDnThreads) void mx_down_combine_kernel(MxProj a, MxCombine cb,
                                                                     int n_sh_tiles) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int R = a.P + a.n_shared * a.T;
  float* yb = reinterpret_cast<float*>(smem);                             // [n_ch][R][COLS]
  int4* til = reinterpret_cast<int4*>(yb + (size_t)cb.n_ch * R * COLS);   // [slots]
  int* n_til = reinterpret_cast<int*>(til + n_sh_tiles + cb.max_tiles);
  int* ppos = n_til + 4;                                                  // [P]
  float* gw = reinterpret_cast<float*>(ppos + a.P);                       // [P]
  float* sg = gw + a.P;                                                   // [T][n_shared]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * COLS;
  const bool wrow = COLS == 16 || (c >> 3) == ((n0 >> 3) & 1);   // this lane's weight row is wanted

  // ---- tile list (expert, first row, end row, shared) and the gate tables
  for (int i = tid; i < a.P; i += kDnThreads) {
    ppos[i] = cb.pair_pos[i];
    gw[i] = cb.topk_w[i];
  }
  const int sh_per = (a.T + kTM - 1) / kTM;
  for (int i = tid; i < n_sh_tiles; i += kDnThreads) {
    const int e = i / sh_per, r = (i - e * sh_per) * kTM;
    til[i] = make_int4(e, a.P + e * a.T + r, a.P + e * a.T + min(a.T, r + kTM), 1);
  }
  for (int i = tid; i < a.T * a.n_shared; i += kDnThreads)
    sg[i] = cb.sh_gate ? shared_gate_weight(cb.sh_gate[i]) : 1.0f;
  if (wave == kDnWaves - 1) {
    auto list = [&](auto t) {
      t.load(a.offsets, a.E, a.P);
      int at = n_sh_tiles + t.pre - t.cnt;
      constexpr int PER = sizeof(t.lo) / sizeof(int);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        for (int r = t.lo[i]; r < t.hi[i] && at < n_sh_tiles + cb.max_tiles; r += kTM)
          til[at++] = make_int4(lane * PER + i, r, min(t.hi[i], r + kTM), 0);
      if (lane == 63) *n_til = n_sh_tiles + min(t.pre, cb.max_tiles);
    };
    if (a.E <= 128) list(MxTiles<kTM, 2>());
    else list(MxTiles<kTM, 8>());
  }
  __syncthreads();

  // ---- items (tile, part of K), kDnItems per wave at a time
  const int n_items = *n_til * cb.n_ch;
  const mx_u32x4 zero = {0, 0, 0, 0};
  for (int base = wave; base < n_items; base += kDnWaves * kDnItems) {
    mx_u32x4 w[kDnItems][1][kDnNB], x[kDnItems][kDnNB][4];
    uint32_t sw[kDnItems][1];
    int4 tl[kDnItems];
#pragma unroll
    for (int i = 0; i < kDnItems; ++i) {
      const int item = base + i * kDnWaves;
      const bool ok = item < n_items;
      const int slot = ok ? item / cb.n_ch : 0, s = ok ? (item - slot * cb.n_ch) * kDnNB : 0;
      tl[i] = ok ? til[slot] : make_int4(0, 0, 0, 0);
      const int K = tl[i].w ? a.K_sh : a.K;
      const int nblk = K / kMxBlock, pieces = mx_pieces(K), words = (pieces + 3) / 4;
      const uint8_t* wq = (tl[i].w ? a.w_sh : a.w) + tl[i].x * mx_code_bytes(a.U, K);
      const uint8_t* ws = (tl[i].w ? a.ws_sh : a.ws) + tl[i].x * mx_scale_bytes(a.U, K);
      const size_t rb = n0 / 16;
      const mx_u32x4* q = reinterpret_cast<const mx_u32x4*>(wq) + rb * pieces * 64 + lane;
#pragma unroll
      for (int j = 0; j < kDnNB; ++j)
        w[i][0][j] = ok && wrow && s + j < pieces ? __builtin_nontemporal_load(q + (s + j) * 64) : zero;
      sw[i][0] = ok && s < pieces
                     ? load_scales<kDnNB>(ws + ((rb * words + (s >> 2)) * 64 + lane) * 4, s)
                     : 0u;
      const bool have = tl[i].y + c < tl[i].z;
      const mx_u32x4* px =
          reinterpret_cast<const mx_u32x4*>(a.x + (size_t)(have ? tl[i].y + c : 0) * a.ld_in);
#pragma unroll
      for (int j = 0; j < kDnNB; ++j) {
        const int b = 4 * (s + j) + g;
#pragma unroll
        for (int t = 0; t < 4; ++t) x[i][j][t] = have && b < nblk ? px[b * 4 + t] : zero;
      }
    }
#pragma unroll
    for (int i = 0; i < kDnItems; ++i) {
      const int item = base + i * kDnWaves;
      if (item >= n_items) break;
      mx_f32x4 acc[1] = {{0, 0, 0, 0}};
      products<ACT4, kDnNB, 1>(w[i], sw[i], x[i], acc);
      mx_keep(acc[0]);
      const int ch = item % cb.n_ch;
      // lane: row c, weight rows 4g .. 4g + 3
      if (tl[i].y + c < tl[i].z && (COLS == 16 || (g >> 1) == ((n0 >> 3) & 1)))
        *reinterpret_cast<mx_f32x4*>(yb + ((size_t)ch * R + tl[i].y + c) * COLS +
                                     (4 * g & (COLS - 1))) = acc[0];
    }
  }
  __syncthreads();

  // ---- the parts of K of every row (rows that no tile wrote are not read below)
  const int part = R * COLS;
  if (cb.n_ch > 1) {
    for (int i = tid; i < part; i += kDnThreads) {
      float y = yb[i];
      for (int c0 = 1; c0 < cb.n_ch; c0 += 4) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = yb[min(c0 + q, cb.n_ch - 1) * part + i];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c0 + q < cb.n_ch) y += v[q];
      }
      yb[i] = y;
    }
    __syncthreads();
  }

  // ---- out[t][n] = sum_j w_j y_j + sum_s g_s y_s, in that order
  for (int i = tid; i < a.T * COLS; i += kDnThreads) {
    const int t = i / COLS, n = i & (COLS - 1);
    // eight pairs at a time: their LDS reads, then the sum in order
    float o = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      int p[8];
      float y[8], w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = t * a.k + min(j0 + j, a.k - 1);
        p[j] = j0 + j < a.k ? ppos[q] : -1;
        w[j] = gw[q];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = yb[max(p[j], 0) * COLS + n];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (p[j] >= 0) o = fmaf(w[j], y[j], o);
    }
    for (int s = 0; s < a.n_shared; ++s)
      o = fmaf(sg[t * a.n_shared + s], yb[(a.P + s * a.T + t) * COLS + n], o);
    if (cb.out_f32) static_cast<float*>(cb.out)[(size_t)t * a.U + n0 + n] = o;
    else static_cast<uint16_t*>(cb.out)[(size_t)t * a.U + n0 + n] = (uint16_t)mx_bf16(o);
  }
}

int dn_parts(const MxProj& a) {
  const int K = a.n_shared > 0 && a.K_sh > a.K ? a.K_sh : a.K;
  return (mx_pieces(K) + kDnNB - 1) / kDnNB;
}

int dn_cols(const MxProj& a) { return a.U / 16 < 256 ? 8 : 16; }

size_t dn_lds(const MxProj& a, int max_tiles, int n_sh_tiles) {
  const size_t R = (size_t)a.P + (size_t)a.n_shared * a.T;
  return dn_parts(a) * R * dn_cols(a) * 4 + (size_t)(n_sh_tiles + max_tiles) * 16 + 16 + (size_t)a.P * 8 +
         (size_t)a.T * a.n_shared * 4;
}

}  // namespace

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

bool mx_down_combine_ok(const MxProj& a) {
  const int max_tiles = moe_permute_max_tiles(a.T, a.k, a.E, kTM);
  const int n_sh_tiles = a.n_shared * ((a.T + kTM - 1) / kTM);
  return n_sh_tiles + max_tiles <= kDnSlots && dn_lds(a, max_tiles, n_sh_tiles) <= 64 * 1024;
}

hipError_t launch_mx_down_combine(const MxProj& a, int act4, const float* topk_w,
                                  const int32_t* pair_pos, const float* sh_gate, void* out,
                                  int out_f32, hipStream_t st) {
  MxCombine cb = {topk_w, pair_pos, sh_gate, out, out_f32,
                  moe_permute_max_tiles(a.T, a.k, a.E, kTM), dn_parts(a)};
  const int n_sh_tiles = a.n_shared * ((a.T + kTM - 1) / kTM);
  const size_t lds = dn_lds(a, cb.max_tiles, n_sh_tiles);
  const bool half = dn_cols(a) == 8;
  auto kern = act4 ? (half ? mx_down_combine_kernel<true, 8> : mx_down_combine_kernel<true, 16>)
                   : (half ? mx_down_combine_kernel<false, 8> : mx_down_combine_kernel<false, 16>);
  kern<<<a.U / dn_cols(a), kDnThreads, lds, st>>>(a, cb, n_sh_tiles);
  return hipGetLastError();
}

}  // namespace moe
