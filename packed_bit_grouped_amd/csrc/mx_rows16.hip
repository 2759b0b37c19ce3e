// Grouped MXFP4 projections on tiles of at most 16 activation rows.
//
//   gate/up: h[r][i] = SiLU(g) * u, g = x_r . W[i], u = x_r . W[I + i]
//   down:    y[r][n] = h_r . W[n]
//
// Few rows per expert: bound by streaming the packed weights (0.53 bytes per
// weight, read once), so a workgroup is small and loads everything it needs
// at once.  It owns 16 units (a gate and an up row each, or 2 x 16 down rows)
// of one tile; its four waves split K and meet in LDS.  Both operands go from
// memory straight into the matrix instruction's registers, the weights as
// tiled pieces (a contiguous kilobyte per load), the activations as the same
// blocks of their rows.  A16 expands a block to bf16 by the conversion
// instruction that takes the scale (exact) and runs four 16x16x32 bf16 steps;
// A4 feeds codes and scale bytes to the scaled 16x16x128 instruction as they
// are.
#include "mx_common.h"

namespace moe {

namespace {

constexpr int kTM = 16;        // rows per tile
constexpr int kWaves = 4;
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

template <int NB, int J = 0>
__device__ __forceinline__ void fp4_steps(const mx_u32x4 (&w0)[NB], uint32_t s0,
                                          const mx_u32x4 (&w1)[NB], uint32_t s1,
                                          const mx_u32x4 (&x)[NB], uint32_t sx, mx_f32x4& a0,
                                          mx_f32x4& a1) {
  if constexpr (J < NB) {
    a0 = mx_mfma_fp4<J>(w0[J], s0, x[J], sx, a0);
    a1 = mx_mfma_fp4<J>(w1[J], s1, x[J], sx, a1);
    fp4_steps<NB, J + 1>(w0, s0, w1, s1, x, sx, a0, a1);
  }
}

template <int MODE, bool ACT4, int NB>
__global__ __launch_bounds__(kThreads) void mx_rows16_kernel(MxProj a, int n_sh_tiles, int n_ub) {
  __shared__ float red[kWaves][2][kTM * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slot = blockIdx.x / n_ub, ub = blockIdx.x - slot * n_ub;
  const int c = lane & 15, g = lane >> 4;

  // ---- the tile: shared experts' first
  bool is_sh = false;
  int e, r0, r1;
  const int per = (a.T + kTM - 1) / kTM;
  if (slot < n_sh_tiles) {
    is_sh = true;
    e = slot / per;
    r0 = (slot - e * per) * kTM;
    r1 = min(a.T, r0 + kTM);
  } else if (!mx_find_tile<kTM>(a.offsets, a.E, a.P, slot - n_sh_tiles, e, r0, r1)) {
    return;
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
    } else {
      const int p = a.sorted_pair[r0 + c];
      have = (unsigned)p < (unsigned)a.P;
      xrow = have ? p / a.k : 0;
    }
  }

  mx_f32x4 a0 = {0, 0, 0, 0}, a1 = {0, 0, 0, 0};
  const mx_u32x4 zero = {0, 0, 0, 0};
  for (int s = wave * NB; s < pieces; s += kWaves * NB) {
    mx_u32x4 w0[NB], w1[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
      w0[j] = s + j < pieces ? __builtin_nontemporal_load(q0 + (s + j) * 64) : zero;
#pragma unroll
    for (int j = 0; j < NB; ++j)
      w1[j] = s + j < pieces ? __builtin_nontemporal_load(q1 + (s + j) * 64) : zero;
    const uint32_t s0 = load_scales<NB>(sw0 + (s >> 2) * 256, s);
    const uint32_t s1 = load_scales<NB>(sw1 + (s >> 2) * 256, s);
    if (ACT4) {
      // rows of whole words, zeros behind K
      const int KP = mx_pad_k(a.ld_in);
      mx_u32x4 x[NB];
      const mx_u32x4* px = reinterpret_cast<const mx_u32x4*>(a.q + xrow * (KP / 2)) + 4 * s + g;
#pragma unroll
      for (int j = 0; j < NB; ++j) x[j] = have && s + j < pieces ? px[4 * j] : zero;
      const uint32_t sx =
          have ? load_scales<NB>(a.s + xrow * (KP / kMxBlock) + (s >> 2) * 16 + 4 * g, s) : 0u;
      fp4_steps<NB>(w0, s0, w1, s1, x, sx, a0, a1);
    } else {
      const mx_u32x4* px = reinterpret_cast<const mx_u32x4*>(a.x + xrow * a.ld_in);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int b = 4 * (s + j) + g;
        mx_u32x4 x[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = have && b < nblk ? px[b * 4 + t] : zero;
        const float f0 = mx_scale_f32((s0 >> (8 * j)) & 255u);
        const float f1 = mx_scale_f32((s1 >> (8 * j)) & 255u);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const mx_bf16x8 xv = __builtin_bit_cast(mx_bf16x8, x[t]);
          a0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_word_to_bf16(w0[j][t], f0), xv, a0, 0, 0, 0);
          a1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_word_to_bf16(w1[j][t], f1), xv, a1, 0, 0, 0);
        }
      }
    }
  }

  // ---- the waves' parts of K meet: word [unit][row]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    red[wave][0][(4 * g + i) * kPitch + c] = a0[i];
    red[wave][1][(4 * g + i) * kPitch + c] = a1[i];
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
    if (u0 + u < U) static_cast<uint16_t*>(a.out)[o] = (uint16_t)mx_bf16(silu_mul(v0, v1));
  } else {
    if (u0 + u < U) static_cast<float*>(a.out)[o] = v0;
    if (u0 + 16 + u < U) static_cast<float*>(a.out)[o + 16] = v1;
  }
}

template <int MODE, bool ACT4>
hipError_t launch(const MxProj& a, hipStream_t st) {
  const int n_sh_tiles = a.n_shared * ((a.T + kTM - 1) / kTM);
  const int step = MODE == 0 ? 16 : 32;
  const int U = a.n_shared > 0 && a.U_sh > a.U ? a.U_sh : a.U;
  const int n_ub = (U + step - 1) / step;
  const long long grid =
      (long long)(n_sh_tiles + moe_permute_max_tiles(a.T, a.k, a.E, kTM)) * n_ub;
  if (grid >= (1LL << 31)) return hipErrorInvalidValue;
  const int K = a.n_shared > 0 && a.K_sh > a.K ? a.K_sh : a.K;
  const int pieces = mx_pieces(K);
  // the longest run per lane that still gives every wave a chunk of K
  auto kern = pieces >= kWaves * 4   ? mx_rows16_kernel<MODE, ACT4, 4>
              : pieces >= kWaves * 2 ? mx_rows16_kernel<MODE, ACT4, 2>
                                     : mx_rows16_kernel<MODE, ACT4, 1>;
  kern<<<(int)grid, kThreads, 0, st>>>(a, n_sh_tiles, n_ub);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_rows16(const MxProj& a, int mode, int act4, hipStream_t st) {
  if (mode == 0) return act4 ? launch<0, true>(a, st) : launch<0, false>(a, st);
  return act4 ? launch<1, true>(a, st) : launch<1, false>(a, st);
}

}  // namespace moe
