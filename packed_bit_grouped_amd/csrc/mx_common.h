// Shared pieces of the microscaled 4-bit (MXFP4) kernels: E2M1 codes, two a
// byte with the even index in the low nibble, and one E8M0 scale byte per 32
// values along K.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef int mx_i32x4 __attribute__((ext_vector_type(4)));
typedef int mx_i32x8 __attribute__((ext_vector_type(8)));
typedef float mx_f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int mx_u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 mx_bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;      // values per scale
constexpr int kMxNanScale = 255;  // scale byte of a block that held inf or NaN
constexpr int kMxMaxLen = 1 << 30;  // H, I, I_shared: 2 I rows and padded rows are ints
constexpr long long kMxMaxGrid = (1LL << 24) - 1;  // workgroups of 256: below 2^32 threads a launch

// Workspace of the projection calls (byte offsets).
struct MxWsLayout {
  size_t qx, sx;     // A4: codes and scales of x, rows of mx_pad_k(H) values;
                     // A16 where rows are not whole steps: qx holds a padded copy of x
  size_t qh, sh;     // the same of h (rows of mx_pad_k(ld_h))
  size_t y;          // fp32 [R][H]
  size_t tiles;      // layer: the sort's tile list and its count
  size_t perm;       // layer: counts of the sort over many workgroups
  size_t total;
};

// Tiled matrices: pieces of 16 rows x 128 K, pieces along K together, as the
// matrix instruction wants them: 16 bytes of codes per lane, lane (row c =
// lane % 16, group g = lane / 16) of piece s holding block 4s + g of row c; and
// the scale bytes of four pieces as one word per lane, byte j the lane's block
// of piece 4S + j.  Blocks past K hold code 0 and scale 0.  A wave's load is
// then one contiguous kilobyte; from plain rows (16 runs of 128 bytes a load)
// the gate/up product of 4096 tokens with MXFP4 activations (H 4096, I 1536,
// 256 experts, k 8) took 716 us where the tiles took 478 (392 now).
constexpr int kMxPieceK = 128;
inline __host__ __device__ int mx_pieces(int K) { return (int)(((uint32_t)K + kMxPieceK - 1) / kMxPieceK); }
inline __host__ __device__ size_t mx_code_bytes(int N, int K) {
  return (size_t)(N / 16) * mx_pieces(K) * 1024;
}
inline __host__ __device__ size_t mx_scale_bytes(int N, int K) {
  return (size_t)(N / 16) * ((mx_pieces(K) + 3) / 4) * 256;
}

// Row length of the activation copies in the workspace: whole scale words, the
// rest zeros (codes 0 with scale 0).  Their scale bytes are in the order of the
// tiles' words: block 16S + 4j + g at byte 16S + 4g + j.
inline __host__ __device__ int mx_pad_k(int K) { return (K + 511) & ~511; }

// Arguments of the grouped projections.
struct MxProj {
  const uint16_t* x;       // A16: bf16 rows (x by token, or h by sorted row)
  const uint8_t* q;        // A4: their codes, rows of mx_pad_k(ld_in) values
  const uint8_t* s;        // A4: their scales
  int ld_in;               // row stride of x in values
  const uint8_t* w;        // routed experts' codes [E][mx_code_bytes(N, K)], tiled
  const uint8_t* ws;       // and scales [E][mx_scale_bytes(N, K)]
  const uint8_t* w_sh;     // shared experts'
  const uint8_t* ws_sh;
  int K, K_sh;
  int U, U_sh;             // gate/up: I pairs of rows; down: H rows
  int T, k, P, E, n_shared;
  const int32_t* offsets;      // [E + 1]
  const int32_t* sorted_pair;  // [P] (gate/up)
  void* out;               // gate/up: h bf16; down: y fp32
  int ld_out;
};

// fp32 -> bf16 bits, to nearest even, NaN kept.
__device__ __forceinline__ uint32_t mx_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// h = SiLU(g) * u of N values with the hardware's exp2 and reciprocal: a few
// units of fp32 of relative error, and |g| of them in the exponential, far below
// the rounding to bf16 behind it; 8 instructions instead of about 40.  The
// reciprocal gives 0 where its result is subnormal (g below -87.3), though u may
// bring the product back into bf16's range.  There 1 + e^-g is e^-g in fp32, and
// g u e^g is formed from two factors of e^(g/2): the products leave fp32's range
// only where h does (e^(g/2) is subnormal, in steps of 2^-149, from g = -174.7
// on; the largest u reaches h's smallest step at -187, where it still has 14
// bits).  One test for the N values of a lane's row: gate/up of 4096 tokens (H
// 4096, I 1536, 256 experts, A4) 377 us without any test, 379 so, 384 with a test
// for each value.
template <int N>
__device__ __forceinline__ void mx_silu_mul(const float (&g)[N], const float (&u)[N], float (&h)[N]) {
  float low = g[0];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * g[i]);
    h[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + e) * u[i];
    low = fminf(low, g[i]);
  }
  if (__builtin_expect(low < -64.0f, 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = expf(0.5f * g[i]);
      if (g[i] < -64.0f) h[i] = (g[i] * s) * (u[i] * s);
    }
  }
}

// Scale byte of a block from its largest magnitude (as fp32 bits without the
// sign): floor(log2 a) - 2, held above -127; 255 when a is inf or NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;   // floor(log2 a) + 127 of a normal a
  if (e == 255) return kMxNanScale;
  return e > 2 ? e - 2 : 0;             // a below 2^-124, subnormals and 0: 2^-127
}
// The scale as the conversion instructions take it: fp32 with the byte as its
// exponent field (they read that field alone: 0 is 2^-127, 255 is NaN).
__device__ __forceinline__ float mx_scale_f32(uint32_t byte) {
  return __uint_as_float(byte << 23);
}

// Eight codes (one word, K order) to eight bf16: code * 2^(byte - 127), exact
// for byte >= 1 and below bf16's overflow.
__device__ __forceinline__ mx_bf16x8 mx_word_to_bf16(uint32_t w, float scale) {
  const mx_bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const mx_bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const mx_bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const mx_bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return mx_bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 16 rows x 128 K of codes against 128 K x 16 columns of codes, each lane with
// 32 consecutive codes of its row (lane % 16) and its scale byte in byte J of
// the scale word: exact products, fp32 sums.
template <int J>
__device__ __forceinline__ mx_f32x4 mx_mfma_fp4(mx_u32x4 a, uint32_t sa, mx_u32x4 b, uint32_t sb,
                                                mx_f32x4 c) {
  const mx_i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const mx_i32x8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  // formats 4, 4: E2M1 on both sides
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, J, (int)sa, J, (int)sb);
}

// Keeps v's computation before this point.  A matrix instruction reads all lanes'
// registers whatever the execution mask, but the compiler may move a scaled one
// (and the conversions that feed it) into a branch that only some lanes take,
// if only those use its result: whatever stands before such a branch is kept
// before it by this.
__device__ __forceinline__ void mx_keep(mx_f32x4& v) { __asm__ volatile("" : "+v"(v)); }

// The sorted rows cut into tiles of at most TM rows, experts in order, empty
// experts skipped, by one wave from the offsets alone: lane l owns the experts
// [PER * l, PER * l + PER) (E <= 64 * PER), all its offsets loaded at once, and
// a prefix sum over the lanes numbers the tiles.  Rows are held inside [0, P]
// whatever the table says.
template <int TM, int PER>
struct MxTiles {
  int lo[PER], hi[PER], cnt, pre;   // row ranges; tiles of this lane, and up to it

  __device__ __forceinline__ void load(const int32_t* __restrict__ offsets, int E, int P) {
    const int lane = threadIdx.x & 63;
    int o[PER + 1];
#pragma unroll
    for (int i = 0; i <= PER; ++i) o[i] = offsets[min(lane * PER + i, E)];
    cnt = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      lo[i] = max(o[i], 0);
      hi[i] = max(min(o[i + 1], P), lo[i]);   // past the last expert: empty
      cnt += (hi[i] - lo[i] + TM - 1) / TM;
    }
    pre = cnt;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(pre, d);
      if (lane >= d) pre += v;
    }
  }
  // Tile j: its expert, the expert's rows, and which of its tiles it is; false
  // past the last.
  __device__ __forceinline__ bool find(int j, int& e, int& first, int& end, int& k) const {
    const uint64_t past = __ballot(pre > j);
    if (past == 0) return false;
    const int owner = __builtin_ctzll(past);
    int left = j - (__builtin_amdgcn_readlane(pre, owner) - __builtin_amdgcn_readlane(cnt, owner));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int l = __builtin_amdgcn_readlane(lo[i], owner), h = __builtin_amdgcn_readlane(hi[i], owner);
      const int nt = (h - l + TM - 1) / TM;
      if (left >= 0 && left < nt) {
        e = owner * PER + i;
        first = l;
        end = h;
        k = left;
      }
      left -= nt;
    }
    return true;
  }
  // The same as rows [r0, r1) of full tiles.
  __device__ __forceinline__ bool find(int j, int& e, int& r0, int& r1) const {
    int l, h, k;
    if (!find(j, e, l, h, k)) return false;
    r0 = l + k * TM;
    r1 = min(h, r0 + TM);
    return true;
  }
};

// R rows of C values (row stride ld) to rows of CP >= C values, zeros behind
// the C: codes [R][CP/2] and scale bytes [R][CP/32]; words: the scale bytes in
// the order of the tiles' words (CP % 512 == 0).
hipError_t launch_mx_quant(const void* src, int is_f32, int R, int C, int ld, uint8_t* q,
                           uint8_t* s, int CP, bool words, hipStream_t st);
// n matrices [N][K] of plain rows to tiled ones.
hipError_t launch_mx_tile(const uint8_t* codes, const uint8_t* scales, int n, int N, int K,
                          uint8_t* dst_codes, uint8_t* dst_scales, hipStream_t st);
hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* s, int R, int C, void* dst,
                             int is_f32, int ld, hipStream_t st);
// R bf16 rows of C values (stride ld, 16-byte aligned) to rows of CP, zeros
// behind the C.
hipError_t launch_mx_pad_rows(const uint16_t* src, int R, int C, int ld, uint16_t* dst, int CP,
                              hipStream_t st);
// Grouped projections; mode 0: gate/up with SiLU*mul to h, 1: down to y.
// Tiles of 16 rows, K split over the workgroup's waves:
long long mx_rows16_grid(const MxProj& a, int mode);   // its workgroups, at most kMxMaxGrid
hipError_t launch_mx_rows16(const MxProj& a, int mode, int act4, hipStream_t st);
// The same for a few tokens with their routing and sort in the launch:
bool mx_route_gateup_ok(int T, int k, int E, int H);
hipError_t launch_mx_route_gateup(const MxProj& a, int act4, const float* logits, int renorm,
                                  int32_t* ids, float* w, int32_t* counts, int32_t* offsets,
                                  int32_t* sorted_pair, int32_t* pair_pos, hipStream_t st);
// Tiles of up to 160 rows (A16: rows of whole steps, K % 256 == 0 or a padded copy):
bool mx_gemm_ok(const MxProj& a, int mode, int act4);
int mx_gemm_tile_rows(const MxProj& a, int mode, int act4);   // 144 or 160
hipError_t launch_mx_gemm(const MxProj& a, int mode, int act4, hipStream_t st);

}  // namespace moe
