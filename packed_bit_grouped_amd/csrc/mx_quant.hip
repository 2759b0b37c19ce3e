// Rows to MXFP4 and back.
//
// quantise: a block of 32 values v with a = max|v| is held as
// q_i = RNE_e2m1(v_i / s), |q_i| <= 6, s = 2^(floor(log2 a) - 2): the largest
// magnitude lands in [4, 8), whose top (6, 8) is rounded to 6.  Dividing by a
// power of two is exact, so the only rounding is the one to the code, done by
// the conversion instruction (all 2^16 bf16 inputs and the codes' midpoints
// were compared with the definition at 12 scales).  Bound by memory: 2 or 4
// bytes read and 0.53 written per value, no reuse.  Measured (kernel trace, medians
// of 30): 201 M fp32 weights to codes 206 us (4.4 TB/s read and written together),
// back to bf16 85 us (6.0 TB/s), to fp32 248 us (3.7 TB/s, 7/8 of it written); 4096
// rows of 4096 bf16 values 9.4 us and 8.8 back (4.5 and 4.8 TB/s, partly the cache),
// to fp32 15.4; 12 rows of 2048 2.5 us, the launch.
#include "mx_common.h"

namespace moe {

namespace {

constexpr int kQuantThreads = 256;

// Four lanes share a block, eight values each: one 16-byte (bf16) or two
// 16-byte loads (fp32) per lane, the maximum by two DPP steps, one 4-byte
// store of codes per lane.  VEC: every row is 16-byte aligned; else the values
// are loaded one by one.  64-bit indices: a bank of experts passes 2^32 bytes.
template <bool F32, bool VEC>
__global__ __launch_bounds__(kQuantThreads) void mx_quant_kernel(
    const void* __restrict__ src, int R, int C8, int ld, uint8_t* __restrict__ q,
    uint8_t* __restrict__ s, int CP8, int words) {
  const long long n = (long long)R * CP8;   // eights of values, the padding's too
  for (long long i = (long long)blockIdx.x * kQuantThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kQuantThreads) {
    const long long r = i / CP8;
    const int c = (int)(i - r * CP8);   // CP8, C8: multiples of 4, a block's four lanes stay together
    float v[8];
    if (c >= C8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    } else if (F32) {
      const float* p = static_cast<const float*>(src) + r * ld + c * 8;
      if (VEC) {
        const mx_f32x4 a = reinterpret_cast<const mx_f32x4*>(p)[0];
        const mx_f32x4 b = reinterpret_cast<const mx_f32x4*>(p)[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p[j];
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(src) + r * ld + c * 8;
      if (VEC) {
        const mx_u32x4 a = *reinterpret_cast<const mx_u32x4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = __uint_as_float(a[j] << 16);
          v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = bf16_to_f32(p[j]);
      }
    }
    // magnitudes compare as integers; inf and NaN come out on top
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)dpp_i<kDppXor1>((int)m, (int)m));
    m = max(m, (uint32_t)dpp_i<kDppXor2>((int)m, (int)m));
    const uint32_t sb = mx_scale_byte(m);
    uint32_t w = 0;
    if (sb != kMxNanScale) {   // such a block holds codes 0: the scale says it all
      const float sc = mx_scale_f32(sb);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
    }
    reinterpret_cast<uint32_t*>(q)[i] = w;
    if ((c & 3) == 0) {
      long long b = i >> 2;   // block; words: bytes 4j + g of sixteen change places with 4g + j
      if (words) b = (b & ~15LL) | ((b & 3) << 2) | ((b >> 2) & 3);
      s[b] = (uint8_t)sb;
    }
  }
}

// Eight codes per lane to 16 (bf16) or 32 (fp32) bytes.  A value beyond the
// type's range becomes inf, one of a block marked 255 NaN.
template <bool F32, bool VEC>
__global__ __launch_bounds__(kQuantThreads) void mx_dequant_kernel(
    const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int R, int C8,
    void* __restrict__ dst, int ld) {
  const long long n = (long long)R * C8;
  for (long long i = (long long)blockIdx.x * kQuantThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kQuantThreads) {
    const long long r = i / C8;
    const int c = (int)(i - r * C8);
    const uint32_t w = reinterpret_cast<const uint32_t*>(q)[i];   // rows are contiguous
    const float sc = mx_scale_f32(s[i >> 2]);
    if (F32) {
      float* p = static_cast<float*>(dst) + r * ld + c * 8;
      float v[8];
#define MX_PAIR(j)                                                               \
  {                                                                              \
    const auto t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, j);           \
    v[2 * j] = t[0];                                                             \
    v[2 * j + 1] = t[1];                                                         \
  }
      MX_PAIR(0) MX_PAIR(1) MX_PAIR(2) MX_PAIR(3)
#undef MX_PAIR
      if (VEC) {
        reinterpret_cast<mx_f32x4*>(p)[0] = mx_f32x4{v[0], v[1], v[2], v[3]};
        reinterpret_cast<mx_f32x4*>(p)[1] = mx_f32x4{v[4], v[5], v[6], v[7]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = v[j];
      }
    } else {
      uint16_t* p = static_cast<uint16_t*>(dst) + r * ld + c * 8;
      const mx_u32x4 o = __builtin_bit_cast(mx_u32x4, mx_word_to_bf16(w, sc));
      if (VEC) {
        *reinterpret_cast<mx_u32x4*>(p) = o;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

// bf16 rows to longer ones, 16 bytes per lane.
__global__ __launch_bounds__(kQuantThreads) void mx_pad_kernel(const uint16_t* __restrict__ src,
                                                               int R, int C8, int ld,
                                                               uint16_t* __restrict__ dst,
                                                               int CP8) {
  const long long n = (long long)R * CP8;
  for (long long i = (long long)blockIdx.x * kQuantThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kQuantThreads) {
    const long long r = i / CP8;
    const int c = (int)(i - r * CP8);
    const mx_u32x4 zero = {0, 0, 0, 0};
    reinterpret_cast<mx_u32x4*>(dst)[i] =
        c < C8 ? *reinterpret_cast<const mx_u32x4*>(src + r * ld + c * 8) : zero;
  }
}

// One workgroup wave per piece: lane (c, g) copies block 4s + g of its row; the
// wave of a word's first piece gathers the four scale bytes of its lanes.
__global__ __launch_bounds__(kQuantThreads) void mx_tile_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long n_pieces,
    int pieces, int nblk, uint8_t* __restrict__ dst, uint8_t* __restrict__ dst_s) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  for (long long p = (long long)blockIdx.x * (kQuantThreads / 64) + (threadIdx.x >> 6);
       p < n_pieces; p += (long long)gridDim.x * (kQuantThreads / 64)) {
    const long long rb = p / pieces;   // 16-row block, over all matrices
    const int s = (int)(p - rb * pieces);
    const long long row = rb * 16 + c;
    const int b = 4 * s + g;
    const mx_u32x4 zero = {0, 0, 0, 0};
    reinterpret_cast<mx_u32x4*>(dst)[p * 64 + lane] =
        b < nblk ? *reinterpret_cast<const mx_u32x4*>(codes + (row * nblk + b) * 16) : zero;
    if ((s & 3) == 0) {
      uint32_t w = 0;
      for (int j = 0; j < 4; ++j)
        if (b + 4 * j < nblk) w |= (uint32_t)scales[row * nblk + b + 4 * j] << (8 * j);
      reinterpret_cast<uint32_t*>(dst_s)[(rb * ((pieces + 3) / 4) + (s >> 2)) * 64 + lane] = w;
    }
  }
}

int quant_blocks(long long eights) {
  const long long b = (eights + kQuantThreads - 1) / kQuantThreads;
  return (int)(b < 16384 ? b : 16384);
}

bool rows_aligned(const void* p, int ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) | ((uintptr_t)ld * elem)) % 16 == 0;
}

}  // namespace

hipError_t launch_mx_quant(const void* src, int is_f32, int R, int C, int ld, uint8_t* q,
                           uint8_t* s, int CP, bool words, hipStream_t st) {
  const int blocks = quant_blocks((long long)R * (CP / 8));
  const bool vec = rows_aligned(src, ld, is_f32 ? 4 : 2);
  auto k = is_f32 ? (vec ? mx_quant_kernel<true, true> : mx_quant_kernel<true, false>)
                  : (vec ? mx_quant_kernel<false, true> : mx_quant_kernel<false, false>);
  k<<<blocks, kQuantThreads, 0, st>>>(src, R, C / 8, ld, q, s, CP / 8, words);
  return hipGetLastError();
}

hipError_t launch_mx_tile(const uint8_t* codes, const uint8_t* scales, int n, int N, int K,
                          uint8_t* dst_codes, uint8_t* dst_scales, hipStream_t st) {
  const int pieces = mx_pieces(K);
  const long long n_pieces = (long long)n * (N / 16) * pieces;
  mx_tile_kernel<<<quant_blocks(n_pieces * 64), kQuantThreads, 0, st>>>(
      codes, scales, n_pieces, pieces, K / kMxBlock, dst_codes, dst_scales);
  return hipGetLastError();
}

hipError_t launch_mx_pad_rows(const uint16_t* src, int R, int C, int ld, uint16_t* dst, int CP,
                              hipStream_t st) {
  mx_pad_kernel<<<quant_blocks((long long)R * (CP / 8)), kQuantThreads, 0, st>>>(src, R, C / 8, ld,
                                                                                 dst, CP / 8);
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* s, int R, int C, void* dst,
                             int is_f32, int ld, hipStream_t st) {
  const int blocks = quant_blocks((long long)R * (C / 8));
  const bool vec = rows_aligned(dst, ld, is_f32 ? 4 : 2);
  auto k = is_f32 ? (vec ? mx_dequant_kernel<true, true> : mx_dequant_kernel<true, false>)
                  : (vec ? mx_dequant_kernel<false, true> : mx_dequant_kernel<false, false>);
  k<<<blocks, kQuantThreads, 0, st>>>(q, s, R, C / 8, dst, ld);
  return hipGetLastError();
}

}  // namespace moe
