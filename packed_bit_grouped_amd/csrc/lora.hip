// Low-rank adapters of many requests beside the experts' projections.
//
// Build log "Two 96 GB Ascend cards run Qwen3.8 Flash-Next", sections "Keep
// low-bit weights packed, do the work on the NPU" (expert weights stay packed:
// adapters cannot be merged into them, so they run beside the projections all
// requests share) and "Optimise serving, not isolated kernels" (one batch of
// many requests).
//
// A row is a (token, expert) pair in sorted order or a shared expert's token.
// Its adapter's pair of matrices for that expert is (A, B):
//   shrink  v = scale A in       (in: x of the token, or the row's h)
//   expand  gate/up: h = SiLU(g + Bg vg) * (u + Bu vu)
//           down:    out[t] = base[t] + sum over the token's rows of w B v
// v is held in fp32 between the two.  All products run on the matrix cores in
// bf16 with fp32 sums: x, A and B are bf16, and an fp32 operand (v; h of 8-bit
// activations) goes in as three bf16 numbers that sum to it exactly, so nothing
// is rounded on the way.  A few tokens' products are bound by the latency of
// sorted pair -> token -> table entry -> matrix, a decode batch by reading each
// (adapter, expert)'s matrices once, a prefill chunk by g, u and h.
//
// Windows.  A workgroup looks at a window of 16 or 64 neighbouring rows and
// splits it into groups of rows of one (adapter, expert); each group runs as
// fragments of 16 rows against that pair's matrices.  Sorted rows of a prompt
// that share an expert are neighbours, so a window holds few groups; a decode
// batch has up to one per row, and there a workgroup takes one group.
#include <type_traits>

#include "lora_common.h"
#include "mx_common.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;

typedef mx_f32x4 f32x4;
typedef mx_u32x4 u32x4;
typedef mx_bf16x8 bf16x8;

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// fp32 as three bf16 numbers that sum to it: cut off, cut off, the rest (8 bits
// at most).  Infinities and NaN are in the first alone.
__device__ __forceinline__ void split3(float f, uint32_t& a, uint32_t& b, uint32_t& c) {
  uint32_t u = __float_as_uint(f);
  const uint32_t mag = u & 0x7FFFFFFFu;
  if (mag > 0x7F800000u) u |= 0x00400000u;   // a NaN stays one
  a = u >> 16;
  const float r = mag >= 0x7F800000u ? 0.0f : f - __uint_as_float(u & 0xFFFF0000u);
  b = __float_as_uint(r) >> 16;
  c = __float_as_uint(r - __uint_as_float(__float_as_uint(r) & 0xFFFF0000u)) >> 16;
}
__device__ __forceinline__ void split3(const float (&f)[8], u32x4 (&s)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a0, b0, c0, a1, b1, c1;
    split3(f[2 * i], a0, b0, c0);
    split3(f[2 * i + 1], a1, b1, c1);
    s[0][i] = a0 | (a1 << 16);
    s[1][i] = b0 | (b1 << 16);
    s[2][i] = c0 | (c1 << 16);
  }
}

// Keys of rows without an adapter (routed and shared ones differ in width), and
// of places without a row.
constexpr int kBaseShared = -1, kBaseRouted = -2, kNoRow = -3;

// A lane's row of the window: its token, width and number in the adapters' table.
struct Row {
  int token, key;
};
__device__ __forceinline__ Row window_row(const LoraArgs& a, int r, bool in) {
  Row w = {0, kNoRow};
  if (!in || r >= a.R) return w;
  int e;
  if (r < a.P) {
    const int p = a.sorted_pair[r];
    if ((unsigned)p >= (unsigned)a.P) return w;
    e = a.topk_ids[p];
    if ((unsigned)e >= (unsigned)a.E) return w;
    w.token = p / a.k;
  } else {
    const int q = r - a.P, s = q / a.T;
    w.token = q - s * a.T;
    e = a.E + s;
  }
  const int d = a.adapter[w.token];
  w.key = (unsigned)d < (unsigned)a.n ? d * (a.E + a.n_shared) + e
          : e < a.E                   ? kBaseRouted
                                      : kBaseShared;
  return w;
}

// The pair of matrices of a table entry; rank 0 where there is none.
struct Pair {
  const uint16_t* a;
  const uint16_t* b;
  int rank;
  float scale;
};
__device__ __forceinline__ Pair pair_of(const LoraArgs& a, int key, int N, int K) {
  Pair p = {nullptr, nullptr, 0, 0.0f};
  if (key < 0) return p;
  const moe_lora d = a.table[key];
  if (d.rank == 0) return p;
  const bool ok = d.rank > 0 && d.rank <= a.max_rank && d.rank % 8 == 0 && d.N == N && d.K == K &&
                  d.a != nullptr && d.b != nullptr &&
                  ((reinterpret_cast<uintptr_t>(d.a) | reinterpret_cast<uintptr_t>(d.b)) & 15) == 0;
  if (!ok) {
    if (threadIdx.x == 0) atomicOr(a.err, 1);
    return p;
  }
  p.a = d.a;
  p.b = d.b;
  p.rank = d.rank;
  p.scale = d.scale;
  return p;
}

// The window's groups in turn, the same in every wave: the rows (bits) and key
// of one; `slot` of `slots` workgroups takes every slots-th.
struct Groups {
  uint64_t todo;
  int ord;
  __device__ __forceinline__ void init(int key, int from) {
    todo = __ballot(key >= from);
    ord = 0;
  }
  __device__ __forceinline__ bool next(int key, int slot, int slots, uint64_t& rows, int& k) {
    while (todo) {
      k = __builtin_amdgcn_readlane(key, __builtin_ctzll(todo));
      rows = __ballot(key == k);
      todo &= ~rows;
      if (ord++ % slots == slot) return true;
    }
    return false;
  }
};

// The n-th set lanes of `rows` in LDS (a wave's own 64 words), n from 0.
__device__ __forceinline__ int list_rows(uint64_t rows, int* list) {
  const int lane = threadIdx.x & 63;
  __builtin_amdgcn_wave_barrier();
  if ((rows >> lane) & 1) list[__popcll(rows & ((1ull << lane) - 1))] = lane;
  __builtin_amdgcn_wave_barrier();
  return __popcll(rows);
}

// ---------------------------------------------------------------------
// shrink: v[row][j] = scale sum_K A[j][K] in[row][K]
//
// The workgroup's waves (and, for few rows, `splits` workgroups) share K; a
// wave's fragments go from memory to registers, 16 bytes per lane, since every
// byte of A and of the rows is read by one wave only.
template <int NF, int CT, bool F32>
__device__ __forceinline__ void shrink_group(const LoraArgs& a, const Pair& p, int K, int C, int ct0,
                                             int split, const void* const (&rows)[NF],
                                             const int (&row)[NF], int n, float* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int steps = K >> 5, workers = kWaves * a.splits, me = split * kWaves + wave;
  const int per = (steps + workers - 1) / workers;
  const int s0 = min(me * per, steps), s1 = min(s0 + per, steps);
  const uint16_t* pa[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j)   // columns past the last are computed and dropped
    pa[j] = p.a + (size_t)min(16 * (ct0 + j) + c, C - 1) * K + 8 * g;
  f32x4 acc[NF][CT];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[f][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = F32 ? 2 : 4;
  int s = s0;
  auto step = [&](int n_st) {
    u32x4 wa[U][CT], wx[U][NF][F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i >= n_st) break;
#pragma unroll
      for (int j = 0; j < CT; ++j)
        wa[i][j] = *reinterpret_cast<const u32x4*>(pa[j] + (size_t)(s + i) * 32);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if constexpr (F32) {
          const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(rows[f]) +
                                                          (size_t)(s + i) * 32 + 8 * g);
          wx[i][f][0] = q[0];
          wx[i][f][1] = q[1];
        } else {
          wx[i][f][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(rows[f]) +
                                                        (size_t)(s + i) * 32 + 8 * g);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (i >= n_st) break;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if constexpr (F32) {
          float t[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] = __uint_as_float(wx[i][f][e / 4][e % 4]);
          u32x4 sp[3];
          split3(t, sp);
#pragma unroll
          for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int e = 0; e < 3; ++e) acc[f][j] = mfma(wa[i][j], sp[e], acc[f][j]);
        } else {
#pragma unroll
          for (int j = 0; j < CT; ++j) acc[f][j] = mfma(wa[i][j], wx[i][f][0], acc[f][j]);
        }
      }
    }
  };
  for (; s + U <= s1; s += U) step(U);
  for (; s < s1; ++s) step(1);

  // the waves' parts meet: wave w adds those of tiles w, w + 4, ...
  __syncthreads();   // the last group's parts have been read
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < CT; ++j)
      *reinterpret_cast<f32x4*>(red + ((wave * NF * CT + f * CT + j) * 64 + lane) * 4) = acc[f][j];
  __syncthreads();
  const int VL = a.halves * a.max_rank;
  float* v = a.v + (size_t)split * a.R * VL;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      if ((f * CT + j) % kWaves != wave) continue;
      f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        t += *reinterpret_cast<const f32x4*>(red + ((w * NF * CT + f * CT + j) * 64 + lane) * 4);
      const int col = 16 * (ct0 + j) + 4 * g;
      if (16 * f + c < n && col < C)
        *reinterpret_cast<f32x4*>(v + (size_t)row[f] * VL + col) = t * p.scale;
    }
}

template <int NW, int CT, bool F32>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(LoraArgs a, int slots) {
  constexpr int NFM = NW / 16;
  __shared__ int list[kWaves][64];
  __shared__ __align__(16) float red[kWaves * NFM * CT * 256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15;
  const int win = blockIdx.x / slots, slot = blockIdx.x - win * slots;
  const int ct0 = blockIdx.y * CT, split = blockIdx.z;
  const int r0 = win * NW;
  const Row w = window_row(a, r0 + lane, lane < NW);
  Groups gr;
  gr.init(w.key, 0);
  uint64_t rows;
  int key;
  while (gr.next(w.key, slot, slots, rows, key)) {
    const int e = key % (a.E + a.n_shared);
    const int width = e < a.E ? a.I : a.I_sh;
    const int K = a.halves == 2 ? a.H : width, N = a.halves == 2 ? 2 * width : a.H;
    const Pair p = pair_of(a, key, N, K);
    const int C = a.halves * p.rank;
    if (16 * ct0 >= C) continue;   // no adapter, or a lower rank than the largest
    const int n = list_rows(rows, list[wave]);
    auto run = [&](auto nf) {
      constexpr int NF = decltype(nf)::value;
      const void* src[NF];
      int row[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        // fragments' rows past the group's end are computed and dropped
        const int l = list[wave][min(16 * f + c, n - 1)];
        row[f] = r0 + l;
        const int token = __shfl(w.token, l);
        if (a.halves == 2) src[f] = static_cast<const uint16_t*>(a.in) + (size_t)token * a.H;
        else if (F32) src[f] = static_cast<const float*>(a.in) + (size_t)row[f] * a.ld_h;
        else src[f] = static_cast<const uint16_t*>(a.in) + (size_t)row[f] * a.ld_h;
      }
      shrink_group<NF, CT, F32>(a, p, K, C, ct0, split, src, row, n, red);
    };
    if constexpr (NFM == 1) {
      run(std::integral_constant<int, 1>{});
    } else {
      if (n <= 16) run(std::integral_constant<int, 1>{});
      else if (n <= 32) run(std::integral_constant<int, 2>{});
      else run(std::integral_constant<int, 4>{});
    }
  }
}

// The row's v from j on, 8 values: the parts of K added in order.
__device__ __forceinline__ void load_v(const LoraArgs& a, size_t row, int j, float (&f)[8]) {
  const int VL = a.halves * a.max_rank;
  f32x4 lo = {0.0f, 0.0f, 0.0f, 0.0f}, hi = lo;
  for (int s = 0; s < a.splits; ++s) {
    const f32x4* q = reinterpret_cast<const f32x4*>(a.v + ((size_t)s * a.R + row) * VL + j);
    lo += q[0];
    hi += q[1];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = lo[i];
    f[4 + i] = hi[i];
  }
}

// SiLU(g) * u in fp32 for outputs in fp32: where e^-g leaves the type, the
// product of two factors of e^(g/2) does not until the result does.
__device__ __forceinline__ float silu_mul_wide(float g, float u) {
  if (g > -64.0f) return g / (1.0f + expf(-g)) * u;
  const float s = expf(0.5f * g);
  return (g * s) * (u * s);
}

// ---------------------------------------------------------------------
// expand, gate/up.  A wave owns 32 columns: two fragments of gate rows of B and
// two of up rows, dealt so that a lane ends with 8 neighbouring columns of its
// row: whole 16-byte loads of g and u and stores of h.
template <int NF>
__device__ __forceinline__ void expand_group(const LoraArgs& a, const Pair& p, int width, int i0,
                                             const int (&row)[NF], int n) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int col = i0 + 8 * g;
  f32x4 gu[NF][4];   // gate, gate, up, up
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const float* q = a.gu + (size_t)row[f] * 2 * a.ld_h + col;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        gu[f][2 * h + i] = *reinterpret_cast<const f32x4*>(q + h * a.ld_h + 4 * i);
  }
  f32x4 acc[NF][4];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[f][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int k0 = 0; k0 < p.rank; k0 += 32) {
    const int j = k0 + 8 * g;
    const bool in = j < p.rank;
    u32x4 b[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int br = h * width + i0 + 8 * (c >> 2) + 4 * i + (c & 3);
        b[2 * h + i] =
            in ? *reinterpret_cast<const u32x4*>(p.b + (size_t)br * p.rank + j) : zero;
      }
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float t[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (in) load_v(a, row[f], h * p.rank + j, t);
        u32x4 sp[3];
        split3(t, sp);
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          acc[f][2 * h] = mfma(b[2 * h], sp[e], acc[f][2 * h]);
          acc[f][2 * h + 1] = mfma(b[2 * h + 1], sp[e], acc[f][2 * h + 1]);
        }
      }
  }
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) mx_keep(acc[f][i]);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    float gv[8], uv[8], hv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gv[i] = gu[f][i / 4][i % 4] + acc[f][i / 4][i % 4];
      uv[i] = gu[f][2 + i / 4][i % 4] + acc[f][2 + i / 4][i % 4];
    }
    if (16 * f + c >= n) continue;
    const size_t o = (size_t)row[f] * a.ld_h + col;
    if (a.out_f32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[i] = silu_mul_wide(gv[i], uv[i]);
      float* h = static_cast<float*>(a.out) + o;
      *reinterpret_cast<f32x4*>(h) = f32x4{hv[0], hv[1], hv[2], hv[3]};
      *reinterpret_cast<f32x4*>(h + 4) = f32x4{hv[4], hv[5], hv[6], hv[7]};
    } else {
      mx_silu_mul(gv, uv, hv);
      u32x4 s;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = mx_bf16(hv[2 * i]) | (mx_bf16(hv[2 * i + 1]) << 16);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + o) = s;
    }
  }
}

template <int NW>
__global__ __launch_bounds__(kThreads) void lora_expand_gateup_kernel(LoraArgs a, int slots) {
  __shared__ int list[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15;
  const int win = blockIdx.x / slots, slot = blockIdx.x - win * slots;
  const int i0 = (blockIdx.y * kWaves + wave) * 32;
  const int r0 = win * NW;
  const Row w = window_row(a, r0 + lane, lane < NW);
  Groups gr;
  gr.init(w.key, kBaseRouted);
  uint64_t rows;
  int key;
  while (gr.next(w.key, slot, slots, rows, key)) {
    const bool sh = key >= 0 ? key % (a.E + a.n_shared) >= a.E : key == kBaseShared;
    const int width = sh ? a.I_sh : a.I;
    const Pair p = pair_of(a, key, 2 * width, a.H);
    if (i0 >= width) continue;
    const int n = list_rows(rows, list[wave]);
    auto run = [&](auto nf) {
      constexpr int NF = decltype(nf)::value;
      int row[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) row[f] = r0 + list[wave][min(16 * f + c, n - 1)];
      expand_group<NF>(a, p, width, i0, row, n);
    };
    if constexpr (NW == 16) {
      run(std::integral_constant<int, 1>{});
    } else {
      if (n <= 16) run(std::integral_constant<int, 1>{});
      else if (n <= 32) run(std::integral_constant<int, 2>{});
      else run(std::integral_constant<int, 4>{});
    }
  }
}

// ---------------------------------------------------------------------
// expand, down, by tokens: out[t][n] = base + sum over the token's rows of
// w B v.  The rows' ranks form one long axis, in pieces of 8 that each have a
// matrix of their own; a matrix product over 32 of it takes four pieces, whatever
// rows they are of.  The other operand's columns 0, 1, 2 are the three parts of w v.
constexpr int kPieces = 128;   // of a pass

__global__ __launch_bounds__(kThreads) void lora_expand_down_kernel(LoraArgs a) {
  __shared__ const uint16_t* src[kPieces];   // B + the piece's first rank
  __shared__ int stride[kPieces];            // the matrix's rank, 0: nothing
  __shared__ __align__(16) u32x4 vs[3][kPieces];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int t = blockIdx.x;
  const int n0 = (blockIdx.y * kWaves + wave) * 16;
  const int per = a.max_rank / 8;            // pieces of a row
  const int choices = a.k + a.n_shared;
  const int total = choices * per;
  const int d = a.adapter[t];
  const bool has = (unsigned)d < (unsigned)a.n;
  const int nc = min(n0 + c, a.H - 1);
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int q0 = 0; has && q0 < total; q0 += kPieces) {
    const int m = min(total - q0, kPieces);
    if (q0) __syncthreads();
    if (tid < kPieces) {
      const int q = q0 + tid, ch = q / per, j = 8 * (q - ch * per);
      const uint16_t* sp = nullptr;
      int rank = 0;
      u32x4 parts[3] = {zero, zero, zero};
      if (tid < m) {
        int row, e;
        float wt;
        if (ch < a.k) {
          row = a.pair_pos[t * a.k + ch];
          e = a.topk_ids[t * a.k + ch];
          wt = a.topk_w[t * a.k + ch];
        } else {
          const int s = ch - a.k;
          row = a.P + s * a.T + t;
          e = a.E + s;
          wt = a.shared_gate ? shared_gate_weight(a.shared_gate[(size_t)t * a.n_shared + s]) : 1.0f;
        }
        const bool ok = (unsigned)row < (unsigned)a.R && (unsigned)e < (unsigned)(a.E + a.n_shared);
        if (ok) {
          const int width = e < a.E ? a.I : a.I_sh;
          const moe_lora* dp = a.table + (size_t)d * (a.E + a.n_shared) + e;
          const Pair p = pair_of(a, (int)(dp - a.table), a.H, width);
          if (j < p.rank) {
            rank = p.rank;
            sp = p.b + j;
            float f[8];
            load_v(a, row, j, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= wt;
            split3(f, parts);
          }
        }
      }
      src[tid] = sp;
      stride[tid] = rank;
#pragma unroll
      for (int i = 0; i < 3; ++i) vs[i][tid] = parts[i];
    }
    __syncthreads();
    const int groups = (m + 3) / 4;
#pragma unroll 4
    for (int s = 0; s < groups; ++s) {
      const int q = 4 * s + g, rank = stride[q];
      const u32x4 b =
          rank ? *reinterpret_cast<const u32x4*>(src[q] + (size_t)nc * rank) : zero;
      const u32x4 v = c < 3 ? vs[c][q] : zero;
      acc = mfma(b, v, acc);
    }
  }
  // the three parts' sums: lanes 1 and 2 of the 16 to lane 0
  f32x4 sum;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    sum[i] = acc[i] + (__shfl(acc[i], lane + 1) + __shfl(acc[i], lane + 2));
  const int n = n0 + 4 * g;
  if (c != 0 || n >= a.H) return;
  const size_t o = (size_t)t * a.H + n;
  const f32x4 b = *reinterpret_cast<const f32x4*>(a.base + o);
  sum += b;
  if (a.out_f32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o) = sum;
  } else {
    uint2 s;
    s.x = mx_bf16(sum[0]) | (mx_bf16(sum[1]) << 16);
    s.y = mx_bf16(sum[2]) | (mx_bf16(sum[3]) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = s;
  }
}

template <int CT>
hipError_t launch_shrink(const LoraArgs& a, hipStream_t st) {
  const int tiles = (a.halves * a.max_rank + 15) / 16;
  const int rows = a.large ? kLoraLargeRows : kLoraSmallRows, slots = a.large ? 1 : kLoraSmallRows;
  const dim3 grid((a.R + rows - 1) / rows * slots, (tiles + CT - 1) / CT, a.splits);
  if (a.large) {
    if (a.in_f32) lora_shrink_kernel<kLoraLargeRows, CT, true><<<grid, kThreads, 0, st>>>(a, slots);
    else lora_shrink_kernel<kLoraLargeRows, CT, false><<<grid, kThreads, 0, st>>>(a, slots);
  } else {
    if (a.in_f32) lora_shrink_kernel<kLoraSmallRows, CT, true><<<grid, kThreads, 0, st>>>(a, slots);
    else lora_shrink_kernel<kLoraSmallRows, CT, false><<<grid, kThreads, 0, st>>>(a, slots);
  }
  return hipGetLastError();
}

hipError_t shrink(const LoraArgs& a, hipStream_t st) {
  const int tiles = (a.halves * a.max_rank + 15) / 16;
  if (!a.large || tiles == 1) return launch_shrink<1>(a, st);
  return launch_shrink<2>(a, st);
}

}  // namespace

void lora_plan(int R, int halves, int max_rank, int& splits, bool& large) {
  large = R > 2048;
  splits = 1;
  const int tiles = (halves * max_rank + 15) / 16;
  while (!large && splits < kLoraMaxSplits && (long long)R * tiles * splits * 2 <= 512) splits *= 2;
}

hipError_t launch_lora_gateup(const LoraArgs& a, hipStream_t st) {
  hipError_t e = shrink(a, st);
  if (e != hipSuccess) return e;
  const int rows = a.large ? kLoraLargeRows : kLoraSmallRows, slots = a.large ? 1 : kLoraSmallRows;
  const dim3 grid((a.R + rows - 1) / rows * slots, (a.ld_h + 32 * kWaves - 1) / (32 * kWaves));
  if (a.large) lora_expand_gateup_kernel<kLoraLargeRows><<<grid, kThreads, 0, st>>>(a, slots);
  else lora_expand_gateup_kernel<kLoraSmallRows><<<grid, kThreads, 0, st>>>(a, slots);
  return hipGetLastError();
}

hipError_t launch_lora_down(const LoraArgs& a, hipStream_t st) {
  hipError_t e = shrink(a, st);
  if (e != hipSuccess) return e;
  const dim3 grid(a.T, (a.H + 16 * kWaves - 1) / (16 * kWaves));
  lora_expand_down_kernel<<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
