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
// A and B are tiled (moe_lora_tile): a fragment's 64 loads of 16 bytes are
// neighbours, a kilobyte together.  From plain rows every lane's load is a cache
// access of its own: one token's A of 131 KB took 4.5 us in one compute unit.
//
// Windows.  The rows of a window of neighbours are split into groups of one
// (adapter, expert); each group runs as fragments of 16 rows against that pair's
// matrices.  Sorted rows of a prompt that share an expert are neighbours, so a
// window of 256 holds few groups; a decode batch has up to one per row, and there
// a workgroup takes one group of a window of 16, from K to h.
//
// What the calls measured (H 2048, I 512, 256 experts and a shared one, 8 a token,
// rank 16; in a graph): one token gate/up 9.7 us, down 7.9; 64 tokens over 32
// adapters 26 and 14 (the matrices at 3.5 and 3.2 TB/s); 4096 tokens over 4
// adapters 110 (3.4 TB/s of what has to be moved) and 116 (1.5); with h in fp32 125
// and 130.
#include <algorithm>
#include <cmath>
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
// at most; below 2^-133, bf16's smallest step, it is dropped).  Infinities and NaN
// are in the first alone.
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

// The i-th of n workgroups as a place in order such that an XCD's (i mod 8) are neighbours.
__device__ __forceinline__ int xcd_order(int i, int n) {
  const int x = i & 7, per = n >> 3, more = n & 7;
  return x * per + min(x, more) + (i >> 3);
}

// A lane's row of the window: its token and number in the adapters' table, and
// (WEIGHT) what its output joins the token's with.
struct Row {
  int token, key;
  float weight;
};
template <bool WEIGHT>
__device__ __forceinline__ Row window_row(const LoraArgs& a, int r, int p, const int* topk_ids,
                                          const int* adapter) {
  Row w = {0, kNoRow, 1.0f};
  if (r >= a.R) return w;
  int e;
  if (r < a.P) {
    if ((unsigned)p >= (unsigned)a.P) return w;
    e = topk_ids[p];
    const int back = WEIGHT ? a.pair_pos[p] : r;   // -1: the pair adds nothing
    if ((unsigned)e >= (unsigned)a.E || back != r) return w;
    w.token = p / a.k;
    if (WEIGHT) w.weight = a.topk_w[p];
  } else {
    const int q = r - a.P, s = q / a.T;
    w.token = q - s * a.T;
    e = a.E + s;
    if (WEIGHT && a.shared_gate)
      w.weight = shared_gate_weight(a.shared_gate[(size_t)w.token * a.n_shared + s]);
  }
  const int d = adapter[w.token];
  w.key = (unsigned)d < (unsigned)a.n ? d * (a.E + a.n_shared) + e
          : e < a.E                   ? kBaseRouted
                                      : kBaseShared;
  return w;
}

template <bool WEIGHT>
__device__ __forceinline__ Row window_row(const LoraArgs& a, int r) {
  return window_row<WEIGHT>(a, r, r < a.P ? a.sorted_pair[r] : 0, a.topk_ids, a.adapter);
}

// Columns of h of a key's rows.
__device__ __forceinline__ bool width_is_shared(const LoraArgs& a, int key) {
  return key >= 0 ? key % (a.E + a.n_shared) >= a.E : key == kBaseShared;
}
__device__ __forceinline__ int width_of(const LoraArgs& a, int key) {
  return width_is_shared(a, key) ? a.I_sh : a.I;
}

// The pair of matrices of a table entry; rank 0 where there is none.
struct Pair {
  const uint16_t* a;
  const uint16_t* b;
  int rank;
  float scale;
};
__device__ __forceinline__ bool entry_ok(const LoraArgs& a, const moe_lora& d, int N, int K) {
  return d.rank > 0 && d.rank <= a.max_rank && d.rank % 8 == 0 && d.N == N && d.K == K &&
         d.a != nullptr && d.b != nullptr &&
         ((reinterpret_cast<uintptr_t>(d.a) | reinterpret_cast<uintptr_t>(d.b)) & 15) == 0;
}
__device__ __forceinline__ Pair pair_of(const LoraArgs& a, int key, int N, int K) {
  Pair p = {nullptr, nullptr, 0, 0.0f};
  if (key < 0) return p;
  const moe_lora d = a.table[key];
  if (d.rank == 0) return p;
  if (!entry_ok(a, d, N, K)) {
    atomicOr(a.err, 1);
    return p;
  }
  p.a = d.a;
  p.b = d.b;
  p.rank = d.rank;
  p.scale = d.scale;
  return p;
}

// The window's groups in turn, the same in every wave: the rows (bits) and key of one.
struct Groups {
  uint64_t todo;
  __device__ __forceinline__ void init(int key, int from) { todo = __ballot(key >= from); }
  __device__ __forceinline__ bool next(int key, uint64_t& rows, int& k) {
    if (!todo) return false;
    k = __builtin_amdgcn_readlane(key, __builtin_ctzll(todo));
    rows = __ballot(key == k);
    todo &= ~rows;
    return true;
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
constexpr int kFragments = 2;                   // of 16 rows that run together
constexpr int kUnitRows = 16 * kFragments;

// shrink: v[row][j] = scale sum_K A[j][K] in[row][K]
//
// The workgroup's waves share K; a wave's fragments go from memory to registers,
// 16 bytes per lane, since every byte of A and of the rows is read by one wave only.
// The loads of U steps are in flight together; what is left goes in 8, 4, 2, 1 (a
// step count that varies in the loop made the compiler wait for each load: 22 us
// became 50).
template <int U, bool F32, int NF, int CT>
__device__ __forceinline__ void shrink_part(const Pair& p, int K, int C, int ct0, int me, int workers,
                                            const void* const (&rows)[NF], f32x4 (&acc)[NF][CT]) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int steps = K >> 5, per = (steps + workers - 1) / workers;
  const int s0 = min(me * per, steps), s1 = min(s0 + per, steps);
  // tiles and steps are the same for all lanes, a lane's place in a step for all steps
  const uint16_t* pa[CT];
  uint32_t mine[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) {   // rows past the last are computed and dropped
    const int t = min(ct0 + j, (C - 1) / 16), h = min(C - 16 * t, 16);
    pa[j] = p.a + (size_t)16 * t * K + (size_t)s0 * 512;
    mine[j] = 8 * (g * 16 + min(c, h - 1));
  }
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[f][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int s = s0;
  auto step = [&](auto n_steps) {
    constexpr int N = decltype(n_steps)::value;
    u32x4 wa[N][CT], wx[N][NF][F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < CT; ++j)
        wa[i][j] = *reinterpret_cast<const u32x4*>(pa[j] + i * 512 + mine[j]);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if constexpr (F32) {
          const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(rows[f]) +
                                                          (size_t)s * 32 + i * 32 + 8 * g);
          wx[i][f][0] = q[0];
          wx[i][f][1] = q[1];
        } else {
          wx[i][f][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(rows[f]) +
                                                        (size_t)s * 32 + i * 32 + 8 * g);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
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
    s += N;
#pragma unroll
    for (int j = 0; j < CT; ++j) pa[j] += N * 512;
  };
  while (s + U <= s1) step(std::integral_constant<int, U>{});
  if constexpr (U > 8)
    if (s + 8 <= s1) step(std::integral_constant<int, 8>{});
  if constexpr (U > 4)
    if (s + 4 <= s1) step(std::integral_constant<int, 4>{});
  if constexpr (U > 2)
    if (s + 2 <= s1) step(std::integral_constant<int, 2>{});
  if (s < s1) step(std::integral_constant<int, 1>{});
}

// The same with the rows through LDS, a wave's own part of it: the lanes of a
// fragment each hold another row, and read so every 16 bytes are an access of their
// own to the cache.  Here a load takes 64 bytes of a row with neighbouring lanes;
// rows[f] is row 16 f + lane / 4.  (Gate/up of 4096 tokens, H 2048: 55 us without,
// 49 so.  fp32 rows go the other way: a lane's 32 bytes of a step are half a line.)
template <bool F32>
struct RowOf {
  typedef uint16_t type;
};
template <>
struct RowOf<true> {
  typedef void type;
};
constexpr int kStagedSteps = 2;
constexpr int kStagedPitch = 80;   // bytes of a row's step: rows spread over the banks
constexpr int kStagedBytes = 16 * kStagedPitch;
template <int U, int NF, int CT>
__device__ __forceinline__ void shrink_staged(const Pair& p, int K, int C, int ct0, int me, int workers,
                                              const uint16_t* const (&rows)[NF], char* stage,
                                              f32x4 (&acc)[NF][CT]) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int steps = K >> 5, per = (steps + workers - 1) / workers;
  const int s0 = min(me * per, steps), s1 = min(s0 + per, steps);
  const uint16_t* pa[CT];
  uint32_t mine[CT];
#pragma unroll
  for (int j = 0; j < CT; ++j) {   // rows past the last are computed and dropped
    const int t = min(ct0 + j, (C - 1) / 16), h = min(C - 16 * t, 16);
    pa[j] = p.a + (size_t)16 * t * K + (size_t)s0 * 512;
    mine[j] = 8 * (g * 16 + min(c, h - 1));
  }
  const uint16_t* px[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) px[f] = rows[f] + (size_t)s0 * 32 + 8 * (lane & 3);
  char* put = stage + (lane >> 2) * kStagedPitch + 16 * (lane & 3);
  const char* get = stage + c * kStagedPitch + 16 * g;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[f][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int s = s0;
  auto step = [&](auto n_steps) {
    constexpr int N = decltype(n_steps)::value;
    u32x4 wa[N][CT], wx[N][NF];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int f = 0; f < NF; ++f) wx[i][f] = *reinterpret_cast<const u32x4*>(px[f] + i * 32);
#pragma unroll
      for (int j = 0; j < CT; ++j)
        wa[i][j] = *reinterpret_cast<const u32x4*>(pa[j] + i * 512 + mine[j]);
    }
    constexpr int kAt = N < kStagedSteps ? N : kStagedSteps;
#pragma unroll
    for (int i0 = 0; i0 < N; i0 += kAt) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < kAt; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f)
          *reinterpret_cast<u32x4*>(put + (i * NF + f) * kStagedBytes) = wx[i0 + i][f];
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < kAt; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const u32x4 w = *reinterpret_cast<const u32x4*>(get + (i * NF + f) * kStagedBytes);
#pragma unroll
          for (int j = 0; j < CT; ++j) acc[f][j] = mfma(wa[i0 + i][j], w, acc[f][j]);
        }
    }
    s += N;
#pragma unroll
    for (int j = 0; j < CT; ++j) pa[j] += N * 512;
#pragma unroll
    for (int f = 0; f < NF; ++f) px[f] += N * 32;
  };
  while (s + U <= s1) step(std::integral_constant<int, U>{});
  if constexpr (U > 4)
    if (s + 4 <= s1) step(std::integral_constant<int, 4>{});
  if constexpr (U > 2)
    if (s + 2 <= s1) step(std::integral_constant<int, 2>{});
  if (s < s1) step(std::integral_constant<int, 1>{});
}

// v of a unit goes out as three bf16 parts (it would else be split once per slab of
// columns), in pieces of 8 ranks of the rows in a window's order: what a fragment of
// the expanding kernels loads.  to[f]: a row's place in the first piece; a piece has
// `places`.  Down's v goes out times the row's weight.
template <int NF, int CT, bool F32, bool DOWN>
__device__ __forceinline__ void shrink_unit(const LoraArgs& a, const Pair& p, int K, int C, int ct0,
                                            const typename RowOf<F32>::type* const (&rows)[NF],
                                            int places, uint16_t* const (&to)[NF],
                                            const float (&weight)[NF], int n, char* stage,
                                            float* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  f32x4 acc[NF][CT];
  if constexpr (F32) shrink_part<2, F32>(p, K, C, ct0, wave, kWaves, rows, acc);
  else shrink_staged<8>(p, K, C, ct0, wave, kWaves, rows, stage, acc);
  // the waves' parts meet: wave w adds those of tiles w, w + 4, ...
  __syncthreads();   // the last group's parts have been read
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < CT; ++j)
      *reinterpret_cast<f32x4*>(red + ((wave * NF * CT + f * CT + j) * 64 + lane) * 4) = acc[f][j];
  __syncthreads();
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
      if (16 * f + c >= n) continue;
      if (col >= C || (DOWN && !to[f])) continue;
      t *= p.scale;
      uint32_t q[4][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) split3(DOWN ? t[i] * weight[f] : t[i], q[i][0], q[i][1], q[i][2]);
      // gate/up: up's ranks from max_rank on
      const int at = DOWN || col < p.rank ? col : col - p.rank + a.max_rank;
      uint16_t* o = to[f] + (at >> 3) * places * 8 + (at & 7);
#pragma unroll
      for (int e = 0; e < 3; ++e)
        *reinterpret_cast<uint2*>(o + e * places * (DOWN ? 1 : 2) * a.max_rank) =
            make_uint2(q[0][e] | (q[1][e] << 16), q[2][e] | (q[3][e] << 16));
    }
}

// An expert's rows [lo, hi), in the order of their pairs: the first ones whose pair
// is at least p and q.  Both searches at once, a trip to memory for each step.
__device__ __forceinline__ int2 first_pairs(const int32_t* sorted_pair, int lo, int hi, int p, int q) {
  int2 at = make_int2(lo, lo), end = make_int2(hi, hi);
  while (at.x < end.x || at.y < end.y) {   // a search that is done stays where it is
    const int i = (at.x + end.x) >> 1, j = (at.y + end.y) >> 1;
    const int u = sorted_pair[min(i, hi - 1)], v = sorted_pair[min(j, hi - 1)];
    if (at.x < end.x) {
      if (u < p) at.x = i + 1;
      else end.x = i;
    }
    if (at.y < end.y) {
      if (v < q) at.y = j + 1;
      else end.y = j;
    }
  }
  return make_int2(at.x, max(at.x, at.y));
}

// The plan of the accumulating kernel: the rows of one block of tokens, experts
// in order, in windows of 64; a window's rows reordered by (adapter, expert) and
// cut into units.  v lies in that order, so that a unit's rows are neighbours and a
// unit is one place, not sixteen.  Workgroup `part` of a block makes 8 windows.
constexpr int kPlanWindows = 8;
struct PlanLds {
  int lo[kLoraPlanMaxE], pos[kLoraPlanMaxE + 1], wave_sum[kWaves];
};
__device__ void make_plan(const LoraArgs& a, int b, int part, PlanLds& L) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int NE = a.E + a.n_shared;
  const int t0 = b * a.block, t1 = min(a.T, t0 + a.block);
  for (int e = tid; e < NE; e += kThreads) {
    int lo, hi;
    if (e < a.E) {
      const int o0 = min(max(a.offsets[e], 0), a.P), o1 = min(max(a.offsets[e + 1], o0), a.P);
      const int2 r = first_pairs(a.sorted_pair, o0, o1, t0 * a.k, t1 * a.k);
      lo = r.x;
      hi = r.y;
    } else {
      lo = a.P + (e - a.E) * a.T + t0;
      hi = lo + t1 - t0;
    }
    L.lo[e] = lo;
    L.pos[e] = hi - lo;
  }
  __syncthreads();
  // exclusive sums: a thread owns PER experts
  constexpr int PER = (kLoraPlanMaxE + kThreads - 1) / kThreads;
  int cnt[PER], own = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    cnt[i] = e < NE ? L.pos[e] : 0;
    own += cnt[i];
  }
  int pre = own;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(pre, d);
    if (lane >= d) pre += v;
  }
  if (lane == 63) L.wave_sum[wave] = pre;
  __syncthreads();
  int total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += L.wave_sum[w];
    total += L.wave_sum[w];
  }
  int at = before + pre - own;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e < NE) L.pos[e] = at;
    at += cnt[i];
  }
  __syncthreads();
  const size_t base = (size_t)b * a.win;
  for (int i = wave; i < kPlanWindows; i += kWaves) {
    const int w = part * kPlanWindows + i;
    if (w >= a.win) break;
    const int q = 64 * w + lane;
    int key = -1, row = 0, token = 0, rank = 0, e = -1;
    const uint16_t* bp = nullptr;
    if (q < total) {
      int hi = NE;   // the last expert whose rows start at q or before
      e = 0;
      while (hi - e > 1) {
        const int mid = (e + hi) >> 1;
        if (L.pos[mid] <= q) e = mid;
        else hi = mid;
      }
      row = L.lo[e] + q - L.pos[e];
      bool counts = true;
      if (e < a.E) {
        const int p = a.sorted_pair[row];
        token = (unsigned)p < (unsigned)a.P ? p / a.k : -1;
        counts = token >= 0 && a.pair_pos[p] == row;   // -1: the pair adds nothing
      } else {
        token = row - a.P - (e - a.E) * a.T;
      }
      if (counts && token >= t0 && token < t1) {
        const int d = a.adapter[token];
        if ((unsigned)d < (unsigned)a.n) {
          const moe_lora m = a.table[(size_t)d * NE + e];
          if (entry_ok(a, m, a.H, e < a.E ? a.I : a.I_sh)) {
            key = d * NE + e;
            rank = m.rank;
            bp = m.b;
          }
        }
      }
    }
    // a token that lists an expert twice has neighbouring rows: each time apart
    const int token1 = __shfl_up(token, 1), e1 = __shfl_up(e, 1);
    const bool same = lane > 0 && token1 == token && e1 == e;
    const uint64_t first = ~__ballot(same) & ((2ull << lane) - 1);
    const int again = lane - (63 - __builtin_clzll(first));
    uint64_t todo = __ballot(key >= 0);
    int units = 0, placed = 0;
    while (todo) {
      const int lead = __builtin_ctzll(todo);
      const uint64_t rows = __ballot(key == __builtin_amdgcn_readlane(key, lead) &&
                                     again == __builtin_amdgcn_readlane(again, lead));
      todo &= ~rows;
      const int n = __popcll(rows), nu = (n + 15) / 16;
      const uint64_t bits = reinterpret_cast<uint64_t>(bp);
      const uint32_t b_hi = (uint32_t)__builtin_amdgcn_readlane((int)(bits >> 32), lead);
      const uint32_t b_lo = (uint32_t)__builtin_amdgcn_readlane((int)bits, lead);
      const uint32_t rank8 = (uint32_t)__builtin_amdgcn_readlane(rank, lead) / 8;
      const size_t first_unit = (base + w) * 64 + units;
      const uint32_t at = (uint32_t)(base + w) * 64 + placed;
      const uint32_t place = ((uint32_t)(base + w) * 3 * (a.max_rank / 8) * 64 + placed) * 16;
      if (lane < nu)
        reinterpret_cast<u32x4*>(a.plan)[first_unit + lane] =
            u32x4{b_lo, b_hi, rank8, place + 256u * lane};
      if ((rows >> lane) & 1) {
        const int t = token - t0, i = __popcll(rows & ((1ull << lane) - 1));
        a.plan_sums[first_unit * 16 + i] = (uint32_t)(t * 256 + (t & 15) * 16);
        a.place[row] = at + i;
        a.row_at[at + i] = (uint32_t)row;
      }
      // lanes without a row add behind the block
      if (n + lane < 16 * nu) a.plan_sums[first_unit * 16 + n + lane] = (uint32_t)a.block * 256;
      units += nu;
      placed += n;
    }
    if (lane == 0) a.plan_count[base + w] = units;
  }
}

// ---------------------------------------------------------------------
// Many rows: three launches.  The first sorts a window of 256 rows by
// (adapter, expert) and cuts the groups into units of up to 32 rows; rows without
// an adapter come last.  A unit's products of K and its expansion then read that
// pair's matrices once.  What bounded both was how often the matrices came in and
// how few rows a fragment had: from windows of 64 rows, sorted by every workgroup
// for itself, 4096 tokens of 9 rows over 4 adapters took 62 us of products of K and
// 85 of expansion; so, 6.6 + 49 + 54 (the last two move their 151 and 230 MB at 3.1
// and 4.3 TB/s).  A wave finds its groups with ballots, the four waves' lists are
// then compared (every row with every other one: 10.7 us, so 6.6).
struct SortLds {
  int2 group[kWaves][64];   // of a wave's rows: key, rows
  int start[kWaves * 64], count[kWaves], wave_sum[2][kWaves];
};
template <bool DOWN>
__global__ __launch_bounds__(kLoraWindow) void lora_sort_kernel(LoraArgs a, int n_win) {
  static_assert(kLoraWindow == kThreads, "a thread per row");
  __shared__ union {
    SortLds sort;
    PlanLds plan;
  } lds;
  if constexpr (DOWN) {
    if ((int)blockIdx.x >= n_win) {
      const int per = (a.win + kPlanWindows - 1) / kPlanWindows, q = (int)blockIdx.x - n_win;
      make_plan(a, q / per, q % per, lds.plan);
      return;
    }
  }
  SortLds& L = lds.sort;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r0 = blockIdx.x * kLoraWindow;
  const Row w = window_row<DOWN>(a, r0 + tid);
  // groups of the wave's rows; a group's first lane stands for it
  int lead = lane, before = 0, groups = 0;
  uint64_t todo = __ballot(w.key != kNoRow);
  while (todo) {
    const int l = __builtin_ctzll(todo);
    const uint64_t rows = __ballot(w.key == __builtin_amdgcn_readlane(w.key, l));
    todo &= ~rows;
    if ((rows >> lane) & 1) {
      lead = l;
      before = __popcll(rows & ((1ull << lane) - 1));
    }
    if (lane == l) L.group[wave][groups] = make_int2(w.key, __popcll(rows));
    ++groups;
  }
  if (lane == 0) L.count[wave] = groups;
  const bool stands = lead == lane && w.key != kNoRow;
  Pair p = {nullptr, nullptr, 0, 0.0f};
  int shared = 0;
  if (stands) {
    shared = width_is_shared(a, w.key);
    if (w.key >= 0) {
      const moe_lora d = a.table[w.key];
      if (d.rank != 0) {
        const int width = shared ? a.I_sh : a.I;
        if (entry_ok(a, d, DOWN ? a.H : 2 * width, DOWN ? width : a.H)) p = Pair{d.a, d.b, d.rank, d.scale};
        else atomicOr(a.err, 1);
      }
    }
  }
  __syncthreads();
  // the same key in other waves: the first one's group holds all its rows
  int n = 0, prior = 0, home = -1;
  if (stands)
    for (int v = 0; v < kWaves; ++v)
      for (int i = 0; i < L.count[v]; ++i) {
        const int2 q = L.group[v][i];
        if (q.x != w.key) continue;
        if (home < 0) home = 64 * v + i;
        if (v < wave) prior += q.y;
        n += q.y;
      }
  const bool first = stands && prior == 0;
  // exclusive sums of rows and units, with an adapter and without
  const int nu = first ? (n + kUnitRows - 1) / kUnitRows : 0, mine = first ? n | (nu << 16) : 0;
  int sum[2] = {p.rank ? mine : 0, p.rank ? 0 : mine}, own[2] = {sum[0], sum[1]};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(sum[h], d);
      if (lane >= d) sum[h] += v;
    }
    if (lane == 63) L.wave_sum[h][wave] = sum[h];
  }
  __syncthreads();
  int total[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      if (v < wave) sum[h] += L.wave_sum[h][v];
      total[h] += L.wave_sum[h][v];
    }
  const int at = p.rank ? sum[0] - own[0] : total[0] + sum[1] - own[1];
  const size_t base = (size_t)blockIdx.x * kLoraWindow;
  if (first) {
    L.start[home] = at & 0xFFFF;
    for (int u = 0; u < nu; ++u)
      a.units[base + (at >> 16) + u] =
          LoraGroupUnit{p.a, p.b, p.scale, (uint16_t)p.rank, (uint16_t)shared,
                        (uint16_t)((at & 0xFFFF) + u * kUnitRows), (uint16_t)min(n - u * kUnitRows, kUnitRows), 0};
  }
  if (tid == 0) a.unit_count[blockIdx.x] = make_int2(total[0] >> 16, (total[0] + total[1]) >> 16);
  __syncthreads();
  const int start = __shfl(stands ? L.start[home] + prior : 0, lead);
  if (w.key != kNoRow) {
    a.order[base + start + before] = (uint32_t)w.token | ((uint32_t)tid << 24);
    if (DOWN) a.weight[base + start + before] = w.weight;
  }
}

template <int CT, bool F32, bool DOWN>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(LoraArgs a, int n_win, int slots) {
  __shared__ __align__(16) float red[kWaves * kFragments * CT * 256];
  __shared__ __align__(16) char stage[F32 ? 1 : kWaves][kStagedSteps * kFragments * kStagedBytes];
  const int lane = threadIdx.x & 63, c = lane & 15;
  const int ct0 = blockIdx.y * CT;
  // neighbouring windows, which share matrices, on one XCD (workgroup mod 8)
  const int i = xcd_order(blockIdx.x, n_win * slots), win = i / slots;
  const size_t base = (size_t)win * kLoraWindow;
  const int n_units = a.unit_count[win].x;
  for (int u = i - win * slots; u < n_units; u += slots) {
    const LoraGroupUnit m = a.units[base + u];
    const Pair p = {m.a, m.b, m.rank, m.scale};
    const int C = (DOWN ? 1 : 2) * p.rank, n = m.n;
    const int K = !DOWN ? a.H : m.shared ? a.I_sh : a.I;
    if (16 * ct0 >= C) continue;   // a lower rank than the largest
    auto run = [&](auto nf) {
      constexpr int NF = decltype(nf)::value;
      const typename RowOf<F32>::type* src[NF];
      uint16_t* to[NF];
      float weight[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        // fragments' rows past the unit's end are computed and dropped
        const int at = m.first + min(16 * f + c, n - 1);
        const int from = F32 ? at : m.first + min(16 * f + (lane >> 2), n - 1);
        const uint32_t row = a.order[base + from];
        const size_t off = DOWN ? (base + (row >> 24)) * a.ld_h : (size_t)(row & 0xFFFFFF) * a.H;
        if constexpr (F32) src[f] = static_cast<const float*>(a.in) + off;
        else src[f] = static_cast<const uint16_t*>(a.in) + off;
        weight[f] = 1.0f;
        if constexpr (DOWN) {
          const uint32_t place = a.place[base + (a.order[base + at] >> 24)];
          to[f] = a.parts + (size_t)(place >> 6) * 64 * 3 * a.max_rank + (place & 63) * 8;
          weight[f] = a.weight[base + at];
          // a row that the plan left out (lists that contradict each other) has
          // whatever place an earlier call left: only a place of its own counts
          const uint32_t places = (uint32_t)a.n_blocks * a.win * 64;
          if (a.row_at[min(place, places - 1)] != (uint32_t)base + (a.order[base + at] >> 24) || place >= places)
            to[f] = nullptr;
        } else {
          to[f] = a.parts + base * 6 * a.max_rank + at * 8;
        }
      }
      shrink_unit<NF, CT, F32, DOWN>(a, p, K, C, ct0, src, DOWN ? 64 : kLoraWindow, to, weight, n,
                                     stage[F32 ? 0 : threadIdx.x >> 6], red);
    };
    if (n > 16) run(std::integral_constant<int, 2>{});
    else run(std::integral_constant<int, 1>{});
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
__device__ __forceinline__ void load_gu(const LoraArgs& a, int row, int col, f32x4 (&gu)[4]) {
  const float* q = a.gu + (size_t)row * 2 * a.ld_h + col;
#pragma unroll
  for (int i = 0; i < 4; ++i)   // gate, gate, up, up
    gu[i] = *reinterpret_cast<const f32x4*>(q + (i >> 1) * a.ld_h + 4 * (i & 1));
}
// Row `row` of a tiled B, ranks [j, j + 8).
__device__ __forceinline__ size_t b_at(int row, int j, int rank) {
  return (size_t)(row & ~31) * rank + 32 * j + 8 * (row & 31);
}
// B's fragments of ranks [k0, k0 + 32): the lane's row of each, zeros past the rank.
__device__ __forceinline__ void load_b(const Pair& p, int width, int i0, int k0, u32x4 (&b)[4]) {
  const int lane = threadIdx.x & 63, c = lane & 15, j = k0 + 8 * (lane >> 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int br = (i >> 1) * width + i0 + 8 * (c >> 2) + 4 * (i & 1) + (c & 3);
    b[i] = u32x4{0u, 0u, 0u, 0u};
    if (j < p.rank) b[i] = *reinterpret_cast<const u32x4*>(p.b + b_at(br, j, p.rank));
  }
}
// v: 8 values each of the gate's and up's.
__device__ __forceinline__ void expand_step(const u32x4 (&b)[4], const float (&vg)[8],
                                            const float (&vu)[8], f32x4 (&acc)[4]) {
  u32x4 g[3], u[3];
  split3(vg, g);
  split3(vu, u);
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    acc[0] = mfma(b[0], g[e], acc[0]);
    acc[1] = mfma(b[1], g[e], acc[1]);
    acc[2] = mfma(b[2], u[e], acc[2]);
    acc[3] = mfma(b[3], u[e], acc[3]);
  }
}
__device__ __forceinline__ void store_h(const LoraArgs& a, int row, int col, bool there,
                                        const f32x4 (&gu)[4], f32x4 (&acc)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) mx_keep(acc[i]);
  if (!there) return;
  float gv[8], uv[8], hv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gv[i] = gu[i / 4][i % 4] + acc[i / 4][i % 4];
    uv[i] = gu[2 + i / 4][i % 4] + acc[2 + i / 4][i % 4];
  }
  const size_t o = (size_t)row * a.ld_h + col;
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

// Many rows: a wave takes 64 columns of every `slots`-th unit, 16 rows at a time,
// and the fragments' parts are exchanged: a lane ends with four neighbouring
// columns of four rows, so that loads of g and u are whole runs of 256 bytes.
// Ranks, rows and columns past the last are offsets out of range: zeros that
// touch no line.
constexpr int kExpandCols = 64;
constexpr uint32_t kOut = 0x80000000u;   // no buffer here is larger

__global__ __launch_bounds__(kThreads) void lora_expand_gateup_kernel(LoraArgs a, int n_win, int slots) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int i0 = (blockIdx.y * kWaves + wave) * kExpandCols;
  if (i0 >= a.ld_h) return;
  const int idx = xcd_order(blockIdx.x, n_win * slots), win = idx / slots;
  const size_t base = (size_t)win * kLoraWindow;
  const int r0 = win * kLoraWindow, n_units = a.unit_count[win].y;
  const int col = i0 + 4 * c;
  const uint32_t v_part = (uint32_t)(a.max_rank * 2 * kLoraWindow * 2);   // bytes
  const __amdgpu_buffer_rsrc_t vrs = __builtin_amdgcn_make_buffer_rsrc(
      a.parts + base * 6 * a.max_rank, 0, (int)(3 * v_part), 0x00020000);
  const __amdgpu_buffer_rsrc_t grs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(a.gu) + (size_t)r0 * 2 * a.ld_h, 0,
      (int)((uint32_t)min(kLoraWindow, a.R - r0) * 8u * a.ld_h), 0x00020000);
  for (int u = idx - win * slots; u < n_units; u += slots) {
    const LoraGroupUnit m = a.units[base + u];
    const int rank = m.rank, width = m.shared ? a.I_sh : a.I;
    if (i0 >= width) continue;
    const __amdgpu_buffer_rsrc_t brs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(m.b), 0, 4 * width * rank, 0x00020000);
    for (int f0 = 0; f0 < m.n; f0 += 16) {
      const uint32_t* order = a.order + base + m.first + f0 + 4 * g;
      int row[4];
      f32x4 gu[4][2], acc[2][4];   // row 4 g + i; gate, up
#pragma unroll
      for (int i = 0; i < 4; ++i) row[i] = (int)(order[i] >> 24);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          gu[i][h] = __builtin_bit_cast(
              f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         grs, f0 + 4 * g + i < m.n && col < width ? 4u * ((row[i] * 2 + h) * a.ld_h + col) : kOut, 0, 0));
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[h][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int k0 = 0; k0 < rank; k0 += 32) {
        const int j = k0 + 8 * g;
        u32x4 v[2][3], b[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t vo = j < rank ? 16u * ((h * a.max_rank + j) / 8 * kLoraWindow + m.first + f0 + c) : kOut;
          const uint32_t br = h * width + col;
          const uint32_t bo = j < rank && col < width ? 2u * ((br & ~31u) * rank + 32 * j + 8 * (br & 31)) : kOut;
#pragma unroll
          for (int e = 0; e < 3; ++e)
            v[h][e] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(vrs, vo, e * v_part, 0));
#pragma unroll
          for (int q = 0; q < 4; ++q)   // column 4 c + q
            b[h][q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(brs, bo + 16 * q, 0, 0));
        }
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[h][q] = mfma(v[h][e], b[h][q], acc[h][q]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (f0 + 4 * g + i >= m.n || col >= width) continue;
        float x[4], y[4], h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x[q] = gu[i][0][q] + acc[0][q][i];
          y[q] = gu[i][1][q] + acc[1][q][i];
        }
        const size_t o = (size_t)(r0 + row[i]) * a.ld_h + col;
        if (a.out_f32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = silu_mul_wide(x[q], y[q]);
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o) = f32x4{h[0], h[1], h[2], h[3]};
        } else {
          mx_silu_mul(x, y, h);
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) =
              make_uint2(mx_bf16(h[0]) | (mx_bf16(h[1]) << 16), mx_bf16(h[2]) | (mx_bf16(h[3]) << 16));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------
// Few rows, gate/up: one launch.  A workgroup takes one group of a window of 16
// rows; its waves share K, v stays in LDS, and each wave then takes blocks of 32
// columns, the first one's g, u and B asked for before the products of K.  A few
// tokens' time is trips to memory, so what depends on nothing is read at once:
// the window's pairs with all tokens' experts and adapters, then the table's
// entry, then the matrices.  Eight waves share the trips of a workgroup that has
// a compute unit to itself, four leave room for three workgroups: 9 rows 9.7 us by
// eight, 11.8 by four, 231 rows 11.6 and 14.4, 576 rows 32.6 and 26.4.
constexpr int kSmallTiles = 2;   // of 16 ranks at a time

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void lora_gateup_small_kernel(LoraArgs a) {
  constexpr int kVPitch = 2 * kLoraMaxRank + 4;
  __shared__ int list[WAVES][64];
  __shared__ int ids[kLoraManyRows], adapter[kLoraManyRows];
  __shared__ __align__(16) float red[WAVES * kSmallTiles * 256];
  __shared__ __align__(16) float v[16 * kVPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
  const int win = blockIdx.x / kLoraSmallRows, slot = blockIdx.x - win * kLoraSmallRows;
  const int r0 = win * kLoraSmallRows, r = r0 + lane;
  const int pr = lane < kLoraSmallRows && r < a.P ? a.sorted_pair[r] : 0;
  for (int i = tid; i < a.P; i += 64 * WAVES) ids[i] = a.topk_ids[i];
  for (int i = tid; i < a.T; i += 64 * WAVES) adapter[i] = a.adapter[i];
  __syncthreads();
  const Row w = window_row<false>(a, lane < kLoraSmallRows ? r : a.R, pr, ids, adapter);
  Groups gr;
  gr.init(w.key, kBaseRouted);
  uint64_t rows;
  int key;
  for (int i = 0; i <= slot; ++i)   // its slot-th group
    if (!gr.next(w.key, rows, key)) return;
  const int width = width_of(a, key);
  const Pair p = pair_of(a, key, 2 * width, a.H);
  const int n = list_rows(rows, list[wave]);
  const int l = list[wave][min(c, n - 1)];   // past the group's end: computed and dropped
  const int row[1] = {r0 + l};
  const void* src[1] = {static_cast<const uint16_t*>(a.in) + (size_t)__shfl(w.token, l) * a.H};

  // blocks of columns: their g, u and first 32 ranks of B
  struct Block {
    f32x4 gu[4];
    u32x4 b[4];
  };
  constexpr int kStep = WAVES * 32, kBlocks = WAVES == 8 ? 4 : 2;
  Block blk[kBlocks];
  auto load = [&](int i0, Block& x) {
    if (i0 >= width) return;
    load_gu(a, row[0], i0 + 8 * g, x.gu);
    load_b(p, width, i0, 0, x.b);
  };
  load(wave * 32, blk[0]);
  const int C = 2 * p.rank;
  for (int ct0 = 0; 16 * ct0 < C; ct0 += kSmallTiles) {
    f32x4 acc[1][kSmallTiles];
    shrink_part<8, false>(p, a.H, C, ct0, wave, WAVES, src, acc);
    if (ct0) __syncthreads();   // the last tiles' parts have been read
#pragma unroll
    for (int j = 0; j < kSmallTiles; ++j)
      *reinterpret_cast<f32x4*>(red + ((wave * kSmallTiles + j) * 64 + lane) * 4) = acc[0][j];
    __syncthreads();
    if (wave < kSmallTiles) {
      f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < WAVES; ++k)
        t += *reinterpret_cast<const f32x4*>(red + ((k * kSmallTiles + wave) * 64 + lane) * 4);
      const int col = 16 * (ct0 + wave) + 4 * g;
      if (col < C) *reinterpret_cast<f32x4*>(v + c * kVPitch + col) = t * p.scale;
    }
  }
  __builtin_amdgcn_sched_barrier(0);   // the registers of A's loads are free
#pragma unroll
  for (int k = 1; k < kBlocks; ++k) load(wave * 32 + k * kStep, blk[k]);
  __syncthreads();
  for (int i0 = wave * 32; i0 < width; i0 += kBlocks * kStep) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      const int col = i0 + k * kStep;
      if (col >= width) break;
      f32x4 acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int k0 = 0; k0 < p.rank; k0 += 32) {
        const int j = k0 + 8 * g;
        if (k0) load_b(p, width, col, k0, blk[k].b);
        float t[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            t[h][i] = j < p.rank ? v[c * kVPitch + h * p.rank + j + i] : 0.0f;
        expand_step(blk[k].b, t[0], t[1], acc);
      }
      store_h(a, row[0], col + 8 * g, c < n, blk[k].gu, acc);
    }
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) load(i0 + (kBlocks + k) * kStep, blk[k]);
  }
}

// ---------------------------------------------------------------------
// Few tokens, down: one launch.  A workgroup takes a token and 192 NT columns.
// It makes v of all the token's rows (a wave a row; a row's h and A are small next
// to B, and the other workgroups of the token find them in the cache), then
// out[t][n] = base[t][n] + sum over the rows of w B v.  There the rows' ranks form
// one long axis, in pieces of 8 that each have a matrix of their own; a matrix
// product over 32 of it takes four pieces, whatever rows they are of.  The other
// operand's columns 0, 1, 2 are the three parts of w v.  The first steps' B is
// asked for with A, a trip to memory earlier.
constexpr int kPieces = 128;      // of a pass
constexpr int kDownWaves = 12;

template <int NT, bool F32>
__global__ __launch_bounds__(64 * kDownWaves) void lora_down_small_kernel(LoraArgs a) {
  __shared__ Pair pair[kPieces];
  __shared__ int row_of[kPieces];
  __shared__ float weight_of[kPieces];
  // [part][row][rank]: one part, or no more than kDownWaves rows of them
  __shared__ __align__(16) float sums[kDownWaves * kLoraMaxRank > 8 * kPieces ? kDownWaves * kLoraMaxRank
                                                                              : 8 * kPieces];
  __shared__ __align__(16) u32x4 vs[3][kPieces];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int t = blockIdx.x;
  const int n0 = (blockIdx.y * kDownWaves + wave) * 16 * NT;
  const int per = a.max_rank / 8;            // pieces of a row
  const int choices = a.k + a.n_shared, at_once = kPieces / per;
  const int d = a.adapter[t];
  const u32x4 zero = {0u, 0u, 0u, 0u};
  constexpr int kAhead = NT == 1 ? 5 : 8 / NT;   // steps of B asked for with A
  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = 0; c0 < choices; c0 += at_once) {
    const int m = min(choices - c0, at_once), pieces = m * per;
    int row = 0, e = -1;
    float wt = 1.0f;
    if (tid < m) {
      const int ch = c0 + tid;
      if (ch < a.k) {
        row = a.pair_pos[(size_t)t * a.k + ch];
        e = a.topk_ids[(size_t)t * a.k + ch];
        wt = a.topk_w[(size_t)t * a.k + ch];
      } else {
        const int s = ch - a.k;
        row = a.P + s * a.T + t;
        e = a.E + s;
        if (a.shared_gate) wt = shared_gate_weight(a.shared_gate[(size_t)t * a.n_shared + s]);
      }
    }
    if ((unsigned)d >= (unsigned)a.n) break;   // after the loads: one trip with d's
    if (c0) __syncthreads();                   // the last pass is done
    if (tid < m) {
      // a routed choice has an expert and a row among the pairs
      const bool ok = (unsigned)row < (unsigned)(c0 + tid < a.k ? a.P : a.R) &&
                      (unsigned)e < (unsigned)(c0 + tid < a.k ? a.E : a.E + a.n_shared);
      const int key = ok ? d * (a.E + a.n_shared) + e : kNoRow;
      pair[tid] = pair_of(a, key, a.H, ok ? width_of(a, key) : 0);
      row_of[tid] = ok ? row : 0;
      weight_of[tid] = wt;
    }
    __syncthreads();
    auto load_b = [&](int s, u32x4 (&b)[NT]) {   // pieces s + g, s a multiple of 4
      const int q = min(s + g, pieces - 1), ch = q / per, j = 8 * (q - ch * per);
      const int rank = s + g < pieces ? pair[ch].rank : 0;
      const auto* bp = (const __attribute__((address_space(1))) uint16_t*)pair[ch].b;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        b[i] = zero;
        if (j < rank)
          b[i] = *(const __attribute__((address_space(1))) u32x4*)(
              bp + b_at(min(n0 + 16 * i + c, a.H - 1), j, rank));
      }
    };
    u32x4 ahead[kAhead][NT];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_b(4 * i, ahead[i]);
    // v of the pass's rows: the waves share them, and a row's K where there are
    // more waves than rows
    const int parts = m < kDownWaves ? kDownWaves / m : 1;
    for (int q = wave; q < m * parts; q += kDownWaves) {
      const int ch = q / parts, part = q - ch * parts;
      Pair p;
      p.rank = __builtin_amdgcn_readfirstlane(pair[ch].rank);
      const uint64_t at = reinterpret_cast<uint64_t>(pair[ch].a);
      p.a = reinterpret_cast<const uint16_t*>(
          ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(at >> 32)) << 32) |
          (uint32_t)__builtin_amdgcn_readfirstlane((int)at));
      const int r = __builtin_amdgcn_readfirstlane(row_of[ch]);
      const int K = r < a.P ? a.I : a.I_sh;
      const void* in[1] = {F32 ? (const void*)(static_cast<const float*>(a.in) + (size_t)r * a.ld_h)
                               : (const void*)(static_cast<const uint16_t*>(a.in) + (size_t)r * a.ld_h)};
      float* to = sums + (part * m + ch) * per * 8 + 4 * g;
      auto tiles = [&](auto n, int ct) {
        constexpr int CT = decltype(n)::value;
        f32x4 x[1][CT];
        shrink_part<(F32 ? 4 : 8) / CT, F32>(p, K, p.rank, ct, part, parts, in, x);
#pragma unroll
        for (int i = 0; i < CT; ++i) {
          mx_keep(x[0][i]);
          const int j = 16 * (ct + i);
          // every column is the same; the last tile may be half
          if (c == 0 && j + 4 * g < p.rank) *reinterpret_cast<f32x4*>(to + j) = x[0][i];
        }
      };
      int ct = 0;
      for (; 16 * ct + 16 < p.rank; ct += 2) tiles(std::integral_constant<int, 2>{}, ct);
      if (16 * ct < p.rank) tiles(std::integral_constant<int, 1>{}, ct);
    }
    __syncthreads();
    for (int i = tid; i < 8 * pieces; i += 64 * kDownWaves) {
      const int q = i / 8, ch = q / per, j = i - 8 * ch * per;
      float x = 0.0f;
      if (j < pair[ch].rank) {
        for (int k = 0; k < parts; ++k) x += sums[8 * k * pieces + i];
        x = x * pair[ch].scale * weight_of[ch];
      }
      uint32_t f[3];
      split3(x, f[0], f[1], f[2]);
#pragma unroll
      for (int e = 0; e < 3; ++e)
        reinterpret_cast<uint16_t*>(&vs[e][q])[i & 7] = (uint16_t)f[e];
    }
    __syncthreads();
    auto add = [&](int s, const u32x4 (&b)[NT]) {
      const u32x4 x = c < 3 && s + g < pieces ? vs[c][s + g] : zero;
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = mfma(b[i], x, acc[i]);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) add(4 * i, ahead[i]);
    for (int s = 4 * kAhead; s < pieces; s += 4) {
      u32x4 b[NT];
      load_b(s, b);
      add(s, b);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    // the three parts' sums: lanes 1 and 2 of the 16 to lane 0
    f32x4 sum;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sum[e] = acc[i][e] + (__shfl(acc[i][e], lane + 1) + __shfl(acc[i][e], lane + 2));
    const int n = n0 + 16 * i + 4 * g;
    if (c != 0 || n >= a.H) continue;
    const size_t o = (size_t)t * a.H + n;
    sum += *reinterpret_cast<const f32x4*>(a.base + o);
    if (a.out_f32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o) = sum;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) =
          make_uint2(mx_bf16(sum[0]) | (mx_bf16(sum[1]) << 16), mx_bf16(sum[2]) | (mx_bf16(sum[3]) << 16));
    }
  }
}

// ---------------------------------------------------------------------
// expand, down, of many tokens.  A workgroup owns 64 columns of a block of
// tokens and keeps their sums in LDS (fp32), starting from base; it passes the
// block's units (make_plan) and adds each unit's products B v to its tokens'.  A
// wave owns 16 of the columns of all the tokens, so no two waves meet in a sum,
// and a unit holds a token once, so no two lanes do: plain reads and writes in a
// wave's own order, the same result every time.  4096 tokens, H 2048: 88 us, 17 of
// them base, out and the units on their way; LDS additions without return were five times slower (500 us),
// sums by tokens without any reuse of B four times (381), and rows of y through
// memory as in the shared projection would be 600 MB.  What bounds it is no rate but
// the way of a unit through a wave, some 165 ns of 434 units a block: 80 MB at the
// device's memory are 0.9 TB/s, LDS is busy for 31% of the cycles, the matrix cores
// for 11%; a SIMD's one wave issues 25 vector instructions a unit, 24% of its cycles,
// and waits in 41%.  Without B's loads it took 85 us, without v's 89, without either
// 81, without the sums' reads and writes 86.  128 columns of 256 tokens (101 to 128
// us), 64 columns of 256 with two workgroups a compute unit (114), waves that divide
// the adapters (104), v through LDS once for all waves (102), products over 16 ranks
// with 8-byte loads (119) and batches of 8 units (99) were slower; two parts of v in
// one product for ranks up to 16 gained 2 us and is not worth a variant.
// A token's 64 sums are 16 chunks of 4; chunk q lies at q ^ (token % 16), so that
// the 16 tokens of a unit spread over the banks.
constexpr int kUnitsAtOnce = 128;  // in LDS; a segment of a prompt has about 100 (segments of 8 windows 96 us, 16 88, 32 95)
constexpr int kUnitsAhead = 16;    // and behind them some that do nothing: what the loop reads past its end

template <int KB>   // steps of 32 ranks
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 2)))
void lora_accumulate_kernel(LoraArgs a, int n_slabs) {
  extern __shared__ f32x4 sums[];                // [block + 1][16]
  __shared__ u32x4 unit_mem[5 * (kUnitsAtOnce + kUnitsAhead)];   // a unit, and its rows' places
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;
  // the workgroups of an XCD (b mod 8) share slabs: B's rows of a slab stay in its L2
  const int xcd = blockIdx.x & 7, li = blockIdx.x >> 3;
  const int slab = xcd + 8 * (li / a.n_blocks), b = li % a.n_blocks;
  if (slab >= n_slabs) return;
  const int n0 = slab * kLoraSlab, t0 = b * a.block, nt = min(a.block, a.T - t0);

  // The units of a segment of windows, `first` on, on their way to LDS: thread t
  // takes pieces t, t + 256, ... of 16 bytes (a unit has 5).
  constexpr int kPer = (5 * kUnitsAtOnce + kThreads - 1) / kThreads;
  const size_t base = (size_t)b * a.win;
  struct Chunk {
    u32x4 piece[kPer];
    int n;   // units
  };
  auto load_counts = [&](int w0) { return a.plan_count[base + w0 + (lane & (kLoraSegment - 1))]; };
  auto load_chunk = [&](int w0, int counts, int first, Chunk& x) {
    int before[kLoraSegment + 1];   // units of the windows before
    before[0] = 0;
#pragma unroll
    for (int w = 0; w < kLoraSegment; ++w)
      before[w + 1] = before[w] + __builtin_amdgcn_readlane(counts, w);
    x.n = min(before[kLoraSegment] - first, kUnitsAtOnce);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = tid + i * kThreads, u = min(p / 5, x.n - 1), q = p - p / 5 * 5, at = first + u;
      int w = 0, start = 0;
#pragma unroll
      for (int k = 1; k < kLoraSegment; ++k)
        if (at >= before[k]) {
          w = k;
          start = before[k];
        }
      const size_t slot = (base + w0 + w) * 64 + (at - start);
      if (x.n > 0)
        x.piece[i] = q == 0 ? reinterpret_cast<const u32x4*>(a.plan)[slot]
                            : reinterpret_cast<const u32x4*>(a.plan_sums)[slot * 4 + q - 1];
    }
    return before[kLoraSegment];
  };
  Chunk next;
  int w0 = 0, first = 0;
  int counts = load_counts(0);
  int counts1 = kLoraSegment < a.win ? load_counts(kLoraSegment) : 0;
  int total = load_chunk(0, counts, 0, next);

  const int q0 = tid & 15, nq = min(n0 + 4 * q0, a.H - 4);   // columns past H: never stored
  for (int i0 = tid >> 4; i0 < nt; i0 += 8 * (kThreads / 16)) {
    f32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = *reinterpret_cast<const f32x4*>(
          a.base + (size_t)(t0 + min(i0 + i * (kThreads / 16), nt - 1)) * a.H + nq);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = i0 + i * (kThreads / 16);
      if (t < nt) sums[t * 16 + (q0 ^ (t & 15))] = v[i];
    }
  }
  const uint32_t col = min(n0 + 16 * wave + c, a.H - 1);   // B's row of the lane
  const uint32_t mine = (uint32_t)(4 * wave + g) * 16;
  const uint32_t part_bytes = 64 * a.max_rank * 2;   // of a window's v
  const __amdgpu_buffer_rsrc_t vrs = __builtin_amdgcn_make_buffer_rsrc(
      a.parts, 0, (int)((uint32_t)a.n_blocks * a.win * 3 * part_bytes), 0x00020000);
  // One wave a SIMD: what bounds it is the instructions of a unit.  None branches, so
  // that the loads of later units stay in flight behind the products of earlier
  // ones.  Ranks past the last are offsets out of range, which load zeros and touch
  // no line; lanes without a row load any and add behind the block.
  constexpr int kBatch = 4 / KB;   // units fetched together
  struct Data {
    u32x4 b[KB], v[KB][3];
    uint32_t place;
  };
  struct Unit {
    u32x4 u;
    uint32_t place;
  };
  auto look = [&](int i, Unit& m) {
    m.u = unit_mem[5 * i];
    m.place = reinterpret_cast<const uint32_t*>(unit_mem + 5 * i + 1)[c];
  };
  auto fetch = [&](const Unit& m, Data& d) {
    const uint64_t at = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)m.u.y) << 32) |
                        (uint32_t)__builtin_amdgcn_readfirstlane((int)m.u.x);
    const __amdgpu_buffer_rsrc_t brs =
        __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), 0, (int)kOut, 0x00020000);
    d.place = m.place ^ mine;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const uint32_t q = 4 * k + g;
      const bool in = q < m.u.z;
      const uint32_t bo = in ? m.u.z * (16 * (col & ~31u)) + 16 * (32 * q + (col & 31)) : kOut;
      const uint32_t vo = in ? m.u.w + 16 * (q * 64 + c) : kOut;
      d.b[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(brs, bo, 0, 0));
#pragma unroll
      for (int e = 0; e < 3; ++e)
        d.v[k][e] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(vrs, vo, e * part_bytes, 0));
    }
  };
  auto add = [&](const Data (&d)[kBatch]) {
    f32x4 acc[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) acc[i] = mfma(d[i].b[k], d[i].v[k][e], acc[i]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      *reinterpret_cast<f32x4*>(reinterpret_cast<char*>(sums) + d[i].place) += acc[i];
  };
  while (true) {
    const int n = next.n;
    const uint32_t behind = (uint32_t)a.block * 256;
    __syncthreads();   // the last units have been read, base is in
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = tid + i * kThreads;
      if (p < 5 * n) unit_mem[p] = next.piece[i];
    }
    if (tid < 5 * kUnitsAhead)   // no rank, behind the block
      unit_mem[5 * n + tid] = tid % 5 ? u32x4{behind, behind, behind, behind} : u32x4{0u, 0u, 0u, 0u};
    __syncthreads();
    first += kUnitsAtOnce;
    bool more = true;
    if (first >= total) {
      first = 0;
      w0 += kLoraSegment;
      counts = counts1;
      more = w0 < a.win;
      if (w0 + kLoraSegment < a.win) counts1 = load_counts(w0 + kLoraSegment);
    }
    if (more) total = load_chunk(w0, counts, first, next);
    if (n > 0) {
      Unit u[kBatch];
      Data cur[kBatch], nxt[kBatch];
      auto look_all = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) look(i0 + i, u[i]);
      };
      auto fetch_all = [&](Data (&d)[kBatch]) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) fetch(u[i], d[i]);
      };
      look_all(0);
      fetch_all(cur);
      look_all(kBatch);
      for (int i = 0; i < n; i += 2 * kBatch) {
        fetch_all(nxt);
        __builtin_amdgcn_sched_barrier(0);
        look_all(i + 2 * kBatch);
        add(cur);
        __builtin_amdgcn_sched_barrier(0);
        fetch_all(cur);
        __builtin_amdgcn_sched_barrier(0);
        look_all(i + 3 * kBatch);
        add(nxt);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (!more) break;
  }
  __syncthreads();
  for (int i = tid; i < nt * 16; i += kThreads) {
    const int t = i >> 4, q = i & 15, n = n0 + 4 * q;
    if (n >= a.H) continue;
    const f32x4 v = sums[t * 16 + (q ^ (t & 15))];
    const size_t o = (size_t)(t0 + t) * a.H + n;
    if (a.out_f32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o) = v;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) =
          make_uint2(mx_bf16(v[0]) | (mx_bf16(v[1]) << 16), mx_bf16(v[2]) | (mx_bf16(v[3]) << 16));
    }
  }
}

// One 16-byte piece of a matrix per thread, to its place in the tiled layout.
__global__ __launch_bounds__(kThreads) void lora_tile_kernel(const uint16_t* __restrict__ src, long long pieces,
                                                             int rows, int cols, int is_b,
                                                             uint16_t* __restrict__ dst) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= pieces) return;
  const int per_row = cols / 8;
  const long long m = i / ((long long)rows * per_row);
  const int in = (int)(i - m * ((long long)rows * per_row)), r = in / per_row, q = in - r * per_row;
  const size_t at = is_b ? b_at(r, 8 * q, cols)
                         : (size_t)(r & ~15) * cols + (size_t)(q / 4) * 512 + 8 * ((q & 3) * 16 + (r & 15));
  const int held = is_b ? rows : (rows + 15) & ~15;
  *reinterpret_cast<u32x4*>(dst + (size_t)m * held * cols + at) =
      reinterpret_cast<const u32x4*>(src)[i];
}

template <bool DOWN>
hipError_t launch_shrink(const LoraArgs& a, int n_win, int slots, hipStream_t st) {
  const int plans = DOWN ? a.n_blocks * ((a.win + kPlanWindows - 1) / kPlanWindows) : 0;
  lora_sort_kernel<DOWN><<<n_win + plans, kLoraWindow, 0, st>>>(a, n_win);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int tiles = ((DOWN ? 1 : 2) * a.max_rank + 15) / 16;
  if (tiles == 1) {
    const dim3 grid(n_win * slots);
    if (DOWN && a.in_f32) lora_shrink_kernel<1, true, true><<<grid, kThreads, 0, st>>>(a, n_win, slots);
    else lora_shrink_kernel<1, false, DOWN><<<grid, kThreads, 0, st>>>(a, n_win, slots);
  } else {
    const dim3 grid(n_win * slots, (tiles + 1) / 2);
    if (DOWN && a.in_f32) lora_shrink_kernel<2, true, true><<<grid, kThreads, 0, st>>>(a, n_win, slots);
    else lora_shrink_kernel<2, false, DOWN><<<grid, kThreads, 0, st>>>(a, n_win, slots);
  }
  return hipGetLastError();
}

// A window's units are dealt to as many workgroups as fill the device some times
// over: of 144 windows to 14 each 55 + 54 us (products of K, expansion), to 8 each
// 61 + 59, to 28 each 55 + 56.
int windows(const LoraArgs& a) { return (a.R + kLoraWindow - 1) / kLoraWindow; }
int unit_slots(const LoraArgs& a) {
  return std::min(kLoraWindow, std::max(8, 2048 / windows(a)));
}

template <int NT>
hipError_t launch_down_small(const LoraArgs& a, hipStream_t st) {
  const dim3 grid(a.T, (a.H + 16 * kDownWaves * NT - 1) / (16 * kDownWaves * NT));
  if (a.in_f32) lora_down_small_kernel<NT, true><<<grid, 64 * kDownWaves, 0, st>>>(a);
  else lora_down_small_kernel<NT, false><<<grid, 64 * kDownWaves, 0, st>>>(a);
  return hipGetLastError();
}

template <int KB>
hipError_t launch_accumulate(const LoraArgs& a, hipStream_t st) {
  const size_t lds = (size_t)(a.block + 1) * kLoraSlab * 4;
  const int n_slabs = (a.H + kLoraSlab - 1) / kLoraSlab;
  const int grid = 8 * ((n_slabs + 7) / 8) * a.n_blocks;
  lora_accumulate_kernel<KB><<<grid, kThreads, lds, st>>>(a, n_slabs);
  return hipGetLastError();
}

}  // namespace

// Three launches or one.
//
// gate/up: one reads a pair's matrices for every window of 16 rows that holds it.
// Three cost about 45 us and read them far less often where rows share a pair:
// 1026 rows of 4 adapters of rank 64 on 33 experts (H 2048, I 512) 48 us against 75,
// 576 rows 62 against 51; without sharing (32 adapters of rank 16 on 257 experts)
// 1440 rows 87 against 62, 2052 rows 109 against 83.
//
// down: one reads a row's matrices from the cache at 4.6 TB/s, whatever they share;
// three cost about 35 us and 0.2 for each 32 ranks of a unit of a block of tokens
// (a block has the adapters of its share of the tokens: a request's are neighbours).
// 32 adapters on 257 experts: 4104 rows 102 us in one, 146 in three, 11700 rows 235
// and 302, 18432 rows 348 and 261, 36864 rows 662 and 302; 4 adapters: 4104 rows 83
// and 90, 8208 rows 138 and 106, 36864 rows 590 and 115; on 33 experts, rank 64: 576
// rows 37 and 67, 1440 rows 71 and 53, 4104 rows 157 and 52.
//
// The constants come from H 2048, I 512.  At H 4096 with I 1536 and 14336, 8 to 256
// experts and ranks 16, 64 and 128 (22 sizes of 720 to 32768 rows) both rules took the
// faster way, or one within 5% of it, at 20: 2000 rows of one adapter of rank 128 on
// 8 experts 64 against 510 gate/up, 50 against 406 down.  They miss at 800 rows of rank
// 16 on 8 experts (one launch: 68 and 60, three 31 and 22) and 2000 of rank 16 on
// 256 (129 and 124, three 104 and 74).
void lora_choose(LoraArgs& a, bool most) {
  a.block = a.n_blocks = a.win = 0;
  a.large = a.R > kLoraFewRows;
  const double experts = (double)a.E + a.n_shared;
  if (a.halves == 2) {
    const double pairs = experts * std::min(a.n, a.T);
    const double bytes = 4.0 * a.R * a.max_rank * ((double)a.H + a.I);
    if (!most && a.R <= kLoraManyRows && (a.R <= 5 * pairs || bytes < 450e6)) a.large = false;
    return;
  }
  if (a.E + a.n_shared > kLoraPlanMaxE) a.large = false;
  if (!a.large) return;
  const int n_slabs = (a.H + kLoraSlab - 1) / kLoraSlab;
  a.block = kLoraMaxBlock;
  while (a.block > 64 && (long long)((a.T + a.block - 1) / a.block) * n_slabs < 256) a.block /= 2;
  a.n_blocks = (a.T + a.block - 1) / a.block;
  // whole segments
  const double rows = (double)a.block * (a.k + a.n_shared);
  const long long windows = ((long long)a.block * (a.k + a.n_shared) + 63) / 64;
  a.win = (int)((windows + kLoraSegment - 1) / kLoraSegment) * kLoraSegment;
  // offsets into v: 31 bits
  if ((long long)a.n_blocks * a.win * 64 * a.max_rank * 6 >= (1LL << 31)) a.large = false;
  if (most || !a.large) return;
  const double adapters = std::ceil((double)a.n * std::min(a.T, a.block) / a.T);
  const double pairs = experts * std::min(adapters, (double)a.block);
  const double units = pairs * (1.0 - std::exp(-rows / std::max(pairs, 1.0))) + rows / 16;
  const double one = 2.0 * a.R * a.max_rank * ((double)a.H + a.I) / 4.6e6;
  const double rounds = std::max(1.0, (double)a.n_blocks * n_slabs / 256);
  if (a.n == 0 || one < 35.0 + 0.2 * ((a.max_rank + 31) / 32) * rounds * units) a.large = false;
}

hipError_t launch_lora_tile(const uint16_t* src, int n, int rows, int cols, int is_b, uint16_t* dst,
                            hipStream_t st) {
  const long long pieces = (long long)n * rows * (cols / 8);
  const long long grid = (pieces + kThreads - 1) / kThreads;
  if (grid >= 1 << 24) return hipErrorInvalidValue;
  lora_tile_kernel<<<(int)grid, kThreads, 0, st>>>(src, pieces, rows, cols, is_b, dst);
  return hipGetLastError();
}

size_t lora_carve(LoraArgs& a, char* ws) {
  const auto up256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    char* p = ws ? ws + off : nullptr;
    off += up256(bytes);
    return p;
  };
  if (!a.large) return off;
  const size_t n_win = (size_t)(a.R + kLoraWindow - 1) / kLoraWindow, rows = n_win * kLoraWindow;
  a.unit_count = reinterpret_cast<int2*>(take(n_win * sizeof(int2)));
  a.units = reinterpret_cast<LoraGroupUnit*>(take(rows * sizeof(LoraGroupUnit)));
  a.order = reinterpret_cast<uint32_t*>(take((rows + kUnitRows) * 4));   // read past a unit's end
  if (a.halves == 2) {
    a.parts = reinterpret_cast<uint16_t*>(take(rows * 2 * a.max_rank * 6));
  } else {
    const size_t win = (size_t)a.n_blocks * a.win;
    a.weight = reinterpret_cast<float*>(take(rows * 4));
    a.place = reinterpret_cast<uint32_t*>(take(rows * 4));
    a.row_at = reinterpret_cast<uint32_t*>(take(win * 64 * 4));
    a.parts = reinterpret_cast<uint16_t*>(take(win * 64 * a.max_rank * 6));
    a.plan_count = reinterpret_cast<int*>(take(win * 4));
    a.plan = reinterpret_cast<LoraUnit*>(take(win * 64 * sizeof(LoraUnit)));
    a.plan_sums = reinterpret_cast<uint32_t*>(take(win * 64 * 16 * 4));
  }
  return off;
}

hipError_t launch_lora_gateup(const LoraArgs& a, hipStream_t st) {
  if (!a.large) {
    const int grid = (a.R + kLoraSmallRows - 1) / kLoraSmallRows * kLoraSmallRows;
    if (a.R <= 256) lora_gateup_small_kernel<8><<<grid, 512, 0, st>>>(a);
    else lora_gateup_small_kernel<4><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  const int n_win = windows(a), slots = unit_slots(a);
  const hipError_t e = launch_shrink<false>(a, n_win, slots, st);
  if (e != hipSuccess) return e;
  constexpr int kCols = kExpandCols * kWaves;
  const dim3 grid(n_win * slots, (a.ld_h + kCols - 1) / kCols);
  lora_expand_gateup_kernel<<<grid, kThreads, 0, st>>>(a, n_win, slots);
  return hipGetLastError();
}

hipError_t launch_lora_down(const LoraArgs& a, hipStream_t st) {
  if (a.large) {
    const hipError_t e = launch_shrink<true>(a, windows(a), unit_slots(a), st);
    if (e != hipSuccess) return e;
    if (a.max_rank <= 32) return launch_accumulate<1>(a, st);
    if (a.max_rank <= 64) return launch_accumulate<2>(a, st);
    return launch_accumulate<4>(a, st);
  }
  // columns of a workgroup: as few as leave a compute unit to each (192, 384 or 768:
  // one token 7.9 us by 192, 9.2 by 768; 64 tokens 24 and 14.6; 77 tokens, H 1056,
  // fp32 15.8, 9.5 by 384, 10.7)
  const auto groups = [&](int nt) { return (long long)a.T * ((a.H + 16 * kDownWaves * nt - 1) / (16 * kDownWaves * nt)); };
  if (groups(1) <= 256) return launch_down_small<1>(a, st);
  if (groups(2) <= 256) return launch_down_small<2>(a, st);
  return launch_down_small<4>(a, st);
}

}  // namespace moe
