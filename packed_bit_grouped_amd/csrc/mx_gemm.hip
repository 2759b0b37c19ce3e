// Grouped MXFP4 projections for tiles of many activation rows.
//
// The same products as mx_rows16.hip where an expert has tens of rows or
// more: the packed weights are still read once per tile, and the matrix cores
// now matter.  Workgroup = one tile (up to 160 sorted rows of one expert, cut
// evenly) x 128 gate/up units or 256 down rows; 4 waves, one per SIMD (512
// registers).  Wave w owns 64 weight rows - the gate and the up rows of 32
// units, so SiLU*mul pairs registers of one lane, or 64 down rows - as four
// 16-row fragments (NF) against all of the tile's rows.  A4 with few rows per
// expert: tiles of 144, two fragments per wave, two workgroups per compute unit.
//
//  * Weights go from memory into a register ring kD steps of 256 K ahead, two
//    tiled pieces per fragment and step (a contiguous kilobyte per load).
//  * Activations go from memory straight into a ring of LDS buffers (loads
//    that write LDS; rows gathered by token).  A4: 128 bytes of codes per row
//    and step, chunk q of row m in slot q ^ ((m >> 1) & 7); the scale bytes of
//    the whole tile are staged once.  A16: 256 bytes of bf16 per row and
//    sub-step, chunk q in slot q ^ swizzle16(m).  Both spread the 16 lanes that
//    a 128-bit LDS access serves at a time over all banks; the counters show no
//    conflicts for A16, and conflicts in 16% of A4's LDS cycles, which reads the
//    scales by two bytes a lane as well (not separated by a measurement).
//  * A4 feeds codes and scales to the scaled 16x16x128 instruction; A16
//    expands a fragment's 8 codes to bf16 by four conversions (exact) for one
//    16x16x32 step against every row fragment.
//  * Activation rows are whole steps, zeros behind K, by the pass that
//    quantises or copies them, and the tiles' scales behind K are 0 (never
//    255), so K's tail needs no cases.
//
// Measured (4096 tokens, H 4096, I 1536, 256 experts, k 8: 128 rows an expert;
// kernel trace, median and fastest of 30 calls on three sets of weights):
//  * A16 gate/up 768 / 745 us (739 a call in a row of calls: 1.12 PFLOP/s): the
//    matrix pipes are busy 54% of the cycles, the conversions of the weights share
//    the issue slots.  A library bf16 product of 8192^3 random values reaches 1.20.
//    Down 519 / 497, pipes 36% busy: half the work, and 0.54 GB of y.
//  * A4 gate/up 392 / 387 us, 1.71 GB of weights at 4.4 TB/s, matrix pipes 24% busy;
//    down 338 / 334 us, 0.86 GB of weights and 0.54 GB of y.  By clock stamps the loop
//    reads at 6.3 TB/s (22.7 of a workgroup's 30.6 us, down 9.6 of 20.0): the
//    rest is finding the tile (1.6), its rows (0.5 to 1.4), the first loads (2.6
//    to 4.2) and the stores (2.0 to 3.8), which one workgroup per compute unit
//    does not overlap.  64 rows an expert, two workgroups: gate/up 333 / 319 us,
//    down 243 / 239, pipes 17% and 11% busy.
//  * A tile of 160 rows reads the weights once for nearly every expert here; with
//    tiles of 128 an expert in two needs a second pass.
//  * Tried: a tile's codes kept in LDS while several blocks of weights pass
//    (A4 down here 343 -> 305 us, but 32 experts 211 -> 255, gate/up with K 1024
//    75 -> 114); columns of down in parts, so that y stays in the cache (460 ->
//    522 us for parts of 1024); a grid of the likely tiles whose workgroups walk
//    to further ones (398 -> 418 us); several blocks of columns per workgroup, the
//    next one's first loads before the stores (397 -> 434 us: the accumulators
//    then move between the register files in every turn).
#include "mx_common.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsMax = 160;      // rows per tile
constexpr int kRowsNarrow = 144;   // of the kernel with two workgroups per compute unit
constexpr int kKS = 256;        // K per weight step
constexpr int kXcd = 8;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// At most N vector-memory operations of this wave in flight, every LDS access
// done, then the workgroup barrier; nothing is scheduled across it.
template <int N>
__device__ __forceinline__ void vm_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}

template <int N>
struct Int {
  static constexpr int value = N;
};

// A16: chunk q of row m of a stage lies in slot q ^ swizzle16(m) of its 16.  A
// 128-bit LDS access serves 16 lanes at a time, but not 16 in a row: lanes 0-3
// and 12-15 of one quarter of the wave go with 4-11 of the next, so the two
// quarters (chunks 4g + q and 4g + 4 + q) have to differ in the low two bits
// for those rows.  (With slot q ^ (m & 15) half of the LDS cycles were
// conflicts.)
__device__ __forceinline__ int swizzle16(int m) { return ((m & 3) << 2) | ((m >> 2) & 3); }

struct GemmArgs {
  MxProj p;
  int KP;              // row length of the activation copy
  int n_ub;            // workgroups per tile
  int max_tiles;       // host bound of the routed tiles
  int sh_per;          // tiles per shared expert
  int sc_pitch;        // A4: LDS bytes per row of scales
};

// A4 has one activation stage per weight step, A16 two of 128 K.  kBufs stages
// of LDS; kD weight steps in registers.
template <bool ACT4>
struct Ring {
  static constexpr int kStages = ACT4 ? 1 : 2;
  static constexpr int kBufs = 3;
  static constexpr int kD = ACT4 ? 3 : 2;
  static constexpr int kRowChunks = ACT4 ? 8 : 16;   // 16-byte chunks per row and stage
  // a stage's chunks; the waves load them 64 at a time, an equal number each:
  // what goes past an odd number of fragments lands behind the ring (spill), or
  // where LDS is not short, in a buffer rounded up
  static constexpr int buf_chunks(int mt, int nf) {
    return kRowChunks * 16 * (nf == 2 ? mt : (mt + 1) & ~1);
  }
  static constexpr int spill(int nf) { return nf == 2 ? 128 : 0; }
  static constexpr int chunks(int mt_max, int nf) { return kBufs * buf_chunks(mt_max, nf) + spill(nf); }
};

// NF: weight fragments of 16 rows per wave.
template <int NF>
struct WStep {
  u32x4 c[NF][2];
  uint32_t s[NF];
};

struct Tile {
  const uint8_t* act;   // padded activation rows
  uint32_t act_bytes;
  int row_bytes;        // of one padded row
  int K, U, n_st;
  int u0;               // first unit / row of this wave
  int orow;             // first output row
};

// The wave's weights: four 16-row blocks; blocks and steps past the end lie past
// the buffer (at most 2^30 bytes), where nothing is read.  Offsets are unsigned:
// a step past the end of a block past the end is twice kNone.
constexpr uint32_t kNone = 0x40000000;
static_assert(2ull * kNone <= UINT32_MAX, "no offset comes round to a valid one");

template <int NF>
struct Weights {
  __amdgpu_buffer_rsrc_t crs, srs;
  uint32_t coff[NF], soff[NF];
  int n_st;

  template <int MODE>
  __device__ __forceinline__ void init(const Tile& t, const uint8_t* w, const uint8_t* ws, int e) {
    const int lane = threadIdx.x & 63;
    const int N = MODE != 1 ? 2 * t.U : t.U;
    const size_t cb = mx_code_bytes(N, t.K), sb = mx_scale_bytes(N, t.K);
    crs = make_rsrc(w + e * cb, (uint32_t)cb);
    srs = make_rsrc(ws + e * sb, (uint32_t)sb);
    n_st = t.n_st;
    const int pieces = mx_pieces(t.K), words = (pieces + 3) / 4;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int u = MODE != 1 ? t.u0 + 16 * (f % (NF / 2)) : t.u0 + 16 * f;
      const int rb = ((MODE != 1 && f >= NF / 2 ? t.U : 0) + u) / 16;
      coff[f] = u < t.U ? rb * pieces * 1024 + lane * 16 : kNone;
      soff[f] = u < t.U ? rb * words * 256 + lane * 4 : kNone;
    }
  }
  __device__ __forceinline__ void load_c(int st, int j, WStep<NF>& w) const {
    const uint32_t o = st < n_st ? st * 2048 + j * 1024 : kNone;
#pragma unroll
    for (int f = 0; f < NF; ++f)
      w.c[f][j] = __builtin_amdgcn_raw_buffer_load_b128(crs, (int)(coff[f] + o), 0, 2);
  }
  __device__ __forceinline__ void load_s(int st, WStep<NF>& w) const {
    const uint32_t o = st < n_st ? (st >> 1) * 256 + (st & 1) * 2 : kNone;
#pragma unroll
    for (int f = 0; f < NF; ++f)
      w.s[f] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(srs, (int)(soff[f] + o), 0, 0);
  }
  __device__ __forceinline__ void load(int st, WStep<NF>& w) const {
    load_c(st, 0, w);
    load_c(st, 1, w);
    load_s(st, w);
    __builtin_amdgcn_sched_barrier(0);
  }
};

// w0: the weights of the first step, already on their way.
template <int MODE, bool ACT4, int NF, int TM, int MT>
__device__ __forceinline__ void body(const GemmArgs& ga, const Tile& t, const Weights<NF>& wt, WStep<NF>& w0,
                                     u32x4* As, const int* tok, const uint8_t* sc, int nrows) {
  using R = Ring<ACT4>;
  constexpr int kBuf = R::buf_chunks(MT, NF);
  constexpr int nA = (kBuf + 255) / 256;       // activation loads per wave and stage
  constexpr int kSpill = R::kBufs * R::buf_chunks((TM + 15) / 16, NF);
  static_assert(nA * 256 - kBuf <= R::spill(NF), "the loads' last chunks");
  constexpr int kD = R::kD, kBufs = R::kBufs;
  constexpr int nS = NF, nW = 2 * NF + nS;      // weight loads per step
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int n_st = t.n_st, n_stage = n_st * R::kStages;
  auto load_c = [&](int st, int j, WStep<NF>& w) { wt.load_c(st, j, w); };
  auto load_s = [&](int st, WStep<NF>& w) { wt.load_s(st, w); };

  // ---- activation pieces of this lane: LDS slot q of a stage holds the chunk
  // that the swizzle puts there
  const __amdgpu_buffer_rsrc_t ars = make_rsrc(t.act, t.act_bytes);
  int aoff[nA];
#pragma unroll
  for (int i = 0; i < nA; ++i) {
    const int q = (wave * nA + i) * 64 + lane;
    const int m = q / R::kRowChunks;
    if (ACT4) {
      aoff[i] = tok[m] * t.row_bytes + (((q & 7) ^ ((m >> 1) & 7)) * 16);
    } else {
      aoff[i] = tok[m] * t.row_bytes + (((q & 15) ^ swizzle16(m)) * 16);
    }
  }
  auto dma = [&](int sg, int buf) {
    sg = min(sg, n_stage - 1);                 // past the end: the last stage once more
    const int o = sg * (ACT4 ? 128 : 256);
#pragma unroll
    for (int i = 0; i < nA; ++i) {
      const int q = (wave * nA + i) * 64;
      const int to = nA * 256 == kBuf || q < kBuf ? buf * kBuf + q : kSpill + q - kBuf;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ars, (__attribute__((address_space(3))) void*)(As + to), 16, aoff[i], o, 0, 0);
    }
  };

  mx_f32x4 acc[NF][MT];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[f][m] = mx_f32x4{0, 0, 0, 0};

  // Sub-steps of a stage: A4 two of 128 K (block 2g + q of every lane), A16
  // four of 32 K (word q of block 2g + j).  A row fragment's register is
  // refilled from LDS for the next sub-step as soon as its four matrix
  // instructions are issued: the other fragments' instructions (64 cycles
  // each) cover the read.  A16 expands the next sub-step's weights meanwhile.
  // Before a stage's last sub-step every wave has read all of its buffer, so
  // the stage's one barrier stands there: it frees the buffer for the stage
  // kBufs on, and covers the next stage's loads, which the last sub-step reads.
  constexpr int kQ = ACT4 ? 2 : 4;
  const int sw = ACT4 ? (c >> 1) & 7 : swizzle16(c);
  const u32x4* Ac = As + c * R::kRowChunks;
  u32x4 x[MT];
  mx_bf16x8 wv[2][NF];
  uint32_t sx[MT];
  auto x_at = [&](int b, int q) {
    return Ac + b * kBuf + ((ACT4 ? 4 * q + g : 4 * g + q) ^ sw);
  };
  auto sx_at = [&](int st) {
    st = min(st, n_st - 1);
    return sc + c * ga.sc_pitch + (st >> 1) * 16 + 4 * g + (st & 1) * 2;
  };
  auto expand = [&](int j, int q, const WStep<NF>& w, mx_bf16x8(&v)[NF]) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
      v[f] = mx_word_to_bf16(w.c[f][j][q], mx_scale_f32((w.s[f] >> (8 * j)) & 255u));
  };
  // issue order of a sub-step: per row fragment four matrix instructions with
  // the conversions and memory loads between them, then its LDS reads
  auto spread = [&](auto n_ds, auto n_ld) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (NF * m + f < n_ld.value) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, ACT4 ? 1 : 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, n_ds.value, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int buf = 0;
  // After the loads of stage a + 1 (issued behind the barrier of stage a + 1 -
  // kBufs) and before the barrier of stage a come the weight loads of kBufs - 1
  // stages (the prologue's: at least as many) and the activation loads of
  // kBufs - 2.
  constexpr int kAfter = (kBufs - 2) * nA + (ACT4 ? (kBufs - 1) * nW : nW);

  // stage (st, j) from buffer buf with w; wn holds the next step's weights
  auto stage = [&](int st, int j, WStep<NF>& w, const WStep<NF>& wn) {
    const int a = st * R::kStages + j;
    const int nb = buf == kBufs - 1 ? 0 : buf + 1;
    if constexpr (ACT4) {
      uint32_t sws[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) sws[f] = w.s[f];
      const u32x4* p = x_at(buf, 1);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[f][m] = mx_mfma_fp4<0>(w.c[f][0], sws[f], x[m], sx[m], acc[f][m]);
        x[m] = p[m * 16 * R::kRowChunks];
      }
      spread(Int<1>(), Int<0>());
      vm_barrier<kAfter>();
      dma(a + kBufs, buf);
      load_c(st + kD, 0, w);
      load_s(st + kD, w);
      p = x_at(nb, 0);
      const uint8_t* ps = sx_at(st + 1);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[f][m] = mx_mfma_fp4<1>(w.c[f][1], sws[f], x[m], sx[m], acc[f][m]);
        x[m] = p[m * 16 * R::kRowChunks];
        sx[m] = *reinterpret_cast<const uint16_t*>(ps + 16 * m * ga.sc_pitch);
      }
      spread(Int<2>(), Int<nA + NF + nS>());
      load_c(st + kD, 1, w);
      __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const int cur = q & 1, nxt = cur ^ 1;
        const u32x4* p;
        if (q < kQ - 1) {
          p = x_at(buf, q + 1);
          expand(j, q + 1, w, wv[nxt]);
        } else {
          vm_barrier<kAfter>();
          dma(a + kBufs, buf);
          p = x_at(nb, 0);
          if (j == 0) expand(1, 0, w, wv[nxt]);
          else expand(0, 0, wn, wv[nxt]);
          load_c(st + kD, j, w);
          if (j == 1) load_s(st + kD, w);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int f = 0; f < NF; ++f)
            acc[f][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                wv[cur][f], __builtin_bit_cast(mx_bf16x8, x[m]), acc[f][m], 0, 0, 0);
          x[m] = p[m * 16 * R::kRowChunks];
        }
        if (q < kQ - 1) spread(Int<1>(), Int<0>());
        else if (j == 0) spread(Int<1>(), Int<nA + NF>());
        else spread(Int<1>(), Int<nA + NF + nS>());
      }
    }
    buf = nb;
  };
  auto step = [&](int st, WStep<NF>& w, const WStep<NF>& wn) {
    stage(st, 0, w, wn);
    if constexpr (!ACT4) stage(st, 1, w, wn);
  };

  // Prologue: the loads in an order for which kAfter holds in the first stages
  // too (the first step's weights went before).
  WStep<NF> w1, w2;
  dma(0, 0);
  dma(1, 1);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (ACT4) {
    wt.load(1, w1);
    dma(2, 2);
    __builtin_amdgcn_sched_barrier(0);
    wt.load(2, w2);
  } else {
    dma(2, 2);
    __builtin_amdgcn_sched_barrier(0);
    wt.load(1, w1);
  }
  vm_barrier<2 * nA + (kD - 1) * nW>();   // stage 0 (and the scales) in LDS
  {
    const u32x4* p = x_at(0, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = p[m * 16 * R::kRowChunks];
    if constexpr (ACT4) {
      const uint8_t* ps = sx_at(0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        sx[m] = *reinterpret_cast<const uint16_t*>(ps + 16 * m * ga.sc_pitch);
    } else {
      expand(0, 0, w0, wv[0]);
    }
  }

  // Whole turns of the ring, then the steps that are left (a condition inside
  // the turn would keep two sets of accumulators alive).  The weight loads of
  // those last steps have no reader and may be dropped: the barriers that count
  // them are the first of the rest, whose loads went out in the turns before,
  // and the last, which nothing needs to wait for.
  int base = 0;
#pragma unroll 1
  for (; base + kD <= n_st; base += kD) {
    step(base, w0, w1);
    if constexpr (ACT4) {
      step(base + 1, w1, w2);
      step(base + 2, w2, w0);
    } else {
      step(base + 1, w1, w0);
    }
  }
  if (base < n_st) step(base, w0, w1);
  if constexpr (ACT4)
    if (base + 1 < n_st) step(base + 1, w1, w2);
  __builtin_amdgcn_s_waitcnt(0);   // nothing writes LDS after this

  // ---- lane: row 16 m + c, four consecutive units of every fragment
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = 16 * m + c;
#pragma unroll
    for (int f = 0; f < NF; ++f) mx_keep(acc[f][m]);
    if (row >= nrows) continue;
    if (MODE == 0) {
      uint16_t* h = static_cast<uint16_t*>(ga.p.out) + (size_t)(t.orow + row) * ga.p.ld_out;
      float gv[2 * NF], uv[2 * NF], hv[2 * NF];
#pragma unroll
      for (int i = 0; i < 2 * NF; ++i) {
        gv[i] = acc[i / 4][m][i % 4];
        uv[i] = acc[i / 4 + NF / 2][m][i % 4];
      }
      mx_silu_mul(gv, uv, hv);
#pragma unroll
      for (int f = 0; f < NF / 2; ++f) {
        const int u = t.u0 + 16 * f + 4 * g;
        if (u >= t.U) continue;
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mx_bf16(hv[4 * f + i]);
        *reinterpret_cast<uint2*>(h + u) = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
      }
    } else if (MODE == 2) {
      // the gate and up sums as they are, up behind the row's first half
      float* y = static_cast<float*>(ga.p.out) + (size_t)(t.orow + row) * ga.p.ld_out;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int u = t.u0 + 16 * (f % (NF / 2)) + 4 * g;
        if (u < t.U)
          *reinterpret_cast<mx_f32x4*>(y + u + (f < NF / 2 ? 0 : ga.p.ld_out / 2)) = acc[f][m];
      }
    } else {
      float* y = static_cast<float*>(ga.p.out) + (size_t)(t.orow + row) * ga.p.ld_out;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int u = t.u0 + 16 * f + 4 * g;
        if (u < t.U) *reinterpret_cast<mx_f32x4*>(y + u) = acc[f][m];
      }
    }
  }
}

// Routed rows: an expert with n rows has ceil(n / TM) tiles of even size.
__device__ __forceinline__ void cut(int first, int end, int n, int k, int& r0, int& r1) {
  const int rows = ((end - first + n - 1) / n + 15) & ~15;
  r0 = min(first + k * rows, end);
  r1 = min(r0 + rows, end);
}

template <int TM, int PER>
__device__ __forceinline__ bool pick_tile(const GemmArgs& ga, bool& is_sh, int& e, int& r0, int& r1,
                                          int& ub) {
  const MxProj& a = ga.p;
  MxTiles<TM, PER> tl;
  tl.load(a.offsets, a.E, a.P);
  const int n_sh = a.n_shared * ga.sh_per;
  const int n_slots = n_sh + min(__builtin_amdgcn_readlane(tl.pre, 63), ga.max_tiles);
  // XCD blockIdx % 8 takes a contiguous range of tiles: the workgroups of one
  // tile share its activation rows in one L2, the tiles of one expert its weights
  const int b = blockIdx.x, xcd = b % kXcd, li = b / kXcd;
  const int per_xcd = (n_slots + kXcd - 1) / kXcd;
  const int local = li / ga.n_ub, slot = xcd * per_xcd + local;
  ub = li - local * ga.n_ub;
  if (local >= per_xcd || slot >= n_slots) return false;
  is_sh = slot < n_sh;
  if (is_sh) {
    e = slot / ga.sh_per;
    cut(0, a.T, ga.sh_per, slot - e * ga.sh_per, r0, r1);
    return r0 < r1;
  }
  int first, end, k;
  if (!tl.find(slot - n_sh, e, first, end, k)) return false;
  cut(first, end, (end - first + TM - 1) / TM, k, r0, r1);
  return r0 < r1;
}

template <int MODE, bool ACT4, int NF, int TM>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4 / NF, 4 / NF)))
void mx_gemm_kernel(GemmArgs ga) {
  extern __shared__ __align__(16) unsigned char smem[];
  const MxProj& a = ga.p;
  int* tok = reinterpret_cast<int*>(smem);                   // [kRowsMax]
  u32x4* As = reinterpret_cast<u32x4*>(smem + kRowsMax * 4);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  bool is_sh;
  int e, r0, r1, ub;
  if (!(a.E <= 128 ? pick_tile<TM, 2>(ga, is_sh, e, r0, r1, ub) : pick_tile<TM, 8>(ga, is_sh, e, r0, r1, ub)))
    return;
  const int nrows = r1 - r0;

  Tile t;
  t.K = is_sh ? a.K_sh : a.K;
  t.U = is_sh ? a.U_sh : a.U;
  t.n_st = (t.K + kKS - 1) / kKS;
  const int ublk = ub * (MODE != 1 ? 32 : 64) * NF;
  if (ublk >= t.U) return;
  t.u0 = ublk + wave * (MODE != 1 ? 8 : 16) * NF;
  t.orow = is_sh ? a.P + e * a.T + r0 : r0;
  // gate/up gathers rows of x by token; down reads its own rows, the shared
  // experts' behind the routed ones
  const int arow = MODE != 1 ? 0 : (is_sh ? a.P : 0);
  const size_t stride = ACT4 ? (size_t)ga.KP / 2 : (size_t)a.ld_in * 2;
  t.row_bytes = (int)stride;
  t.act = (ACT4 ? a.q : reinterpret_cast<const uint8_t*>(a.x)) + arow * stride;
  const int act_rows = MODE != 1 ? a.T : (is_sh ? a.n_shared * a.T : a.P);
  t.act_bytes = (uint32_t)(act_rows * stride);
  // the first step's weights need only the tile: on their way before its rows
  // are looked up
  Weights<NF> wt;
  wt.template init<MODE>(t, is_sh ? a.w_sh : a.w, is_sh ? a.ws_sh : a.ws, e);
  WStep<NF> w0;
  wt.load(0, w0);

  if (tid < kRowsMax) {
    const int m = tid < nrows ? tid : 0;   // padding rows repeat row 0 (not stored)
    int row;
    if (MODE == 1) {
      row = is_sh ? e * a.T + r0 + m : r0 + m;
    } else if (is_sh) {
      row = r0 + m;
    } else {
      const int p = a.sorted_pair[r0 + m];
      row = (unsigned)p < (unsigned)a.P ? p / a.k : 0;
    }
    tok[tid] = row;
  }
  __syncthreads();
  const int mt = (nrows + 15) / 16;
  uint8_t* sc = nullptr;
  if (ACT4) {
    // the tile's scale bytes, by loads that write LDS, ahead of every activation
    // load: rows of an odd number of 16-byte chunks, so that 16 rows' words lie
    // on different banks (an even number is followed by a chunk that is not read)
    sc = smem + kRowsMax * 4 + Ring<true>::chunks((TM + 15) / 16, NF) * 16;
    const int row = ga.KP / kMxBlock, chunks = ga.sc_pitch / 16;
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc(a.s + (size_t)arow * row, (uint32_t)((size_t)act_rows * row));
    const int n = mt * 16 * chunks;
    for (int i = wave * 64; i < n; i += kThreads) {
      const int q = min(i + lane, n - 1), m = q / chunks, ch = min(q - m * chunks, row / 16 - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void*)(sc + i * 16), 16, tok[m] * row + ch * 16, 0, 0,
          0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#define MX_BODY(MT) body<MODE, ACT4, NF, TM, MT>(ga, t, wt, w0, As, tok, sc, nrows)
  if (mt <= 2) MX_BODY(2);
  else if (mt <= 4) MX_BODY(4);
  else if (mt <= 6) MX_BODY(6);
  else if (mt == 7) MX_BODY(7);
  else if (mt == 8) MX_BODY(8);
  else if (TM <= 144 || mt == 9) MX_BODY(9);
  else if constexpr (TM > 144) MX_BODY(10);
#undef MX_BODY
}

int sc_pitch(int KP) { return (KP / kMxBlock) | 16; }   // KP / 32 is a multiple of 16

size_t lds_bytes(bool act4, int KP, int tm, int nf) {
  const size_t ring = act4 ? Ring<true>::chunks((tm + 15) / 16, nf) : Ring<false>::chunks((tm + 15) / 16, nf);
  return kRowsMax * 4 + ring * 16 + (act4 ? (size_t)tm * sc_pitch(KP) + 1024 : 0);
}

// The launch's tiles and grid.
struct Plan {
  bool narrow;
  int KP, tm, sh_per, max_tiles, n_ub;
  long long grid;
};

Plan plan(const MxProj& a, int mode, int act4) {
  Plan p;
  p.KP = mx_pad_k(a.ld_in);   // row length of the activation copy
  // Two workgroups per compute unit, each with half the weight rows per wave: one's
  // start and stores pass behind the other's loop (by clock stamps 8 of 31 us of a
  // gate/up workgroup, 10 of 20 of down, whose loop alone reads 6.3 TB/s), but the
  // activations are read twice as often.  A4 calls (down with the sum), us, one /
  // two workgroups, by rows per expert.  H 4096, I 1536: 256 experts, 12 rows gate/up
  // 280/264, down 206/195, 32 rows 295/279, 243/231, 64 rows 322/309, 309/289, 80 rows
  // 340/326, 350/323; 32 experts, 96 rows 57/54, 53/52; 8 experts, 96 rows 28/21,
  // 26/22.  H 2048, I 768, 128 experts: 32 rows 48/47, 49/46, 96 rows 59/58, 76/75.
  // In eight layers with 12 to 96 rows it was never more than 1% slower.  Beyond 96
  // the two win in turn, gate/up and down alike, as the tiles fall into rounds of the
  // chip: 256 experts, 128 rows 398/400, 460/437; 32 experts, 192 rows 87/91, 84/93;
  // 8 experts, 128 rows 31/33, 30/30, 384 rows 55/48, 50/47; H 2048, 128 experts, 128
  // rows 65/68, 89/95; I 14336, 8 experts, 128 rows gate/up 124/182.
  p.narrow = act4 && a.P <= 96LL * a.E && lds_bytes(true, p.KP, kRowsNarrow, 2) <= 80 * 1024;
  p.tm = p.narrow ? kRowsNarrow : kRowsMax;
  p.sh_per = (a.T + p.tm - 1) / p.tm;
  p.max_tiles = moe_permute_max_tiles(a.T, a.k, a.E, p.tm);
  const int step = (mode == 0 ? 32 : 64) * (p.narrow ? 2 : 4);
  const int U = a.n_shared > 0 && a.U_sh > a.U ? a.U_sh : a.U;
  p.n_ub = (U + step - 1) / step;
  const long long slots = (long long)a.n_shared * p.sh_per + p.max_tiles;
  p.grid = (slots + kXcd - 1) / kXcd * kXcd * p.n_ub;
  return p;
}

}  // namespace

bool mx_gemm_ok(const MxProj& a, int mode, int act4) {
  const int KP = mx_pad_k(a.K > a.K_sh ? a.K : a.K_sh);
  if (lds_bytes(act4, KP, kRowsMax, 4) > 160 * 1024) return false;
  // 32-bit offsets into one matrix and into the activation rows
  const long long rows = mode == 0 ? a.T : (long long)a.P + (long long)a.n_shared * a.T;
  const long long stride = act4 ? mx_pad_k(a.ld_in) / 2 : 2LL * mx_pad_k(a.ld_in);
  if (rows * stride >= (1LL << 31)) return false;
  const int per = mode == 0 ? 2 : 1;
  return mx_code_bytes(per * a.U, a.K) < (1u << 30) && mx_code_bytes(per * a.U_sh, a.K_sh) < (1u << 30) &&
         plan(a, mode, act4).grid <= kMxMaxGrid;
}

int mx_gemm_tile_rows(const MxProj& a, int mode, int act4) { return plan(a, mode, act4).tm; }

hipError_t launch_mx_gemm(const MxProj& a, int mode, int act4, hipStream_t st) {
  const Plan p = plan(a, mode, act4);
  const GemmArgs ga = {a, p.KP, p.n_ub, p.max_tiles, p.sh_per, sc_pitch(p.KP)};
  const size_t lds = lds_bytes(act4, p.KP, p.tm, p.narrow ? 2 : 4);
#define MX_GO(MODE, ACT4, NF, TM) \
  mx_gemm_kernel<MODE, ACT4, NF, TM><<<(int)p.grid, kThreads, lds, st>>>(ga)
  if (mode == 0 && a.raw) {
    if (p.narrow) MX_GO(2, true, 2, kRowsNarrow);
    else if (act4) MX_GO(2, true, 4, kRowsMax);
    else MX_GO(2, false, 4, kRowsMax);
  } else if (p.narrow) {
    if (mode == 0) MX_GO(0, true, 2, kRowsNarrow);
    else MX_GO(1, true, 2, kRowsNarrow);
  } else if (act4) {
    if (mode == 0) MX_GO(0, true, 4, kRowsMax);
    else MX_GO(1, true, 4, kRowsMax);
  } else {
    if (mode == 0) MX_GO(0, false, 4, kRowsMax);
    else MX_GO(1, false, 4, kRowsMax);
  }
#undef MX_GO
  return hipGetLastError();
}

}  // namespace moe
