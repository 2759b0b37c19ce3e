// C ABI of the MXFP4 layer: host-side argument checks, workspace layout and
// dispatch (the same rules as api.cpp: nothing allocates, synchronizes or
// reads device memory).
#include <hip/hip_runtime.h>

#include <cstring>

#include "mx_common.h"

using namespace moe;

namespace {

constexpr int kSortTile = 4096;   // the sort's own tile list is not used

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_E_DEVICE; }
int ld_h_of(int I, int n_shared, int I_shared) {
  return n_shared > 0 && I_shared > I ? I_shared : I;
}

// Sizes of the projections (pointers null).
MxProj gateup_dims(int T, int H, int I, int E, int k, int n_shared, int I_shared) {
  MxProj a;
  std::memset(&a, 0, sizeof(a));
  a.T = T;
  a.k = k;
  a.P = T * k;
  a.E = E;
  a.n_shared = n_shared;
  a.ld_in = H;
  a.K = a.K_sh = H;
  a.U = I;
  a.U_sh = n_shared > 0 ? I_shared : 0;
  a.ld_out = ld_h_of(I, n_shared, I_shared);
  return a;
}

MxProj down_dims(int T, int H, int I, int E, int k, int n_shared, int I_shared) {
  MxProj a = gateup_dims(T, H, I, E, k, n_shared, I_shared);
  a.ld_in = ld_h_of(I, n_shared, I_shared);
  a.K = I;
  a.K_sh = n_shared > 0 ? I_shared : I;
  a.U = a.U_sh = a.ld_out = H;
  return a;
}

// n matrices of one size, 0 beyond any memory (a matrix has fewer than 2^62 bytes).
size_t bank_bytes(int n, size_t one) {
  size_t all;
  return __builtin_mul_overflow((size_t)n, one, &all) ? 0 : all;
}

bool bank_ok(const moe_mxbank* b) {
  return b && b->codes && b->scales && aligned(b->codes, 16) && aligned(b->scales, 4);
}

// A16 rows that are not whole steps of the matrix kernel are copied to padded ones.
bool pad_x(int H) { return H % 256 != 0; }
bool pad_h(int I, int n_shared, int I_shared) {
  return I % 256 != 0 || (n_shared > 0 && I_shared % 256 != 0);
}

// Whether a projection runs on tiles of up to 160 rows or of 16.  A tile of 160
// costs its workgroup a long pass whatever its rows (so there have to be enough
// of them to fill the chip: the first test, in pieces of weights, an expert's
// last tile counted as half), one of 16 reads the weights anew for every 16 rows
// and converts them for 16.
//  * A16 expands the weights on the vector units, so it is the work that decides:
//    rows x blocks of columns x pieces of K.  us, 16 rows / 160 rows, H 2048,
//    I 768, 128 experts, k 8: gate/up of 16 tokens 34/40, of 24 41/41, of 32
//    45/42, of 256 88/45; down of 64 tokens 33/35, of 128 38/37, of 256 55/40.
//    H 4096, I 1536, 256 experts, k 8: gate/up of 4 tokens 46/47, of 8 (one row
//    an expert) 83/77, of 16 132/121, of 64 296/257; down of 16 84/77, of 64
//    187/167.
//    But not with fewer workgroups than half the compute units (the experts that
//    P pairs are likely to touch, about E P / (E + P), x blocks of columns) until
//    an expert's rows fill a tile of 16: H 4096, I 1536, 8 experts, k 2: gate/up
//    of 32 tokens (8 rows) 17/22, of 48 20/22, of 64 26/22; down of 48 14/15, of
//    64 18/16.  H 8192, I 2048: gate/up of 24 tokens 34/39, of 48 41/39; down,
//    with twice the blocks, of 24 24/19.  H 4096, I 14336: down of 24 tokens
//    55/65, of 48 72/67.
//    (Of 448 sizes measured 69 still run more than 5% longer than on the other
//    kernel: 1.1x to 1.2x for 16 tokens on 64 experts, whose 41 tiles take a third
//    round of the chip, two shared experts of H 2048 and I 1408, down of 80 tokens,
//    experts chosen by a Zipf prior, down of 128; 1.4x for gate/up of 4 tokens with
//    I 14336 and for down of 96 to 192 tokens on 8 or 32 experts; 1.4x to 1.8x at
//    short K, H 512, 512 experts, 16 to 64 tokens.  The rule knows neither how tiles
//    fall on the chip nor how rows on the experts.)
//  * A4 takes codes on both sides and gains from the rows of an expert alone.
//    The same sizes: gate/up of 128 tokens (8 rows an expert) 41/42, of 256
//    54/43; down of 192 tokens 35/36, of 256 41/38; 8 experts, 32 tokens (8 rows)
//    gate/up 14/16, down 12/13, 64 tokens 18/17, 16/14; 256 experts, 256 tokens
//    (8 rows) 287/260, 214/187, 512 tokens 434/262, 293/202 (with that many
//    experts the larger tiles win from 6 rows an expert on, which the rule leaves).
//  * Few workgroups: H 1056, I 352, 8 experts, k 3, A16 gate/up of 512 tokens
//    (351 pieces) 19/21, of 1024 (621) 29/26.
bool large_tiles(const MxProj& a, bool act4, int mode) {
  const long long n_ub = mode == 0 ? (a.U + 127) / 128 : (a.U + 255) / 256;
  const long long work = n_ub * mx_pieces(a.K);
  const long long tiles = a.P / 160 + (a.E < a.P ? a.E : a.P) / 2;
  if (tiles * work < 500) return false;
  if (act4) {
    if (a.P < 16LL * a.E) return false;
  } else {
    const long long touched = (long long)a.E * a.P / (a.E + a.P);
    if (a.P * work < (mode == 0 ? 24576 : 40960)) return false;
    if (touched * n_ub < 128 && a.P < 12LL * a.E) return false;
  }
  return mx_gemm_ok(a, mode, act4);
}

// Pieces of weight blocks that all workgroups on tiles of 16 rows pass, at most:
// what quantising the rows in each of them costs.
long long rows16_work(const MxProj& a, int mode) {
  const long long n_ub = mode == 0 ? (a.U + 15) / 16 : (a.U + 31) / 32;
  const long long slots = a.n_shared * ((a.T + 15LL) / 16) + moe_permute_max_tiles(a.T, a.k, a.E, 16);
  return slots * n_ub * mx_pieces(a.K);
}

// A4 on tiles of 16 rows: whether the rows are quantised once, by a launch of
// their own, or by every workgroup that reads them (the same codes).  us, in the
// workgroups / by a launch: H 2048, I 768, 128 experts, k 8, gate/up of 1 token
// (work 6144) 6.8/7.2, of 2 (12288) 9.4/9.4, of 4 15.9/13.3, of 16 38/28; down of
// 2 tokens (6144) 8.7/9.7, of 4 (12288) 12.3/12.2, of 16 24.7/21.1; H 1024,
// I 512, 64 experts, k 4, gate/up of 8 tokens (8192) 6.5/7.7, of 16 10.8/10.5.
constexpr long long kCodesWork = 12288;

bool codes_first(const MxProj& a, int mode) { return rows16_work(a, mode) > kCodesWork; }

// Whether a few tokens are routed and sorted by every workgroup of gate/up: one
// or two launches less, for the passes over the logits in each and, A4, the
// quantisation there.  Layer, us, by a launch / in the workgroups: H 2048, I 768,
// 128 experts, k 8, one shared, A16 1 token 19.0/14.7, 3 tokens 29.6/26.7, A4 the
// same 20.7/16.3, 28.9/27.8; H 4096, I 1536, 256 experts, A16 1 token 31.4/31.0
// (work 24576), 2 tokens 47.9/47.1, 3 tokens 63.4/66.3, A4 1 token 31.0/32.3.
bool route_inside(const MxProj& a, bool act4) {
  return mx_route_gateup_ok(a.T, a.k, a.E, a.ld_in) && !large_tiles(a, act4, 0) &&
         rows16_work(a, 0) < (act4 ? 2 : 5) * kCodesWork;
}

moe_status check_shape(int act, int T, int H, int I, int E, int k, int n_shared, int I_shared) {
  if (act != MOE_A16 && act != MOE_A4) return MOE_E_INVAL;
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0 || n_shared < 0) return MOE_E_INVAL;
  if (k > E) return MOE_E_INVAL;
  if (n_shared > 0 && I_shared <= 0) return MOE_E_INVAL;
  if (H % kMxBlock || I % kMxBlock || (n_shared > 0 && I_shared % kMxBlock))
    return MOE_E_UNSUPPORTED;
  if (H >= kMxMaxLen || I >= kMxMaxLen || (n_shared > 0 && I_shared >= kMxMaxLen))
    return MOE_E_UNSUPPORTED;
  if (E > kPermMaxE || T > 65535 || n_shared > 65535) return MOE_E_UNSUPPORTED;
  if ((long long)T * k >= (1LL << 24)) return MOE_E_UNSUPPORTED;
  const long long rows = (long long)T * ((long long)k + n_shared);
  if (rows * H >= (1LL << 31) || rows * ld_h_of(I, n_shared, I_shared) >= (1LL << 31))
    return MOE_E_UNSUPPORTED;
  // more workgroups than a launch holds (the routed launch has one more than counted)
  const int act4 = act == MOE_A4;
  const MxProj g = gateup_dims(T, H, I, E, k, n_shared, I_shared);
  const MxProj d = down_dims(T, H, I, E, k, n_shared, I_shared);
  if ((mx_rows16_grid(g, 0) >= kMxMaxGrid && !large_tiles(g, act4, 0)) ||
      (mx_rows16_grid(d, 1) >= kMxMaxGrid && !large_tiles(d, act4, 1)))
    return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

MxWsLayout layout(int act, int T, int H, int I, int E, int k, int n_shared, int I_shared) {
  MxWsLayout L;
  const size_t R = (size_t)T * (k + n_shared);
  const int ld_h = ld_h_of(I, n_shared, I_shared);
  size_t off = 0;
  const size_t xp = mx_pad_k(H), hp = mx_pad_k(ld_h);
  L.qx = off;
  if (act == MOE_A4) off += up256((size_t)T * (xp / 2));
  else if (pad_x(H)) off += up256((size_t)T * xp * 2);
  L.sx = off;
  if (act == MOE_A4) off += up256((size_t)T * (xp / kMxBlock));
  L.qh = off;
  if (act == MOE_A4) off += up256(R * (hp / 2));
  else if (pad_h(I, n_shared, I_shared)) off += up256(R * hp * 2);
  L.sh = off;
  if (act == MOE_A4) off += up256(R * (hp / kMxBlock));
  L.y = off;
  off += up256(R * H * 4);
  L.tiles = off;
  off += 256 + up256((size_t)moe_permute_max_tiles(T, k, E, kSortTile) * 16);
  L.perm = off;
  off += up256((size_t)permute_multi_blocks(T * k) * E * 4);
  L.total = off;
  return L;
}

moe_status check_ws(const void* ws, size_t bytes, const MxWsLayout& L) {
  return ws && aligned(ws, 256) && bytes >= L.total ? MOE_OK : MOE_E_WORKSPACE;
}

void set_banks(MxProj& a, const moe_mxbank* w, const moe_mxbank* w_sh) {
  a.w = w->codes;
  a.ws = w->scales;
  if (a.n_shared > 0) {
    a.w_sh = w_sh->codes;
    a.ws_sh = w_sh->scales;
  }
}

// The projections' launches, every argument checked.
moe_status gateup(int act, MxProj a, const MxWsLayout& L, const int32_t* offsets,
                  const int32_t* sorted_pair, char* ws, hipStream_t s) {
  const int act4 = act == MOE_A4, H = a.K;
  a.offsets = offsets;
  a.sorted_pair = sorted_pair;
  const bool gemm = large_tiles(a, act4, 0);
  hipError_t e = hipSuccess;
  if (act4 && (gemm || codes_first(a, 0))) {
    uint8_t* q = reinterpret_cast<uint8_t*>(ws + L.qx);
    uint8_t* sc = reinterpret_cast<uint8_t*>(ws + L.sx);
    e = launch_mx_quant(a.x, 0, a.T, H, H, q, sc, mx_pad_k(H), true, s);
    a.q = q;
    a.s = sc;
  } else if (gemm && pad_x(H)) {
    uint16_t* xp = reinterpret_cast<uint16_t*>(ws + L.qx);
    e = launch_mx_pad_rows(a.x, a.T, H, H, xp, mx_pad_k(H), s);
    a.x = xp;
    a.ld_in = mx_pad_k(H);
  }
  if (e != hipSuccess) return MOE_E_DEVICE;
  return from_hip(gemm ? launch_mx_gemm(a, 0, act4, s) : launch_mx_rows16(a, 0, act4, s));
}

moe_status down(int act, const uint16_t* h, int T, int H, int I, int E, int k,
                const moe_mxbank* w2, const moe_mxbank* w2_shared, int n_shared, int I_shared,
                const float* shared_gate, const float* topk_w, const int32_t* offsets,
                const int32_t* pair_pos, void* out, int out_f32, char* ws, hipStream_t s) {
  const MxWsLayout L = layout(act, T, H, I, E, k, n_shared, I_shared);
  const int act4 = act == MOE_A4, ld_h = ld_h_of(I, n_shared, I_shared), hp = mx_pad_k(ld_h);
  const int P = T * k, R_sh = n_shared * T;
  if (n_shared == 0) shared_gate = nullptr;
  MxProj a = down_dims(T, H, I, E, k, n_shared, I_shared);
  set_banks(a, w2, w2_shared);
  a.x = h;
  a.offsets = offsets;
  float* y = reinterpret_cast<float*>(ws + L.y);
  a.out = y;
  hipError_t e = hipSuccess;
  const bool gemm = large_tiles(a, act4, 1);
  const uint16_t* h_sh = h + (size_t)P * ld_h;
  if (act4 && (gemm || codes_first(a, 1))) {
    uint8_t* q = reinterpret_cast<uint8_t*>(ws + L.qh);
    uint8_t* sc = reinterpret_cast<uint8_t*>(ws + L.sh);
    // rows of one length are one launch
    const bool one = n_shared == 0 || I_shared == I;
    e = launch_mx_quant(h, 0, one ? P + R_sh : P, I, ld_h, q, sc, hp, true, s);
    if (e == hipSuccess && !one)
      e = launch_mx_quant(h_sh, 0, R_sh, I_shared, ld_h, q + (size_t)P * (hp / 2),
                          sc + (size_t)P * (hp / kMxBlock), hp, true, s);
    a.q = q;
    a.s = sc;
  } else if (gemm && pad_h(I, n_shared, I_shared)) {
    uint16_t* pd = reinterpret_cast<uint16_t*>(ws + L.qh);
    e = launch_mx_pad_rows(h, P, I, ld_h, pd, hp, s);
    if (e == hipSuccess && n_shared > 0)
      e = launch_mx_pad_rows(h_sh, R_sh, I_shared, ld_h, pd + (size_t)P * hp, hp, s);
    a.x = pd;
    a.ld_in = hp;
  }
  if (e == hipSuccess) e = gemm ? launch_mx_gemm(a, 1, act4, s) : launch_mx_rows16(a, 1, act4, s);
  if (e != hipSuccess) return MOE_E_DEVICE;
  return from_hip(launch_combine(y, H, topk_w, pair_pos, T, k, H, P, n_shared, shared_gate, out,
                                 out_f32, s));
}

}  // namespace

extern "C" {

moe_status moe_mx4_quant_rows(const void* src, int src_is_f32, int R, int C, int ld,
                              uint8_t* codes, uint8_t* scales, void* stream) {
  if (R < 0 || C <= 0 || ld < C) return MOE_E_INVAL;
  if (src_is_f32 != 0 && src_is_f32 != 1) return MOE_E_INVAL;
  if (C % kMxBlock) return MOE_E_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!src || !codes || !scales) return MOE_E_INVAL;
  if (!aligned(src, src_is_f32 ? 4 : 2) || !aligned(codes, 4)) return MOE_E_INVAL;
  const moe_status d = device_usable();
  if (d != MOE_OK) return d;
  return from_hip(launch_mx_quant(src, src_is_f32, R, C, ld, codes, scales, C, false,
                                  static_cast<hipStream_t>(stream)));
}

moe_status moe_mx4_dequant_rows(const uint8_t* codes, const uint8_t* scales, int R, int C,
                                void* dst, int dst_is_f32, int ld, void* stream) {
  if (R < 0 || C <= 0 || ld < C) return MOE_E_INVAL;
  if (dst_is_f32 != 0 && dst_is_f32 != 1) return MOE_E_INVAL;
  if (C % kMxBlock) return MOE_E_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!dst || !codes || !scales) return MOE_E_INVAL;
  if (!aligned(dst, dst_is_f32 ? 4 : 2) || !aligned(codes, 4)) return MOE_E_INVAL;
  const moe_status d = device_usable();
  if (d != MOE_OK) return d;
  return from_hip(launch_mx_dequant(codes, scales, R, C, dst, dst_is_f32, ld,
                                    static_cast<hipStream_t>(stream)));
}

size_t moe_mx4_bank_code_bytes(int n, int N, int K) {
  if (n <= 0 || N <= 0 || K <= 0 || N % 16 || K % kMxBlock) return 0;
  return bank_bytes(n, mx_code_bytes(N, K));
}

size_t moe_mx4_bank_scale_bytes(int n, int N, int K) {
  if (n <= 0 || N <= 0 || K <= 0 || N % 16 || K % kMxBlock) return 0;
  return bank_bytes(n, mx_scale_bytes(N, K));
}

moe_status moe_mx4_tile_bank(const uint8_t* codes, const uint8_t* scales, int n, int N, int K,
                             uint8_t* dst_codes, uint8_t* dst_scales, void* stream) {
  if (n < 0 || N <= 0 || K <= 0) return MOE_E_INVAL;
  if (N % 16 || K % kMxBlock) return MOE_E_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!codes || !scales || !dst_codes || !dst_scales) return MOE_E_INVAL;
  if (codes == dst_codes || scales == dst_scales) return MOE_E_INVAL;
  if (!aligned(codes, 16) || !aligned(dst_codes, 16) || !aligned(dst_scales, 4)) return MOE_E_INVAL;
  const moe_status d = device_usable();
  if (d != MOE_OK) return d;
  return from_hip(launch_mx_tile(codes, scales, n, N, K, dst_codes, dst_scales,
                                 static_cast<hipStream_t>(stream)));
}

size_t moe_mx4_workspace_bytes(int act, int T, int H, int I, int E, int k, int n_shared,
                               int I_shared) {
  if (check_shape(act, T, H, I, E, k, n_shared, I_shared) != MOE_OK) return 0;
  return layout(act, T, H, I, E, k, n_shared, I_shared).total;
}

int moe_mx4_tile_rows(int act, int T, int H, int I, int E, int k, int n_shared, int I_shared,
                      int down) {
  if (check_shape(act, T, H, I, E, k, n_shared, I_shared) != MOE_OK) return 0;
  if (down != 0 && down != 1) return 0;
  const int act4 = act == MOE_A4;
  const MxProj a = down ? down_dims(T, H, I, E, k, n_shared, I_shared)
                        : gateup_dims(T, H, I, E, k, n_shared, I_shared);
  return large_tiles(a, act4, down) ? mx_gemm_tile_rows(a, down, act4) : 16;
}

moe_status moe_mx4_gateup_silu(int act, const uint16_t* x, int T, int H, int I, int E, int k,
                               const moe_mxbank* w13, const moe_mxbank* w13_shared, int n_shared,
                               int I_shared, const int32_t* offsets, const int32_t* sorted_pair,
                               uint16_t* h, void* workspace, size_t ws_bytes, int flags,
                               void* stream) {
  moe_status st = check_shape(act, T, H, I, E, k, n_shared, I_shared);
  if (st != MOE_OK) return st;
  if (flags) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (!x || !offsets || !sorted_pair || !h || !aligned(x, 16) || !aligned(h, 16))
    return MOE_E_INVAL;
  if (!bank_ok(w13) || (n_shared > 0 && !bank_ok(w13_shared))) return MOE_E_INVAL;
  const MxWsLayout L = layout(act, T, H, I, E, k, n_shared, I_shared);
  st = check_ws(workspace, ws_bytes, L);
  if (st != MOE_OK) return st;
  st = device_usable();
  if (st != MOE_OK) return st;
  MxProj a = gateup_dims(T, H, I, E, k, n_shared, I_shared);
  set_banks(a, w13, w13_shared);
  a.x = x;
  a.out = h;
  return gateup(act, a, L, offsets, sorted_pair, static_cast<char*>(workspace),
                static_cast<hipStream_t>(stream));
}

moe_status moe_mx4_down_combine(int act, const uint16_t* h, int T, int H, int I, int E, int k,
                                const moe_mxbank* w2, const moe_mxbank* w2_shared, int n_shared,
                                int I_shared, const float* shared_gate, const float* topk_w,
                                const int32_t* offsets, const int32_t* pair_pos, void* out,
                                void* workspace, size_t ws_bytes, int flags, void* stream) {
  moe_status st = check_shape(act, T, H, I, E, k, n_shared, I_shared);
  if (st != MOE_OK) return st;
  if (flags & ~MOE_OUT_F32) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (!h || !topk_w || !offsets || !pair_pos || !out) return MOE_E_INVAL;
  if (!aligned(h, 16) || !aligned(out, 16)) return MOE_E_INVAL;
  if (!bank_ok(w2) || (n_shared > 0 && !bank_ok(w2_shared))) return MOE_E_INVAL;
  st = check_ws(workspace, ws_bytes, layout(act, T, H, I, E, k, n_shared, I_shared));
  if (st != MOE_OK) return st;
  st = device_usable();
  if (st != MOE_OK) return st;
  return down(act, h, T, H, I, E, k, w2, w2_shared, n_shared, I_shared, shared_gate, topk_w,
              offsets, pair_pos, out, (flags & MOE_OUT_F32) ? 1 : 0,
              static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
}

moe_status moe_mx4_layer(int act, const float* logits, const uint16_t* x, int T, int H, int I,
                         int E, int k, int renormalize, const moe_mxbank* w13,
                         const moe_mxbank* w2, const moe_mxbank* w13_shared,
                         const moe_mxbank* w2_shared, int n_shared, int I_shared,
                         const float* shared_gate, int32_t* topk_ids, float* topk_w,
                         int32_t* counts, int32_t* offsets, int32_t* sorted_pair,
                         int32_t* pair_pos, uint16_t* h, void* out, void* workspace,
                         size_t ws_bytes, int flags, void* stream) {
  moe_status st = check_shape(act, T, H, I, E, k, n_shared, I_shared);
  if (st != MOE_OK) return st;
  if ((flags & ~MOE_OUT_F32) || (renormalize != 0 && renormalize != 1)) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (!logits || !x || !topk_ids || !topk_w || !counts || !offsets || !sorted_pair || !pair_pos ||
      !h || !out)
    return MOE_E_INVAL;
  if (!aligned(x, 16) || !aligned(h, 16) || !aligned(out, 16)) return MOE_E_INVAL;
  if (!bank_ok(w13) || !bank_ok(w2)) return MOE_E_INVAL;
  if (n_shared > 0 && (!bank_ok(w13_shared) || !bank_ok(w2_shared))) return MOE_E_INVAL;
  const MxWsLayout L = layout(act, T, H, I, E, k, n_shared, I_shared);
  st = check_ws(workspace, ws_bytes, L);
  if (st != MOE_OK) return st;
  st = device_usable();
  if (st != MOE_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  MxProj a = gateup_dims(T, H, I, E, k, n_shared, I_shared);
  set_banks(a, w13, w13_shared);
  a.x = x;
  a.out = h;
  if (route_inside(a, act == MOE_A4)) {
    // a few tokens: routing, sort and gate/up in one launch
    st = from_hip(launch_mx_route_gateup(a, act == MOE_A4, logits, renormalize, topk_ids, topk_w,
                                         counts, offsets, sorted_pair, pair_pos, s));
  } else {
    int32_t* n_tiles = reinterpret_cast<int32_t*>(ws + L.tiles);
    int32_t* tiles = reinterpret_cast<int32_t*>(ws + L.tiles + 256);
    hipError_t e;
    if (T <= kFusedRouteMaxT && a.P <= kFusedRouteMaxP) {
      e = launch_route_permute(logits, T, E, k, renormalize, kSortTile, topk_ids, topk_w, counts,
                               offsets, sorted_pair, pair_pos, tiles, n_tiles, s);
    } else {
      e = launch_route_topk(logits, T, E, k, renormalize, topk_ids, topk_w, s);
      if (e == hipSuccess && permute_multi_blocks(a.P) > 0)
        e = launch_permute_multi(topk_ids, a.P, E, kSortTile, counts, offsets, sorted_pair,
                                 pair_pos, tiles, n_tiles,
                                 reinterpret_cast<int32_t*>(ws + L.perm), s);
      else if (e == hipSuccess)
        e = launch_permute(topk_ids, a.P, E, kSortTile, counts, offsets, sorted_pair, pair_pos,
                           tiles, n_tiles, s);
    }
    if (e != hipSuccess) return MOE_E_DEVICE;
    st = gateup(act, a, L, offsets, sorted_pair, ws, s);
  }
  if (st != MOE_OK) return st;
  return down(act, h, T, H, I, E, k, w2, w2_shared, n_shared, I_shared, shared_gate, topk_w,
              offsets, pair_pos, out, (flags & MOE_OUT_F32) ? 1 : 0, ws, s);
}

}  // extern "C"
