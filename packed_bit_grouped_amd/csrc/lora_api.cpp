// C ABI of the low-rank adapters: host-side argument checks, workspace layout
// and dispatch (the same rules as api.cpp: nothing allocates, synchronizes or
// reads device memory).
#include <hip/hip_runtime.h>

#include <cstring>

#include "lora_common.h"

using namespace moe;

namespace {

constexpr int kLoraMaxLen = 1 << 20;   // H, I, I_shared

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_E_DEVICE; }
int ld_h_of(int I, int n_shared, int I_shared) {
  return n_shared > 0 && I_shared > I ? I_shared : I;
}

moe_status check_shape(int T, int H, int I, int E, int k, int n_shared, int I_shared,
                       int n_adapters, int max_rank) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0 || n_shared < 0) return MOE_E_INVAL;
  if (k > E || n_adapters < 0 || max_rank <= 0 || max_rank % 8) return MOE_E_INVAL;
  if (n_shared > 0 && I_shared <= 0) return MOE_E_INVAL;
  if (H % 32 || I % 32 || (n_shared > 0 && I_shared % 32)) return MOE_E_UNSUPPORTED;
  if (H > kLoraMaxLen || I > kLoraMaxLen || (n_shared > 0 && I_shared > kLoraMaxLen))
    return MOE_E_UNSUPPORTED;
  if (max_rank > kLoraMaxRank || E > kRouteMaxE || n_shared > 65535) return MOE_E_UNSUPPORTED;
  if ((long long)n_adapters * ((long long)E + n_shared) >= (1LL << 31)) return MOE_E_UNSUPPORTED;
  const long long rows = (long long)T * ((long long)k + n_shared);
  if (T > (1 << 22) || (long long)T * k >= (1LL << 24) || rows >= (1LL << 26))
    return MOE_E_UNSUPPORTED;
  if (rows * H >= (1LL << 31) || rows * ld_h_of(I, n_shared, I_shared) >= (1LL << 31))
    return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

LoraArgs args_of(int T, int H, int I, int E, int k, int n_shared, int I_shared,
                 const int32_t* adapter, int n_adapters, int max_rank, const moe_lora* table,
                 const int32_t* topk_ids, const int32_t* sorted_pair, char* ws, int halves) {
  LoraArgs a;
  std::memset(&a, 0, sizeof(a));
  a.T = T;
  a.k = k;
  a.P = T * k;
  a.R = T * (k + n_shared);
  a.E = E;
  a.n_shared = n_shared;
  a.n = n_adapters;
  a.max_rank = max_rank;
  a.adapter = adapter;
  a.topk_ids = topk_ids;
  a.sorted_pair = sorted_pair;
  a.table = table;
  a.halves = halves;
  a.H = H;
  a.I = I;
  a.I_sh = n_shared > 0 ? I_shared : I;
  a.ld_h = ld_h_of(I, n_shared, I_shared);
  a.err = reinterpret_cast<int32_t*>(ws);
  lora_choose(a, ws == nullptr);
  lora_carve(a, ws ? ws + 256 : nullptr);
  return a;
}

// The larger of the two calls' needs (neither depends on the table).
size_t workspace_bytes(int T, int H, int I, int E, int k, int n_shared, int I_shared,
                       int max_rank) {
  size_t most = 0;
  for (int halves = 1; halves <= 2; ++halves) {
    LoraArgs a = args_of(T, H, I, E, k, n_shared, I_shared, nullptr, 0, max_rank, nullptr, nullptr,
                         nullptr, nullptr, halves);
    const size_t n = lora_carve(a, nullptr);
    most = n > most ? n : most;
  }
  return 256 + most;
}

}  // namespace

extern "C" {

size_t moe_lora_workspace_bytes(int T, int H, int I, int E, int k, int n_shared, int I_shared,
                                int max_rank) {
  if (check_shape(T, H, I, E, k, n_shared, I_shared, 0, max_rank) != MOE_OK) return 0;
  return workspace_bytes(T, H, I, E, k, n_shared, I_shared, max_rank);
}

int moe_lora_block(int T, int H, int I, int E, int k, int n_shared, int I_shared, int n_adapters,
                   int max_rank, int down) {
  const moe_status st = check_shape(T, H, I, E, k, n_shared, I_shared, n_adapters, max_rank);
  if (st != MOE_OK) return st;
  if (down != 0 && down != 1) return MOE_E_INVAL;
  LoraArgs a = args_of(T, H, I, E, k, n_shared, I_shared, nullptr, n_adapters, max_rank, nullptr,
                       nullptr, nullptr, nullptr, down ? 1 : 2);
  lora_choose(a, false);
  return !a.large ? 0 : down ? a.block : kLoraWindow;
}

moe_status moe_lora_tile(const uint16_t* src, int n, int rows, int cols, int is_b, uint16_t* dst,
                         void* stream) {
  if (n < 0 || rows <= 0 || cols <= 0 || (is_b != 0 && is_b != 1)) return MOE_E_INVAL;
  if (rows % (is_b ? 32 : 8) || cols % (is_b ? 8 : 32)) return MOE_E_UNSUPPORTED;
  if ((long long)rows * cols >= (1LL << 31) ||
      (__int128)n * rows * cols >= (__int128)(1LL << 34))
    return MOE_E_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!src || !dst || src == dst || !aligned(src, 16) || !aligned(dst, 16)) return MOE_E_INVAL;
  const moe_status st = device_usable();
  if (st != MOE_OK) return st;
  return from_hip(
      launch_lora_tile(src, n, rows, cols, is_b, dst, static_cast<hipStream_t>(stream)));
}

moe_status moe_lora_gateup_silu(const uint16_t* x, int T, int H, int I, int E, int k,
                                int n_shared, int I_shared, const int32_t* adapter,
                                int n_adapters, int max_rank, const moe_lora* table,
                                const int32_t* topk_ids, const int32_t* sorted_pair,
                                const float* gu, void* h, void* workspace, size_t ws_bytes,
                                int flags, void* stream) {
  moe_status st = check_shape(T, H, I, E, k, n_shared, I_shared, n_adapters, max_rank);
  if (st != MOE_OK) return st;
  if (flags & ~MOE_H_F32) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (!x || !adapter || !topk_ids || !sorted_pair || !gu || !h || gu == h) return MOE_E_INVAL;
  if (n_adapters > 0 && (!table || !aligned(table, 8))) return MOE_E_INVAL;
  if (!aligned(x, 16) || !aligned(gu, 16) || !aligned(h, 16)) return MOE_E_INVAL;
  if (!workspace || !aligned(workspace, 256) ||
      ws_bytes < workspace_bytes(T, H, I, E, k, n_shared, I_shared, max_rank))
    return MOE_E_WORKSPACE;
  st = device_usable();
  if (st != MOE_OK) return st;
  LoraArgs a = args_of(T, H, I, E, k, n_shared, I_shared, adapter, n_adapters, max_rank, table,
                       topk_ids, sorted_pair, static_cast<char*>(workspace), 2);
  a.in = x;
  a.gu = gu;
  a.out = h;
  a.out_f32 = (flags & MOE_H_F32) ? 1 : 0;
  return from_hip(launch_lora_gateup(a, static_cast<hipStream_t>(stream)));
}

moe_status moe_lora_down_combine(const void* h, int T, int H, int I, int E, int k,
                                 int n_shared, int I_shared, const int32_t* adapter,
                                 int n_adapters, int max_rank, const moe_lora* table,
                                 const float* shared_gate, const float* topk_w,
                                 const int32_t* topk_ids, const int32_t* offsets,
                                 const int32_t* sorted_pair, const int32_t* pair_pos,
                                 const float* base, void* out, void* workspace,
                                 size_t ws_bytes, int flags, void* stream) {
  moe_status st = check_shape(T, H, I, E, k, n_shared, I_shared, n_adapters, max_rank);
  if (st != MOE_OK) return st;
  if (flags & ~(MOE_H_F32 | MOE_OUT_F32)) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (!h || !adapter || !topk_w || !topk_ids || !offsets || !sorted_pair || !pair_pos || !base ||
      !out)
    return MOE_E_INVAL;
  if (out == base && !(flags & MOE_OUT_F32)) return MOE_E_INVAL;
  if (n_adapters > 0 && (!table || !aligned(table, 8))) return MOE_E_INVAL;
  if (!aligned(h, 16) || !aligned(base, 16) || !aligned(out, (flags & MOE_OUT_F32) ? 16 : 8))
    return MOE_E_INVAL;
  if (!workspace || !aligned(workspace, 256) ||
      ws_bytes < workspace_bytes(T, H, I, E, k, n_shared, I_shared, max_rank))
    return MOE_E_WORKSPACE;
  st = device_usable();
  if (st != MOE_OK) return st;
  LoraArgs a = args_of(T, H, I, E, k, n_shared, I_shared, adapter, n_adapters, max_rank, table,
                       topk_ids, sorted_pair, static_cast<char*>(workspace), 1);
  a.in = h;
  a.in_f32 = (flags & MOE_H_F32) ? 1 : 0;
  a.offsets = offsets;
  a.pair_pos = pair_pos;
  a.topk_w = topk_w;
  a.shared_gate = n_shared > 0 ? shared_gate : nullptr;
  a.base = base;
  a.out = out;
  a.out_f32 = (flags & MOE_OUT_F32) ? 1 : 0;
  return from_hip(launch_lora_down(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
