// Low-rank adapters of many requests beside the experts' projections: launch
// interface between the C ABI (lora_api.cpp) and the kernels (lora.hip).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraSmallRows = 16;    // rows of a window, small calls
constexpr int kLoraLargeRows = 64;    // and large ones
constexpr int kLoraMaxSplits = 4;

// Rows of a layer (sorted pairs, then the shared experts' tokens) with their
// tokens' adapters.
struct LoraArgs {
  int T, k, P, R, E, n_shared, n, max_rank;
  const int32_t* adapter;       // [T]
  const int32_t* topk_ids;      // [T * k]
  const int32_t* offsets;       // [E + 1]
  const int32_t* sorted_pair;   // [P]
  const moe_lora* table;        // [n][E + n_shared]
  int halves;                   // 2: gate/up, 1: down
  int H, I, I_sh, ld_h;
  const void* in;               // gate/up: x bf16 [T][H]; down: h [R][ld_h]
  int in_f32;
  float* v;                     // [splits][R][halves * max_rank]
  int splits;                   // parts of K
  bool large;                   // windows of 64 rows, one workgroup each
  const float* gu;              // gate/up: [R][2 ld_h]
  const float* base;            // down: [T][H]
  const float* topk_w;          // down
  const float* shared_gate;     // down: [T][n_shared] or null
  const int32_t* pair_pos;      // down
  void* out;                    // gate/up: h [R][ld_h]; down: out [T][H]
  int out_f32;
  int32_t* err;
};

// Splits of K and the window size for R rows (the workspace is sized by it).
void lora_plan(int R, int halves, int max_rank, int& splits, bool& large);

hipError_t launch_lora_gateup(const LoraArgs& a, hipStream_t st);
hipError_t launch_lora_down(const LoraArgs& a, hipStream_t st);

}  // namespace moe
