// Low-rank adapters of many requests beside the experts' projections: launch
// interface between the C ABI (lora_api.cpp) and the kernels (lora.hip).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraSmallRows = 16;    // rows of a window: gate/up, small calls
constexpr int kLoraWindow = 256;      // large ones
constexpr int kLoraFewRows = 640;     // rows up to which a call is one launch
constexpr int kLoraManyRows = 2048;   // gate/up: up to which it may be
constexpr int kLoraPlanMaxE = 1088;   // routed and shared experts of a plan
constexpr int kLoraSlab = 64;         // columns of a workgroup of the accumulating kernel
constexpr int kLoraMaxBlock = 512;    // and tokens
constexpr int kLoraSegment = 16;      // windows of 64 rows that it takes at a time

// A unit: up to 16 rows of one (adapter, expert) with tokens of one block; v: the
// byte of parts where the first one's lies, the others' behind it.
struct alignas(16) LoraUnit {
  const uint16_t* b;
  uint32_t rank8, v;
};

// Up to 32 rows of one (adapter, expert) of a window, neighbours in the window's
// order; rank 0 without an adapter.
struct alignas(32) LoraGroupUnit {
  const uint16_t* a;
  const uint16_t* b;
  float scale;
  uint16_t rank, shared, first, n;
  uint32_t unused;
};

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
  // large calls: windows of 256 rows
  int2* unit_count;             // [window] units with an adapter, and in all
  LoraGroupUnit* units;         // [window][256], those with an adapter first
  uint32_t* order;              // [window][256] token | row of the window << 24
  // v (down: times the gate weight) as three bf16 parts that sum to it; gate/up:
  // [window][3][2 max_rank / 8][256][8], down: [plan's window][3][max_rank / 8][64][8]
  uint16_t* parts;
  // down, large calls: the plan of the accumulating kernel, per block of `block`
  // tokens: its rows in win windows of 64, each with its units
  float* weight;                // [window][256] in the window's order
  uint32_t* place;              // [R] plan's window * 64 + place in it
  uint32_t* row_at;             // [n_blocks][win][64] and back
  int block, n_blocks, win;
  int* plan_count;              // [n_blocks][win] units of a window
  LoraUnit* plan;               // [n_blocks][win][64]
  uint32_t* plan_sums;          // [n_blocks][win][64][16] byte of a row's token's chunk 0 in LDS
  bool large;                   // three launches
  const float* gu;              // gate/up: [R][2 ld_h]
  const float* base;            // down: [T][H]
  const float* topk_w;          // down
  const float* shared_gate;     // down: [T][n_shared] or null
  const int32_t* pair_pos;      // down
  void* out;                    // gate/up: h [R][ld_h]; down: out [T][H]
  int out_f32;
  int32_t* err;
};

// How a call of these sizes runs: fills large and, for down, the accumulating
// kernel's block, n_blocks and win.  most: of any adapters, the way that needs the
// most workspace.  Host only.
void lora_choose(LoraArgs& a, bool most);
// The workspace behind the error word, in bytes; with ws, sets the pointers.
size_t lora_carve(LoraArgs& a, char* ws);

// n matrices [rows][cols] to the layout of A (rows % 8 == 0, cols % 32 == 0) or of
// B (rows % 32 == 0, cols % 8 == 0).
hipError_t launch_lora_tile(const uint16_t* src, int n, int rows, int cols, int is_b, uint16_t* dst,
                            hipStream_t st);
hipError_t launch_lora_gateup(const LoraArgs& a, hipStream_t st);
hipError_t launch_lora_down(const LoraArgs& a, hipStream_t st);

}  // namespace moe
