// Low-rank adapters of many requests beside the experts' projections: launch
// interface between the C ABI (lora_api.cpp) and the kernels (lora.hip).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraSmallRows = 16;    // rows of a window: gate/up, small calls
constexpr int kLoraWindow = 256;      // gate/up, large ones
constexpr int kLoraLargeRows = 64;    // down, large ones
constexpr int kLoraManyRows = 2048;   // rows up to which a call is small
constexpr int kLoraPlanMaxE = 1088;   // routed and shared experts of a plan
constexpr int kLoraSlab = 64;         // columns of a workgroup of the accumulating kernel
constexpr int kLoraMaxBlock = 512;    // and tokens
constexpr int kLoraSegment = 8;       // windows of 64 rows that it takes at a time

// A unit: up to 16 rows of one (adapter, expert) with tokens of one block, and
// its rows: the row of v, and the byte of LDS where chunk 0 of the token's sums
// lies (behind the block's where there is no row).
struct alignas(16) LoraUnit {
  const uint16_t* b;
  int rank8, unused;
};
struct alignas(8) LoraUnitRow {
  uint32_t row, place;
};

// gate/up: up to 32 rows of one (adapter, expert) of a window, neighbours in the
// window's order; rank 0 without an adapter.
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
  // large calls: v (down: times the gate weight) as three bf16 parts that sum to
  // it; gate/up: [window][3][2 max_rank / 8][256][8], down: [3][max_rank / 8][R][8]
  uint16_t* parts;
  // gate/up, large calls: windows of 256 rows
  int2* unit_count;             // [window] units with an adapter, and in all
  LoraGroupUnit* units;         // [window][256], those with an adapter first
  uint32_t* order;              // [window][256] token | row of the window << 24
  // down, large calls: the plan of the accumulating kernel, per block of `block`
  // tokens: its rows in win windows of 64, each with its units
  int block, n_blocks, win;
  int* plan_count;              // [n_blocks][win] units of a window
  LoraUnit* plan;               // [n_blocks][win][64]
  LoraUnitRow* plan_rows;       // [n_blocks][win][64][16]
  bool large;                   // two launches
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
// kernel's block (0: not taken), n_blocks and win.  Host only.
void lora_choose(LoraArgs& a);
// The workspace behind the error word, in bytes; with ws, sets the pointers.
size_t lora_carve(LoraArgs& a, char* ws);

// n matrices [rows][cols] to the layout of A (rows % 8 == 0, cols % 32 == 0) or of
// B (rows % 32 == 0, cols % 8 == 0).
hipError_t launch_lora_tile(const uint16_t* src, int n, int rows, int cols, int is_b, uint16_t* dst,
                            hipStream_t st);
hipError_t launch_lora_gateup(const LoraArgs& a, hipStream_t st);
hipError_t launch_lora_down(const LoraArgs& a, hipStream_t st);

}  // namespace moe
