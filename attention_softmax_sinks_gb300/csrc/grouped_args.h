// Launcher interface of the grouped expert products (grouped.cu).  Arguments arrive already
// validated by abi.cu.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sa {

constexpr int kMaxExperts = 256;
constexpr int kBoxRows = 16;  // rows of one TMA box of x (cap / 4 with pairs: two make a CTA's half)
constexpr int kScaleBoxRows = 112;  // rows of one TMA box of x's scales: half of a pair's tile
constexpr int kScaleBoxCols = 3;    // 16 bytes of a row's scales, so many times, in one TMA box
constexpr int kGroupedFeatures = 128;  // features of one tile (the tcgen05.mma M)

struct GroupedArgs {
  const uint8_t* x;          // [x_rows, K] bf16 or codes (read directly when rows are gathered)
  const uint16_t* bias;      // bf16 [E, N] or nullptr
  uint16_t* out;             // bf16 [rows, N], or [rows, N / 2] with swiglu
  const int32_t* offsets;    // [E + 1], or nullptr: one group of all rows
  const int32_t* row_token;  // [rows], or nullptr: row r reads row r of x
  const uint8_t* x_scales;   // MXFP4: [x_rows, scale_stride]
  const uint8_t* w_scales;   // MXFP4: [E, N, scale_stride]
  int scale_stride;
  int x_rows, rows, num_experts, N, K;
  int n_out;    // features written per row: N, or N / 2 with swiglu
  int tiles_f;  // feature tiles (of N)
  int pair;     // tiles of CTA pairs: 2 x 128 features
  int width;    // features of a single CTA's tile: a multiple of 16, at most 128
  int cap;      // most rows of a tile
  int sub;      // blocks of 128 bytes of K per ring stage (1 with pairs)
  // set by the launcher
  int stages;        // ring stages
  uint32_t f_magic;  // x / tiles_f = x * f_magic >> f_shift
  int f_shift;
  int swiglu;
  float alpha, limit;
  unsigned* status;
  unsigned long long timeout_ns;
};

// The tiling (pair, width, cap, sub, tiles_f) for a.rows, a.num_experts and a.N.  cap is
// 16, 64 or, for pairs, 256 in bf16 and 224 in MXFP4 (whose scales take TMEM columns beside
// the accumulators).
void grouped_plan(GroupedArgs& a, bool mxfp4, int sms);
// w: {K, N, E} in boxes of 128 bytes x width x 1;  x: [x_rows, K] in boxes of 128 bytes x kBoxRows
// (cap / 4 with pairs);  MXFP4 scales, with pairs only: [E N, scale_stride] in boxes of
// 16 kScaleBoxCols bytes x width and [x_rows, scale_stride] in as many bytes x kScaleBoxRows.
struct GroupedMaps {
  CUtensorMap w, x, w_scales, x_scales;
};
cudaError_t launch_grouped(const GroupedMaps& m, const GroupedArgs& a, bool mxfp4, int sms, cudaStream_t stream);

}  // namespace sa
