// Launcher interface of the grouped expert products (grouped.cu).  Arguments arrive already
// validated by abi.cu.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sa {

constexpr int kMaxExperts = 256;
constexpr int kGroupedFeatures = 128;  // features of one sub-tile (one tcgen05.mma M)

struct GroupedArgs {
  const uint16_t* bias;      // bf16 [E, N] or nullptr
  uint16_t* out;             // bf16 [rows, N], or [rows, N / 2] with swiglu
  const int32_t* offsets;    // [E + 1], or nullptr: one group of all rows
  const int32_t* row_token;  // [rows], or nullptr: row r reads row r of x
  const uint8_t* x_scales;   // MXFP4: [x_rows, scale_stride]
  const uint8_t* w_scales;   // MXFP4: [E, N, scale_stride]
  int scale_stride;
  int x_rows, rows, num_experts, N, K;
  int n_out;    // features written per row: N, or N / 2 with swiglu
  int subs;     // 128-feature sub-tiles per tile: 2, or 1 when few tiles (always 2 with swiglu)
  int tiles_f;  // feature tiles
  int swiglu;
  float alpha, limit;
  unsigned* status;
  unsigned long long timeout_ns;
};

// Token rows of one tile (the largest MMA N): 128 in bf16, fewer in MXFP4, whose scales take
// TMEM columns beside the accumulators.
int grouped_tile_rows(bool mxfp4);
// wmap: w as {K, gate/up (1 without swiglu), features, E} in boxes of 128 bytes x 1 x 128 x 1;
// xmap: x [x_rows, K] in boxes of 128 bytes x 16 rows, or x 1 row when row_token gathers.
cudaError_t launch_grouped(const CUtensorMap& wmap, const CUtensorMap& xmap, const GroupedArgs& a, bool mxfp4,
                           int sms, cudaStream_t stream);

}  // namespace sa
