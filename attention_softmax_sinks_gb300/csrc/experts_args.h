// Launcher interface of the pair grouping and the weighted combine (experts.cu) and of the
// MXFP4 conversions (mxfp4.cu).  Arguments arrive already validated by abi.cu.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace sa {

// Position of a thread that walks over [rows, width] elements in steps of a whole grid, without
// a division per step: `step` = step_row * width + step_col.
struct GridWalk {
  long long row;
  int col;
#ifdef __CUDACC__
  __device__ __forceinline__ GridWalk(long long i, int width) : row(i / width), col(static_cast<int>(i - row * width)) {}
  __device__ __forceinline__ void advance(long long step_row, int step_col, int width) {
    row += step_row;
    col += step_col;
    if (col >= width) {
      col -= width;
      ++row;
    }
  }
#endif
};

struct GroupRowsArgs {
  const int32_t* topk_idx;  // [T, k]
  int32_t* offsets;         // [E + 1]
  int32_t* row_token;       // [T * k]
  int32_t* pair_row;        // [T, k]
  int pairs, top_k, num_experts;
  unsigned* status;
};

struct CombineArgs {
  const uint16_t* y;        // bf16 [R, H]
  const int32_t* pair_row;  // [T, k]
  const uint16_t* weight;   // bf16 [T, k]
  uint16_t* out;            // bf16 [T, H]
  int num_rows, num_tokens, top_k, hidden;
  unsigned* status;
};

cudaError_t launch_group_rows(const GroupRowsArgs& a, cudaStream_t stream);
cudaError_t launch_combine(const CombineArgs& a, int sms, cudaStream_t stream);

struct Mxfp4Args {
  const void* in;     // bf16 or fp32 [rows, k] (quantise), codes (dequantise)
  uint8_t* codes;     // [rows, k / 2] (quantise)
  uint8_t* scales;    // [rows, stride]: written (quantise) or read (dequantise)
  uint16_t* out;      // bf16 [rows, k] (dequantise)
  long long rows;
  int k, stride, is_fp32;
};

cudaError_t launch_mxfp4_quantize(const Mxfp4Args& a, int sms, cudaStream_t stream);
cudaError_t launch_mxfp4_dequantize(const Mxfp4Args& a, int sms, cudaStream_t stream);

}  // namespace sa
