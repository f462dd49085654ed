// Launcher interface of the linear layer with low-rank adapters (lora.cu).  Arguments arrive
// already validated by abi.cu.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sa {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = 1024;
constexpr int kLoraTileRows = 128;  // tokens of a CTA's tile
struct LoraArgs {
  const uint16_t* x;         // bf16 [M, K]
  const uint16_t* w;         // bf16 [N, K]
  const uint16_t* lora_a;    // bf16 [L, R, K]
  const uint16_t* lora_b;    // bf16 [L, N, R]
  const int32_t* adapter;    // [M]
  const float* scale;        // [L] or nullptr (1)
  const uint16_t* bias;      // bf16 [N] or nullptr
  uint16_t* out;             // bf16 [M, N]
  // workspace, s_a x A_a^T: bf16 [M, R] (many tokens, else nullptr), or fp32 parts [splits, M, R]
  uint16_t* t;
  float* t_parts;
  int M, N, K, R, num_adapters;
  int splits;                // parts of K of the first product
  int block_n, tiles_m, tiles_n;  // tiles_m: of 128 tokens
  int k_parts;               // CTAs of a cluster that share a tile's K (1, 2, 4 or 8)
  int plan_tiles;            // 128-token tiles per tile of the product (2: pairs of CTAs)
  int box_rows;              // rows of an x box
  unsigned* status;
  unsigned long long timeout_ns;
};

// x in boxes of box_rows x 64; W [N, K] in boxes of block_n / plan_tiles rows x 64; lora_a [L R, K] in
// boxes of R x 64; lora_b [L, N, R] in boxes of 1 x block_n / plan_tiles x 16 (32-byte swizzle).
struct LoraMaps {
  CUtensorMap x, w, a, b;
};

// Tiles for the sizes in a: block_n, tiles_m, tiles_n, plan_tiles, k_parts, box_rows, splits.
void lora_plan(LoraArgs& a, int sms);
cudaError_t launch_lora(const LoraMaps& m, const LoraArgs& a, int sms, cudaStream_t stream);

}  // namespace sa
