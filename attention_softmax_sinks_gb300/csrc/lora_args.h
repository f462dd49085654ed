// Launcher interface of the linear layer with low-rank adapters (lora.cu).  Arguments arrive
// already validated by abi.cu.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sa {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = 1024;
constexpr int kLoraTileRows = 128;  // tokens of an output tile
// Per 128 tokens: the number of distinct adapters, which ones (ascending), and each token's place
// among them (-1: none).
constexpr int kLoraPlanInts = 264;
constexpr int kLoraPlanList = 8;
constexpr int kLoraPlanSlot = kLoraPlanList + kLoraTileRows;

struct LoraArgs {
  const uint16_t* x;         // bf16 [M, K]
  const uint16_t* w;         // bf16 [N, K]
  const uint16_t* lora_a;    // bf16 [L, R, K]
  const uint16_t* lora_b;    // bf16 [L, N, R]
  const int32_t* adapter;    // [M]
  const float* scale;        // [L] or nullptr (1)
  const uint16_t* bias;      // bf16 [N] or nullptr
  uint16_t* out;             // bf16 [M, N]
  int32_t* plan;             // workspace: [tiles_m, kLoraPlanInts]
  float* t;                  // workspace: [splits, M, R]
  int M, N, K, R, num_adapters;
  int splits;                // parts of K whose products are added up by their reader
  int block_n, tiles_m, tiles_n;
  int box_rows;              // rows of an x box
  unsigned* status;
  unsigned long long timeout_ns;
};

// Parts of K for the adapters' first product (fixed by the sizes: the workspace holds them).
int lora_splits(int m, int k);
// Columns of an output tile (a multiple of 16, at most 224).
int lora_tile_n(int m, int n, int k, int sms);
// xmap: x in boxes of box_rows x 64; wmap: W [N, K] in boxes of block_n x 64; bmap: lora_b
// [L, N, R] in boxes of 1 x block_n x 16 (32-byte swizzle).
cudaError_t launch_lora(const CUtensorMap& xmap, const CUtensorMap& wmap, const CUtensorMap& bmap, const LoraArgs& a,
                        int sms, cudaStream_t stream);

}  // namespace sa
