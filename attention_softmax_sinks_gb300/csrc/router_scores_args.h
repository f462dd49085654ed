// Launcher interface of the router by scores, groups and balance (router_scores.cu).  Arguments
// arrive already validated by abi.cu.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace sa {

constexpr int kRouterMaxGroups = 32;

struct RouterScoresArgs {
  const void* logits;      // bf16 or fp32 [T, E]
  const float* bias;       // [E] or nullptr
  int32_t* topk_idx;       // [T, k]
  uint16_t* topk_w;        // bf16 [T, k]
  int32_t* counts;         // [E] (already zeroed) or nullptr
  long long num_tokens;
  int num_experts, top_k, num_groups, top_groups;
  int fp32, sigmoid, renormalize;
  int vec4;                // rows read four logits at a time
  float scale;
};

cudaError_t launch_router_scores(const RouterScoresArgs& a, int sms, cudaStream_t stream);

}  // namespace sa
