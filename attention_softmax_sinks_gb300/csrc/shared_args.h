// Launcher interface of the decode of a batch that shares prompts (shared.cu for the shared
// pages, decode.cu for each sequence's own ones).  Arguments arrive already validated by abi.cu.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace sa {

// Which pages a batch shares: group g is sequences [group_offsets[g], group_offsets[g + 1]), and
// its sequences' first shared_pages[g] pages are the same.
struct SharedPlan {
  const int32_t* group_offsets;  // [num_groups + 1]
  const int32_t* shared_pages;   // [num_groups]
  int num_groups;
  int max_shared_pages;          // bound on shared_pages
  int shared_splits, own_splits; // slots of a row's partial results: shared ones first
};

struct SharedArgs {
  const uint16_t* q;             // bf16 [B, Hq, 64]
  const int32_t* page_table;     // [B, max_pages]
  float* partial_o;              // [B, shared_splits + own_splits, Hq, 64]
  float* partial_lse;            // [B, shared_splits + own_splits, Hq]
  SharedPlan plan;
  int batch, hq, hkv, group, max_pages, num_pages;
  int ctas;                      // of the shared part's grid
  float scale_log2;              // sm_scale * log2(e)
  unsigned* status;
  unsigned long long timeout_ns;
};

// Pairs of row tiles of the batch per KV head: at most, however it is divided into num_groups groups.
long long shared_row_tiles(int batch, int num_groups, int group);
// CTAs for the shared part, so that it and the own parts (which get the other SMs) end together as
// far as the bounds on their lengths tell.
int shared_ctas(int batch, int num_groups, int group, int hkv, int max_shared_pages, int max_pages,
                long long own_ctas, int sms);
// Attention of every group's rows over its shared pages, into slots [0, shared_splits) (slots not
// used: lse = -inf, the output not written; nothing for groups that share no pages).
cudaError_t launch_shared(const CUtensorMap& kmap, const CUtensorMap& vmap, const SharedArgs& a, cudaStream_t stream);
// Every sequence's own pages and its sink, into the slots behind; launched after launch_shared
// (decode.cu).  Where a sequence shares nothing, its shared slots get lse = -inf.  a.num_splits = plan.own_splits, a.out and a.lse are the partial results.
cudaError_t launch_decode_own(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeArgs& a,
                              const SharedPlan& plan, cudaStream_t stream);

// Adds the slots up; launched after launch_decode_own.
cudaError_t launch_shared_merge(const MergeArgs& a, cudaStream_t stream);

}  // namespace sa
