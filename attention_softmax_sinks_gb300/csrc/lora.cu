// Linear layer with the low-rank adapters of many requests beside it: for token m with adapter a,
//
//     out[m] = x[m] W^T + b + s_a (x[m] A_a^T) B_a^T        A_a [R, K], B_a [N, R]
//
// (page "GPT-OSS on day 0": the projections carry bias terms; the adapters are what requests of
// one server differ in).  Two kernels, in one call:
//
// 1. lora_shrink_kernel: t[m] = s_a x[m] A_a^T, on tcgen05 (few tokens: lora_shrink_few_kernel,
//    below).  A CTA takes 128 tokens, a part of K and up to 256 columns: the A_a of as many of the
//    tile's distinct adapters as fit, one behind the other (found by a bit per adapter and
//    population counts).  Every token meets every one of them, and its row keeps its own adapter's
//    R columns.  That is wasted work for a tile of many adapters, but the tile is short of nothing
//    else: what bounds it is the operands' way
//    in, which is A once per tile and x once per 256 columns.  The CTAs of a tile's parts of K are
//    a cluster: each sends its rows to the one that adds them up, in order, and rounds once to
//    bf16 for the second product, as x is: a relative error of 2^-8 at most per term of a sum
//    over the ranks, of the adapters' part only (which the bf16 output rounds once more anyway).
//    (With fp32 parts added by the second kernel, 8192 tokens of rank 64 took 27 us longer than
//    without adapters, and of rank 128 115 us: its loads of t were longer than a tile.)
// 2. lora_linear_kernel: the product with W on tcgen05, tokens x block_n features per tile,
//    accumulator seeded with the bias, and then on the same accumulator one more product per
//    adapter of the tile: T_i B_i^T, where T_i holds s t for the tokens of adapter i and zeros for
//    the others.  T_i is the A operand in TMEM, written by warps of its own (a thread per row),
//    which run ahead of the product; B_i comes by TMA in boxes of 16 ranks.  So any mix of
//    adapters in a tile is right, and a tile of one adapter costs R more columns of K.
//    Zeros do not keep out an infinity or NaN of another request's B_i: an element that comes out
//    not finite is computed once more by itself, from its own operands only, unless its row has a
//    NaN of its own.
//    Many tokens: pairs of CTAs (cta_group::2, 256 tokens), which stage half of W's columns each.
//    Few tiles: clusters of 2, 4 or 8 CTAs share one tile's K and adapters and add their accumulators
//    up through each other's shared memory.  What bounds them is not W's way from memory but the
//    operands' way into an SM (2 cycles per row and 64 values of K) and the tensor core's reading
//    of 128 rows of x, live or not; larger tiles with a part of K each need less of both.
//
// The second kernel starts while the first runs (programmatic dependent launch): the product with
// W needs nothing from it, and only the roles of the adapters' part wait for it.
//
// 2880 -> 5120 with rank 64, 8192 tokens: 159 us, 1.6 PFLOP/s of all products (the second kernel some
// 147, its tensor cores busy 78% of the time under the power limit; the first, 12, runs before pairs
// have an SM).  1 token 4096 -> 2880, rank 16: 11.1 us, 64 tokens 2880 -> 5120 with nearly as many adapters
// 18.5, 333 tokens 4096 -> 2880 of rank 32 23.1: a launch (about 4 us), one way of the operands through
// each SM (W is spread over the SMs, x goes into all of them), and the adding up.
#include <atomic>
#include <cstdint>

#include "lora_args.h"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr unsigned long long kDrainTimeoutNs = 2000000000ull;
constexpr int kBM = kLoraTileRows;
constexpr int kBK = 64;

__device__ __forceinline__ uint64_t sw128_kmajor(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(1024 >> 4) << 16;  // leading byte offset (unused)
  d |= static_cast<uint64_t>(1024 >> 4) << 32;  // stride byte offset: next 8-row group
  d |= 1ull << 46;                               // tcgen05 descriptor version
  d |= 2ull << 61;                               // 128-byte swizzle
  return d;
}
__device__ __forceinline__ uint64_t sw32_kmajor(uint32_t saddr) {  // rows of 16 values
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(256 >> 4) << 16;   // leading byte offset (unused)
  d |= static_cast<uint64_t>(256 >> 4) << 32;   // stride byte offset: next 8-row group
  d |= 1ull << 46;
  d |= 6ull << 61;                               // 32-byte swizzle
  return d;
}
__device__ __forceinline__ uint32_t idesc_bf16_kk(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// Waits of a whole warp; the result is the same in all lanes.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > timeout_ns)) {
      *abort_flag = 1;
      return false;
    }
  }
}

// Position in the ring: stage index and number of rounds made.
struct RingPos {
  int stage = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      ++round;
    }
  }
};

// One lane of a converged warp, always the same one: what it issues stays in a warp-uniform region
// (from a divergent branch an MMA takes about 125 cycles to issue; 4096 -> 2880 for one token went
// from 28.5 to 13.6 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// ------------------------------------------------------------------ which adapters a tile has
// The distinct adapters of a tile's rows, ascending (`slots` of them, slot by slot).
struct TilePlan {
  uint32_t bits[kLoraMaxAdapters / 32];
  int word_rank[kLoraMaxAdapters / 32];  // adapters in the words before
  int list[2 * kBM];                     // adapter of a slot
  int slots;
};

__device__ __forceinline__ void plan_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool plan_barrier_and(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, r;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred r, 1, 128, p;\n\tselp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}

// By the 128 threads (four warps) that share named barrier 1: thread i brings rows first_row + i
// and, of 256 rows, first_row + 128 + i; returns the slot of row first_row + own_row + i (own_row
// 0 or 128), -1 without adapter.  An adapter that does not exist counts as none and is reported.
template <int kRows>
__device__ __forceinline__ int make_plan(const LoraArgs& a, TilePlan& plan, int i, int first_row, int own_row) {
  int id[kRows / 128];
#pragma unroll
  for (int h = 0; h < kRows / 128; ++h) {
    const int row = first_row + 128 * h + i;
    id[h] = row < a.M ? __ldg(a.adapter + row) : -1;
    if (id[h] >= a.num_adapters) {
      raise_status(a.status, kStatusBadPage);
      id[h] = -1;
    }
  }
  if (i < kLoraMaxAdapters / 32) plan.bits[i] = 0;
  plan_barrier();
#pragma unroll
  for (int h = 0; h < kRows / 128; ++h)
    if (id[h] >= 0) atomicOr(&plan.bits[id[h] >> 5], 1u << (id[h] & 31));
  plan_barrier();
  if (i < 32) {
    const int n = __popc(plan.bits[i]);
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (i >= off) incl += v;
    }
    plan.word_rank[i] = incl - n;
    if (i == 31) plan.slots = incl;
  }
  plan_barrier();
  int slot = -1;
#pragma unroll
  for (int h = 0; h < kRows / 128; ++h) {
    if (id[h] < 0) continue;
    const int s = plan.word_rank[id[h] >> 5] + __popc(plan.bits[id[h] >> 5] & ((1u << (id[h] & 31)) - 1));
    plan.list[s] = id[h];  // the same value from all of its rows
    if (128 * h == own_row) slot = s;
  }
  return slot;
}

// ------------------------------------------------------------------ first product, few tokens
// lora_shrink_few_kernel.  A CTA sorts the 128 tokens of a tile by adapter and takes its share of the
// units (adapter, up to 64 of its tokens) and of K.  Warp-level matrix instructions with the ranks
// as M = 16 and the tokens as N = 8: a unit of one token costs what its adapter's rows cost to read.
// Fragments come straight from memory in 16-byte loads: a lane's eight values of K serve two
// instructions, in the same order for both operands.  It is small enough (20 KB, half of the
// registers) to run beside the second kernel's CTAs.  The parts of K are added by their reader.
constexpr int kFewWarps = 8;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kUnitTokens = 64;
constexpr int kRed = 6 * 16 * 32;  // floats: partial sums of the warps that do not add up

struct FewSmem {
  float red[kRed];
  uint32_t bits[kLoraMaxAdapters / 32];
  int word_rank[kLoraMaxAdapters / 32];  // adapters in the words before
  int list[kLoraTileRows];               // adapter of a slot
  int warp_count[4][kLoraTileRows];      // its tokens among each 32 of the tile
  int count[kLoraTileRows];              // its tokens
  int start[kLoraTileRows + 1];          // where they begin in `order`
  int unit_start[kLoraTileRows + 1];     // units before a slot
  int order[kLoraTileRows];              // the tile's tokens by slot
  int slots;
};

// Sorts the tile's tokens by adapter.  All threads.
__device__ __forceinline__ void sort_tokens(const LoraArgs& a, FewSmem& sm, int tile) {
  const int tid = threadIdx.x;
  const int m = tile * kLoraTileRows + tid;
  if (tid < kLoraMaxAdapters / 32) sm.bits[tid] = 0;
  if (tid < kLoraTileRows)
    for (int w = 0; w < 4; ++w) sm.warp_count[w][tid] = 0;
  int id = -1;
  if (tid < kLoraTileRows && m < a.M) {
    id = __ldg(a.adapter + m);
    if (id >= a.num_adapters) {
      raise_status(a.status, kStatusBadPage);
      id = -1;
    }
  }
  __syncthreads();
  if (id >= 0) atomicOr(&sm.bits[id >> 5], 1u << (id & 31));
  __syncthreads();
  if (tid < 32) {  // ranks of the words
    const int n = __popc(sm.bits[tid]);
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (tid >= off) incl += v;
    }
    sm.word_rank[tid] = incl - n;
    if (tid == 31) sm.slots = incl;
  }
  __syncthreads();
  int slot = -1, before = 0;
  if (tid < kLoraTileRows) {
    if (id >= 0) slot = sm.word_rank[id >> 5] + __popc(sm.bits[id >> 5] & ((1u << (id & 31)) - 1));
    const unsigned same = __match_any_sync(0xffffffffu, slot);
    before = __popc(same & ((1u << (tid & 31)) - 1));
    if (slot >= 0 && before == 0) {  // the first of the warp's tokens with this adapter
      sm.list[slot] = id;            // the same value from every warp
      sm.warp_count[tid >> 5][slot] = __popc(same);
    }
  }
  __syncthreads();
  if (tid < sm.slots) {
    int n = 0;
    for (int w = 0; w < 4; ++w) n += sm.warp_count[w][tid];
    sm.count[tid] = n;
  }
  __syncthreads();
  if (tid < 32) {  // where each slot's tokens and units begin
    int tokens = 0, units = 0;
    for (int s0 = 0; s0 < sm.slots; s0 += 32) {
      const int s = s0 + tid;
      const int n = s < sm.slots ? sm.count[s] : 0, u = (n + kUnitTokens - 1) / kUnitTokens;
      int in = n, iu = u;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int vn = __shfl_up_sync(0xffffffffu, in, off), vu = __shfl_up_sync(0xffffffffu, iu, off);
        if (tid >= off) {
          in += vn;
          iu += vu;
        }
      }
      if (s < sm.slots) {
        sm.start[s] = tokens + in - n;
        sm.unit_start[s] = units + iu - u;
      }
      tokens += __shfl_sync(0xffffffffu, in, 31);
      units += __shfl_sync(0xffffffffu, iu, 31);
    }
    if (tid == 0) {
      sm.start[sm.slots] = tokens;
      sm.unit_start[sm.slots] = units;
    }
  }
  __syncthreads();
  if (slot >= 0) {  // the tokens of a slot in their own order, the same in every CTA
    for (int w = 0; w < (tid >> 5); ++w) before += sm.warp_count[w][slot];
    sm.order[sm.start[slot] + before] = m;
  }
  __syncthreads();
}

// t of one unit: `n` tokens (order[0..n)) of one adapter over k in [k0, k1), ranks [r0, r0 + 16 RC).
// TG token groups of 8 per warp: TG = 1: the eight warps split K; TG = 4: four parts of K times
// two halves of the tokens.
template <int RC, int TG>
__device__ __forceinline__ void few_unit(const LoraArgs& a, FewSmem& sm, const uint16_t* adapter_rows, const int* order,
                                            int n, int r0, int k0, int k1, float scale, float* out) {
  constexpr int kParts = TG == 1 ? kFewWarps : kFewWarps / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % kParts, half = warp / kParts;
  const int g = lane >> 2, q = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // lane's rows: ranks g, g + 8 of each chunk of 16; token g of each group
  const uint16_t* arow[RC][2];
  bool aok[RC][2];
#pragma unroll
  for (int c = 0; c < RC; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + 16 * c + 8 * h + g;
      aok[c][h] = r < a.R;
      arow[c][h] = adapter_rows + static_cast<long long>(aok[c][h] ? r : 0) * a.K;
    }
  const uint16_t* xrow[TG];
  bool xok[TG];
#pragma unroll
  for (int i = 0; i < TG; ++i) {
    const int j = (half * TG + i) * 8 + g;
    xok[i] = j < n;
    xrow[i] = a.x + static_cast<long long>(order[xok[i] ? j : 0]) * a.K;
  }
  float acc[RC][TG][4];
#pragma unroll
  for (int c = 0; c < RC; ++c)
#pragma unroll
    for (int i = 0; i < TG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[c][i][e] = 0.0f;
#pragma unroll 2
  for (int kb = k0 + 32 * part; kb < k1; kb += 32 * kParts) {
    const int k = kb + 8 * q;
    const bool in = k < k1;
    uint4 av[RC][2], xv[TG];
#pragma unroll
    for (int c = 0; c < RC; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        av[c][h] = in && aok[c][h] ? __ldg(reinterpret_cast<const uint4*>(arow[c][h] + k)) : zero;
#pragma unroll
    for (int i = 0; i < TG; ++i) xv[i] = in && xok[i] ? __ldg(reinterpret_cast<const uint4*>(xrow[i] + k)) : zero;
#pragma unroll
    for (int c = 0; c < RC; ++c)
#pragma unroll
      for (int i = 0; i < TG; ++i) {
        mma_bf16_16816(acc[c][i], av[c][0].x, av[c][1].x, av[c][0].y, av[c][1].y, xv[i].x, xv[i].y);
        mma_bf16_16816(acc[c][i], av[c][0].z, av[c][1].z, av[c][0].w, av[c][1].w, xv[i].z, xv[i].w);
      }
  }
  // the parts of K are added in order by the first part's warps, a few chunks at a time
  constexpr int kWarpFloats = 16 * 8 * TG;  // of one chunk of ranks
  static_assert((kParts - 1) * (kFewWarps / kParts) * kWarpFloats <= kRed, "partial sums fit");
#pragma unroll
  for (int c = 0; c < RC; ++c) {
    float* mine = sm.red + ((part - 1) * (kFewWarps / kParts) + half) * kWarpFloats;
    if (part > 0) {
#pragma unroll
      for (int i = 0; i < TG; ++i)
        *reinterpret_cast<float4*>(mine + (i * 32 + lane) * 4) = make_float4(acc[c][i][0], acc[c][i][1], acc[c][i][2], acc[c][i][3]);
    }
    __syncthreads();
    if (part == 0) {
      for (int p = 0; p < kParts - 1; ++p) {
        const float* other = sm.red + (p * (kFewWarps / kParts) + half) * kWarpFloats;
#pragma unroll
        for (int i = 0; i < TG; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(other + (i * 32 + lane) * 4);
          acc[c][i][0] += v.x;
          acc[c][i][1] += v.y;
          acc[c][i][2] += v.z;
          acc[c][i][3] += v.w;
        }
      }
      // accumulator element e: rank g + 8 (e / 2), token 2 q + e % 2
#pragma unroll
      for (int i = 0; i < TG; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 16 * c + g + 8 * (e >> 1), j = (half * TG + i) * 8 + 2 * q + (e & 1);
          if (r < a.R && j < n) out[static_cast<long long>(order[j]) * a.R + r] = scale * acc[c][i][e];
        }
    }
    __syncthreads();
  }
}

template <int RC>
__global__ void __launch_bounds__(kFewThreads, 2) lora_shrink_few_kernel(const LoraArgs a) {
  __shared__ __align__(16) FewSmem sm;
  const int tile = blockIdx.z, split = blockIdx.y;
  // The next kernel starts only when every CTA has passed this wait, so it may read the call's
  // inputs without waiting for this grid.
  pdl_wait_primary();
  pdl_launch_dependents();
  sort_tokens(a, sm, tile);
  // this CTA's part of K, in steps of 32
  const int steps = (a.K + 31) / 32;
  const int k0 = static_cast<int>(static_cast<long long>(steps) * split / a.splits) * 32;
  const int k1 = min(static_cast<int>(static_cast<long long>(steps) * (split + 1) / a.splits) * 32, a.K);
  float* out = a.t_parts + static_cast<long long>(split) * a.M * a.R;
  const int units = sm.unit_start[sm.slots];
  int s = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    while (sm.unit_start[s + 1] <= u) ++s;  // units ascend
    const int first = sm.start[s] + (u - sm.unit_start[s]) * kUnitTokens;
    const int n = min(sm.start[s + 1] - first, kUnitTokens);
    const int id = sm.list[s];
    const float scale = a.scale ? __ldg(a.scale + id) : 1.0f;
    const uint16_t* rows = a.lora_a + static_cast<long long>(id) * a.R * a.K;
    for (int r0 = 0; r0 < a.R; r0 += 16 * RC) {
      if (n <= 8) few_unit<RC, 1>(a, sm, rows, sm.order + first, n, r0, k0, k1, scale, out);
      else few_unit<RC, 4>(a, sm, rows, sm.order + first, n, r0, k0, k1, scale, out);
    }
  }
}

// ------------------------------------------------------------------ first product, many tokens
constexpr int kShrinkThreads = 256;  // loads, products, plan; warps 4..7 epilogue
constexpr int kShrinkCols = 256;     // columns of an accumulator
constexpr int kShrinkMaxStages = 8;
// Three stages of all columns, or more of a tile's few adapters: one of 64 ranks (24 KB) has six.
constexpr int kShrinkRingBytes = 3 * (kBM + kShrinkCols) * kBK * 2;
// rows that this CTA adds up: from each part of K, together 128 rows of up to 128 ranks
constexpr int kShrinkRecvBytes = kBM * kLoraMaxRank * 4;
constexpr size_t kShrinkSmem = 1024 + kShrinkRingBytes + kShrinkRecvBytes + 4096;

struct ShrinkShared {
  uint64_t full[kShrinkMaxStages], empty[kShrinkMaxStages], acc_full, acc_empty, drain;
  uint32_t tmem_base;
  int abort_flag;
  int issued;
  int slot[kBM];
  TilePlan plan;
};
static_assert(sizeof(ShrinkShared) <= 4096, "fits behind the ring");

__global__ void __launch_bounds__(kShrinkThreads, 1)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap amap, const LoraArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ShrinkShared& sb = *reinterpret_cast<ShrinkShared*>(tiles + kShrinkRingBytes + kShrinkRecvBytes);
  volatile int* abort_flag = &sb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x, split = blockIdx.y, side = blockIdx.z;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&amap);
    for (int s = 0; s < kShrinkMaxStages; ++s) {
      mbar_init(smem_u32(&sb.full[s]), 1);
      mbar_init(smem_u32(&sb.empty[s]), 1);
    }
    mbar_init(smem_u32(&sb.acc_full), 1);
    mbar_init(smem_u32(&sb.acc_empty), 4);
    mbar_init(smem_u32(&sb.drain), 1);
    sb.abort_flag = 0;
    sb.issued = 0;
    fence_barrier_init();
  }
  // The next kernel starts only when every CTA has passed this wait, so it may read the call's
  // inputs without waiting for this grid.
  pdl_wait_primary();
  pdl_launch_dependents();
  int mine = -1;  // slot of the epilogue thread's row
  if (warp >= 4) sb.slot[threadIdx.x - 128] = mine = make_plan<kBM>(a, sb.plan, threadIdx.x - 128, tile * kBM, 0);
  __syncthreads();
  const int slots = sb.plan.slots;
  const int per_pass = kShrinkCols / a.R;  // adapters side by side
  const int passes = (slots + per_pass - 1) / per_pass;
  if (side >= passes) return;  // the whole cluster, before TMEM is taken
  cluster_arrive_relaxed();  // waited for before the first store into another CTA
  const int owner_rows = kBM / a.splits;  // of the tile: CTA `split` adds up [split * owner_rows, ..)
  float* recv = reinterpret_cast<float*>(tiles + kShrinkRingBytes);  // [part][R / 4][row], four each
  // this CTA's part of K, in steps of 64
  const int steps = (a.K + kBK - 1) / kBK;
  const int k0 = static_cast<int>(static_cast<long long>(steps) * split / a.splits);
  const int k_steps = static_cast<int>(static_cast<long long>(steps) * (split + 1) / a.splits) - k0;
  if (warp == 1) {
    tmem_alloc(smem_u32(&sb.tmem_base), kShrinkCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;
  const uint32_t ring = smem_u32(tiles);
  const int xbytes = a.box_rows * kBK * 2;
  // (multiples of 1 KB, as the swizzled operands need: rows in eights)
  const int stage_bytes = kBM * kBK * 2 + min(per_pass, slots) * a.R * kBK * 2;
  const int stages = min(kShrinkRingBytes / stage_bytes, kShrinkMaxStages);
  cluster_wait();  // every CTA of the cluster runs

  if (warp == 0) {
    RingPos p;
    int issued = 0;
    bool ok = true;
    for (int pass = side; pass < passes && ok; pass += gridDim.z) {
      const int first = pass * per_pass, n = min(per_pass, slots - first);
      for (int ks = 0; ks < k_steps; ++ks, p.next(stages)) {
        ok = p.round == 0 || wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        const uint32_t bar = smem_u32(&sb.full[p.stage]), dst = ring + p.stage * stage_bytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, xbytes + n * a.R * kBK * 2);
          tma_load_2d(dst, &xmap, (k0 + ks) * kBK, tile * kBM, bar, l2_policy_evict_last());
          sb.issued = ++issued;
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32)  // a box of R rows per adapter
          tma_load_2d(dst + kBM * kBK * 2 + i * a.R * kBK * 2, &amap, (k0 + ks) * kBK, sb.plan.list[first + i] * a.R, bar,
                      l2_policy_evict_last());
      }
    }
    if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
  } else if (warp == 1) {
    RingPos p;
    int i = 0;
    bool ok = true;
    for (int pass = side; pass < passes && ok; pass += gridDim.z, ++i) {
      const int n = min(per_pass, slots - pass * per_pass);
      const uint32_t idesc = idesc_bf16_kk(kBM, (n * a.R + 15) / 16 * 16);
      if (i > 0) ok = wait_or_abort(smem_u32(&sb.acc_empty), (i - 1) & 1, a.timeout_ns, abort_flag);
      if (!ok) break;
      tc_fence_after();
      for (int ks = 0; ks < k_steps; ++ks, p.next(stages)) {
        ok = wait_or_abort(smem_u32(&sb.full[p.stage]), p.round & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t stage = ring + p.stage * stage_bytes;
          const uint64_t xd = sw128_kmajor(stage), ad = sw128_kmajor(stage + kBM * kBK * 2);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) tc_mma_ss(tmem, xd + 2 * kk, ad + 2 * kk, idesc, (ks | kk) != 0);
          tc_commit(smem_u32(&sb.empty[p.stage]));
        }
      }
      if (ok && elect_one()) tc_commit(smem_u32(&sb.acc_full));
    }
    if (elect_one()) {
      if (!ok) raise_status(a.status, kStatusTimeout);
      tc_commit(smem_u32(&sb.drain));
      if (!mbar_wait(smem_u32(&sb.drain), 0, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, r = 32 * q + lane;
    const uint32_t acc = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const float scale = mine >= 0 && a.scale ? __ldg(a.scale + sb.plan.list[mine]) : 1.0f;
    const uint32_t out = dsmem_addr(smem_u32(recv + (split * (a.R / 4) * owner_rows + r % owner_rows) * 4), r / owner_rows);
    int i = 0;
    for (int pass = side; pass < passes; pass += gridDim.z, ++i) {
      const int first = pass * per_pass, n = min(per_pass, slots - first);
      if (!wait_or_abort(smem_u32(&sb.acc_full), i & 1, a.timeout_ns, abort_flag)) break;
      tc_fence_after();
      for (int s = 0; s < n; ++s) {
        const bool own = mine == first + s;
        if (!__any_sync(0xffffffffu, own)) continue;
        for (int c = 0; c < a.R; c += 8) {
          uint32_t v[8];
          tmem_ld8(acc + s * a.R + c, v);
          tc_wait_ld();
          if (own) {
            float f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] = scale * __uint_as_float(v[u]);
            dsmem_st4(out + 4 * c * owner_rows, f[0], f[1], f[2], f[3]);
            dsmem_st4(out + 4 * (c + 4) * owner_rows, f[4], f[5], f[6], f[7]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sb.acc_empty));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {  // copies still in flight land before the shared memory is released
    for (int s = 0; s < stages && s < sb.issued; ++s) {
      const int last = sb.issued - 1 - ((sb.issued - 1 - s) % stages);
      if (!mbar_wait(smem_u32(&sb.full[s]), (last / stages) & 1, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
  }
  cluster_sync();  // every part of the rows has arrived
  const int parts = a.splits;
  for (int i = threadIdx.x; i < owner_rows * (a.R / 8); i += kShrinkThreads) {
    const int r = i % owner_rows, c = i / owner_rows * 8, s = sb.slot[split * owner_rows + r];
    if (s < 0 || s / per_pass % static_cast<int>(gridDim.z) != side) continue;  // none, or another cluster's
    float sum[8] = {};
    for (int p = 0; p < parts; ++p) {
      const float4* v = reinterpret_cast<const float4*>(recv) + (p * (a.R / 4) + c / 4) * owner_rows + r;
      const float4 v0 = v[0], v1 = v[owner_rows];
      sum[0] += v0.x;
      sum[1] += v0.y;
      sum[2] += v0.z;
      sum[3] += v0.w;
      sum[4] += v1.x;
      sum[5] += v1.y;
      sum[6] += v1.z;
      sum[7] += v1.w;
    }
    *reinterpret_cast<uint4*>(a.t + static_cast<long long>(tile * kBM + split * owner_rows + r) * a.R + c) =
        make_uint4(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]), pack_bf16x2(sum[4], sum[5]),
                   pack_bf16x2(sum[6], sum[7]));
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kShrinkCols);
  }
}

// ------------------------------------------------------------------ product with W, adapters added
constexpr int kThreads = 384;   // 4 control warps, 4 epilogue warps, 4 warps that write T
constexpr int kMaxStages = 16;
constexpr int kMaxTBufs = 8;
constexpr int kMaxBlockN = 224;
constexpr int kTCols = 32;      // TMEM columns of a T buffer: 64 values of K, four chunks of 16 ranks
constexpr int kChunks = 4;      // chunks of 16 ranks per ring stage
constexpr int kStageTarget = 24 * 1024;  // bytes of a ring stage, where blocks are smaller
constexpr uint32_t kTmemCols = 512;
// A tile per CTA (persistent), per pair of CTAs (persistent), per cluster that shares K.
constexpr int kModeSingle = 0, kModePair = 1, kModeSplit = 2;
// Pairs have the SM to themselves; the others leave room for the first kernel's CTAs.
__host__ __device__ constexpr int ring_bytes(int mode) { return (mode == kModePair ? 196 : 176) * 1024; }
// An MMA reads 128 rows of x also where a box has fewer: behind the last stage, too, that stays
// inside the allocation (what it reads there goes to accumulator rows that are never stored).
constexpr size_t smem_bytes(int mode) { return 1024 + ring_bytes(mode) + kBM * kBK * 2 + 4096; }

struct LoraBarriers {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], t_full[kMaxTBufs], t_empty[kMaxTBufs];
  uint64_t plan_full[2], plan_empty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
  int issued;
  TilePlan plan[2];  // of this tile's tokens and the next's
};
static_assert(sizeof(LoraBarriers) <= 4096, "barriers and plans fit");

// The tcgen05 instructions and copies for one CTA or for a pair (an M = 256 MMA on both SMs,
// issued by the leading CTA; operands and accumulator halves lie at the same places in both).
template <bool kPair>
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(ad), "l"(bd), "r"(idesc)
        : "memory");
  else
    tc_mma_ss(d, ad, bd, idesc, 1u);
}
template <bool kPair>
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(at), "l"(bd), "r"(idesc)
        : "memory");
  else
    tc_mma_ts(d, at, bd, idesc, 1u);
}
// Arrive on `bar` (in a pair: on both CTAs') when all tcgen05 work issued so far is done.
template <bool kPair>
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    tc_commit(bar);
}
// Barriers of the leading CTA (`bar`: a shared::cluster address in a pair).  None of these arrivals
// publishes memory to the other CTA's threads: copies report themselves, accumulators and T are
// handed over by tcgen05 fences.
template <bool kPair>
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
  if constexpr (kPair) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
  else mbar_arrive(bar);
}
template <bool kPair>
__device__ __forceinline__ void pair_expect_tx(uint32_t bar, uint32_t bytes) {
  if constexpr (kPair)
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  else
    mbar_arrive_expect_tx(bar, bytes);
}
template <bool kPair>
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
        : "memory");
  else
    tma_load_2d(dst, map, x, y, bar, policy);
}
template <bool kPair>
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar, uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar),
        "l"(policy)
        : "memory");
  else
    tma_load_3d(dst, map, x, y, z, bar, policy);
}

// Write bias[n0 + c] (c < bn, zero past N) into every lane of the accumulator columns of this
// warp's TMEM lane quarter.
__device__ __forceinline__ void seed_bias(uint32_t taddr, const uint16_t* bias, int n0, int N, int bn) {
#pragma unroll 1
  for (int c = 0; c < bn; c += 16) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = n0 + c + i;
      const uint32_t bits = (bias != nullptr && n < N) ? static_cast<uint32_t>(__ldg(bias + n)) : 0u;
      r[i] = bits << 16;  // bf16 -> fp32 bit pattern
    }
    tmem_st16(taddr + c, r);
  }
}

__device__ __forceinline__ bool bf16_nan(uint32_t pair) {  // one of two
  return (pair & 0x7FFFu) > 0x7F80u || (pair & 0x7FFF0000u) > 0x7F800000u;
}

// Part (of 32 lanes) of x[m] W^T for columns n .. n + kCols - 1 of W, and of t B^T behind it.
template <int kCols, typename St>
__device__ __forceinline__ void row_products(const LoraArgs& a, const uint16_t* x, int id, int n, St&& st, float (&sum)[kCols]) {
  const int lane = threadIdx.x & 31;
  const uint16_t* w = a.w + static_cast<long long>(n) * a.K;
#pragma unroll kCols == 1 ? 4 : 1
  for (int k = 8 * lane; k < a.K; k += 256) {
    const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x + k));
    const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(w + static_cast<long long>(i) * a.K + k));
      const uint32_t ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[i] = fmaf(__uint_as_float(xs[j] << 16), __uint_as_float(ws[j] << 16), sum[i]);
        sum[i] = fmaf(__uint_as_float(xs[j] & 0xFFFF0000u), __uint_as_float(ws[j] & 0xFFFF0000u), sum[i]);
      }
    }
  }
  if (id >= 0) {
    const uint16_t* b = a.lora_b + (static_cast<long long>(id) * a.N + n) * a.R;
    for (int r = lane; r < a.R; r += 32) {
      const float t = __uint_as_float(st(r) << 16);
#pragma unroll
      for (int i = 0; i < kCols; ++i) sum[i] = fmaf(t, __uint_as_float(static_cast<uint32_t>(__ldg(b + i * a.R + r)) << 16), sum[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kCols; ++i)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
}

// Outputs that are not finite once more, each from the operands of its own token alone: an adapter of
// another token in the tile may have made them so (0 times infinity).  By a whole warp, whose lane i
// has stored row row0 + i; bit c of its `odd`: columns n0 + 8 c .. + 7 are not all finite.  A row with a NaN
// of its own is NaN throughout already and stays: a batch may be padded with such rows (4096 -> 2880, 333
// tokens, one of them NaN: as without; a lane by itself for each element, 5.9 ms).  An adapter with a NaN
// in one output feature costs the others' rows a column: 2880 -> 5120, 64 tokens, 0.15 ms.
__device__ __noinline__ void repair_rows(const LoraArgs& a, unsigned odd, int row0, int n0) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // the other lanes' stores are visible
  for (unsigned rows = __ballot_sync(0xffffffffu, odd != 0); rows; rows &= rows - 1) {
    const int i = __ffs(rows) - 1, m = row0 + i;
    const uint16_t* x = a.x + static_cast<long long>(m) * a.K;
    int id = __ldg(a.adapter + m);
    if (id >= a.num_adapters) id = -1;
    auto st = [&](int r) -> uint32_t {  // as the tensor core gets it
      if (a.t) return __ldcg(a.t + static_cast<long long>(m) * a.R + r);
      float v = 0.0f;
      for (int s = 0; s < a.splits; ++s) v += __ldcg(a.t_parts + (static_cast<long long>(s) * a.M + m) * a.R + r);
      return pack_bf16x2(v, 0.0f) & 0xFFFFu;
    };
    bool looked = false;
    for (unsigned blocks = __shfl_sync(0xffffffffu, odd, i); blocks; blocks &= blocks - 1) {
      const int n = n0 + 8 * (__ffs(blocks) - 1);
      uint16_t* out = a.out + static_cast<long long>(m) * a.N + n;
      const uint32_t now = lane < 8 ? *reinterpret_cast<const volatile uint16_t*>(out + lane) : 0;
      const unsigned which = __ballot_sync(0xffffffffu, (now & 0x7F80u) == 0x7F80u);
      if (!looked && __ballot_sync(0xffffffffu, bf16_nan(now)) == 0xFFu) {
        bool nan = false;
        for (int k = 8 * lane; k < a.K; k += 256) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + k));
          nan |= bf16_nan(v.x) || bf16_nan(v.y) || bf16_nan(v.z) || bf16_nan(v.w);
        }
        if (id >= 0)
          for (int r = lane; r < a.R; r += 32) nan |= bf16_nan(st(r));
        if (__any_sync(0xffffffffu, nan)) break;
        looked = true;
      }
      float mine = 0.0f;
      if (which == 0) continue;
      if ((which & (which - 1)) == 0) {  // one column
        float sum[1] = {};
        row_products(a, x, id, n + __ffs(which) - 1, st, sum);
        mine = sum[0];
      } else {
        float sum[8] = {};
        row_products(a, x, id, n, st, sum);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (lane == c) mine = sum[c];
      }
      if (which >> lane & 1) {
        if (a.bias) mine += __uint_as_float(static_cast<uint32_t>(__ldg(a.bias + n + lane)) << 16);
        out[lane] = static_cast<uint16_t>(pack_bf16x2(mine, 0.0f) & 0xFFFFu);
      }
    }
  }
}

// A ring stage holds `sub` blocks of 64 values of K: small tiles' blocks are a few KB, and a stage's
// way round the ring costs the same for one as for four.  wrows: rows of W that a CTA stages.
__host__ __device__ constexpr int block_bytes(int box_rows, int wrows) { return (box_rows + wrows) * kBK * 2; }
__host__ __device__ constexpr int stage_blocks(int box_rows, int wrows) {
  const int n = kStageTarget / block_bytes(box_rows, wrows);
  return n >= 4 ? 4 : n >= 2 ? 2 : 1;
}
__host__ __device__ constexpr int stage_bytes(int box_rows, int wrows) {
  return stage_blocks(box_rows, wrows) * block_bytes(box_rows, wrows);
}
__host__ __device__ constexpr int stage_count(int mode, int box_rows, int wrows) {
  const int n = ring_bytes(mode) / stage_bytes(box_rows, wrows);
  return n > kMaxStages ? kMaxStages : n;
}
// Accumulators r of row m, columns n .. n + 7, to the output (where n < N; N is a multiple of 8).
// Is one of them not finite: a bit for the block of columns (the c-th of a tile, of eight).
__device__ __forceinline__ unsigned store8(const LoraArgs& a, int m, int n, int c, const float (&r)[8]) {
  float odd = 0.0f;  // NaN if some element is not finite
#pragma unroll
  for (int v = 0; v < 8; ++v) odd = fmaf(r[v], 0.0f, odd);
  *reinterpret_cast<uint4*>(a.out + static_cast<long long>(m) * a.N + n) =
      make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7]));
  return odd != 0.0f ? 1u << c : 0u;
}

__host__ __device__ constexpr int acc_columns(int bn) { return (bn + 31) / 32 * 32; }
__host__ __device__ constexpr int t_bufs(int bn) {
  const int n = (static_cast<int>(kTmemCols) - 2 * acc_columns(bn)) / kTCols;
  return n > kMaxTBufs ? kMaxTBufs : n;
}
static_assert(kMaxBlockN / 8 <= 32, "a bit for eight columns");
static_assert(t_bufs(kMaxBlockN) >= 2, "two buffers of T behind the accumulators");

// RC: chunks of 16 ranks (a rank in between counts as the next size: the boxes behind R read zeros).
// Outside pairs 80 registers (two blocks' worth), so that a CTA of the first kernel fits beside.
template <int RC, int kMode>
__global__ void __launch_bounds__(kThreads, kMode == kModePair || RC > 4 ? 1 : 2)
    lora_linear_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap bmap, const LoraArgs a) {
  constexpr bool kPair = kMode == kModePair, kSplit = kMode == kModeSplit;
  constexpr int kCtas = kPair ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LoraBarriers& sb = *reinterpret_cast<LoraBarriers*>(tiles + ring_bytes(kMode) + kBM * kBK * 2);
  volatile int* abort_flag = &sb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const int tiles_m = (a.tiles_m + kCtas - 1) / kCtas, tiles_total = tiles_m * a.tiles_n;
  // parts of K and of the adapters, and this CTA's (the whole, part 0, without clusters)
  const int parts = kSplit ? a.k_parts : 1, part = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int t_first = blockIdx.x / (kCtas * parts), t_step = gridDim.x / (kCtas * parts);
  const int bn = a.block_n, wrows = bn / kCtas;
  const int sub = stage_blocks(a.box_rows, wrows), stages = stage_count(kMode, a.box_rows, wrows);
  const int xbytes = a.box_rows * kBK * 2, bbytes = block_bytes(a.box_rows, wrows), sbytes = sub * bbytes;
  const int all_blocks = (a.K + kBK - 1) / kBK, k_first = all_blocks * part / parts;
  const int k_blocks = all_blocks * (part + 1) / parts - k_first, k_stages = (k_blocks + sub - 1) / sub;
  const int tbufs = t_bufs(bn);
  const uint32_t acc_stride = acc_columns(bn), t_col = 2 * acc_stride;
  // the leading CTA's barriers
  auto lead = [&](uint64_t& bar) { return kPair ? dsmem_addr(smem_u32(&bar), 0) : smem_u32(&bar); };
  const uint32_t full0 = lead(sb.full[0]), acc_empty0 = lead(sb.acc_empty[0]), t_full0 = lead(sb.t_full[0]);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&sb.full[s]), kCtas);
      mbar_init(smem_u32(&sb.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sb.acc_full[b]), 1);
      mbar_init(smem_u32(&sb.acc_empty[b]), 4 * kCtas);
    }
    for (int b = 0; b < tbufs; ++b) {
      mbar_init(smem_u32(&sb.t_full[b]), 4 * kCtas);
      mbar_init(smem_u32(&sb.t_empty[b]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sb.plan_full[b]), 128);
      mbar_init(smem_u32(&sb.plan_empty[b]), rank == 0 ? 2 : 1);  // the loads, and the products
    }
    mbar_init(smem_u32(&sb.drain), 1);
    sb.abort_flag = 0;
    sb.issued = 0;
    fence_barrier_init();
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&bmap);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sb.tmem_base)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(smem_u32(&sb.tmem_base), kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // the other CTA's barriers exist
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;
  const uint32_t ring = smem_u32(tiles);
  pdl_launch_dependents();  // (they wait for this grid's end)
  // Ring stages of a tile behind those of K: four chunks of 16 ranks each.
  auto adapter_stages = [&](int slots) { return (slots * RC + kChunks - 1) / kChunks; };
  // The plans, one per row block that this CTA passes: made by the warps that write T, read by those
  // that load and multiply, two at a time.
  struct PlanPos {
    int mt = -1, n = -1;  // row block; plans so far less one
  };
  // the plan of row block mt is there (all lanes agree); releases the one before
  auto next_plan = [&](PlanPos& p, int mt) {
    if (p.mt == mt) return true;
    if (p.n >= 0 && elect_one()) mbar_arrive(smem_u32(&sb.plan_empty[p.n & 1]));
    __syncwarp();
    p.mt = mt;
    ++p.n;
    return wait_or_abort(smem_u32(&sb.plan_full[p.n & 1]), (p.n >> 1) & 1, a.timeout_ns, abort_flag);
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    const uint64_t policy = l2_policy_evict_last();  // x is read for every column tile, W for every row block
    RingPos p;
    int issued = 0;
    PlanPos plan;
    bool ok = true;
    auto free_stage = [&]() {
      return p.round == 0 || wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
    };
    for (int t = t_first; t < tiles_total && ok; t += t_step) {
      const int m0 = (t / a.tiles_n * kCtas + rank) * kBM, n0 = (t % a.tiles_n) * bn + rank * wrows;
      for (int ks = 0; ks < k_stages; ++ks, p.next(stages)) {
        ok = free_stage();
        if (!ok) break;
        const int blocks = min(sub, k_blocks - ks * sub);
        if (elect_one()) {
          const uint32_t bar = full0 + 8 * p.stage;
          pair_expect_tx<kPair>(bar, blocks * bbytes);
          for (int u = 0; u < blocks; ++u) {
            const uint32_t dst = ring + p.stage * sbytes + u * bbytes;
            const int x = (k_first + ks * sub + u) * kBK;
            pair_load_2d<kPair>(dst, &xmap, x, m0, bar, policy);  // rows past M are zero-filled
            pair_load_2d<kPair>(dst + xbytes, &wmap, x, n0, bar, policy);
          }
          sb.issued = ++issued;
        }
        __syncwarp();
      }
      if (!ok) break;
      ok = next_plan(plan, t / a.tiles_n);
      if (!ok) break;
      const TilePlan& tp = sb.plan[plan.n & 1];
      const int slots = tp.slots;
      for (int e = part; e < adapter_stages(slots); e += parts, p.next(stages)) {
        const int first = e * kChunks, n = min(kChunks, slots * RC - first);
        ok = free_stage();
        if (!ok) break;
        int id[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) id[c] = tp.list[min((first + c) / RC, slots - 1)];
        if (elect_one()) {
          const uint32_t bar = full0 + 8 * p.stage;
          pair_expect_tx<kPair>(bar, n * wrows * 32);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < n)
              pair_load_3d<kPair>(ring + p.stage * sbytes + c * wrows * 32, &bmap, (first + c) % RC * 16, n0, id[c], bar, policy);
          sb.issued = ++issued;
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------------ products
    const uint32_t idesc = idesc_bf16_kk(kCtas * kBM, bn);
    RingPos p, tb;
    int i = 0;
    PlanPos plan;
    bool ok = true;
    for (int t = t_first; t < tiles_total && ok; t += t_step, ++i) {
      const int b = i & 1;
      ok = wait_or_abort(smem_u32(&sb.acc_empty[b]), (i >> 1) & 1, a.timeout_ns, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * acc_stride;
      for (int ks = 0; ks < k_stages; ++ks, p.next(stages)) {
        ok = wait_or_abort(smem_u32(&sb.full[p.stage]), p.round & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t stage = ring + p.stage * sbytes;
        const int blocks = min(sub, k_blocks - ks * sub);
        if (elect_one()) {
#pragma unroll 1
          for (int u = 0; u < blocks; ++u) {
            const uint64_t xd = sw128_kmajor(stage + u * bbytes), wd = sw128_kmajor(stage + u * bbytes + xbytes);
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) pair_mma_ss<kPair>(d, xd + 2 * kk, wd + 2 * kk, idesc);
          }
          pair_commit<kPair>(smem_u32(&sb.empty[p.stage]));
        }
      }
      if (!ok) break;
      ok = next_plan(plan, t / a.tiles_n);
      if (!ok) break;
      const int slots = sb.plan[plan.n & 1].slots;
      for (int e = part; e < adapter_stages(slots); e += parts, p.next(stages), tb.next(tbufs)) {
        const int n = min(kChunks, slots * RC - e * kChunks);
        ok = wait_or_abort(smem_u32(&sb.t_full[tb.stage]), tb.round & 1, a.timeout_ns, abort_flag) &&
             wait_or_abort(smem_u32(&sb.full[p.stage]), p.round & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t t_addr = tmem + t_col + tb.stage * kTCols;
          const uint64_t bd = sw32_kmajor(ring + p.stage * sbytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < n) pair_mma_ts<kPair>(d, t_addr + c * 8, bd + 2 * c * wrows, idesc);
          pair_commit<kPair>(smem_u32(&sb.t_empty[tb.stage]));
          pair_commit<kPair>(smem_u32(&sb.empty[p.stage]));
        }
      }
      if (ok && elect_one()) pair_commit<kPair>(smem_u32(&sb.acc_full[b]));
    }
    if (elect_one()) {
      if (!ok) raise_status(a.status, kStatusTimeout);
      // every product issued by this thread has finished before TMEM is released
      pair_commit<kPair>(smem_u32(&sb.drain));
      if (!mbar_wait(smem_u32(&sb.drain), 0, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ T
    const int q = warp & 3;  // TMEM lane quarter
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    RingPos tb;
    int held_mt = -1, plans = 0, slots = 0, my_slot = -1;
    uint32_t tp[8 * RC];  // s t of this thread's row, bf16 pairs
#pragma unroll
    for (int e = 0; e < 8 * RC; ++e) tp[e] = 0;
    // A warp that gave up still comes to the next plan's barrier, where all four learn of it: none
    // is left waiting there.
    bool ok = true;
    for (int t = t_first; t < tiles_total; t += t_step) {
      const int mt = t / a.tiles_n;
      if (mt != held_mt) {
        held_mt = mt;
        if (ok && plans >= 2) ok = wait_or_abort(smem_u32(&sb.plan_empty[plans & 1]), ((plans >> 1) - 1) & 1, a.timeout_ns, abort_flag);
        ok = plan_barrier_and(ok);  // all four warps go on, or none
        if (!ok) break;
        TilePlan& plan = sb.plan[plans & 1];
        const int i = 32 * q + lane, row = (mt * kCtas + rank) * kBM + i;
        if constexpr (kPair) my_slot = make_plan<2 * kBM>(a, plan, i, mt * 2 * kBM, rank * kBM);
        else my_slot = make_plan<kBM>(a, plan, i, mt * kBM, 0);
        plan_barrier();
        slots = plan.slots;
        mbar_arrive(smem_u32(&sb.plan_full[plans & 1]));
        if (plans == 0) pdl_wait_primary();  // t
        ++plans;
        if (my_slot >= 0) {
          if constexpr (kPair) {
            const uint4* src = reinterpret_cast<const uint4*>(a.t + static_cast<long long>(row) * a.R);
#pragma unroll
            for (int c = 0; c < 2 * RC; ++c) {  // eight ranks at a time (R is a multiple of 8)
              const uint4 v = 8 * c < a.R ? __ldcg(src + c) : make_uint4(0, 0, 0, 0);
              tp[4 * c] = v.x;
              tp[4 * c + 1] = v.y;
              tp[4 * c + 2] = v.z;
              tp[4 * c + 3] = v.w;
            }
          } else {
            const float* src = a.t_parts + static_cast<long long>(row) * a.R;
            const long long stride = static_cast<long long>(a.M) * a.R;
#pragma unroll
            for (int c = 0; c < 4 * RC; ++c) {  // four ranks at a time
              float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
              if (4 * c < a.R) {
                for (int s = 0; s < a.splits; ++s) {
                  const float4 u = __ldcg(reinterpret_cast<const float4*>(src + s * stride + 4 * c));
                  v.x += u.x;
                  v.y += u.y;
                  v.z += u.z;
                  v.w += u.w;
                }
              }
              tp[2 * c] = pack_bf16x2(v.x, v.y);
              tp[2 * c + 1] = pack_bf16x2(v.z, v.w);
            }
          }
        }
      }
      for (int e = part; e < adapter_stages(slots); e += parts, tb.next(tbufs)) {
        if (ok && tb.round != 0) ok = wait_or_abort(smem_u32(&sb.t_empty[tb.stage]), (tb.round - 1) & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t r[32];
        if constexpr (RC <= kChunks) {  // whole slots per buffer
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const bool own = my_slot == e * (kChunks / RC) + c / RC;
#pragma unroll
            for (int w = 0; w < 8; ++w) r[8 * c + w] = own ? tp[8 * (c % RC) + w] : 0u;
          }
        } else {  // a slot takes RC / kChunks buffers
          const bool own = my_slot == e / (RC / kChunks);
          const bool upper = e % (RC / kChunks) != 0;
#pragma unroll
          for (int w = 0; w < 32; ++w) r[w] = own ? (upper ? tp[32 + w] : tp[w]) : 0u;
        }
        const uint32_t dst = lane_base + t_col + tb.stage * kTCols;
        tmem_st16_at<0>(dst, r);
        tmem_st16_at<16>(dst + 16, r);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair_arrive<kPair>(t_full0 + 8 * tb.stage);
      }
    }
    if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lane quarter
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    for (int j = 0; j < 2; ++j) {  // both accumulators start from the bias of this CTA's first tiles
      const int t = t_first + j * t_step;
      if (t < tiles_total) seed_bias(lane_base + j * acc_stride, part == 0 ? a.bias : nullptr, (t % a.tiles_n) * bn, a.N, bn);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive<kPair>(acc_empty0 + 8 * j);
    }
    pdl_wait_primary();  // no output before the first kernel's end, which may still read what it overwrites
    int i = 0;
    for (int t = t_first; t < tiles_total; t += t_step, ++i) {
      const int b = i & 1;
      const int m0 = (t / a.tiles_n * kCtas + rank) * kBM, n0 = (t % a.tiles_n) * bn;
      const int row = m0 + 32 * q + lane;
      if (!wait_or_abort(smem_u32(&sb.acc_full[b]), (i >> 1) & 1, a.timeout_ns, abort_flag)) break;
      tc_fence_after();
      if constexpr (kSplit) break;  // the one tile: added up below
      const uint32_t acc = lane_base + b * acc_stride;
      unsigned odd = 0;
      if (m0 + 32 * q < a.M) {  // some row of this warp exists
#pragma unroll 1
        for (int c = 0; c < bn; c += 16) {
          uint32_t r[16];
          tmem_ld16(acc + c, r);
          tc_wait_ld();
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            float f[8];
#pragma unroll
            for (int v = 0; v < 8; ++v) f[v] = __uint_as_float(r[h + v]);
            if (row < a.M && n0 + c + h < a.N) odd |= store8(a, row, n0 + c + h, (c + h) / 8, f);
          }
        }
      }
      const int t2 = t + 2 * t_step;  // this buffer's next tile starts from its bias
      if (t2 < tiles_total) seed_bias(acc, a.bias, (t2 % a.tiles_n) * bn, a.N, bn);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive<kPair>(acc_empty0 + 8 * b);
      if (__any_sync(0xffffffffu, odd != 0)) repair_rows(a, odd, m0 + 32 * q, n0);
    }
  }

  if constexpr (kSplit) {
    // Part p adds up and stores columns [p cw, (p + 1) cw) of the tile.  The others' go into its
    // ring, whose operands every CTA has consumed behind the first barrier; warps 4..7 and 8..11
    // take turns of 8 columns.
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const int cw = (bn + 8 * parts - 1) / (8 * parts) * 8;
    const int q = warp & 3, r = 32 * q + lane, half = warp >= 8 ? 1 : 0;
    const int mt = t_first / a.tiles_n, n0 = (t_first % a.tiles_n) * bn, row = mt * kBM + r;
    const uint32_t acc = tmem + (static_cast<uint32_t>(32 * q) << 16);
    // [part][cw / 4][row], four columns each: a warp's stores are 512 bytes in a row
    const float4* recv = reinterpret_cast<const float4*>(tiles);
    const bool warp_live = warp >= 4 && mt * kBM + 32 * q < a.M;
    if (warp_live) {
#pragma unroll 1
      for (int c = 8 * half; c < bn; c += 16) {
        const int owner = c / cw;
        if (owner == part) continue;
        uint32_t v[8];
        tmem_ld8(acc + c, v);
        tc_wait_ld();
        if (row < a.M) {
          const uint32_t to = dsmem_addr(ring + 16 * ((part * (cw / 4) + (c - owner * cw) / 4) * kBM + r), owner);
          dsmem_st4(to, __uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
          dsmem_st4(to + 16 * kBM, __uint_as_float(v[4]), __uint_as_float(v[5]), __uint_as_float(v[6]), __uint_as_float(v[7]));
        }
      }
    }
    __syncwarp();
    cluster_sync();
    if (warp_live && !__any_sync(0xffffffffu, *abort_flag != 0)) {
      unsigned odd = 0;
#pragma unroll 1
      for (int c = part * cw + 8 * half; c < min((part + 1) * cw, bn); c += 16) {
        uint32_t v[8];
        tmem_ld8(acc + c, v);
        tc_wait_ld();
        if (row < a.M && n0 + c < a.N) {
          float sum[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) sum[u] = 0.0f;
          for (int p = 0; p < parts; ++p) {  // in order, whoever adds
            float4 lo, hi;
            if (p == part) {
              lo = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
              hi = make_float4(__uint_as_float(v[4]), __uint_as_float(v[5]), __uint_as_float(v[6]), __uint_as_float(v[7]));
            } else {
              const float4* from = recv + (p * (cw / 4) + (c - part * cw) / 4) * kBM + r;
              lo = from[0];
              hi = from[kBM];
            }
            sum[0] += lo.x;
            sum[1] += lo.y;
            sum[2] += lo.z;
            sum[3] += lo.w;
            sum[4] += hi.x;
            sum[5] += hi.y;
            sum[6] += hi.z;
            sum[7] += hi.w;
          }
          odd |= store8(a, row, n0 + c, c / 8, sum);
        }
      }
      if (__any_sync(0xffffffffu, odd != 0)) repair_rows(a, odd, mt * kBM + 32 * q, n0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();
  if (threadIdx.x == 0 && rank == 0) {
    // Copies still in flight land before the shared memory is released.  A stage completes once
    // every CTA's producer has arrived; arrivals that an aborted one did not make are made up for.
    auto peer = [&](const int* v, int cta) {
      int x;
      if constexpr (kPair)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(dsmem_addr(smem_u32(v), cta)) : "memory");
      else
        x = *const_cast<const volatile int*>(v);
      return x;
    };
    int aborted = 0, most = 0;
    for (int c = 0; c < kCtas; ++c) {
      aborted |= peer(&sb.abort_flag, c);
      most = max(most, peer(&sb.issued, c));
    }
    if (aborted) {
      for (int c = 0; c < kCtas; ++c)
        for (int g = peer(&sb.issued, c); g < most; ++g) pair_arrive<kPair>(full0 + 8 * (g % stages));
      for (int s = 0; s < stages && s < most; ++s) {
        const int last = most - 1 - ((most - 1 - s) % stages);
        if (!mbar_wait(smem_u32(&sb.full[s]), (last / stages) & 1, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
      }
    }
  }
  if constexpr (kPair) {
    // the leader's last arrival here is behind all its earlier ones: none is still to come
    if (threadIdx.x == 0 && rank != 0 && !mbar_wait(smem_u32(&sb.drain), 0, kDrainTimeoutNs))
      raise_status(a.status, kStatusTimeout);
    __syncthreads();
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    else
      tmem_dealloc(tmem, kTmemCols);
  }
}

// The shared-memory opt-in of a kernel, once per device (host threads may race here: atomic
// flags, and setting the attribute twice is harmless).
template <typename Kern>
cudaError_t opt_in(Kern kern, size_t bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

template <int RC, int kMode>
cudaError_t launch_lora_t(const LoraMaps& m, const LoraArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  cudaError_t e = opt_in(lora_linear_kernel<RC, kMode>, smem_bytes(kMode), done);
  if (e != cudaSuccess) return e;
  constexpr int kCtas = kMode == kModePair ? 2 : 1;
  const int cluster = kMode == kModeSplit ? a.k_parts : kCtas;
  const int total = (a.tiles_m + kCtas - 1) / kCtas * a.tiles_n, slots = kMode == kModeSplit ? total : sms / kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((total < slots ? total : slots) * cluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes(kMode);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kMode == kModeSingle ? 1 : 2;
  e = cudaLaunchKernelEx(&cfg, lora_linear_kernel<RC, kMode>, m.x, m.w, m.b, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int RC>
cudaError_t launch_lora_r(const LoraMaps& m, const LoraArgs& a, int sms, cudaStream_t stream) {
  if (a.plan_tiles == 2) return launch_lora_t<RC, kModePair>(m, a, sms, stream);
  return a.k_parts > 1 ? launch_lora_t<RC, kModeSplit>(m, a, sms, stream) : launch_lora_t<RC, kModeSingle>(m, a, sms, stream);
}

}  // namespace

void lora_plan(LoraArgs& a, int sms) {
  a.tiles_m = (a.M + kBM - 1) / kBM;
  a.box_rows = a.M < kBM ? (a.M + 7) / 8 * 8 : kBM;
  const int k_blocks = (a.K + kBK - 1) / kBK;
  // Parts of K of the first product.  Pairs (many tokens): a CTA per SM, clusters of up to 8 parts of at
  // least two steps; else: a step of K for each of a CTA's eight warps, up to 4 parts.
  int pair_splits = 1;
  while (pair_splits < 8 && 2 * pair_splits * a.tiles_m <= sms && 4 * pair_splits <= k_blocks) pair_splits *= 2;
  // As blocks of K: ranks of half the adapters that a tile of tokens can have.  (The host knows the resident
  // ones only: where 2 of 1000 are present, 64 tokens 2880 -> 5120 of rank 16 take 14.7 us instead of 13.8
  // with 2 resident, 1000 tokens of rank 64 38.2 instead of 33.0.)
  const int most = a.M < kBM ? a.M : kBM;
  const int adapter_blocks = ((a.num_adapters < most ? a.num_adapters : most) * ((a.R + 15) / 16) + 7) / 8;
  // Estimated cycles of tiles of bn columns, by single CTAs, by pairs or by clusters that share K; the
  // factors are fitted to times over 27 sizes (1 to 2000 tokens, 4096 -> 2880, 2880 -> 5120 and 640), where
  // what is chosen took up to 4% more than the best, for six of them 7 to 13%.  A block of 64 values of K takes what is
  // longest: the operands' way in (64 bytes a cycle), the tensor core's reading (128 bytes a cycle, 128
  // rows of x whatever their number), its arithmetic.  Clusters that share K add up at the end, and the
  // GPU holds 76, 36 or 15 of them (GPCs of 18 to 20 SMs), fewer beside the first product's CTAs of
  // more tokens: a second round is not considered.  Pairs need whole SMs: those that the first
  // product's CTAs leave (if enough for there to be pairs among them), or all when they are through.  Single CTAs and clusters pay more for it.
  // (4096 -> 2880, 1 token: single CTAs 12.7 us, clusters of 4 11.0; 2880 -> 5120, 64 tokens: 16.4 and,
  // clusters of 2, 14.0; 512 tokens: 25.2, pairs 23.5.)
  auto cycles = [&](int bn, int ctas, int parts) {
    const long long tiles = static_cast<long long>((a.tiles_m + ctas - 1) / ctas) * ((a.N + bn - 1) / bn);
    const bool few = a.M <= 32;
    const long long slots = parts == 1   ? sms / ctas
                            : parts == 2 ? sms * (few ? 76 : 60) / 152
                            : parts == 4 ? sms * (few ? 36 : 32) / 152
                                         : sms * 15 / 152;
    const long long rounds = (tiles + slots - 1) / slots;
    if (parts > 1 && rounds > 1) return 1LL << 60;
    const long long in = 2LL * (a.box_rows + bn / ctas), read = kBM + bn / ctas, mma = 2LL * bn;
    long long block = in > read ? in : read;
    if (mma > block) block = mma;
    long long tile = (k_blocks + adapter_blocks + parts - 1) / parts * (112 + 7 * block / 10) + 53LL * bn;
    if (parts > 1) tile += 3LL * most * (bn - bn / parts) / 10;
    if (ctas == 1) return rounds * tile + 12LL * a.M + (parts == 8 ? 2000 : 0);
    const long long left = sms - static_cast<long long>(pair_splits) * a.tiles_m, beside = 4 * left >= sms ? left / 2 : 0;
    const long long late = tiles > beside ? 16000 + (tiles - beside + slots - 1) / slots * tile : 0;
    return rounds * tile > late ? rounds * tile : late;
  };
  long long least = 1LL << 60;
  auto offer = [&](int bn, int ctas, int parts) {
    const long long c = cycles(bn, ctas, parts);
    if (c >= least) return;
    least = c;
    a.block_n = bn;
    a.plan_tiles = ctas;
    a.k_parts = parts;
  };
  for (int bn = kMaxBlockN; bn >= 16; bn -= 16) offer(bn, 1, 1);
  if (a.tiles_m >= 2)
    for (int bn = kMaxBlockN; bn >= 32; bn -= 32) offer(bn, 2, 1);
  for (int parts = 2; parts <= 8 && 2 * parts <= k_blocks; parts *= 2)
    for (int bn = kMaxBlockN; bn >= 32; bn -= 16) offer(bn, 1, parts);
  a.tiles_n = (a.N + a.block_n - 1) / a.block_n;
  a.splits = a.plan_tiles == 2 ? pair_splits : (a.K + 255) / 256 < 4 ? (a.K + 255) / 256 : 4;
}

cudaError_t launch_lora(const LoraMaps& m, const LoraArgs& a, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = a.splits;
  attr[1].val.clusterDim.z = 1;
  cfg.stream = stream;
  cfg.attrs = attr;
  int most = a.M < kBM ? a.M : kBM;  // distinct adapters of a tile
  if (most > a.num_adapters) most = a.num_adapters;
  const long long room = 2LL * sms / (static_cast<long long>(a.tiles_m) * a.splits);
  cudaError_t e;
  if (a.plan_tiles == 2) {
    static std::atomic<bool> done[64];
    e = opt_in(lora_shrink_kernel, kShrinkSmem, done);
    if (e != cudaSuccess) return e;
    // CTAs side by side: as many passes of 256 columns as a tile can have
    const int per_pass = kShrinkCols / a.R, passes = (most + per_pass - 1) / per_pass;
    // (those that a tile of fewer adapters leaves without work come last)
    cfg.gridDim = dim3(a.tiles_m, a.splits, static_cast<unsigned>(room < 1 ? 1 : room < passes ? room : passes));
    cfg.blockDim = dim3(kShrinkThreads, 1, 1);
    cfg.dynamicSmemBytes = kShrinkSmem;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel, m.x, m.a, a);
  } else {
    // side by side: the units that a tile can have (a long unit more than its adapters)
    const int units = most + 1;
    cfg.gridDim = dim3(static_cast<unsigned>(room < 2 ? 2 : room < units ? room : units), a.splits, a.tiles_m);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.numAttrs = 1;
    e = a.R <= 16   ? cudaLaunchKernelEx(&cfg, lora_shrink_few_kernel<1>, a)
        : a.R <= 32 ? cudaLaunchKernelEx(&cfg, lora_shrink_few_kernel<2>, a)
                    : cudaLaunchKernelEx(&cfg, lora_shrink_few_kernel<4>, a);
  }
  if (e != cudaSuccess) return e;
  if (a.R <= 16) return launch_lora_r<1>(m, a, sms, stream);
  if (a.R <= 32) return launch_lora_r<2>(m, a, sms, stream);
  if (a.R <= 64) return launch_lora_r<4>(m, a, sms, stream);
  return launch_lora_r<8>(m, a, sms, stream);
}

}  // namespace sa
