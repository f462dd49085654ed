// Linear layer with the low-rank adapters of many requests beside it: for token m with adapter a,
//
//     out[m] = x[m] W^T + b + s_a (x[m] A_a^T) B_a^T        A_a [R, K], B_a [N, R]
//
// (page "GPT-OSS on day 0": the projections carry bias terms; the adapters are what requests of
// one server differ in).  Two kernels, in one call:
//
// 1. lora_shrink_kernel: t[m] = x[m] A_a^T, fp32.  Every CTA sorts the 128 tokens of a tile by
//    adapter (a bit per adapter, ranks by population counts) and takes its share of the units
//    (adapter, up to 64 of its tokens) and of K.  Products by warp-level matrix instructions with
//    the ranks as M = 16 and the tokens as N = 8: a unit of one token costs what its adapter's
//    rows cost to read, one of 64 reads each operand once.  Fragments come straight from memory
//    in 16-byte loads: a lane's eight values of K serve two instructions, in the same order for
//    both operands.  The parts of K are added by the reader, in order: no atomics.
// 2. lora_linear_kernel: the product with W on tcgen05, 128 tokens x block_n features per tile,
//    accumulator seeded with the bias, and then on the same accumulator one more product per
//    adapter of the tile: T_i B_i^T, where T_i holds s t for the tokens of adapter i and zeros for
//    the others.  T_i is the A operand in TMEM, written by the threads that own the rows (the
//    epilogue's); B_i comes by TMA in boxes of 16 ranks.  So any mix of adapters in a tile is
//    right, and a tile of one adapter costs R more columns of K.
//    s t is rounded to bf16 for the tensor core, as x is: a relative error of 2^-8 at most per
//    term of a sum over the ranks, of the adapters' part only (which the bf16 output rounds once
//    more anyway).
//    Zeros do not keep out an infinity or NaN of another request's B_i: an element that comes out
//    not finite is computed once more by itself, from its own operands only.
//
// The second kernel starts while the first runs (programmatic dependent launch): the product with
// W needs nothing from it, and only the roles of the adapters' part wait for it.
#include <atomic>
#include <cstdint>

#include "lora_args.h"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr unsigned long long kDrainTimeoutNs = 2000000000ull;

// ------------------------------------------------------------------ first product
constexpr int kShrinkWarps = 8;
constexpr int kShrinkThreads = 32 * kShrinkWarps;
constexpr int kUnitTokens = 64;
constexpr int kRed = 6 * 16 * 32;  // floats: partial sums of the warps that do not add up

struct ShrinkSmem {
  float red[kRed];
  uint32_t bits[kLoraMaxAdapters / 32];
  int word_rank[kLoraMaxAdapters / 32];  // adapters in the words before
  int list[kLoraTileRows];               // adapter of a slot
  int warp_count[4][kLoraTileRows];      // its tokens among each 32 of the tile
  int count[kLoraTileRows];              // its tokens
  int start[kLoraTileRows + 1];          // where they begin in `order`
  int unit_start[kLoraTileRows + 1];     // units before a slot
  int slot[kLoraTileRows];
  int order[kLoraTileRows];              // the tile's tokens by slot
  int slots;
};

// Sorts the tile's tokens by adapter.  All threads.
__device__ __forceinline__ void make_plan(const LoraArgs& a, ShrinkSmem& sm, int tile) {
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
    sm.slot[tid] = slot;
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
__device__ __forceinline__ void shrink_unit(const LoraArgs& a, ShrinkSmem& sm, const uint16_t* adapter_rows, const int* order,
                                            int n, int r0, int k0, int k1, float* out) {
  constexpr int kParts = TG == 1 ? kShrinkWarps : kShrinkWarps / 2;
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
  static_assert((kParts - 1) * (kShrinkWarps / kParts) * kWarpFloats <= kRed, "partial sums fit");
#pragma unroll
  for (int c = 0; c < RC; ++c) {
    float* mine = sm.red + ((part - 1) * (kShrinkWarps / kParts) + half) * kWarpFloats;
    if (part > 0) {
#pragma unroll
      for (int i = 0; i < TG; ++i)
        *reinterpret_cast<float4*>(mine + (i * 32 + lane) * 4) = make_float4(acc[c][i][0], acc[c][i][1], acc[c][i][2], acc[c][i][3]);
    }
    __syncthreads();
    if (part == 0) {
      for (int p = 0; p < kParts - 1; ++p) {
        const float* other = sm.red + (p * (kShrinkWarps / kParts) + half) * kWarpFloats;
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
          if (r < a.R && j < n) out[static_cast<long long>(order[j]) * a.R + r] = acc[c][i][e];
        }
    }
    __syncthreads();
  }
}

template <int RC>
__global__ void __launch_bounds__(kShrinkThreads, 2) lora_shrink_kernel(const LoraArgs a) {
  __shared__ __align__(16) ShrinkSmem sm;
  // The next kernel starts only when every CTA has passed this wait, so it may read the call's
  // inputs without waiting for this grid.
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tile = blockIdx.z, split = blockIdx.y;
  make_plan(a, sm, tile);
  if (blockIdx.x == 0 && split == 0) {
    int32_t* plan = a.plan + static_cast<long long>(tile) * kLoraPlanInts;
    if (threadIdx.x == 0) plan[0] = sm.slots;
    if (threadIdx.x < kLoraTileRows) {
      if (threadIdx.x < sm.slots) plan[kLoraPlanList + threadIdx.x] = sm.list[threadIdx.x];
      plan[kLoraPlanSlot + threadIdx.x] = sm.slot[threadIdx.x];
    }
  }
  // this CTA's part of K, in steps of 32
  const int steps = (a.K + 31) / 32;
  const int k0 = static_cast<int>(static_cast<long long>(steps) * split / a.splits) * 32;
  const int k1 = min(static_cast<int>(static_cast<long long>(steps) * (split + 1) / a.splits) * 32, a.K);
  float* out = a.t + static_cast<long long>(split) * a.M * a.R;
  const int units = sm.unit_start[sm.slots];
  int s = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    while (sm.unit_start[s + 1] <= u) ++s;  // units ascend
    const int first = sm.start[s] + (u - sm.unit_start[s]) * kUnitTokens;
    const int n = min(sm.start[s + 1] - first, kUnitTokens);
    const uint16_t* rows = a.lora_a + static_cast<long long>(sm.list[s]) * a.R * a.K;
    for (int r0 = 0; r0 < a.R; r0 += 16 * RC) {
      if (n <= 8) shrink_unit<RC, 1>(a, sm, rows, sm.order + first, n, r0, k0, k1, out);
      else shrink_unit<RC, 4>(a, sm, rows, sm.order + first, n, r0, k0, k1, out);
    }
  }
}

// ------------------------------------------------------------------ product with W, adapters added
constexpr int kBM = kLoraTileRows;
constexpr int kBK = 64;
constexpr int kThreads = 256;   // 4 control warps, 4 epilogue warps
constexpr int kMaxStages = 16;
constexpr int kMaxTBufs = 8;
constexpr int kMaxBlockN = 224;
constexpr int kTCols = 32;      // TMEM columns of a T buffer: 64 values of K, four chunks of 16 ranks
constexpr int kChunks = 4;      // chunks of 16 ranks per ring stage
constexpr int kRingBytes = 196 * 1024;
constexpr int kStageTarget = 24 * 1024;  // bytes of a ring stage, where blocks are smaller
constexpr uint32_t kTmemCols = 512;
// An MMA reads 128 rows of x also where a box has fewer: behind the last stage, too, that stays
// inside the allocation (what it reads there goes to accumulator rows that are never stored).
constexpr size_t kSmem = 1024 + kRingBytes + kBM * kBK * 2 + 1024;

struct LoraBarriers {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], t_full[kMaxTBufs], t_empty[kMaxTBufs], drain;
  uint32_t tmem_base;
  int abort_flag;
  int issued;
};

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

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > timeout_ns) {
      *abort_flag = 1;
      return false;
    }
  }
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

// Element (m, n) by itself, from the operands of token m alone: for elements that an adapter of
// another token in the tile made not finite (0 times infinity).  `slot`: its place in the plan.
__device__ __noinline__ float single_element(const LoraArgs& a, const int32_t* plan, int m, int n, int slot) {
  auto dot8 = [](const uint16_t* p, const uint16_t* q, float sum) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p)), v = __ldg(reinterpret_cast<const uint4*>(q));
    const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum = fmaf(__uint_as_float(us[i] << 16), __uint_as_float(vs[i] << 16), sum);
      sum = fmaf(__uint_as_float(us[i] & 0xFFFF0000u), __uint_as_float(vs[i] & 0xFFFF0000u), sum);
    }
    return sum;
  };
  float sum = a.bias ? __uint_as_float(static_cast<uint32_t>(__ldg(a.bias + n)) << 16) : 0.0f;
  for (int k = 0; k < a.K; k += 8)
    sum = dot8(a.x + static_cast<long long>(m) * a.K + k, a.w + static_cast<long long>(n) * a.K + k, sum);
  if (slot >= 0) {
    const int id = __ldcg(plan + kLoraPlanList + slot);
    const float s = a.scale ? __ldg(a.scale + id) : 1.0f;
    const uint16_t* b = a.lora_b + (static_cast<long long>(id) * a.N + n) * a.R;
    for (int r = 0; r < a.R; ++r) {
      float t = 0.0f;
      for (int p = 0; p < a.splits; ++p) t += __ldcg(a.t + (static_cast<long long>(p) * a.M + m) * a.R + r);
      const uint32_t st = pack_bf16x2(s * t, 0.0f) << 16;  // rounded as for the tensor core
      sum = fmaf(__uint_as_float(st), __uint_as_float(static_cast<uint32_t>(__ldg(b + r)) << 16), sum);
    }
  }
  return sum;
}

// A ring stage holds `sub` blocks of 64 values of K: small tiles' blocks are a few KB, and a stage's
// way round the ring costs the same for one as for four.
__host__ __device__ constexpr int block_bytes(int box_rows, int bn) { return (box_rows + bn) * kBK * 2; }
__host__ __device__ constexpr int stage_blocks(int box_rows, int bn) {
  const int n = kStageTarget / block_bytes(box_rows, bn);
  return n >= 4 ? 4 : n >= 2 ? 2 : 1;
}
__host__ __device__ constexpr int stage_bytes(int box_rows, int bn) {
  return stage_blocks(box_rows, bn) * block_bytes(box_rows, bn);
}
__host__ __device__ constexpr int stage_count(int box_rows, int bn) {
  const int n = kRingBytes / stage_bytes(box_rows, bn);
  return n > kMaxStages ? kMaxStages : n;
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
// (from a divergent branch an MMA takes about 125 cycles to issue).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__host__ __device__ constexpr int acc_columns(int bn) { return (bn + 31) / 32 * 32; }
__host__ __device__ constexpr int t_bufs(int bn) {
  const int n = (static_cast<int>(kTmemCols) - 2 * acc_columns(bn)) / kTCols;
  return n > kMaxTBufs ? kMaxTBufs : n;
}

// RC: chunks of 16 ranks (a rank in between counts as the next size: the boxes behind R read zeros)
template <int RC>
__global__ void __launch_bounds__(kThreads, 1)
    lora_linear_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap bmap, const LoraArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LoraBarriers& sb = *reinterpret_cast<LoraBarriers*>(tiles + kRingBytes + kBM * kBK * 2);
  static_assert(sizeof(LoraBarriers) <= 1024, "barriers fit");
  volatile int* abort_flag = &sb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_total = a.tiles_m * a.tiles_n;
  const int bn = a.block_n;
  const int sub = stage_blocks(a.box_rows, bn), stages = stage_count(a.box_rows, bn);
  const int xbytes = a.box_rows * kBK * 2, bbytes = block_bytes(a.box_rows, bn), sbytes = sub * bbytes;
  const int k_blocks = (a.K + kBK - 1) / kBK, k_stages = (k_blocks + sub - 1) / sub;
  const int tbufs = t_bufs(bn);
  const uint32_t acc_stride = acc_columns(bn), t_col = 2 * acc_stride;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&sb.full[s]), 1);
      mbar_init(smem_u32(&sb.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sb.acc_full[b]), 1);
      mbar_init(smem_u32(&sb.acc_empty[b]), 4);
    }
    for (int b = 0; b < tbufs; ++b) {
      mbar_init(smem_u32(&sb.t_full[b]), 128);
      mbar_init(smem_u32(&sb.t_empty[b]), 1);
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
    tmem_alloc(smem_u32(&sb.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;
  const uint32_t ring = smem_u32(tiles);
  // Ring stages of a tile behind those of K: four chunks of 16 ranks each.  Only these, and
  // whatever is written, wait for the first kernel.
  auto adapter_stages = [&](int slots) { return (slots * RC + kChunks - 1) / kChunks; };

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    const uint64_t policy = l2_policy_evict_last();  // x is read for every column tile, W for every row block
    RingPos p;
    int issued = 0;
    bool ok = true;
    // the stage is free (all lanes agree)
    auto free_stage = [&]() {
      return p.round == 0 || wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
    };
    for (int t = blockIdx.x; t < tiles_total && ok; t += gridDim.x) {
      const int mt = t / a.tiles_n;
      const int m0 = mt * kBM, n0 = (t % a.tiles_n) * bn;
      for (int ks = 0; ks < k_stages; ++ks, p.next(stages)) {
        ok = __all_sync(0xffffffffu, free_stage());
        if (!ok) break;
        const int blocks = min(sub, k_blocks - ks * sub);
        if (elect_one()) {
          const uint32_t bar = smem_u32(&sb.full[p.stage]);
          mbar_arrive_expect_tx(bar, blocks * bbytes);
          for (int u = 0; u < blocks; ++u) {
            const uint32_t dst = ring + p.stage * sbytes + u * bbytes;
            const int x = (ks * sub + u) * kBK;
            tma_load_2d(dst, &xmap, x, m0, bar, policy);  // rows past M are zero-filled
            tma_load_2d(dst + xbytes, &wmap, x, n0, bar, policy);
          }
          sb.issued = ++issued;
        }
      }
      if (!ok) break;
      pdl_wait_primary();  // the plan
      const int32_t* plan = a.plan + static_cast<long long>(mt) * kLoraPlanInts;
      const int slots = __ldcg(plan);
      int held = 0;  // adapters of 32 slots, one per lane
      for (int e = 0; e < adapter_stages(slots); ++e, p.next(stages)) {
        const int first = e * kChunks, n = min(kChunks, slots * RC - first);
        if (first % (32 * RC) == 0) {  // entering the next 32 slots
          const int i = first / RC + lane;
          held = i < slots ? __ldcg(plan + kLoraPlanList + i) : 0;
        }
        ok = __all_sync(0xffffffffu, free_stage());
        if (!ok) break;
        int id[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) id[c] = __shfl_sync(0xffffffffu, held, (first + c) / RC % 32);
        if (elect_one()) {
          const uint32_t bar = smem_u32(&sb.full[p.stage]);
          mbar_arrive_expect_tx(bar, n * bn * 32);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < n)
              tma_load_3d(ring + p.stage * sbytes + c * bn * 32, &bmap, (first + c) % RC * 16, n0, id[c], bar, policy);
          sb.issued = ++issued;
        }
      }
    }
    if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    const uint32_t idesc = idesc_bf16_kk(kBM, bn);
    RingPos p, tb;
    int i = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles_total && ok; t += gridDim.x, ++i) {
      const int b = i & 1;
      ok = __all_sync(0xffffffffu, wait_or_abort(smem_u32(&sb.acc_empty[b]), (i >> 1) & 1, a.timeout_ns, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * acc_stride;
      for (int ks = 0; ks < k_stages; ++ks, p.next(stages)) {
        ok = __all_sync(0xffffffffu, wait_or_abort(smem_u32(&sb.full[p.stage]), p.round & 1, a.timeout_ns, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t stage = ring + p.stage * sbytes;
        const int blocks = min(sub, k_blocks - ks * sub);
        if (elect_one()) {
#pragma unroll 1
          for (int u = 0; u < blocks; ++u) {
            const uint64_t xd = sw128_kmajor(stage + u * bbytes), wd = sw128_kmajor(stage + u * bbytes + xbytes);
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) tc_mma_ss(d, xd + 2 * kk, wd + 2 * kk, idesc, 1u);
          }
          tc_commit(smem_u32(&sb.empty[p.stage]));
        }
      }
      if (!ok) break;
      pdl_wait_primary();
      const int slots = __ldcg(a.plan + static_cast<long long>(t / a.tiles_n) * kLoraPlanInts);
      for (int e = 0; e < adapter_stages(slots); ++e, p.next(stages), tb.next(tbufs)) {
        const int n = min(kChunks, slots * RC - e * kChunks);
        ok = wait_or_abort(smem_u32(&sb.t_full[tb.stage]), tb.round & 1, a.timeout_ns, abort_flag) &&
             wait_or_abort(smem_u32(&sb.full[p.stage]), p.round & 1, a.timeout_ns, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t t_addr = tmem + t_col + tb.stage * kTCols;
          const uint64_t bd = sw32_kmajor(ring + p.stage * sbytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < n) tc_mma_ts(d, t_addr + c * 8, bd + 2 * c * bn, idesc, 1u);
          tc_commit(smem_u32(&sb.t_empty[tb.stage]));
          tc_commit(smem_u32(&sb.empty[p.stage]));
        }
      }
      if (ok && elect_one()) tc_commit(smem_u32(&sb.acc_full[b]));
    }
    if (elect_one()) {
      if (!ok) raise_status(a.status, kStatusTimeout);
      // every product issued by this thread has finished before TMEM is released
      tc_commit(smem_u32(&sb.drain));
      if (!mbar_wait(smem_u32(&sb.drain), 0, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ T and epilogue
    const int q = warp & 3;  // TMEM lane quarter
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    for (int j = 0; j < 2; ++j) {  // both accumulators start from the bias of this CTA's first tiles
      const int t = blockIdx.x + j * gridDim.x;
      if (t < tiles_total) seed_bias(lane_base + j * acc_stride, a.bias, (t % a.tiles_n) * bn, a.N, bn);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sb.acc_empty[j]));
    }
    pdl_wait_primary();  // plan and t; and no output before the first kernel's end
    RingPos tb;
    int i = 0, held_mt = -1, slots = 0, my_slot = -1;
    uint32_t tp[8 * RC];  // s t of this thread's row, bf16 pairs
#pragma unroll
    for (int e = 0; e < 8 * RC; ++e) tp[e] = 0;
    for (int t = blockIdx.x; t < tiles_total; t += gridDim.x, ++i) {
      const int b = i & 1;
      const int mt = t / a.tiles_n, m0 = mt * kBM, n0 = (t % a.tiles_n) * bn;
      const int row = m0 + 32 * q + lane;
      bool ok = true;
      if (mt != held_mt) {
        held_mt = mt;
        const int32_t* plan = a.plan + static_cast<long long>(mt) * kLoraPlanInts;
        slots = __ldcg(plan);
        my_slot = __ldcg(plan + kLoraPlanSlot + 32 * q + lane);
        if (my_slot >= 0) {
          const float s = a.scale ? __ldg(a.scale + __ldcg(plan + kLoraPlanList + my_slot)) : 1.0f;
          const float* src = a.t + static_cast<long long>(row) * a.R;
          const long long part = static_cast<long long>(a.M) * a.R;
#pragma unroll
          for (int c = 0; c < 4 * RC; ++c) {  // four ranks at a time (R is a multiple of 8)
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (4 * c < a.R) {
              for (int p = 0; p < a.splits; ++p) {
                const float4 u = __ldcg(reinterpret_cast<const float4*>(src + p * part + 4 * c));
                v.x += u.x;
                v.y += u.y;
                v.z += u.z;
                v.w += u.w;
              }
            }
            tp[2 * c] = pack_bf16x2(s * v.x, s * v.y);
            tp[2 * c + 1] = pack_bf16x2(s * v.z, s * v.w);
          }
        }
      }
      for (int e = 0; e < adapter_stages(slots); ++e, tb.next(tbufs)) {
        if (tb.round != 0 &&
            !wait_or_abort(smem_u32(&sb.t_empty[tb.stage]), (tb.round - 1) & 1, a.timeout_ns, abort_flag)) {
          ok = false;
          break;
        }
        __syncwarp();
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
        mbar_arrive(smem_u32(&sb.t_full[tb.stage]));
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) ok = wait_or_abort(smem_u32(&sb.acc_full[b]), (i >> 1) & 1, a.timeout_ns, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = lane_base + b * acc_stride;
      if (m0 + 32 * q < a.M) {  // some row of this warp exists
        uint16_t* orow = a.out + static_cast<long long>(row) * a.N;
#pragma unroll 1
        for (int c = 0; c < bn; c += 16) {
          uint32_t r[16];
          tmem_ld16(acc + c, r);
          tc_wait_ld();
          float odd = 0.0f;  // NaN if some element is not finite
#pragma unroll
          for (int v = 0; v < 16; ++v) odd = fmaf(__uint_as_float(r[v]), 0.0f, odd);
          if (odd != 0.0f && slots > 0 && row < a.M) {
            const int32_t* plan = a.plan + static_cast<long long>(mt) * kLoraPlanInts;
#pragma unroll
            for (int v = 0; v < 16; ++v)
              if (n0 + c + v < a.N && !(fabsf(__uint_as_float(r[v])) <= 3.402823466e38f))
                r[v] = __float_as_uint(single_element(a, plan, row, n0 + c + v, my_slot));
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int n = n0 + c + 8 * v;
            if (row < a.M && n < a.N)
              *reinterpret_cast<uint4*>(orow + n) =
                  make_uint4(pack_bf16x2(__uint_as_float(r[8 * v]), __uint_as_float(r[8 * v + 1])),
                             pack_bf16x2(__uint_as_float(r[8 * v + 2]), __uint_as_float(r[8 * v + 3])),
                             pack_bf16x2(__uint_as_float(r[8 * v + 4]), __uint_as_float(r[8 * v + 5])),
                             pack_bf16x2(__uint_as_float(r[8 * v + 6]), __uint_as_float(r[8 * v + 7])));
          }
        }
      }
      const int t2 = t + 2 * gridDim.x;  // this buffer's next tile starts from its bias
      if (t2 < tiles_total) seed_bias(acc, a.bias, (t2 % a.tiles_n) * bn, a.N, bn);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sb.acc_empty[b]));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    // copies still in flight land before the shared memory is released
    const int issued = sb.issued;
    for (int s = 0; s < stages && s < issued; ++s) {
      const int last = issued - 1 - ((issued - 1 - s) % stages);
      if (!mbar_wait(smem_u32(&sb.full[s]), (last / stages) & 1, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int RC>
cudaError_t launch_lora_t(const CUtensorMap& xmap, const CUtensorMap& wmap, const CUtensorMap& bmap, const LoraArgs& a,
                          int sms, cudaStream_t stream) {
  // the shared-memory opt-in, once per device (host threads may race here: atomic flags)
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(lora_linear_kernel<RC>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // units of a tile side by side: about two CTAs per SM in all, no more than a tile can have
  const int most = a.M < kLoraTileRows ? a.M : kLoraTileRows;
  const long long around = 2LL * sms / (static_cast<long long>(a.tiles_m) * a.splits);
  const int side = static_cast<int>(around < 2 ? 2 : around > most ? most : around);
  cfg.gridDim = dim3(side, a.splits, a.tiles_m);
  cfg.blockDim = dim3(kShrinkThreads, 1, 1);
  e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel<(RC > 4 ? 4 : RC)>, a);
  if (e != cudaSuccess) return e;
  const int total = a.tiles_m * a.tiles_n;
  cfg.gridDim = dim3(total < sms ? total : sms, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  e = cudaLaunchKernelEx(&cfg, lora_linear_kernel<RC>, xmap, wmap, bmap, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

int lora_splits(int m, int k) {
  const int tiles = (m + kLoraTileRows - 1) / kLoraTileRows;
  const int want = tiles <= 16 ? 4 : 2;
  const int steps = (k + 255) / 256;  // a step of K for each of the eight warps
  return want < steps ? want : steps;
}

int lora_tile_n(int m, int n, int k, int sms) {
  // the width with the least rounds x (columns + what a tile costs beside its columns)
  const long long tiles_m = (static_cast<long long>(m) + kBM - 1) / kBM;
  int best = kMaxBlockN;
  long long best_cost = -1;
  for (int bn = kMaxBlockN; bn >= 16; bn -= 16) {
    const long long tiles = tiles_m * ((n + bn - 1) / bn);
    const long long cost = ((tiles + sms - 1) / sms) * (bn + 48);
    if (best_cost < 0 || cost < best_cost) {
      best = bn;
      best_cost = cost;
    }
  }
  return best;
}

cudaError_t launch_lora(const CUtensorMap& xmap, const CUtensorMap& wmap, const CUtensorMap& bmap, const LoraArgs& a,
                        int sms, cudaStream_t stream) {
  if (a.R <= 16) return launch_lora_t<1>(xmap, wmap, bmap, a, sms, stream);
  if (a.R <= 32) return launch_lora_t<2>(xmap, wmap, bmap, a, sms, stream);
  if (a.R <= 64) return launch_lora_t<4>(xmap, wmap, bmap, a, sms, stream);
  return launch_lora_t<8>(xmap, wmap, bmap, a, sms, stream);
}

}  // namespace sa
