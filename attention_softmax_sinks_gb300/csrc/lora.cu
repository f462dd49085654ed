// Linear layer with the low-rank adapters of many requests beside it: for token m with adapter a,
//
//     out[m] = x[m] W^T + b + s_a (x[m] A_a^T) B_a^T        A_a [R, K], B_a [N, R]
//
// (page "GPT-OSS on day 0": the projections carry bias terms; the adapters are what requests of
// one server differ in).  Two kernels, in one call:
//
// 1. lora_shrink_kernel: t[m] = s_a x[m] A_a^T, on tcgen05.  A CTA takes 128 tokens, a part of K
//    and up to 256 columns: the A_a of as many of the tile's distinct adapters as fit, one behind
//    the other (found by a bit per adapter and population counts).  Every token meets every one
//    of them, and its row keeps its own adapter's R columns.  That is wasted work for a tile of
//    many adapters, but the tile is short of nothing else: what bounds it is the operands' way
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
//    not finite is computed once more by itself, from its own operands only.
//    Many tokens: pairs of CTAs (cta_group::2, 256 tokens), which stage half of W's columns each.
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

// ------------------------------------------------------------------ first product
constexpr int kShrinkThreads = 256;  // loads, products, plan; warps 4..7 epilogue
constexpr int kShrinkCols = 256;     // columns of an accumulator
constexpr int kShrinkStages = 3;
constexpr int kShrinkStageBytes = (kBM + kShrinkCols) * kBK * 2;
// rows that this CTA adds up: from each part of K, together 128 rows of up to 128 ranks
constexpr int kShrinkRecvBytes = kBM * kLoraMaxRank * 4;
constexpr size_t kShrinkSmem = 1024 + kShrinkStages * kShrinkStageBytes + kShrinkRecvBytes + 4096;

struct ShrinkShared {
  uint64_t full[kShrinkStages], empty[kShrinkStages], acc_full, acc_empty, drain;
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
  ShrinkShared& sb = *reinterpret_cast<ShrinkShared*>(tiles + kShrinkStages * kShrinkStageBytes + kShrinkRecvBytes);
  volatile int* abort_flag = &sb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.z, split = blockIdx.y;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&amap);
    for (int s = 0; s < kShrinkStages; ++s) {
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
  if (static_cast<int>(blockIdx.x) >= passes) return;  // the whole cluster, before TMEM is taken
  cluster_arrive_relaxed();  // waited for before the first store into another CTA
  const int owner_rows = kBM / a.splits;  // of the tile: CTA `split` adds up [split * owner_rows, ..)
  float* recv = reinterpret_cast<float*>(tiles + kShrinkStages * kShrinkStageBytes);  // [part][row][R]
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
  cluster_wait();  // every CTA of the cluster runs

  if (warp == 0) {
    RingPos p;
    int issued = 0;
    bool ok = true;
    for (int pass = blockIdx.x; pass < passes && ok; pass += gridDim.x) {
      const int first = pass * per_pass, n = min(per_pass, slots - first);
      for (int ks = 0; ks < k_steps; ++ks, p.next(kShrinkStages)) {
        ok = p.round == 0 || wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        const uint32_t bar = smem_u32(&sb.full[p.stage]), dst = ring + p.stage * kShrinkStageBytes;
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
    for (int pass = blockIdx.x; pass < passes && ok; pass += gridDim.x, ++i) {
      const int n = min(per_pass, slots - pass * per_pass);
      const uint32_t idesc = idesc_bf16_kk(kBM, (n * a.R + 15) / 16 * 16);
      if (i > 0) ok = wait_or_abort(smem_u32(&sb.acc_empty), (i - 1) & 1, a.timeout_ns, abort_flag);
      if (!ok) break;
      tc_fence_after();
      for (int ks = 0; ks < k_steps; ++ks, p.next(kShrinkStages)) {
        ok = wait_or_abort(smem_u32(&sb.full[p.stage]), p.round & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t stage = ring + p.stage * kShrinkStageBytes;
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
    const uint32_t out = dsmem_addr(smem_u32(recv + (split * owner_rows + r % owner_rows) * a.R), r / owner_rows);
    int i = 0;
    for (int pass = blockIdx.x; pass < passes; pass += gridDim.x, ++i) {
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
            dsmem_st4(out + 4 * c, f[0], f[1], f[2], f[3]);
            dsmem_st4(out + 4 * c + 16, f[4], f[5], f[6], f[7]);
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
    for (int s = 0; s < kShrinkStages && s < sb.issued; ++s) {
      const int last = sb.issued - 1 - ((sb.issued - 1 - s) % kShrinkStages);
      if (!mbar_wait(smem_u32(&sb.full[s]), (last / kShrinkStages) & 1, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
  }
  cluster_sync();  // every part of the rows has arrived
  const int parts = a.splits;
  for (int i = threadIdx.x; i < owner_rows * (a.R / 8); i += kShrinkThreads) {
    const int r = i / (a.R / 8), c = i % (a.R / 8) * 8, s = sb.slot[split * owner_rows + r];
    if (s < 0 || s / per_pass % gridDim.x != blockIdx.x) continue;  // none, or another cluster's
    float sum[8] = {};
    for (int p = 0; p < parts; ++p) {
      const float4* v = reinterpret_cast<const float4*>(recv + (p * owner_rows + r) * a.R + c);
      const float4 v0 = v[0], v1 = v[1];
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
constexpr int kRingBytes = 196 * 1024;
constexpr int kStageTarget = 24 * 1024;  // bytes of a ring stage, where blocks are smaller
constexpr uint32_t kTmemCols = 512;
// An MMA reads 128 rows of x also where a box has fewer: behind the last stage, too, that stays
// inside the allocation (what it reads there goes to accumulator rows that are never stored).
constexpr size_t kSmem = 1024 + kRingBytes + kBM * kBK * 2 + 4096;

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

// Element (m, n) by itself, from the operands of token m alone: for elements that an adapter of
// another token in the tile made not finite (0 times infinity).
__device__ __noinline__ float single_element(const LoraArgs& a, int m, int n) {
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
  const int id = __ldg(a.adapter + m);
  if (id >= 0 && id < a.num_adapters) {
    const uint16_t* b = a.lora_b + (static_cast<long long>(id) * a.N + n) * a.R;
    for (int r = 0; r < a.R; ++r)
      sum = fmaf(__uint_as_float(static_cast<uint32_t>(__ldcg(a.t + static_cast<long long>(m) * a.R + r)) << 16),
                 __uint_as_float(static_cast<uint32_t>(__ldg(b + r)) << 16), sum);
  }
  return sum;
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
__host__ __device__ constexpr int stage_count(int box_rows, int wrows) {
  const int n = kRingBytes / stage_bytes(box_rows, wrows);
  return n > kMaxStages ? kMaxStages : n;
}
__host__ __device__ constexpr int acc_columns(int bn) { return (bn + 31) / 32 * 32; }
__host__ __device__ constexpr int t_bufs(int bn) {
  const int n = (static_cast<int>(kTmemCols) - 2 * acc_columns(bn)) / kTCols;
  return n > kMaxTBufs ? kMaxTBufs : n;
}

// RC: chunks of 16 ranks (a rank in between counts as the next size: the boxes behind R read zeros)
template <int RC, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    lora_linear_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap bmap, const LoraArgs a) {
  constexpr int kCtas = kPair ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  LoraBarriers& sb = *reinterpret_cast<LoraBarriers*>(tiles + kRingBytes + kBM * kBK * 2);
  volatile int* abort_flag = &sb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const int tiles_m = (a.tiles_m + kCtas - 1) / kCtas, tiles_total = tiles_m * a.tiles_n;
  const int t_first = blockIdx.x / kCtas, t_step = gridDim.x / kCtas;
  const int bn = a.block_n, wrows = bn / kCtas;
  const int sub = stage_blocks(a.box_rows, wrows), stages = stage_count(a.box_rows, wrows);
  const int xbytes = a.box_rows * kBK * 2, bbytes = block_bytes(a.box_rows, wrows), sbytes = sub * bbytes;
  const int k_blocks = (a.K + kBK - 1) / kBK, k_stages = (k_blocks + sub - 1) / sub;
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
            const int x = (ks * sub + u) * kBK;
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
      for (int e = 0; e < adapter_stages(slots); ++e, p.next(stages)) {
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
      for (int e = 0; e < adapter_stages(slots); ++e, p.next(stages), tb.next(tbufs)) {
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
          const uint4* src = reinterpret_cast<const uint4*>(a.t + static_cast<long long>(row) * a.R);
#pragma unroll
          for (int c = 0; c < 2 * RC; ++c) {  // eight ranks at a time (R is a multiple of 8)
            const uint4 v = 8 * c < a.R ? __ldcg(src + c) : make_uint4(0, 0, 0, 0);
            tp[4 * c] = v.x;
            tp[4 * c + 1] = v.y;
            tp[4 * c + 2] = v.z;
            tp[4 * c + 3] = v.w;
          }
        }
      }
      for (int e = 0; e < adapter_stages(slots); ++e, tb.next(tbufs)) {
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
      if (t < tiles_total) seed_bias(lane_base + j * acc_stride, a.bias, (t % a.tiles_n) * bn, a.N, bn);
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
          if (odd != 0.0f && row < a.M) {
#pragma unroll
            for (int v = 0; v < 16; ++v)
              if (n0 + c + v < a.N && !(fabsf(__uint_as_float(r[v])) <= 3.402823466e38f))
                r[v] = __float_as_uint(single_element(a, row, n0 + c + v));
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
      const int t2 = t + 2 * t_step;  // this buffer's next tile starts from its bias
      if (t2 < tiles_total) seed_bias(acc, a.bias, (t2 % a.tiles_n) * bn, a.N, bn);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pair_arrive<kPair>(acc_empty0 + 8 * b);
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

template <int RC, bool kPair>
cudaError_t launch_lora_t(const LoraMaps& m, const LoraArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  cudaError_t e = opt_in(lora_linear_kernel<RC, kPair>, kSmem, done);
  if (e != cudaSuccess) return e;
  constexpr int kCtas = kPair ? 2 : 1;
  const int total = (a.tiles_m + kCtas - 1) / kCtas * a.tiles_n, slots = sms / kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((total < slots ? total : slots) * kCtas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, lora_linear_kernel<RC, kPair>, m.x, m.w, m.b, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int RC>
cudaError_t launch_lora_r(const LoraMaps& m, const LoraArgs& a, int sms, cudaStream_t stream) {
  return a.plan_tiles == 2 ? launch_lora_t<RC, true>(m, a, sms, stream) : launch_lora_t<RC, false>(m, a, sms, stream);
}

}  // namespace

void lora_plan(LoraArgs& a, int sms) {
  a.tiles_m = (a.M + kBM - 1) / kBM;
  // the width with the least rounds x (columns + what a tile costs beside its columns)
  auto cost_of = [&](int bn, int ctas) {
    const long long tiles = static_cast<long long>((a.tiles_m + ctas - 1) / ctas) * ((a.N + bn - 1) / bn);
    return (tiles + sms / ctas - 1) / (sms / ctas) * (bn + 48);
  };
  long long best = -1;
  for (int bn = kMaxBlockN; bn >= 16; bn -= 16) {
    const long long cost = cost_of(bn, 1);
    if (best < 0 || cost < best) {
      best = cost;
      a.block_n = bn;
    }
  }
  // Pairs of CTAs stage half as much of W for the same product; where there are tiles for all pairs
  // and the last round of tiles is not much emptier for them
  a.plan_tiles = 1;
  if (a.tiles_m >= 2) {
    int pair_n = kMaxBlockN;
    long long pair_cost = -1;
    for (int bn = kMaxBlockN; bn >= 128; bn -= 32) {
      const long long cost = cost_of(bn, 2);
      if (pair_cost < 0 || cost < pair_cost) {
        pair_cost = cost;
        pair_n = bn;
      }
    }
    const long long pair_tiles = static_cast<long long>((a.tiles_m + 1) / 2) * ((a.N + pair_n - 1) / pair_n);
    if (pair_tiles >= sms / 2 && 10 * pair_cost <= 11 * best) {
      a.plan_tiles = 2;
      a.block_n = pair_n;
    }
  }
  a.tiles_n = (a.N + a.block_n - 1) / a.block_n;
  a.box_rows = a.M < kBM ? (a.M + 7) / 8 * 8 : kBM;
  // parts of K for the first product: a CTA per SM, up to 8 parts of at least two steps
  a.splits = 1;
  while (a.splits < 8 && 2 * a.splits * a.tiles_m <= sms && 4 * a.splits <= (a.K + kBK - 1) / kBK) a.splits *= 2;
}

cudaError_t launch_lora(const LoraMaps& m, const LoraArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  cudaError_t e = opt_in(lora_shrink_kernel, kShrinkSmem, done);
  if (e != cudaSuccess) return e;
  // CTAs side by side: as many passes of 256 columns as a tile can have
  int most = a.M < kBM ? a.M : kBM;
  if (most > a.num_adapters) most = a.num_adapters;
  const int per_pass = kShrinkCols / a.R, passes = (most + per_pass - 1) / per_pass;
  const long long room = 2LL * sms / (static_cast<long long>(a.tiles_m) * a.splits);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = a.splits;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(room < 1 ? 1 : room < passes ? room : passes), a.splits, a.tiles_m);
  cfg.blockDim = dim3(kShrinkThreads, 1, 1);
  cfg.dynamicSmemBytes = kShrinkSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel, m.x, m.a, a);
  if (e != cudaSuccess) return e;
  if (a.R <= 16) return launch_lora_r<1>(m, a, sms, stream);
  if (a.R <= 32) return launch_lora_r<2>(m, a, sms, stream);
  if (a.R <= 64) return launch_lora_r<4>(m, a, sms, stream);
  return launch_lora_r<8>(m, a, sms, stream);
}

}  // namespace sa
