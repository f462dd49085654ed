// Attention of a decode batch over the pages that its sequences share, once for all of them.
//
// The sequences of a group begin with the same prompt, so the first pages of their page tables
// are the same.  Softmax attention splits over disjoint sets of keys (page "GPT-OSS on day 0",
// section "Kernels for GPT-OSS / Sink Attention": blocks along the sequence, the sink in one of
// them): with o_s, lse_s the attention over the shared keys and o_r, lse_r over the sequence's
// own keys and its sink,
//
//     lse = ln(e^lse_s + e^lse_r),  out = e^(lse_s - lse) o_s + e^(lse_r - lse) o_r.
//
// This kernel computes (o_s, lse_s), in slots along the keys; the decode kernel (decode.cu) does
// the own parts and the merge kernel (merge.cu) adds everything up.  Sequence by sequence a page
// of the prompt is read once per sequence; here the new tokens of a group's sequences stand
// together as the rows of one product (row r of KV head h: sequence r / G of the group, query head
// h G + r % G), so a shared page is read once per 256 rows and the products run on tcgen05 tiles
// of 128 rows.
//
// One CTA per (slot, KV head, pair of row tiles), 12 warps:
//   warp 0        pages by TMA, one per lane, into a ring of four stages of 128 keys
//   warps 1, 2    one elected thread each issues a row tile's products: S = Q K^T (M = 128,
//                 N = 128, K = 64) and O += P V with P from TMEM (M = 128, N = 64, K = 128)
//   warps 4..11   four warps per row tile, a thread per row: it copies its row of Q into shared
//                 memory (any G: rows of neighbouring heads and sequences fill the tiles without
//                 gaps), then for each tile of keys the running maximum and sum and P in bf16
//                 (relative error 2^-9 per weight, as in the other attention kernels; the
//                 sum takes the weights before that rounding); warps without rows only keep step
// O is rescaled only when the maximum grows by more than 2^8 (O / d does not change).
// A slot without keys, or of a group that shares nothing, writes zeros and lse = -inf.
#include <atomic>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "shared_args.h"

namespace sa {
namespace {

constexpr int kBlockQ = 128;
constexpr int kBlockK = 128;
constexpr int kPagesPerTile = kBlockK / kPageSize;
constexpr int kStages = 4;
constexpr int kThreads = 384;
constexpr int kTileBytes = kBlockQ * kHeadDim * 2;  // 16 KiB
constexpr uint32_t kColS = 0, kColO = 256, kColP = 384, kTmemCols = 512;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr unsigned long long kDrainTimeoutNs = 2000000000ull;

struct __align__(1024) SharedSmem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint64_t q_ready[2];         // the row tile's Q is in shared memory        (128 arrivals)
  uint64_t kv_full[kStages];   // K and V of a tile of keys landed            (TMA tx)
  uint64_t kv_empty[kStages];  // every row tile's products on it are done    (1 commit per row tile)
  uint64_t s_full[2];          // S is in TMEM                                (tcgen05.commit)
  uint64_t s_free[2];          // the softmax warps have read S               (128 arrivals)
  uint64_t p_full[2];          // P is written and O rescaled                 (128 arrivals)
  uint64_t pv_done[2];         // O += P V is done                            (tcgen05.commit)
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int issued_kv;
  int found;                   // group of this CTA, -1: none
  int first_tile;              // row tile pairs before that group
  int warp_sum[kThreads / 32];
};

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(1024 >> 4) << 16;  // leading byte offset (unused)
  d |= static_cast<uint64_t>(1024 >> 4) << 32;  // stride byte offset: next 8-row group
  d |= 1ull << 46;                               // descriptor version for tcgen05
  d |= 2ull << 61;                               // 128-byte swizzle
  return d;
}
// kind::f16, bf16 operands, fp32 accumulator, M x N
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
constexpr uint32_t kIdescS = idesc_bf16(128, 128, false);
constexpr uint32_t kIdescPV = idesc_bf16(128, 64, true);

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Bounded wait that also gives up as soon as another role has aborted.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > timeout_ns) {
      *abort_flag = 1;
      return false;
    }
  }
}

// Sequences and shared pages of group g; no rows when they break the declared bounds.
__device__ __forceinline__ bool group_bounds(const SharedArgs& a, int g, int& first, int& count, int& pages) {
  first = __ldg(a.plan.group_offsets + g);
  const int end = __ldg(a.plan.group_offsets + g + 1);
  pages = __ldg(a.plan.shared_pages + g);
  const bool good = first >= 0 && end >= first && end <= a.batch && pages >= 0 && pages <= a.plan.max_shared_pages &&
                    (g > 0 || first == 0) && (g + 1 < a.plan.num_groups || end == a.batch);
  count = good ? end - first : 0;
  return good;
}

// Pairs of row tiles of a group of `count` sequences.
__device__ __forceinline__ int row_tile_pairs(const SharedArgs& a, int count) {
  return (count * a.group + 2 * kBlockQ - 1) / (2 * kBlockQ);
}

// Finds the group whose row tiles contain pair `pair` (sm.found, sm.first_tile), by prefix sums
// over kThreads groups at a time.  All threads; leaves sm.found = -1 behind the last pair.
__device__ __noinline__ void find_group(const SharedArgs& a, SharedSmem& sm, int pair) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool reporter = pair == 0 && blockIdx.x == 0 && blockIdx.y == 0;  // looks at every group
  int before = 0;
  for (int g0 = 0; g0 < a.plan.num_groups; g0 += kThreads) {
    const int g = g0 + static_cast<int>(threadIdx.x);
    int n = 0;
    if (g < a.plan.num_groups) {
      int first, count, pages;
      if (!group_bounds(a, g, first, count, pages) && reporter) raise_status(a.status, kStatusBadLen);
      n = row_tile_pairs(a, count);
    }
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    __syncthreads();  // the last round's sums have been read
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    int total = 0, mine = before;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) mine += sm.warp_sum[w];
      total += sm.warp_sum[w];
    }
    const int start = mine + incl - n;
    if (n > 0 && pair >= start && pair < start + n) {
      sm.found = g;
      sm.first_tile = start;
    }
    before += total;
    if (pair < before && !reporter) break;  // the same for every thread
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const SharedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  SharedSmem& sm = *reinterpret_cast<SharedSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, kvh = blockIdx.y, pair = blockIdx.z;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    sm.found = -1;
  }
  // Launched with programmatic stream serialisation.  Every CTA lets the next kernel start only
  // after its own wait, so that kernel (the own parts) may read the call's inputs without waiting
  // for this one: whatever ran before this grid has completed by then.
  pdl_wait_primary();
  pdl_launch_dependents();

  __syncthreads();
  find_group(a, sm, pair);
  __syncthreads();
  const int g = sm.found;
  if (g < 0) return;  // uniform: no such row tile
  int first_seq, n_seq, n_pages;
  group_bounds(a, g, first_seq, n_seq, n_pages);
  const int row0 = (pair - sm.first_tile) * 2 * kBlockQ;  // first row within the group
  const int rows = min(n_seq * a.group - row0, 2 * kBlockQ);
  const int ntiles = rows > kBlockQ ? 2 : 1;
  // this slot's tiles of keys: an even share of the group's
  const int all_tiles = (n_pages + kPagesPerTile - 1) / kPagesPerTile;
  const int splits = a.plan.shared_splits;
  const int tile0 = static_cast<int>(static_cast<long long>(all_tiles) * split / splits);
  const int n_kv = static_cast<int>(static_cast<long long>(all_tiles) * (split + 1) / splits) - tile0;
  const int n_keys = n_pages * kPageSize;
  const int slots = splits + a.plan.own_splits;
  // where row r of this CTA goes: its sequence and query head
  auto row_index = [&](int r, int& seq, int& head) {
    const int gr = row0 + r;
    seq = first_seq + gr / a.group;
    head = kvh * a.group + gr % a.group;
  };

  if (n_kv == 0) {  // uniform
    for (int i = threadIdx.x; i < rows * (kHeadDim / 4); i += kThreads) {
      int seq, head;
      row_index(i / (kHeadDim / 4), seq, head);
      const size_t out = (static_cast<size_t>(seq) * slots + split) * a.hq + head;
      reinterpret_cast<float4*>(a.partial_o)[out * (kHeadDim / 4) + i % (kHeadDim / 4)] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i % (kHeadDim / 4) == 0) a.partial_lse[out] = kNegInf;
    }
    return;
  }

  volatile int* abort_flag = &sm.abort_flag;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&sm.q_ready[t]), 128);
      mbar_init(smem_u32(&sm.s_full[t]), 1);
      mbar_init(smem_u32(&sm.s_free[t]), 128);
      mbar_init(smem_u32(&sm.p_full[t]), 128);
      mbar_init(smem_u32(&sm.pv_done[t]), 1);
      mbar_init(smem_u32(&sm.drain[t]), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm.kv_full[s]), 1);
      mbar_init(smem_u32(&sm.kv_empty[s]), ntiles);
    }
    sm.abort_flag = 0;
    sm.issued_kv = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  auto tmem_base = [&]() { return *reinterpret_cast<volatile const uint32_t*>(&sm.tmem_base); };

  // 128 * 56 + 256 * 224 = 384 * 168 registers (the launch's total)
  if (warp < 4) {
    regs_dec<56>();
    if (warp == 0) {
      // ------------------------------------------------------------ pages
      const uint64_t policy = l2_policy_evict_last();  // other row tiles read the same pages
      const int32_t* ptab = a.page_table + static_cast<size_t>(first_seq) * a.max_pages;
      const int no_page = a.num_pages * a.hkv * kPageSize;  // a row behind the cache: reads as zeros
      auto load_row = [&](int j) {  // first cache row of box `lane` of tile j (lanes < 8)
        const int lp = (tile0 + j) * kPagesPerTile + lane;
        if (lane >= kPagesPerTile || lp >= n_pages) return no_page;
        const int phys = __ldg(ptab + lp);
        if (phys < 0 || phys >= a.num_pages) {
          raise_status(a.status, kStatusBadPage);
          return no_page;
        }
        return (phys * a.hkv + kvh) * kPageSize;
      };
      int row = load_row(0);
      bool ok = true;
      for (int j = 0; j < n_kv; ++j) {
        const int st = j % kStages;
        const int next = j + 1 < n_kv ? load_row(j + 1) : no_page;  // in flight while tile j is issued
        if (j >= kStages) {
          int r = 1;
          if (lane == 0) r = wait_bar(smem_u32(&sm.kv_empty[st]), ((j / kStages) - 1) & 1, a.timeout_ns, abort_flag) ? 1 : 0;
          if (!__shfl_sync(0xffffffffu, r, 0)) {
            ok = false;
            break;
          }
        }
        const uint32_t bar = smem_u32(&sm.kv_full[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kTileBytes);
        __syncwarp();
        if (lane < kPagesPerTile) {
          tma_load_2d(smem_u32(sm.k[st]) + lane * kPageSize * 128, &kmap, 0, row, bar, policy);
          tma_load_2d(smem_u32(sm.v[st]) + lane * kPageSize * 128, &vmap, 0, row, bar, policy);
        }
        if (lane == 0) sm.issued_kv = j + 1;
        row = next;
      }
      if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
    } else if (warp == 1 || warp == 2) {
      // ------------------------------------------------------------ products
      const int t = warp - 1;
      if (t < ntiles) {
        const uint32_t tmem = tmem_base();
        const uint32_t d_s = tmem + kColS + t * 128, d_o = tmem + kColO + t * 64, a_p = tmem + kColP + t * 64;
        auto wait = [&](uint64_t& bar, int parity) {
          return __all_sync(0xffffffffu, wait_bar(smem_u32(&bar), parity & 1, a.timeout_ns, abort_flag)) != 0;
        };
        bool ok = wait(sm.q_ready[t], 0);
        const uint64_t qd = sw128_desc(smem_u32(sm.q[t]));
        auto s_step = [&](int j) {  // S(j) = Q K_j^T
          ok = wait(sm.kv_full[j % kStages], j / kStages);
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t kd = sw128_desc(smem_u32(sm.k[j % kStages]));
#pragma unroll
            for (int kk = 0; kk < kHeadDim / 16; ++kk) tc_mma_ss(d_s, qd + 2 * kk, kd + 2 * kk, kIdescS, kk > 0);
            tc_commit(smem_u32(&sm.s_full[t]));
          }
        };
        auto pv_step = [&](int j) {  // O += P(j) V_j
          ok = wait(sm.p_full[t], j);
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vd = sw128_desc(smem_u32(sm.v[j % kStages]));
#pragma unroll
            for (int kk = 0; kk < kBlockK / 16; ++kk)
              tc_mma_ts(d_o, a_p + kk * 8, vd + kk * (16 * 128 / 16), kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
            tc_commit(smem_u32(&sm.pv_done[t]));
            tc_commit(smem_u32(&sm.kv_empty[j % kStages]));
          }
        };
        if (ok) s_step(0);
        for (int j = 0; j < n_kv && ok; ++j) {
          if (j >= 1) pv_step(j - 1);
          if (ok && j + 1 < n_kv) {
            ok = wait(sm.s_free[t], j);
            if (ok) s_step(j + 1);
          }
        }
        if (ok) pv_step(n_kv - 1);
        if (elect_one()) {
          if (!ok) raise_status(a.status, kStatusTimeout);
          // whatever happened, every product issued here is done before TMEM is released
          tc_commit(smem_u32(&sm.drain[t]));
          mbar_wait(smem_u32(&sm.drain[t]), 0, kDrainTimeoutNs);
        }
        __syncwarp();
      }
    }
  } else {
    regs_inc<224>();
    // -------------------------------------------------------------- softmax
    const int t = (warp - 4) >> 2;  // row tile of this warpgroup
    const int qw = warp & 3;        // TMEM lane quarter
    const int r = qw * 32 + lane;   // row within the tile
    if (t < ntiles) {
      const uint32_t lane_base = tmem_base() + (static_cast<uint32_t>(qw * 32) << 16);
      const uint32_t s_col = lane_base + kColS + t * 128;
      const uint32_t o_col = lane_base + kColO + t * 64;
      const uint32_t p_col = lane_base + kColP + t * 64;
      const bool live = t * kBlockQ + r < rows;
      const bool warp_live = t * kBlockQ + qw * 32 < rows;
      int seq, head;
      row_index(live ? t * kBlockQ + r : 0, seq, head);
      {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<size_t>(seq) * a.hq + head) * kHeadDim);
        uint4 x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        uint8_t* dst = sm.q[t] + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(dst + ((c ^ (r & 7)) << 4)) = x[c];
        fence_proxy_async_smem();  // the rows are read by the tensor core (async proxy)
        mbar_arrive(smem_u32(&sm.q_ready[t]));
      }
      const uint64_t scale2 = f2(a.scale_log2, a.scale_log2);
      float m = kNegInf, d = 0.0f;  // running maximum (log2 units) and sum
      bool ok = true;
      for (int j = 0; j < n_kv; ++j) {
        if (!wait_bar(smem_u32(&sm.s_full[t]), j & 1, a.timeout_ns, abort_flag)) {
          ok = false;
          break;
        }
        if (!warp_live) {  // rows that nothing reads: keep step with the others, phase by phase
          mbar_arrive(smem_u32(&sm.s_free[t]));
          if (j > 0 && !wait_bar(smem_u32(&sm.pv_done[t]), (j - 1) & 1, a.timeout_ns, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive(smem_u32(&sm.p_full[t]));
          continue;
        }
        tc_fence_after();
        uint32_t sr[128];
        float pm0, pm1, pm2, pm3;  // maxima of the four slices of 32 columns
        tmem_ld32_max_at<0>(s_col + 0, sr, pm0);
        tmem_ld32_max_at<32>(s_col + 32, sr, pm1);
        tmem_ld32_max_at<64>(s_col + 64, sr, pm2);
        tmem_ld32_max_at<96>(s_col + 96, sr, pm3);
        tc_wait_ld();
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.s_free[t]));
        float s[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(sr[c]);
        const int left = n_keys - (tile0 + j) * kBlockK;  // keys from this tile's first on
        float mraw = fmax3(pm0, pm1, fmaxf(pm2, pm3));
        if (left < kBlockK) {  // the prompt ends inside this tile: its missing pages read as zeros
          mraw = kNegInf;
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            if (c >= left) s[c] = kNegInf;
            mraw = fmaxf(mraw, s[c]);
          }
        }
        const float mx = mraw * a.scale_log2;
        const bool grow = mx > m + kRescaleThreshold;
        float factor = 1.0f;
        if (grow) {
          factor = (m == kNegInf) ? 0.0f : ex2(m - mx);
          m = mx;
          d *= factor;
        }
        const float mu = (m == kNegInf) ? 0.0f : m;
        const uint64_t negm2 = f2(-mu, -mu);
        // p = 2^(s * scale - m), packed two per instruction; four partial row sums
        uint32_t pk[64];
        uint64_t acc0 = 0, acc1 = 0, acc2 = 0, acc3 = 0;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float x0, x1;
          f2_split(f2_fma(f2(s[2 * c], s[2 * c + 1]), scale2, negm2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          const uint64_t pp = f2(p0, p1);
          if ((c & 3) == 0) acc0 = f2_add(acc0, pp);
          if ((c & 3) == 1) acc1 = f2_add(acc1, pp);
          if ((c & 3) == 2) acc2 = f2_add(acc2, pp);
          if ((c & 3) == 3) acc3 = f2_add(acc3, pp);
          pk[c] = pack_bf16x2(p0, p1);
        }
        float r0, r1;
        f2_split(f2_add(f2_add(acc0, acc1), f2_add(acc2, acc3)), r0, r1);
        d += r0 + r1;
        // P and O are in use by the previous product until it is done
        if (j > 0 && !wait_bar(smem_u32(&sm.pv_done[t]), (j - 1) & 1, a.timeout_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          const uint64_t f22 = f2(factor, factor);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t u[32];
            tmem_ld32(o_col + c * 32, u);
            tc_wait_ld();
            uint32_t lo[16], hi[16];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float a0, a1;
              f2_split(f2_mul(f2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])), f22), a0, a1);
              lo[e] = __float_as_uint(a0);
              lo[e + 1] = __float_as_uint(a1);
              f2_split(f2_mul(f2(__uint_as_float(u[16 + e]), __uint_as_float(u[17 + e])), f22), a0, a1);
              hi[e] = __float_as_uint(a0);
              hi[e + 1] = __float_as_uint(a1);
            }
            tmem_st16(o_col + c * 32, lo);
            tmem_st16(o_col + c * 32 + 16, hi);
          }
        }
        tmem_st16_at<0>(p_col + 0, pk);
        tmem_st16_at<16>(p_col + 16, pk);
        tmem_st16_at<32>(p_col + 32, pk);
        tmem_st16_at<48>(p_col + 48, pk);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.p_full[t]));
      }
      if (ok) ok = wait_bar(smem_u32(&sm.pv_done[t]), (n_kv - 1) & 1, a.timeout_ns, abort_flag);
      if (ok && warp_live) {
        tc_fence_after();
        uint32_t ou[2][32];
        tmem_ld32(o_col, ou[0]);
        tmem_ld32(o_col + 32, ou[1]);
        tc_wait_ld();
        if (live) {
          const float inv = d > 0.0f ? 1.0f / d : 0.0f;
          const size_t out = (static_cast<size_t>(seq) * slots + split) * a.hq + head;
          float4* o = reinterpret_cast<float4*>(a.partial_o + out * kHeadDim);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint32_t* u = ou[c >> 3] + 4 * (c & 7);
            o[c] = make_float4(__uint_as_float(u[0]) * inv, __uint_as_float(u[1]) * inv, __uint_as_float(u[2]) * inv,
                               __uint_as_float(u[3]) * inv);
          }
          a.partial_lse[out] = d > 0.0f ? (m + lg2(d)) * kLn2 : kNegInf;
        }
      }
      if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag && threadIdx.x == 0) {
    // copies that nobody consumed land before the shared memory is released
    const int issued = sm.issued_kv;
    for (int j = max(0, issued - kStages); j < issued; ++j)
      mbar_wait(smem_u32(&sm.kv_full[j % kStages]), (j / kStages) & 1, kDrainTimeoutNs);
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem_base(), kTmemCols);
}

}  // namespace

long long shared_row_tiles(int batch, int num_groups, int group) {
  const long long rows = static_cast<long long>(batch) * group, block = 2 * kBlockQ;
  const long long groups = num_groups < batch ? num_groups : batch;  // the ones that can have rows
  return (rows + groups * (block - 1)) / block;
}

cudaError_t launch_shared(const CUtensorMap& kmap, const CUtensorMap& vmap, const SharedArgs& a, cudaStream_t stream) {
  const size_t smem = sizeof(SharedSmem) + 1024;
  // the shared-memory opt-in, once per device (host threads may race here: atomic flags, and
  // setting the attribute twice is harmless)
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(shared_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.plan.shared_splits, a.hkv, static_cast<unsigned>(shared_row_tiles(a.batch, a.plan.num_groups, a.group)));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, shared_prefix_kernel, kmap, vmap, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace sa
