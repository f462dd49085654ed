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
// the own parts and shared_merge_kernel adds everything up.  Sequence by sequence a page
// of the prompt is read once per sequence; here the new tokens of a group's sequences stand
// together as the rows of one product (row r of KV head h: sequence r / G of the group, query head
// h G + r % G), so a shared page is read once per 256 rows and the products run on tcgen05 tiles
// of 128 rows.
//
// Work is counted in tiles of 128 keys of a unit (KV head, pair of row tiles), unit behind unit, and
// dealt out in equal runs: one run per CTA, of a grid that leaves SMs to the own parts, which are
// bound by memory where this is bound by arithmetic.  A run covers the end of one unit and the
// beginning of the next, or several; the part of a unit in a run is a slot of its results.  A CTA
// has 12 warps:
//   warp 0        pages by TMA, one per lane, into a ring of four stages of 128 keys
//   warp 3        walks along the run and puts its parts into a ring of four for the other warps
//   warps 1, 2    one elected thread each issues a row tile's products: S = Q K^T (M = 128,
//                 N = 128, K = 64) and O += P V with P from TMEM (M = 128, N = 64, K = 128)
//   warps 4..11   four warps per row tile, a thread per row: it copies its row of Q into shared
//                 memory (any G: rows of neighbouring heads and sequences fill the tiles without
//                 gaps), then for each tile of keys the running maximum and sum and P in bf16
//                 (relative error 2^-8 at most per weight, as in the other attention kernels; the
//                 sum takes the weights before that rounding); warps without rows only keep step
// O is rescaled only when the maximum grows by more than 2^8 (O / d does not change).
// A unit of no more than 128 rows has one row tile, whose steps (product, softmax, product) would
// follow one another: there the two sets of warps take its tiles of keys in turn, as two slots.
// Slots that a unit does not use get lse = -inf and are not read by the merge; those of sequences
// that share nothing are marked by the own parts' kernel.
//
// What bounds it: the chain of a tile's steps (scores, maximum, exponentials, P, product), one row tile's
// beside the other's.  A tile of 128 keys and two row tiles takes 1.28 us of an SM, 0.68 of which the
// tensor core needs; while an SM works, issue slots are taken 40% of the time, the exponentials' pipe
// 39%, the tensor core 39%: none is near its limit (64 sequences of 64/8 heads that share 32768 tokens,
// with 500 of their own each: 57.5 us, of which 46 are this kernel on 128 SMs beside the own parts on
// the others; each sequence by itself would read 64 times as much, 4.3 GB).
// A batch whose own parts are longer than its prompts is bound by memory: 512 sequences in 8 groups,
// 1.1 GB, take 203 us, 5.5 TB/s.  Few short prompts are bound by latency: 4 sequences that share 2048
// tokens 11.9 us, of which 2.6 go by before the first part begins and 2.5 in the merge; such batches
// are left to one launch that reads every sequence's pages (8.1 us).
// Kept out, as slower: units of up to 64 rows twice in a tile, each copy with half of a tile's keys
// (4 x 2048 13.1 us, 37 in 5 groups 31.5); all SMs for both kernels (37 sequences in 5 groups 33 us against 29), units dealt
// out whole (211 us against 203 for 512 sequences), every role walking along the run for itself (its
// registers spilled: a tile of keys took 1.5 us).
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

constexpr int kSegments = 4;
constexpr int kMaxChunks = 176;  // kThreads groups each: up to 65535 groups

// A place in the CTA's run.
struct Walk {
  int at, end;   // the rest of the run
  int in_group;  // work of group g before `at`
  int g, first_seq, count, pages;
};

// A unit's part of a run: rows [row0, row0 + rows) of the group that begins with sequence first_seq,
// KV head kvh, tiles of keys [tile0, tile0 + n_kv) of its n_pages pages.
struct Segment {
  int first_seq, row0, rows, n_pages, kvh, tile0, n_kv;
  int slot;   // where the results go (in turn: 2 slot and 2 slot + 1)
  int turns;  // one row tile, whose tiles of keys both sets of warps take in turn
  int last;   // the unit's last part: slots behind it stay empty
};

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
  uint64_t seg_full[kSegments];   // a part of the run is there               (1 arrival)
  uint64_t seg_empty[kSegments];  // every warp that reads it is through with it (11 arrivals)
  uint64_t stagger;            // row tile 0 has handed over a part's first P  (1 arrival)
  uint32_t tmem_base;
  int abort_flag;
  int issued_kv;
  int total;                   // tiles of keys of all units
  int units;
  int most[2];                 // of one unit: of one row tile in two slots, others
  unsigned warp_sum[kThreads / 32];
  unsigned warp_units[kThreads / 32];
  int warp_most[2][kThreads / 32];
  int chunk[kMaxChunks];       // work before each kThreads groups
  Segment seg[kSegments];      // parts of this CTA's run, in turn; n_kv = 0: its end
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

// Sequences and shared pages of group g; no rows (0, or -1 where the offsets go back) when they
// break the declared bounds.
__device__ __forceinline__ bool group_bounds(const SharedArgs& a, int g, int& first, int& count, int& pages) {
  first = __ldg(a.plan.group_offsets + g);
  const int end = __ldg(a.plan.group_offsets + g + 1);
  pages = __ldg(a.plan.shared_pages + g);
  const bool good = first >= 0 && end >= first && end <= a.batch && pages >= 0 && pages <= a.plan.max_shared_pages &&
                    (g > 0 || first == 0) && (g + 1 < a.plan.num_groups || end == a.batch);
  count = good ? end - first : end < first ? -1 : 0;
  return good;
}

// Pairs of row tiles of a group of `count` sequences, and its tiles of keys.
__device__ __forceinline__ int row_tile_pairs(const SharedArgs& a, int count) {
  return (count * a.group + 2 * kBlockQ - 1) / (2 * kBlockQ);
}
__device__ __forceinline__ int key_tiles(int pages) { return (pages + kPagesPerTile - 1) / kPagesPerTile; }

// A group's work, and its units' length: its tiles of keys, rounded up to a multiple of `each` if
// that is not 0; 0 if it shares nothing.
__device__ __forceinline__ int group_work(const SharedArgs& a, int count, int pages, int each, int& len) {
  const int tiles = count > 0 ? key_tiles(pages) : 0;
  len = each ? (tiles + each - 1) / each * each : tiles;
  return row_tile_pairs(a, count) * a.hkv * len;
}

// Sums up the groups' work, kThreads groups at a time: sm.total, sm.units, sm.most, sm.chunk.  All threads.
// Offsets that go back somewhere can count a sequence many times, each group for itself within its
// bounds.  Then there is no work: the sums, and places in them, would pass 32 bits (without, the
// limit that the call checks holds), and the batch's size would not bound the time.
__device__ __forceinline__ void sum_work(const SharedArgs& a, SharedSmem& sm, int each, bool report) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned before = 0, units = 0;
  int most[2] = {0, 0};
  bool ascend = true;
  for (int g0 = 0; g0 < a.plan.num_groups; g0 += kThreads) {
    const int g = g0 + static_cast<int>(threadIdx.x);
    unsigned n = 0, u = 0;
    int count = 0, tiles[2] = {0, 0};
    if (g < a.plan.num_groups) {
      int first, pages, len;
      if (!group_bounds(a, g, first, count, pages) && report) raise_status(a.status, kStatusBadLen);
      n = group_work(a, count, pages, each, len);
      u = n > 0 ? n / len : 0;
      const int rows = count * a.group;  // its last unit has one row tile, or two; the others two
      if ((rows - 1) % (2 * kBlockQ) < kBlockQ) tiles[0] = len;
      if (rows > kBlockQ) tiles[1] = len;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      n += __shfl_xor_sync(0xffffffffu, n, off);
      u += __shfl_xor_sync(0xffffffffu, u, off);
      tiles[0] = max(tiles[0], __shfl_xor_sync(0xffffffffu, tiles[0], off));
      tiles[1] = max(tiles[1], __shfl_xor_sync(0xffffffffu, tiles[1], off));
    }
    if (__syncthreads_or(count < 0)) ascend = false;  // (the last round's sums have been read)
    if (lane == 0) {
      sm.warp_sum[warp] = n;
      sm.warp_units[warp] = u;
      sm.warp_most[0][warp] = tiles[0];
      sm.warp_most[1][warp] = tiles[1];
    }
    __syncthreads();
    if (threadIdx.x == 0) sm.chunk[g0 / kThreads] = before;
    for (int w = 0; w < kThreads / 32; ++w) {
      before += sm.warp_sum[w];
      units += sm.warp_units[w];
      most[0] = max(most[0], sm.warp_most[0][w]);
      most[1] = max(most[1], sm.warp_most[1][w]);
    }
  }
  if (threadIdx.x == 0) {
    sm.total = ascend ? before : 0;
    sm.units = ascend ? units : 0;
    sm.most[0] = ascend ? most[0] : 0;
    sm.most[1] = ascend ? most[1] : 0;
  }
  __syncthreads();
}

// The walk stands at position `pos` of the work (below sm.total), for `quantum` of it.  The whole warp.
__device__ __forceinline__ void seek(const SharedArgs& a, SharedSmem& sm, Walk& walk, int pos, int quantum, int each) {
  const int lane = threadIdx.x & 31;
  int c = 0;
  while ((c + 1) * kThreads < a.plan.num_groups && sm.chunk[c + 1] <= pos) ++c;
  int before = sm.chunk[c];
  for (int g0 = c * kThreads; g0 < a.plan.num_groups; g0 += 32) {
    const int g = g0 + lane;
    int first = 0, count = 0, pages = 0, len;
    int n = 0;
    if (g < a.plan.num_groups) {
      group_bounds(a, g, first, count, pages);
      n = group_work(a, count, pages, each, len);
    }
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    const int start = before + incl - n;
    const unsigned here = __ballot_sync(0xffffffffu, n > 0 && pos >= start && pos < start + n);
    if (here) {
      const int l = __ffs(here) - 1;
      walk.at = pos;
      walk.end = quantum < sm.total - pos ? pos + quantum : sm.total;
      walk.in_group = pos - __shfl_sync(0xffffffffu, start, l);
      walk.g = g0 + l;
      walk.first_seq = __shfl_sync(0xffffffffu, first, l);
      walk.count = __shfl_sync(0xffffffffu, count, l);
      walk.pages = __shfl_sync(0xffffffffu, pages, l);
      return;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The walk's next part of a unit, if any.
__device__ __forceinline__ bool next_segment(const SharedArgs& a, Walk& w, Segment& s, int quantum, int each, bool turns) {
  bool found = false;
  while (!found && w.at < w.end) {
    int len;
    const int work = group_work(a, w.count, w.pages, each, len);
    if (w.in_group >= work) {  // on to the next group
      if (++w.g >= a.plan.num_groups) break;
      w.in_group = 0;
      group_bounds(a, w.g, w.first_seq, w.count, w.pages);
      continue;
    }
    const int unit = w.in_group / len, off = w.in_group % len;
    const int n = min(len - off, w.end - w.at);
    const int unit_start = w.at - off;
    s.first_seq = w.first_seq;
    s.row0 = unit / a.hkv * 2 * kBlockQ;
    s.rows = min(w.count * a.group - s.row0, 2 * kBlockQ);
    s.n_pages = w.pages;
    s.kvh = unit % a.hkv;
    s.tile0 = off;
    s.n_kv = min(n, key_tiles(w.pages) - off);  // (a unit shorter than `each` leaves the rest idle)
    s.slot = w.at / quantum - unit_start / quantum;
    s.turns = turns && s.rows <= kBlockQ;
    s.last = off + n == len;
    w.at += n;
    w.in_group += n;
    found = s.n_kv > 0;
  }
  return found;
}

__global__ void __launch_bounds__(kThreads, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const SharedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  SharedSmem& sm = *reinterpret_cast<SharedSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  // Launched with programmatic stream serialisation.  Every CTA lets the next kernel start only
  // after its own wait, so that kernel (the own parts) may read the call's inputs without waiting
  // for this one: whatever ran before this grid has completed by then.
  pdl_wait_primary();
  pdl_launch_dependents();

  __syncthreads();
  // Runs of equal length, as long as it takes for the grid to cover the work and for no unit to
  // have more parts than slots.  Where there are at least four CTAs to a unit, units end with a run
  // (their lengths are rounded up), as a CTA spends 3 to 5 us between two parts (16 sequences that
  // share 16384 tokens, 64/8 heads: 28 us with runs of 12 tiles across units of 128, 21 in this
  // way); else a unit meets at most one run more than its length holds.  One slot: runs of whole
  // units, all as long as the longest.
  const int slots = a.plan.shared_splits, grid = gridDim.x;
  sum_work(a, sm, 0, blockIdx.x == 0);
  const int units = sm.units, most1 = sm.most[1], most = max(sm.most[0], most1);
  const bool aligned = slots > 1 && 4 * units <= grid;
  int each = 0, quantum;
  bool turns = false;
  if (slots == 1) {
    each = most;
    if (each > 0) sum_work(a, sm, each, false);
    quantum = each * ((units + grid - 1) / grid);
  } else {
    const int cover = aligned ? (sm.total - units + grid - units - 1) / (grid - units) : (sm.total + grid - 1) / grid;
    quantum = max(cover, aligned ? (most + slots - 1) / slots : (most + slots - 2) / (slots - 1));
    // Units of one row tile: tiles of keys in turn, if the slots (two for each part) are enough for
    // runs not much longer than that, as a tile then takes 0.75 us instead of 1.2; an even number,
    // as many for each set of warps.  Units of two row tiles gain nothing by longer runs.
    const int parts = slots / 2 - (aligned ? 0 : 1);
    if (parts > 0 && sm.most[0] > 0) {
      int in_turn = max((sm.most[0] + parts - 1) / parts, 2);
      if (most1 == 0) in_turn = (max(in_turn, cover) + 1) & ~1;
      turns = most1 > 0 ? in_turn <= quantum : 5 * in_turn <= 8 * quantum;
      if (turns) quantum = max(quantum, in_turn);
    }
    if (aligned) {
      each = max(quantum, 1);
      if (a.plan.num_groups > 1) {
        sum_work(a, sm, each, false);
      } else {
        __syncthreads();
        if (threadIdx.x == 0) sm.total = units * ((most + each - 1) / each * each);
        __syncthreads();
      }
    }
  }
  const int total = sm.total;
  if (quantum < 1) quantum = 1;
  if (static_cast<int>(blockIdx.x) >= total / quantum + (total % quantum != 0)) return;  // uniform, before any barrier or TMEM use

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
    mbar_init(smem_u32(&sm.stagger), 1);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(smem_u32(&sm.seg_full[i]), 1);
      mbar_init(smem_u32(&sm.seg_empty[i]), 11);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm.kv_full[s]), 1);
      mbar_init(smem_u32(&sm.kv_empty[s]), 2);
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

  const int slot_rows = slots + a.plan.own_splits;  // slots of a sequence's results
  // body(part, its tiles of keys, tiles of keys of the parts before) for every part of this CTA's run,
  // until it returns false.  The whole warp; false when something has been given up.
  auto for_segments = [&](auto&& body) {
    int g = 0;
    for (int it = 0;; ++it) {
      if (!__all_sync(0xffffffffu, wait_bar(smem_u32(&sm.seg_full[it % kSegments]), (it / kSegments) & 1, a.timeout_ns, abort_flag)))
        return false;
      const volatile Segment& seg = sm.seg[it % kSegments];
      const int n = seg.n_kv;
      if (n == 0) return true;
      if (!__all_sync(0xffffffffu, body(seg, n, g))) return false;
      if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[it % kSegments]));
      g += n;
    }
  };

  // 128 * 56 + 256 * 224 = 384 * 168 registers (the launch's total)
  if (warp < 4) {
    regs_dec<56>();
    if (warp == 0) {
      // ------------------------------------------------------------ pages
      const uint64_t policy = l2_policy_evict_last();  // other row tiles read the same pages
      const int no_page = a.num_pages * a.hkv * kPageSize;  // a row behind the cache: reads as zeros
      const bool ok = for_segments([&](const volatile Segment& seg, int n_kv, int g) {
        const int32_t* ptab = a.page_table + static_cast<size_t>(seg.first_seq) * a.max_pages;
        const int n_pages = seg.n_pages, tile0 = seg.tile0, kvh = seg.kvh;
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
        for (int j = 0; j < n_kv; ++j) {
          const int gg = g + j, st = gg % kStages;
          const int next = j + 1 < n_kv ? load_row(j + 1) : no_page;  // in flight while tile j is issued
          if (gg >= kStages) {
            int r = 1;
            if (lane == 0) r = wait_bar(smem_u32(&sm.kv_empty[st]), ((gg / kStages) - 1) & 1, a.timeout_ns, abort_flag) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, r, 0)) return false;
          }
          const uint32_t bar = smem_u32(&sm.kv_full[st]);
          if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kTileBytes);
          __syncwarp();
          if (lane < kPagesPerTile) {
            tma_load_2d(smem_u32(sm.k[st]) + lane * kPageSize * 128, &kmap, 0, row, bar, policy);
            tma_load_2d(smem_u32(sm.v[st]) + lane * kPageSize * 128, &vmap, 0, row, bar, policy);
          }
          if (lane == 0) sm.issued_kv = gg + 1;
          row = next;
        }
        return true;
      });
      if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
    } else if (warp == 3) {
      // ------------------------------------------------------------ the run's parts
      Walk walk;
      seek(a, sm, walk, static_cast<int>(blockIdx.x) * quantum, quantum, each);
      bool more = true;
      for (int it = 0; more; ++it) {
        if (it >= kSegments && !__all_sync(0xffffffffu, wait_bar(smem_u32(&sm.seg_empty[it % kSegments]), ((it / kSegments) - 1) & 1,
                                                                 a.timeout_ns, abort_flag))) {
          if (lane == 0) raise_status(a.status, kStatusTimeout);
          break;
        }
        Segment s{};
        more = next_segment(a, walk, s, quantum, each, turns);
        if (!more) s.n_kv = 0;
        if (lane == 0) {
          sm.seg[it % kSegments] = s;  // (n_kv = 0 behind the last)
          mbar_arrive(smem_u32(&sm.seg_full[it % kSegments]));
        }
        __syncwarp();
      }
    } else if (warp == 1 || warp == 2) {
      // ------------------------------------------------------------ products
      const int t = warp - 1;
      const uint32_t tmem = tmem_base();
      const uint32_t d_s = tmem + kColS + t * 128, d_o = tmem + kColO + t * 64, a_p = tmem + kColP + t * 64;
      const uint64_t qd = sw128_desc(smem_u32(sm.q[t]));
      auto wait = [&](uint64_t& bar, int parity) {
        return __all_sync(0xffffffffu, wait_bar(smem_u32(&bar), parity & 1, a.timeout_ns, abort_flag)) != 0;
      };
      bool ok = true;
      int steps = 0, parts = 0, all_parts = 0;  // of this set of warps; of the CTA
      const bool walked = for_segments([&](const volatile Segment& seg, int n_kv, int g) {
        const int part = all_parts++;
        const bool turns = seg.turns;
        if (!turns && t * kBlockQ >= seg.rows) {  // no such row tile: the stages are as good as used
          for (int j = 0; j < n_kv && ok; ++j) {
            ok = wait(sm.kv_full[(g + j) % kStages], (g + j) / kStages);
            if (ok && elect_one()) mbar_arrive(smem_u32(&sm.kv_empty[(g + j) % kStages]));
            __syncwarp();
          }
          return ok;
        }
        // step i works on tile of keys `first + i * stride` of the part
        const int stride = turns ? 2 : 1, first = turns ? t : 0, n = turns ? (n_kv - t + 1) / 2 : n_kv;
        if (n == 0) return true;
        ok = wait(sm.q_ready[t], parts);
        // Row tile 1 begins a softmax phase behind row tile 0, so that one set of warps computes
        // while the other loads and stores.  (Parts longer than the ring only: tile 0 cannot be
        // through with this part, and `stagger` cannot be two phases on, before tile 1 has begun.)
        if (ok && t == 1 && !turns && n_kv > kStages) ok = wait(sm.stagger, part);
        auto s_step = [&](int i) {  // S = Q K^T
          const int j = g + first + i * stride;
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
        auto pv_step = [&](int i) {  // O += P V
          const int j = g + first + i * stride;
          ok = wait(sm.p_full[t], steps + i);
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vd = sw128_desc(smem_u32(sm.v[j % kStages]));
#pragma unroll
            for (int kk = 0; kk < kBlockK / 16; ++kk)
              tc_mma_ts(d_o, a_p + kk * 8, vd + kk * (16 * 128 / 16), kIdescPV, (i > 0 || kk > 0) ? 1u : 0u);
            tc_commit(smem_u32(&sm.pv_done[t]));
            tc_commit(smem_u32(&sm.kv_empty[j % kStages]));
            if (turns) mbar_arrive(smem_u32(&sm.kv_empty[j % kStages]));  // for the other set of warps
          }
        };
        if (ok) s_step(0);
        for (int i = 0; i < n && ok; ++i) {
          if (i >= 1) pv_step(i - 1);
          if (ok && i + 1 < n) {
            ok = wait(sm.s_free[t], steps + i);
            if (ok) s_step(i + 1);
          }
        }
        if (ok) pv_step(n - 1);
        steps += n;
        ++parts;
        return ok;
      });
      if (elect_one()) {
        if (!walked) raise_status(a.status, kStatusTimeout);
        // whatever happened, every product issued here is done before TMEM is released
        tc_commit(smem_u32(&sm.drain[t]));
        mbar_wait(smem_u32(&sm.drain[t]), 0, kDrainTimeoutNs);
      }
      __syncwarp();
    }
  } else {
    regs_inc<224>();
    // -------------------------------------------------------------- softmax
    const int t = (warp - 4) >> 2;  // row tile of this warpgroup
    const int qw = warp & 3;        // TMEM lane quarter
    const uint32_t lane_base = tmem_base() + (static_cast<uint32_t>(qw * 32) << 16);
    const uint32_t s_col = lane_base + kColS + t * 128;
    const uint32_t o_col = lane_base + kColO + t * 64;
    const uint32_t p_col = lane_base + kColP + t * 64;
    const uint64_t scale2 = f2(a.scale_log2, a.scale_log2);
    // sequence and query head of a row of a part
    auto row_index = [&](const volatile Segment& seg, int row, int& seq, int& head) {
      const int gr = seg.row0 + row;
      seq = seg.first_seq + gr / a.group;
      head = seg.kvh * a.group + gr % a.group;
    };
    auto wait = [&](uint64_t& bar, int parity) {  // the same in all lanes: what follows is for the whole warp
      return __all_sync(0xffffffffu, wait_bar(smem_u32(&bar), parity & 1, a.timeout_ns, abort_flag)) != 0;
    };
    int steps = 0;  // of this set of warps
    const bool ok = for_segments([&](const volatile Segment& seg, int n_kv, int) {
      if (!seg.turns && t * kBlockQ >= seg.rows) return true;  // no such row tile
      const int r = (seg.turns ? 0 : t * kBlockQ) + qw * 32 + lane;  // row within the unit
      const int n = seg.turns ? (n_kv - t + 1) / 2 : n_kv;
      // read again where it is used, rather than held in registers that the score row needs
      auto live = [&]() { return r < seg.rows; };
      auto warp_live = [&]() { return (r & ~31) < seg.rows; };
      if (n > 0) {
        // the tile's Q (every product that read the last part's is done: its scores have been waited for)
        int seq, head;
        row_index(seg, live() ? r : 0, seq, head);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<size_t>(seq) * a.hq + head) * kHeadDim);
        uint4 x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = live() ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        uint8_t* dst = sm.q[t] + (r & 127) * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(dst + ((c ^ (r & 7)) << 4)) = x[c];
        fence_proxy_async_smem();  // the rows are read by the tensor core (async proxy)
        mbar_arrive(smem_u32(&sm.q_ready[t]));
      }
      float m = kNegInf, d = 0.0f;  // running maximum (log2 units) and sum
      for (int j = 0; j < n; ++j) {
        if (!wait(sm.s_full[t], steps + j)) return false;
        if (!warp_live()) {  // rows that nothing reads: keep step with the others, phase by phase
          mbar_arrive(smem_u32(&sm.s_free[t]));
          if (j > 0 && !wait(sm.pv_done[t], steps + j - 1)) return false;
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
        float mraw = fmax3(pm0, pm1, fmaxf(pm2, pm3));
        // keys from this tile's first on
        const int left = seg.n_pages * kPageSize - (seg.tile0 + (seg.turns ? 2 * j + t : j)) * kBlockK;
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
        if (j > 0 && !wait(sm.pv_done[t], steps + j - 1)) return false;
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
        if (j == 0 && warp == 4 && lane == 0) mbar_arrive(smem_u32(&sm.stagger));
      }
      steps += n;
      if (n > 0 && !wait(sm.pv_done[t], steps - 1)) return false;
      if (warp_live()) {
        tc_fence_after();
        uint32_t ou[2][32];
        tmem_ld32(o_col, ou[0]);
        tmem_ld32(o_col + 32, ou[1]);
        tc_wait_ld();
        tc_fence_before();  // the next part's products may overwrite O once this thread has handed over its P
        if (live()) {
          const float inv = d > 0.0f ? 1.0f / d : 0.0f;
          int seq, head;
          row_index(seg, r, seq, head);
          const int slot = seg.turns ? 2 * seg.slot + t : seg.slot;
          const size_t out = (static_cast<size_t>(seq) * slot_rows + slot) * a.hq + head;
          if (n > 0) {
            float4* o = reinterpret_cast<float4*>(a.partial_o + out * kHeadDim);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const uint32_t* u = ou[c >> 3] + 4 * (c & 7);
              o[c] = make_float4(__uint_as_float(u[0]) * inv, __uint_as_float(u[1]) * inv, __uint_as_float(u[2]) * inv,
                                 __uint_as_float(u[3]) * inv);
            }
          }
          a.partial_lse[out] = d > 0.0f ? (m + lg2(d)) * kLn2 : d == d ? kNegInf : d;  // NaN stays NaN
          if (seg.last && (t == 0 || !seg.turns)) {  // slots that nothing goes into
            float* lse = a.partial_lse + static_cast<size_t>(seq) * slot_rows * a.hq + head;
            for (int e = seg.turns ? 2 * seg.slot + 2 : seg.slot + 1; e < a.plan.shared_splits; ++e) lse[static_cast<size_t>(e) * a.hq] = kNegInf;
          }
        }
      }
      return true;
    });
    if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
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

// Adds a row's slots up: lse = ln sum e^lse_s, out = sum e^(lse_s - lse) o_s.  Sixteen lanes per row,
// four dimensions each; an empty slot (lse = -inf) is not read.  A slot whose scores were not all numbers
// (lse = NaN) makes the output NaN, and one whose weight vanishes is multiplied all the same: an infinite
// value in it shows, as in the decode of a sequence by itself.  The lse of a NaN row is -inf, as there.
constexpr int kMergeThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPosInf = __builtin_huge_valf();

__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const MergeArgs a) {
  // the partial results come from the two kernels before, whose last CTA has waited for both
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 15;
  const long long row = static_cast<long long>(blockIdx.x) * (kMergeThreads / 16) + (threadIdx.x >> 4);
  if (row >= static_cast<long long>(a.batch) * a.heads) return;
  const long long b = row / a.heads, h = row % a.heads;
  const int S = a.num_splits;
  const float* lse = a.partial_lse + b * S * a.heads + h;
  const float4* o = reinterpret_cast<const float4*>(a.partial_o + (b * S * a.heads + h) * kHeadDim) + lane;
  const unsigned half = 0xffffu << (threadIdx.x & 16);
  // Sixteen slots' values are asked for before any weight is known, so that a row of up to sixteen
  // costs one way to L2 (a slot that was not written holds anything, and is not multiplied).
  float4 v[16];
  auto ask = [&](int s0) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (s0 + i < S) v[i] = o[static_cast<long long>(s0 + i) * a.heads * (kHeadDim / 4)];
  };
  const float first = lane < S ? lse[static_cast<long long>(lane) * a.heads] : kNegInf;
  ask(0);
  float most = first;
  for (int s = lane + 16; s < S; s += 16) most = fmaxf(most, lse[static_cast<long long>(s) * a.heads]);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(half, most, off));
  float z = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < S; s0 += 16) {
    // this lane's slot's weight: the largest term exactly 1;
    const float l = s0 == 0 ? first : s0 + lane < S ? lse[static_cast<long long>(s0 + lane) * a.heads] : kNegInf;
    // an empty slot has weight -1 here.
    const float w = l == kNegInf ? -1.0f : l == most ? 1.0f : l != l ? l : most == kPosInf ? 0.0f : ex2((l - most) * kLog2e);
    if (s0 > 0) ask(s0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float wi = __shfl_sync(half, w, (threadIdx.x & 16) + i);  // (-1 behind the last slot)
      if (!(wi < 0.0f)) {
        z += wi;
        acc.x = fmaf(wi, v[i].x, acc.x);
        acc.y = fmaf(wi, v[i].y, acc.y);
        acc.z = fmaf(wi, v[i].z, acc.z);
        acc.w = fmaf(wi, v[i].w, acc.w);
      }
    }
  }
  const float inv = z > 0.0f ? 1.0f / z : 0.0f;
  uint2 pk;
  pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kHeadDim + 4 * lane) = pk;
  if (a.lse && lane == 0) a.lse[row] = !(z > 0.0f) ? kNegInf : most == kPosInf ? kPosInf : most + lg2(z) * kLn2;
}

}  // namespace

static int key_tiles_of(int pages) { return (pages + kPagesPerTile - 1) / kPagesPerTile; }

long long shared_row_tiles(int batch, int num_groups, int group) {
  const long long rows = static_cast<long long>(batch) * group, block = 2 * kBlockQ;
  const long long groups = num_groups < batch ? num_groups : batch;  // the ones that can have rows
  return (rows + groups * (block - 1)) / block;
}

int shared_ctas(int batch, int num_groups, int group, int hkv, int max_shared_pages, int max_pages,
                long long own_ctas, int sms) {
  // SM time (us) of the shared part, if every group's prompt is the longest: 1.28 for a tile of keys
  // of two row tiles, 0.75 of one.  Of the own parts, if they are half as long as the page table has
  // room for, but of 48 pages at most: three CTAs of 3 us and 35 KB per us beside one another.  A table
  // may be as wide as the model's context, for a step captured once; SMs left to own parts that
  // are not there cost a factor, too few of them little, as own parts run where the shared part has ended
  // (64 sequences that share 32768 tokens, 1024 of their own: 56.5 us with a table of 2108 pages and 57.4 with
  // 8192, without the limit 383; 32 sequences of 32/8 heads in 2 groups on 11200 tokens, own parts
  // to 3000: 41.6 us, 35.3 without).
  const bool one = static_cast<long long>(batch) * group <= static_cast<long long>(kBlockQ) * num_groups;
  const double tiles = static_cast<double>(shared_row_tiles(batch, num_groups, group)) * hkv * key_tiles_of(max_shared_pages);
  const double work = tiles * (one ? 0.75 : 1.28);
  const int own_pages = max_pages - max_shared_pages;
  const double own_bytes = 0.5 * (own_pages < 96 ? own_pages : 96) * kPageSize * 256.0 * hkv * batch;
  const double cta = 3.0 + own_bytes / own_ctas / 35e3;
  const double own = own_ctas * cta / 3.0;
  // x SMs for the shared part: what the own parts have left at its end then has all SMs
  int best = sms;
  double least = 1e30;
  for (int x = sms; x >= 8; x -= 4) {
    const double end = 4.0 + work / x;
    const double left = own - (sms - x) * end;
    const double t = end + (left > 0.0 ? left / sms : 0.0);
    if (t < 0.999 * least) {
      least = t;
      best = x;
    }
  }
  return best;
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
  cfg.gridDim = dim3(a.ctas, 1, 1);
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

cudaError_t launch_shared_merge(const MergeArgs& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.batch) * a.heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kMergeThreads / 16 - 1) / (kMergeThreads / 16)), 1, 1);
  cfg.blockDim = dim3(kMergeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, shared_merge_kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace sa
