// Matrix products grouped by expert, out[r, j] = sum_i x[row_token[r], i] w[e, j, i] + b[e, j]
// for the rows r of expert e, on the 5th-generation tensor cores, with operands in bf16 or
// MXFP4 and an optional clamped SwiGLU on interleaved gate / up features (the experts of the
// page "GPT-OSS on day 0": SwiGLU, bias terms; the models' own format is MXFP4).
//
// Orientation.  The group sizes are ragged and often tiny (a decode step gives an expert one
// or two rows), while the features are many and fixed, so the weights are the A operand (M =
// 128 features) and the rows the B operand, whose N is chosen per tile: a tile of n rows
// issues MMAs of N = n rounded up to 16 (32 in a pair of CTAs, below).  Transposed this way one
// kernel serves one row and thousands without padding rows to an M of 128.  Gathered rows are
// loaded one by one; consecutive ones in whole boxes, of 16 rows in a single CTA and of 64 (bf16)
// or 56 (MXFP4) in each CTA of a pair, with the scales of 112 rows.
//
// A tile is 128 features by up to `cap` rows; with more than a few rows per expert two CTAs on
// neighbouring SMs work as a pair (cta_group::2: one MMA of 256 features on both, each CTA
// staging half of the rows).  Persistent kernel, one CTA per SM, 17 warps (21 in bf16):
//   warp 0        the weights of a ring stage (boxes of 128 features x 128 bytes of K, 128-byte
//                 swizzle) when it is free
//   warp 1        TMEM owner and MMA issuer (one elected thread): 32 bytes of K per MMA
//   warp 2        MXFP4: scale bytes of weights and rows, into a staging place
//   warps 3, 16   in turns of a stage: write them into the ring in the layout that tcgen05.cp
//                 spreads over TMEM (row r of a block of 128: 4 bytes at 16 (r % 32) + 4 (r / 32),
//                 512 bytes per 128 values of K); report them, and gathered rows
//   warps 4..11   epilogue: TMEM lanes are features, columns rows; bias and activation in
//                 fp32, one rounding, 8 x 8 transpositions through shared memory and 16-byte
//                 stores, 64 consecutive bytes per row and warp (32 with SwiGLU, whose gate and
//                 up features are neighbouring lanes)
//   warps 12..15  the rows: consecutive ones in TMA boxes, in turns of a stage; rows gathered by
//                 their indices (bf16: warps 17..20 as well) with 16-byte asynchronous copies (TMA
//                 gathers of four rows cost their warp about 90 cycles each: 32768 tokens took
//                 5.3 ms that way, 2.6 this way)
// What a warp does per stage it does with uniform control flow and one elected lane, so that
// descriptors and addresses stay in uniform registers (MMAs from a divergent branch: 125 cycles
// each to issue, twice what they take).
// Two TMEM accumulators alternate, so the epilogue of a tile overlaps the next tile's MMAs.
//
// Tiles are numbered by expert, then feature tile, then row tile: the row tiles of one weight
// tile run at the same time and share it through L2, so weights come from memory once; experts
// of more than 8 row tiles go in bands of 8, whose rows stay in L2 over all features.  An
// expert's rows are split evenly among its row tiles.  Each CTA derives the numbering from
// the offsets in device memory (a prefix sum over at most 256 experts).
//
// What bounds it, and what it measured (one GB300; 2880 -> 5760 with SwiGLU and gathered rows,
// 128 experts, top 4, unless stated):
//   few rows    the weights' way from memory.  61 tokens 0.51 ms in bf16 (7.0 TB/s), 0.15 ms in
//               MXFP4 (6.5 TB/s); 1 token 25.5 us and 15 us, of which about 6 are launch, first
//               loads and the last tile's end.
//   many rows   bf16: the tensor cores and the power limit; 32768 tokens 2.6 - 2.8 ms, 3.0 back to
//               back (1400 - 1650 TFLOP/s), one group of 32768 rows x 4096 -> 2880 0.42 ms (1830).
//               MXFP4: a stage's way round the ring (free, filled, reported, multiplied) beside an
//               epilogue that competes for issue slots; 1.07 - 1.09 ms (4.0 PFLOP/s), consecutive rows
//               0.88 - 0.93, one group 0.138 (5.6).  With nothing loaded the 0.93 stay, without the
//               epilogue as well 0.70, without the MMAs as well 0.47.
#include <atomic>
#include <cstdint>

#include "grouped_args.h"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr int kFeat = kGroupedFeatures;
constexpr int kStageKBytes = 128;  // bytes of K per ring stage: 64 bf16 or 256 E2M1 values
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kRowWarp0 = kEpiWarp0 + kEpiWarps;
constexpr int kRowWarps = 4;
// Warps that take turns of one stage: those that bring rows in boxes, and those that report what
// threads have brought (warp 3 and kReportWarp1).
constexpr int kTurns = kRowWarps;
constexpr int kReportTurns = 2;
constexpr int kReportWarp1 = kRowWarp0 + kRowWarps;
constexpr int kGatherWarp1 = kReportWarp1 + 1;  // the first of the warps that help with gathered rows
constexpr int kProducers = 1 + kTurns + kReportTurns;  // warps: weights, rows, reports
constexpr int kMaxStages = 16;
constexpr int kMaxSingleRows = 64;  // rows of a single CTA's tile
constexpr int kMaxRawSlots = 6;
constexpr int kBand = 8;             // row tiles of an expert that pass over its features together
constexpr int kSfBlock = 512;        // scales of 128 rows x 128 values of K
constexpr int kPatchBytes = 512;     // of an epilogue warp
constexpr unsigned long long kDrainTimeoutNs = 2000000000ull;

template <bool kFp4>
struct GrpCfg {
  // two accumulators of kRows columns; in MXFP4 two stages' scales beside them
  static constexpr int kRows = kFp4 ? 224 : 256;
  static constexpr int kStageK = kFp4 ? 256 : 64;
  static constexpr int kSfBytes = kFp4 ? 2 * 3 * kSfBlock : 0;  // per 128 values of K: a block of weights, two of rows
  static constexpr int kSfCols = 24;
  // Warps that copy gathered rows: a warp spends about 100 cycles on each of its copies of a stage,
  // so more of them fill it sooner (32768 tokens up, back to back: bf16 3.09 ms with four, 3.02 with
  // eight), but they take issue slots, which MXFP4's short stages miss (1.09 ms, 1.19).
  static constexpr int kGatherWarps = kFp4 ? kRowWarps : 2 * kRowWarps;
  static constexpr int kThreads = 32 * (kGatherWarp1 + kGatherWarps - kRowWarps);
  static constexpr int kTmemCols = 512;
  static_assert(2 * kRows + (kFp4 ? 2 * kSfCols : 0) <= kTmemCols, "TMEM holds 512 columns");
};

// Shared memory: the ring, and places for MXFP4 scale bytes on their way.  A row's 16 bytes serve
// two blocks of K.  With pairs of CTAs a place takes three times 16 bytes of each of 128 features
// and 224 rows: to the copy engine a piece of 16 bytes is a request like one of 128, and 16 at a
// time the scales' requests were 176 a stage beside the operands' 240.  (32768 x 4096 -> 2880: 16
// bytes and six stages 144 us, 48 and five stages 138.  Gathered rows, whose scales threads copy,
// prefer the sixth stage by 2 %.)
template <bool kFp4, bool kPair>
struct GrpSmem {
  static constexpr int kRawCols = kPair ? kScaleBoxCols : 1;  // of 16 bytes
  static constexpr int kRawPitch = 16 * kRawCols;
  static constexpr int kRawSlots = kPair ? 3 : kMaxRawSlots;
  static constexpr int kRawRows = kPair ? GrpCfg<true>::kRows : kMaxSingleRows;
  static constexpr int kRawStep = kRawPitch * (kFeat + kRawRows);
  static constexpr int kRawBytes = kFp4 ? kRawSlots * kRawStep : 0;
  static constexpr int kRingBytes = (kFp4 && kPair ? 165 : 198) * 1024;
  static constexpr size_t kTotal = 1024 /*alignment slack*/ + kRingBytes + kRawBytes + kEpiWarps * kPatchBytes;
};

// A stage holds `sub` blocks of kStageKBytes of K: `width` features and `rows` rows of 128 bytes
// in each (a CTA of a pair stages half of the tile's rows), then the blocks' scales.  width and
// rows are multiples of 16, so the parts start on multiples of 1024 bytes (the swizzle atom).
template <bool kFp4>
__host__ __device__ constexpr int stage_bytes(int width, int rows, int sub) {
  return (sub * ((width + rows) * kStageKBytes + GrpCfg<kFp4>::kSfBytes) + 1023) / 1024 * 1024;
}
// An MMA reads 128 features also where the tile has fewer: at the end of the last stage, too,
// that stays inside the ring (what it reads there goes to accumulator lanes that are never stored).
template <bool kFp4, bool kPair>
__host__ __device__ constexpr int stage_count(int width, int rows, int sub) {
  const int size = stage_bytes<kFp4>(width, rows, sub);
  const int n = (GrpSmem<kFp4, kPair>::kRingBytes - (kFeat - width) * kStageKBytes) / size;
  return n < kMaxStages ? n : kMaxStages;
}

struct GrpShared {
  uint64_t full[kMaxStages], empty[kMaxStages], landed[kMaxStages];
  uint64_t raw_full[kMaxRawSlots], raw_empty[kMaxRawSlots];
  uint64_t acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
  int issued[kProducers];     // stages that each producer warp filled, written when it ends
  int raw_issued;                // places of scales that warp 2 requested, likewise
  int total;                     // row tiles of all experts
  int cum[kMaxExperts + 32];     // row tiles of lower experts (a huge number from E + 1 on)
  int4 group[kMaxExperts];       // first row, rows, row tiles, rows per tile
};
template <bool kFp4, bool kPair>
constexpr size_t smem_bytes() {
  return GrpSmem<kFp4, kPair>::kTotal + sizeof(GrpShared);
}
static_assert(smem_bytes<true, true>() <= 227 * 1024 && smem_bytes<true, false>() <= 227 * 1024 &&
              smem_bytes<false, true>() <= 227 * 1024, "shared memory of one CTA");

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
  __device__ __forceinline__ void skip(int n, int stages) {
    for (stage += n; stage >= stages; stage -= stages) ++round;
  }
};

__device__ __forceinline__ uint64_t sw128_kmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(1024 >> 4) << 16;  // leading byte offset (unused, K-major SW128)
  d |= static_cast<uint64_t>(1024 >> 4) << 32;  // stride byte offset: next 8-row group
  d |= 1ull << 46;                               // tcgen05 descriptor version
  d |= 2ull << 61;                               // 128-byte swizzle
  return d;
}

// 32 rows of 16 bytes, dense (core matrices of 8 rows x 16 bytes, 128 bytes apart).
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= 1ull << 46;
  return d;
}

// M: 128 features, or 256 of a CTA pair.  kind::f16, bf16 operands, both K-major.
template <bool kPair>
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>((kPair ? 2 : 1) * kFeat >> 4) << 24);
}
// kind::mxf4, E2M1 operands, E8M0 scales; which two scale bytes of a TMEM word (`sf`: 0 or 2).
template <bool kPair>
__device__ __forceinline__ uint32_t idesc_mxf4(int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>((kPair ? 2 : 1) * kFeat >> 7) << 27);
}
__device__ __forceinline__ uint32_t idesc_scale_bytes(int sf) {
  return (static_cast<uint32_t>(sf) << 4) | (static_cast<uint32_t>(sf) << 29);
}

// The tcgen05 instructions for one CTA or for a pair (an M = 256 MMA on both SMs, issued by
// the leading CTA; operands, scales and accumulator halves lie at the same places in both).
template <bool kPair>
__device__ __forceinline__ void grp_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  }
}
template <bool kPair>
__device__ __forceinline__ void grp_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tmem_dealloc(taddr, ncols);
}
template <bool kPair>
__device__ __forceinline__ void grp_mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    tc_mma_ss(d_tmem, a_desc, b_desc, idesc, accumulate);
}
template <bool kPair>
__device__ __forceinline__ void grp_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 512 bytes (32 rows x 16) to the same four columns of all four lane quarters; in a pair both
// CTAs copy from their own shared memory.
template <bool kPair>
__device__ __forceinline__ void grp_cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Arrive on `bar` (in a pair: on both CTAs') when all tcgen05 work issued so far is done.
template <bool kPair>
__device__ __forceinline__ void grp_commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    tc_commit(bar);
}

// Barriers of the leading CTA: `bar` is a shared::cluster address in a pair, which threads of
// and TMA copies into either CTA signal.  None of these arrivals publishes memory to the other
// CTA's threads: copies report themselves, accumulators are handed back by tcgen05 fences, and
// what threads write into a stage is read only by their own SM's tensor core, after a proxy
// fence that has put it there.  (At cluster scope, a releasing arrival waits for everything its
// warp has under way and halves the kernel's speed.)
template <bool kPair>
__device__ __forceinline__ void grp_arrive(uint32_t bar) {
  if constexpr (kPair)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
  else
    mbar_arrive(bar);
}
template <bool kPair>
__device__ __forceinline__ void grp_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  if constexpr (kPair)
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
  else
    mbar_arrive_expect_tx(bar, bytes);
}
template <bool kPair>
__device__ __forceinline__ void tma_load_w(uint32_t dst, const CUtensorMap* map, int x, int f, int e, uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(f), "r"(e), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(f), "r"(e), "r"(bar)
        : "memory");
}
template <bool kPair>
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// 16 bytes by a thread of its own: `bytes` of them from src, zeros behind.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// This thread's arrival on `bar` once its copies so far have landed.
__device__ __forceinline__ void copy_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Waits of a whole warp; the result is the same in all lanes.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                              volatile int* abort_flag) {
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

// One lane of the warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

struct Tile {
  int e, f0;  // expert; first feature
  int r0, n;  // first row, number of rows
};

// x / tiles_f for 0 <= x < 2^30 (a.f_magic, a.f_shift: set by the launcher).
__device__ __forceinline__ int over_tiles_f(const GroupedArgs& a, int x) {
  return static_cast<int>((static_cast<uint64_t>(x) * a.f_magic) >> a.f_shift);
}

// Tile t of the numbering in `sb` (all 32 lanes of a warp call this together).  `features`: of
// one tile.  Every role does this once per tile, the MMA warp between two tiles' MMAs: no
// integer division, whose latency would show there.
__device__ __forceinline__ Tile find_tile(const GrpShared& sb, const GroupedArgs& a, int t, int features, int lane) {
  const int q = over_tiles_f(a, t);  // row tiles before it are whole experts' and at most its own expert's
  const unsigned lt = __ballot_sync(0xffffffffu, sb.cum[8 * lane] <= q);
  const int base = 8 * (__popc(lt) - 1);
  const unsigned in = __ballot_sync(0xffffffffu, lane < 8 && sb.cum[base + (lane & 7)] <= q);
  const int e = base + __popc(in) - 1;
  const int4 group = sb.group[e];
  int local = t - sb.cum[e] * a.tiles_f;
  const int band = group.z <= kBand ? 0 : over_tiles_f(a, local) / kBand;
  local -= band * kBand * a.tiles_f;
  const int wide = min(kBand, group.z - band * kBand);  // 1..8
  // local / wide: for x < 2^30 the excess of the factor stays below 2^-4 < 1 / 8
  const uint64_t factor = wide == 1   ? (1ull << 34)
                          : wide == 2 ? (1ull << 33)
                          : wide == 3 ? (1ull << 34) / 3 + 1
                          : wide == 4 ? (1ull << 32)
                          : wide == 5 ? (1ull << 34) / 5 + 1
                          : wide == 6 ? (1ull << 34) / 6 + 1
                          : wide == 7 ? (1ull << 34) / 7 + 1
                                      : (1ull << 31);
  const int ft = static_cast<int>((static_cast<uint64_t>(local) * factor) >> 34);
  const int rt = band * kBand + local - ft * wide;
  // through a reduction, whose result the compiler knows to be the same in all lanes
  Tile r;
  r.n = __reduce_min_sync(0xffffffffu, min(group.w, group.y - rt * group.w));
  r.r0 = __reduce_min_sync(0xffffffffu, group.x + rt * group.w);
  r.e = __reduce_min_sync(0xffffffffu, e);
  r.f0 = __reduce_min_sync(0xffffffffu, ft * features);
  return r;
}

// 16 TMEM lanes x 32 columns: thread t gets, for each group i of 8 columns, lane t / 4 (r[4 i],
// r[4 i + 1]) and lane t / 4 + 8 (r[4 i + 2], r[4 i + 3]) of columns 8 i + 2 (t % 4) + {0, 1}.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit values, each transposed on its way to shared memory: thread
// 8 m + t gives the address of row t of matrix m, 16 bytes.
__device__ __forceinline__ void store_transposed(uint32_t addr, const uint32_t (&m)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(m[0]),
               "r"(m[1]), "r"(m[2]), "r"(m[3])
               : "memory");
}

// Minimum and maximum that let NaN through.
__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
  float2 r;
  f2_split(v, r.x, r.y);
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two of g sigmoid(alpha g) (u + 1) with clamped g and u; minus_alpha2 = -alpha, twice.  The product
// with log2(e) follows that with g: alpha log2(e) may not fit into fp32, and would make NaN of a
// gate of 0.  The epilogue shares the issue slots with the warps that keep the ring turning, so its
// instructions count: packed arithmetic, and results of 2^x and of the reciprocal below 2^-126 taken
// as 0, which saves their rescaling.  A sigmoid below 2^-126 is one of these: |g (u + 1)| 2^-126 of
// the result at most.
__device__ __forceinline__ uint32_t swiglu2(float g0, float g1, float u0, float u1, uint64_t minus_alpha2, float limit) {
  const uint64_t g = f2(min_nan(g0, limit), min_nan(g1, limit));
  const uint64_t u = f2(max_nan(min_nan(u0, limit), -limit), max_nan(min_nan(u1, limit), -limit));
  const float2 x = f2_unpack(f2_mul(f2_mul(g, minus_alpha2), f2(1.4426950408889634f, 1.4426950408889634f)));
  const float2 d = f2_unpack(f2_add(f2(ex2(x.x), ex2(x.y)), f2(1.0f, 1.0f)));
  const uint64_t t = f2_mul(g, f2(rcp_ftz(d.x), rcp_ftz(d.y)));
  // not t u + t, which is NaN for an infinite t and u <= 0
  const float2 y = f2_unpack(f2_mul(t, f2_add(u, f2(1.0f, 1.0f))));
  return pack_bf16x2(y.x, y.y);
}

template <bool kFp4, bool kSwiglu, bool kPair>
__global__ void __launch_bounds__(GrpCfg<kFp4>::kThreads, 1)
grouped_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
               const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap xsmap,
               const GroupedArgs a) {
  using C = GrpCfg<kFp4>;
  using S = GrpSmem<kFp4, kPair>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  GrpShared& sb = *reinterpret_cast<GrpShared*>(tiles + S::kRingBytes + S::kRawBytes + kEpiWarps * kPatchBytes);
  volatile int* abort_flag = &sb.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int k_blocks = (a.K + C::kStageK - 1) / C::kStageK;  // of kStageKBytes
  const int sub = kPair ? 1 : a.sub;                         // blocks per stage
  const int k_steps = (k_blocks + sub - 1) / sub;
  const int stages = a.stages;
  const uint32_t ring = smem_u32(tiles);
  // a pair stages half of a tile's rows in each CTA
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kGrain = 16 * kCtas;
  const int stage_rows = a.cap / kCtas;
  const int width = kPair ? kFeat : a.width;  // features of one CTA's part of a tile
  const uint32_t w_bytes = width * kStageKBytes;
  const uint32_t stage_size = stage_bytes<kFp4>(width, stage_rows, sub);
  const uint32_t x_part = sub * w_bytes, sf_part = x_part + sub * stage_rows * kStageKBytes;  // of a stage
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  // reports of a CTA that a stage is filled: weights, rows in boxes, what threads bring
  const bool gather = a.row_token != nullptr;
  const int producers = 1 + (gather ? 0 : 1) + (kFp4 || gather ? 1 : 0);
  const int t_first = blockIdx.x / kCtas, t_step = gridDim.x / kCtas;
  // the leading CTA's barriers
  const uint32_t full0 = kPair ? dsmem_addr(smem_u32(&sb.full[0]), 0) : smem_u32(&sb.full[0]);
  const uint32_t acc_empty0 = kPair ? dsmem_addr(smem_u32(&sb.acc_empty[0]), 0) : smem_u32(&sb.acc_empty[0]);

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
    if (kFp4 && kPair) {
      tma_prefetch_desc(&wsmap);
      tma_prefetch_desc(&xsmap);
    }
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&sb.full[s]), kCtas * producers);
      mbar_init(smem_u32(&sb.landed[s]), 32 * C::kGatherWarps);
      mbar_init(smem_u32(&sb.empty[s]), 1);
    }
    for (int r = 0; kFp4 && r < kMaxRawSlots; ++r) {
      mbar_init(smem_u32(&sb.raw_full[r]), kPair ? (gather ? 33 : 1) : 32);
      mbar_init(smem_u32(&sb.raw_empty[r]), kReportTurns);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sb.acc_full[b]), 1);
      mbar_init(smem_u32(&sb.acc_empty[b]), kCtas * kEpiWarps);
    }
    mbar_init(smem_u32(&sb.drain), 1);
    sb.abort_flag = 0;
    for (int w = 0; w < kProducers; ++w) sb.issued[w] = 0;
    sb.raw_issued = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    grp_tmem_alloc<kPair>(smem_u32(&sb.tmem_base), C::kTmemCols);
  }
  if (warp == 2) {
    // the groups: validated, and their row tiles summed up (8 experts per lane).  A group
    // counts if it starts at or behind every earlier offset: groups never overlap.
    int off[9], high = 0;
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      const int e = 8 * lane + j;
      off[j] = e > a.num_experts ? 0 : a.offsets ? __ldg(a.offsets + e) : e == 0 ? 0 : a.rows;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) high = max(high, off[j]);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, high, d);
      if (lane >= d) high = max(high, v);
    }
    high = __shfl_up_sync(0xffffffffu, high, 1);  // the largest offset of lower lanes
    if (lane == 0) high = 0;
    int sum = 0, mine[8];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = 8 * lane + j;
      int lo = 0, hi = 0;
      if (e < a.num_experts) {
        lo = off[j];
        hi = off[j + 1];
        if (lo < high || hi < lo || hi > a.rows) {
          bad = true;
          lo = hi = 0;
        }
        high = max(high, off[j]);
      }
      // row tiles, and an even split of the rows among them in multiples of kGrain
      const int rows = hi - lo, count = (rows + a.cap - 1) / a.cap;
      const int per = count ? (rows + count * kGrain - 1) / (count * kGrain) * kGrain : 0;
      sb.group[e] = make_int4(lo, rows, count, per);
      mine[j] = sum;
      sum += count;
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sb.cum[8 * lane + j] = 8 * lane + j <= a.num_experts ? incl - sum + mine[j] : 0x7FFFFFFF;
    if (lane == 31) {
      sb.total = incl;
      sb.cum[kMaxExperts] = 0x7FFFFFFF;
    }
    if (bad) raise_status(a.status, kStatusBadLen);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // the other CTA's barriers exist
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;
  const int tiles_total = sb.total * a.tiles_f;

  if (warp == 0) {
    // Copies first, then the report: the copies' way is the long one, and a phase of `full` is not
    // over before all its arrivals, whatever has landed.
    RingPos p;
    int g = 0;
    bool ok = true;
    for (int t = t_first; t < tiles_total && ok; t += t_step) {
      const Tile tl = find_tile(sb, a, t, kCtas * width, lane);
      for (int kb = 0; kb < k_steps; ++kb, ++g, p.next(stages)) {
        if (p.round != 0)
          ok = wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = full0 + 8 * p.stage;
          const int blocks = kPair ? 1 : min(sub, k_blocks - kb * sub);
          for (int u = 0; u == 0 || (!kPair && u < blocks); ++u)  // features past N are zero-filled
            tma_load_w<kPair>(ring + p.stage * stage_size + u * w_bytes, &wmap,
                              (kb * sub + u) * (kFp4 ? kStageKBytes : kStageKBytes / 2), tl.f0 + rank * kFeat, tl.e,
                              bar);
          grp_arrive_expect_tx<kPair>(bar, blocks * w_bytes);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) raise_status(a.status, kStatusTimeout);
      sb.issued[0] = g;
    }
  } else if (warp == 1 && rank == 0) {
    RingPos p;
    int i = 0, scales = 0;
    bool ok = true;
    for (int t = t_first; t < tiles_total && ok; t += t_step, ++i) {
      const Tile tl = find_tile(sb, a, t, kCtas * width, lane);
      const int n16 = (tl.n + kGrain - 1) / kGrain * kGrain;
      const int b = i & 1;
      if (i >= 2) ok = wait_or_abort(smem_u32(&sb.acc_empty[b]), ((i >> 1) - 1) & 1, a.timeout_ns, abort_flag);
      tc_fence_after();
      const uint32_t d = tmem + b * C::kRows;
      const uint32_t idesc = kFp4 ? idesc_mxf4<kPair>(n16) : idesc_bf16<kPair>(n16);
      for (int kb = 0; kb < k_steps && ok; ++kb, p.next(stages)) {
        ok = wait_or_abort(smem_u32(&sb.full[p.stage]), p.round & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t stage = ring + p.stage * stage_size;
        const int blocks = kPair ? 1 : min(sub, k_blocks - kb * sub);
        if (elect_one()) {
#pragma unroll 1
          for (int u = 0; u == 0 || (!kPair && u < blocks); ++u) {
            const uint64_t wd = sw128_kmajor_desc(stage + u * w_bytes);
            const uint64_t xd = sw128_kmajor_desc(stage + x_part + u * stage_rows * kStageKBytes);
            const int block = kb * sub + u;
            if constexpr (kFp4) {
              // this block's scales: per 128 values of K the weights' and the rows'
              const uint32_t sf = tmem + 2 * C::kRows + (scales & 1) * C::kSfCols;
              const uint64_t sd = scale_desc(stage + sf_part + u * C::kSfBytes);
              ++scales;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                grp_cp_scales<kPair>(sf + 12 * c, sd + (3 * c) * (kSfBlock >> 4));
                grp_cp_scales<kPair>(sf + 12 * c + 4, sd + (3 * c + 1) * (kSfBlock >> 4));
                if (n16 > 128) grp_cp_scales<kPair>(sf + 12 * c + 8, sd + (3 * c + 2) * (kSfBlock >> 4));
              }
              const int left = (a.K - block * C::kStageK + 63) / 64;  // 64-value steps with data
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (kk < left)
                  grp_mma_mxf4<kPair>(d, wd + 2 * kk, xd + 2 * kk, idesc | idesc_scale_bytes(2 * (kk & 1)),
                                      sf + 12 * (kk >> 1), sf + 12 * (kk >> 1) + 4, (block | kk) != 0);
              }
            } else {
              const int left = (a.K - block * C::kStageK + 15) / 16;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (kk < left) grp_mma_bf16<kPair>(d, wd + 2 * kk, xd + 2 * kk, idesc, (block | kk) != 0);
              }
            }
          }
          grp_commit<kPair>(smem_u32(&sb.empty[p.stage]));
          if (kb == k_steps - 1) grp_commit<kPair>(smem_u32(&sb.acc_full[b]));
        }
      }
    }
    if (elect_one()) {
      if (!ok) raise_status(a.status, kStatusTimeout);
      // every MMA issued by this thread has finished before TMEM is released
      grp_commit<kPair>(smem_u32(&sb.drain));
      if (!mbar_wait(smem_u32(&sb.drain), 0, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (kFp4 && warp == 2) {
    if constexpr (kFp4) {
      // Scale bytes on their way, some blocks of K ahead.  In a pair of CTAs they come in boxes of
      // kRawPitch bytes x rows, but for gathered rows: copies by threads, 16 bytes each,
      // neighbouring lanes on the same row.  Small tiles take copies throughout (8 tokens down,
      // 2880 x 2880: 28 us, with boxes 31).
      const int cols = a.scale_stride / 16;
      const int slots = (k_blocks + 2 * S::kRawCols - 1) / (2 * S::kRawCols);
      const uint32_t raw = smem_u32(tiles + S::kRingBytes);
      constexpr int kRowCopies = S::kRawRows * S::kRawCols / 32;
      constexpr uint32_t kRowPart = kFeat * S::kRawPitch;
      RingPos p;
      bool ok = true;
      for (int t = t_first; t < tiles_total && ok; t += t_step) {
        const Tile tl = find_tile(sb, a, t, kCtas * width, lane);
        const int copies = (tl.n * S::kRawCols + 31) / 32;
        const bool by_threads = !kPair || gather;
        int src[kRowCopies];  // row of x of copy j: the piece (32 j + lane) % kRawCols of it
        const uint8_t* wsrc[kPair ? 1 : 4];
#pragma unroll
        for (int j = 0; j < kRowCopies; ++j) {
          const int r = (32 * j + lane) / S::kRawCols;
          src[j] = -1;  // behind the tile's last row: zeros
          if (by_threads && r < tl.n) {
            src[j] = tl.r0 + r;
            if (gather) {
              const int id = __ldg(a.row_token + tl.r0 + r);
              src[j] = id < 0 || id >= a.x_rows ? 0 : id;  // reported by the row warps
            }
          }
        }
        const int f0 = tl.f0 + rank * kFeat;
        if constexpr (!kPair) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 32 * j + lane;
            wsrc[j] = r < width && f0 + r < a.N
                          ? a.w_scales + (static_cast<long long>(tl.e) * a.N + f0 + r) * a.scale_stride
                          : nullptr;
          }
        }
        for (int slot = 0; slot < slots; ++slot, p.next(S::kRawSlots)) {
          if (p.round != 0)
            ok = wait_or_abort(smem_u32(&sb.raw_empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
          if (!ok) break;
          const uint32_t bar = smem_u32(&sb.raw_full[p.stage]);
          const uint32_t dst = raw + p.stage * S::kRawStep;
          if constexpr (kPair) {
            if (elect_one()) {
              // few and large boxes: each costs its warp about 90 cycles to issue
              const int boxes = gather ? 0 : tl.n > kScaleBoxRows ? 2 : 1;
              mbar_arrive_expect_tx(bar, S::kRawPitch * (width + boxes * kScaleBoxRows));
              tma_load_rows<false>(dst, &wsmap, S::kRawPitch * slot, tl.e * a.N + f0, bar);  // E N < 2^31
              for (int i = 0; i < boxes; ++i)
                tma_load_rows<false>(dst + kRowPart + S::kRawPitch * kScaleBoxRows * i, &xsmap, S::kRawPitch * slot,
                                     tl.r0 + kScaleBoxRows * i, bar);
            }
            __syncwarp();  // together again: the copies below are issued once, not once per branch
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (32 * j < width)
                copy_async16(dst + 512 * j + 16 * lane, wsrc[j] ? wsrc[j] + 16 * slot : a.w_scales, wsrc[j] ? 16 : 0);
          }
          if (by_threads) {
#pragma unroll
            for (int j = 0; j < kRowCopies; ++j)
              if (j < copies) {
                const int col = slot * S::kRawCols + (32 * j + lane) % S::kRawCols;
                const bool read = src[j] >= 0 && col < cols;
                copy_async16(dst + kRowPart + 512 * j + 16 * lane,
                             a.x_scales + (read ? static_cast<long long>(src[j]) * a.scale_stride + 16 * col : 0),
                             read ? 16 : 0);
              }
            copy_async_arrive(bar);
          }
        }
      }
      copy_async_wait_all();
      if (lane == 0) {
        if (!ok) raise_status(a.status, kStatusTimeout);
        sb.raw_issued = p.round * S::kRawSlots + p.stage;
      }
    }
  } else if (warp == 3 || warp == kReportWarp1) {
    // What threads have brought becomes the tensor core's: scales are put in their layout,
    // gathered rows have landed; then one proxy fence, by a warp that has no copies under way
    // (with them, a fence takes as long as they do), and the stage is reported.  The two warps take
    // turns of one stage, counted over all tiles: a wait for a parity is sound only if the phase
    // before it is known to be over, which a warp that comes back within one round of the ring
    // knows from its last stage (rows land, and stages become free, in their order).  Four warps
    // were slower: every warp that waits takes issue slots from those that work (gathered rows,
    // 32768 tokens up: 1.25 ms, with two 1.12).
    const int turn = warp == 3 ? 0 : 1;
    RingPos p, pr;
    int base = 0, done = 0;  // stages of earlier tiles; one more than the last stage reported
    bool ok = kFp4 || gather;
    for (int t = t_first; t < tiles_total && ok; t += t_step, base += k_steps) {
      [[maybe_unused]] int quarters = 0, slot = -1;  // of 128 rows; place of scales that is being read
      if constexpr (kFp4) quarters = (find_tile(sb, a, t, kCtas * width, lane).n + 31) / 32;
      auto leave = [&]() {
        __syncwarp();
        if (elect_one()) mbar_arrive(smem_u32(&sb.raw_empty[pr.stage]));
        __syncwarp();
        pr.next(S::kRawSlots);
      };
      auto enter = [&](int next) {
        while (slot < next && ok) {
          if (slot >= 0) leave();
          ++slot;
          ok = wait_or_abort(smem_u32(&sb.raw_full[pr.stage]), pr.round & 1, a.timeout_ns, abort_flag);
        }
      };
      int at = 0;
      for (int kb = (turn - base) & (kReportTurns - 1); kb < k_steps; kb += kReportTurns) {
        p.skip(kb - at, stages);
        at = kb;
        if constexpr (kFp4) {
          const int blocks = kPair ? 1 : min(sub, k_blocks - kb * sub);
          for (int u = 0; u == 0 || (!kPair && u < blocks); ++u) {
            const int block = kb * sub + u;
            enter(block / (2 * S::kRawCols));
            if (!ok) break;
            // The block's 8 bytes of rows lane, lane + 32, lane + 64, lane + 96 of each block of
            // 128.  All that can be there is read, without a branch: what rows behind the tile's last
            // one (or features behind its width) have there scales columns (lanes) that are never stored.
            const uint8_t* raw = tiles + S::kRingBytes + pr.stage * S::kRawStep + S::kRawPitch * lane +
                                 8 * (block - 2 * S::kRawCols * slot);
            constexpr int kQuarters = (kFeat + S::kRawRows) / 32;
            uint2 c[12];
#pragma unroll
            for (int i = 0; i < 12; ++i)
              c[i] = i < kQuarters ? *reinterpret_cast<const uint2*>(raw + 32 * S::kRawPitch * i) : make_uint2(0, 0);
            const int valid = a.K / 32 - 8 * block;  // bytes in use, the rest is padding
            if (valid < 8) {
              const uint32_t mask0 = valid >= 4 ? 0xFFFFFFFFu : valid <= 0 ? 0u : (1u << (8 * valid)) - 1u;
              const uint32_t mask1 = valid <= 4 ? 0u : (1u << (8 * valid - 32)) - 1u;
#pragma unroll
              for (int i = 0; i < kQuarters; ++i) c[i] = make_uint2(c[i].x & mask0, c[i].y & mask1);
            }
            if (u == 0 && p.round != 0)
              ok = wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
            if (!ok) break;
            uint4* sf = reinterpret_cast<uint4*>(tiles + p.stage * stage_size + sf_part + u * C::kSfBytes) + lane;
#pragma unroll
            for (int blk = 0; blk < 3; ++blk) {
              if (blk == 2 && quarters <= 4) break;
              const uint2* v = c + 4 * blk;
              sf[blk * (kSfBlock / 16)] = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
              sf[(3 + blk) * (kSfBlock / 16)] = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
            }
          }
        }
        if (gather && ok) ok = wait_or_abort(smem_u32(&sb.landed[p.stage]), p.round & 1, a.timeout_ns, abort_flag);
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) grp_arrive<kPair>(full0 + 8 * p.stage);
        __syncwarp();
        done = base + kb + 1;
      }
      p.skip(k_steps - at, stages);
      if constexpr (kFp4) {
        if (ok) enter((k_blocks - 1) / (2 * S::kRawCols));
        if (ok) leave();
      }
    }
    if (lane == 0) {
      if (!ok && (kFp4 || gather)) raise_status(a.status, kStatusTimeout);
      sb.issued[1 + kTurns + turn] = done;
    }
  } else if (warp >= kRowWarp0) {
    const int wr = kFp4 || warp < kReportWarp1 ? warp - kRowWarp0 : kRowWarps + warp - kGatherWarp1;
    constexpr int kStepRows = 4 * C::kGatherWarps;  // rows that one copy by each thread brings
    constexpr int kSteps = ((kPair ? C::kRows / 2 : kMaxSingleRows) + kStepRows - 1) / kStepRows;
    RingPos p;
    int g = 0, done = 0;  // stages of earlier tiles; one more than the last stage reported
    bool ok = true;
    if (gather) {
      // Gathered rows: eight threads per row copy its 128 bytes into the places of the 128-byte swizzle.
      const int tid = 32 * wr + lane;
      const int chunk = tid & 7, row0 = tid >> 3;
      const long long row_bytes = kFp4 ? a.K / 2 : 2LL * a.K;
      const uint32_t dst0 = x_part + row0 * kStageKBytes + ((chunk ^ (row0 & 7)) << 4);
      for (int t = t_first; t < tiles_total && ok; t += t_step) {
        const Tile tl = find_tile(sb, a, t, kCtas * width, lane);
        const int half = (tl.n + kGrain - 1) / kGrain * 16;  // rows that this CTA stages
        const int steps = (half + kStepRows - 1) / kStepRows;
        auto mine = [&](int i) { return i < steps && (kStepRows == 16 || kStepRows * i + row0 < half); };
        const uint8_t* src[kSteps];
        uint32_t has = 0;  // zeros behind the tile's last row: no request
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int r = rank * half + kStepRows * i + row0;
          src[i] = a.x;
          if (mine(i) && r < tl.n) {
            int id = __ldg(a.row_token + tl.r0 + r);
            if (id < 0 || id >= a.x_rows) {
              raise_status(a.status, kStatusBadLen);
              id = 0;
            }
            src[i] += id * row_bytes + 16 * chunk;
            has |= 1u << i;
          }
        }
        for (int kb = 0; kb < k_steps; ++kb, p.next(stages)) {
          if (p.round != 0)
            ok = wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
          if (!ok) break;
          const int blocks = kPair ? 1 : min(sub, k_blocks - kb * sub);
#pragma unroll 1
          for (int u = 0; u == 0 || (!kPair && u < blocks); ++u) {
            const int at = (kb * sub + u) * kStageKBytes;
            const bool data = at + 16 * chunk < row_bytes;  // zeros past the row's end
            const uint32_t dst = ring + p.stage * stage_size + dst0 + u * stage_rows * kStageKBytes;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
              if (mine(i)) {
                const bool read = data && (has >> i & 1);
                copy_async16(dst + i * kStepRows * kStageKBytes, src[i] + (read ? at : 0), read ? 16 : 0);
              }
          }
          copy_async_arrive(smem_u32(&sb.landed[p.stage]));
        }
      }
      copy_async_wait_all();
    } else if (kFp4 || wr < kRowWarps) {
      // Boxes of rows, whole stages in turns: a report to the leading CTA's barrier keeps its warp
      // about 220 cycles, a copy's issue 100 and more.
      constexpr int kBox = kPair ? C::kRows / 4 : kBoxRows;
      for (int t = t_first; t < tiles_total && ok; t += t_step, g += k_steps) {
        const Tile tl = find_tile(sb, a, t, kCtas * width, lane);
        const int half = (tl.n + kGrain - 1) / kGrain * 16;  // rows that this CTA stages
        const int units = (half + kBox - 1) / kBox;          // at most 2 in a pair
        const int u = kPair ? 0 : lane / units, unit = lane - u * units;
        const int row0 = tl.r0 + rank * half;
        int at = 0;
        for (int kb = (wr - g) & (kTurns - 1); kb < k_steps; kb += kTurns) {
          p.skip(kb - at, stages);
          at = kb;
          if (p.round != 0)
            ok = wait_or_abort(smem_u32(&sb.empty[p.stage]), (p.round - 1) & 1, a.timeout_ns, abort_flag);
          if (!ok) break;
          const int boxes = (kPair ? 1 : min(sub, k_blocks - kb * sub)) * units;
          const uint32_t bar = full0 + 8 * p.stage, dst = ring + p.stage * stage_size + x_part;
          if constexpr (kPair) {
            if (elect_one()) {
              const int x = kb * (kFp4 ? kStageKBytes : kStageKBytes / 2);
              tma_load_rows<true>(dst, &xmap, x, row0, bar);
              if (units > 1) tma_load_rows<true>(dst + kBox * kStageKBytes, &xmap, x, row0 + kBox, bar);
              grp_arrive_expect_tx<true>(bar, boxes * kBox * kStageKBytes);
            }
          } else {
            if (lane < boxes)
              tma_load_rows<false>(dst + (u * stage_rows + unit * kBox) * kStageKBytes, &xmap,
                                   (kb * sub + u) * (kFp4 ? kStageKBytes : kStageKBytes / 2), row0 + kBox * unit, bar);
            __syncwarp();
            if (elect_one()) grp_arrive_expect_tx<false>(bar, boxes * kBox * kStageKBytes);
          }
          __syncwarp();
          done = g + kb + 1;
        }
        p.skip(k_steps - at, stages);
      }
    }
    if (lane == 0) {
      if (!ok) raise_status(a.status, kStatusTimeout);
      if (kFp4 || wr < kTurns) sb.issued[1 + wr] = done;
    }
  } else if (warp >= kEpiWarp0) {
    const int half = (warp - kEpiWarp0) >> 2;  // the two warps of a lane quarter take turns of 32 columns
    const int q = warp & 3;                    // TMEM lane quarter (a warp reaches lanes 32 (warp % 4) ..)
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    // Rows of 16-byte pieces where the output allows them: the fragment's threads hold pairs of
    // rows (columns) of a feature (lane), an 8 x 8 transposition through this warp's 512 bytes
    // of shared memory makes eight features of a row of them.
    uint8_t* patch = tiles + S::kRingBytes + S::kRawBytes + (warp - kEpiWarp0) * kPatchBytes;
    const uint32_t patch0 = smem_u32(patch);
    const int fr = lane >> 2;
    // pieces of a row in the patch: 4 (2 with SwiGLU), at places that spread over the banks
    const uint32_t put = kSwiglu ? patch0 + ((lane >> 4) * 8 + (lane & 7)) * 32 +
                                       ((((lane >> 3) & 1) ^ ((lane >> 2) & 1)) << 4)
                                 : patch0 + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
    const uint8_t* get = kSwiglu ? patch + (lane >> 1) * 32 + (((lane & 1) ^ ((lane >> 3) & 1)) << 4)
                                 : patch + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    [[maybe_unused]] const uint64_t minus_alpha2 = f2(-a.alpha, -a.alpha);
    auto add2 = [](const uint32_t* v, float b) {  // two accumulators of one feature and its bias
      return f2_unpack(f2_add(f2(__uint_as_float(v[0]), __uint_as_float(v[1])), f2(b, b)));
    };
    const bool wide = a.n_out % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
    int i = 0;
    for (int t = t_first; t < tiles_total; t += t_step, ++i) {
      const Tile tl = find_tile(sb, a, t, kCtas * width, lane);
      const int b = i & 1;
      const int f0 = tl.f0 + rank * kFeat + 32 * q;  // first feature of this warp
      const int most = min(width - 32 * q, a.N - f0);  // features that are the tile's and exist
      const uint32_t acc = tmem + lane_base + b * C::kRows;
      const uint16_t* bias = a.bias ? a.bias + static_cast<long long>(tl.e) * a.N + f0 : nullptr;
      auto bias_of = [&](int f) {
        return bias && f < most ? __uint_as_float(static_cast<uint32_t>(__ldg(bias + f)) << 16) : 0.0f;
      };
      uint16_t* out = a.out + static_cast<long long>(tl.r0) * a.n_out + (kSwiglu ? f0 >> 1 : f0);
      if (wide) {
        const float b0 = bias_of(fr), b1 = bias_of(fr + 8), b2 = bias_of(fr + 16), b3 = bias_of(fr + 24);
        if (!wait_or_abort(smem_u32(&sb.acc_full[b]), (i >> 1) & 1, a.timeout_ns, abort_flag)) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 32 * half; c < tl.n; c += 64) {
          uint32_t lo[16], hi[16];  // features 0..15 and 16..31
          tmem_ld_16x32(acc + c, lo);
          tmem_ld_16x32(acc + (16u << 16) + c, hi);
          tc_wait_ld();
          if constexpr (kSwiglu) {
            // Gate and up are neighbouring lanes, threads 4 apart.  The one with gates (even)
            // finishes the outputs of its lower lane, the other those of its upper lane: of
            // 8 outputs, thread row fr has number fr / 2 + 4 (fr % 2).
            const bool odd = fr & 1;
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
              uint32_t m[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t* v = ((j & 1) ? hi : lo) + 4 * (2 * i2 + (j >> 1));
                const float2 l = add2(v, (j & 1) ? b2 : b0), h = add2(v + 2, (j & 1) ? b3 : b1);
                const float t0 = __shfl_xor_sync(0xffffffffu, odd ? l.x : h.x, 4);
                const float t1 = __shfl_xor_sync(0xffffffffu, odd ? l.y : h.y, 4);
                m[j] = swiglu2(odd ? t0 : l.x, odd ? t1 : l.y, odd ? h.x : t0, odd ? h.y : t1, minus_alpha2, a.limit);
              }
              store_transposed(put, m);
              __syncwarp();
              const uint4 w = *reinterpret_cast<const uint4*>(get);
              __syncwarp();
              const int row = c + 16 * i2 + (lane >> 1), f = 8 * (lane & 1);
              if (row < tl.n && 2 * f < most)  // outputs 0 4 | 1 5 | 2 6 | 3 7 put in order
                *reinterpret_cast<uint4*>(out + static_cast<long long>(row) * a.n_out + f) =
                    make_uint4(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.z, w.w, 0x5410),
                               __byte_perm(w.x, w.y, 0x7632), __byte_perm(w.z, w.w, 0x7632));
            }
          } else {
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              uint32_t m[4];
              const uint32_t *vl = lo + 4 * i4, *vh = hi + 4 * i4;
              const float2 y[4] = {add2(vl, b0), add2(vl + 2, b1), add2(vh, b2), add2(vh + 2, b3)};
#pragma unroll
              for (int j = 0; j < 4; ++j) m[j] = pack_bf16x2(y[j].x, y[j].y);
              store_transposed(put, m);
              __syncwarp();
              const uint4 w = *reinterpret_cast<const uint4*>(get);
              __syncwarp();
              const int row = c + 8 * i4 + (lane >> 2), f = 8 * (lane & 3);
              if (row < tl.n && f < most)
                *reinterpret_cast<uint4*>(out + static_cast<long long>(row) * a.n_out + f) = w;
            }
          }
        }
      } else {
        // Any N and any address: a thread per feature, 2 bytes at a time.  With few rows that costs
        // nothing (61 tokens up: within 3 %), with many what the epilogue's issue slots do: 32768
        // gathered tokens up, 5758 features beside 5760, SwiGLU 1.36 / 1.07 ms in MXFP4 and 2.79 / 2.54
        // in bf16, without it 1.16 / 1.10 and 2.64 / 2.59.
        const bool mine = lane < most;
        const float b0 = bias_of(lane);
        out += kSwiglu ? lane >> 1 : lane;
        if (!wait_or_abort(smem_u32(&sb.acc_full[b]), (i >> 1) & 1, a.timeout_ns, abort_flag)) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 16 * half; c < tl.n; c += 32) {
          uint32_t r[16];
          tmem_ld16(acc + c, r);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float y = __uint_as_float(r[j]) + b0;
            uint32_t bits;
            if constexpr (kSwiglu) {
              // both lanes of a pair compute the output, the even one stores it
              const float theirs = __shfl_xor_sync(0xffffffffu, y, 1);
              const float g = (lane & 1) ? theirs : y, u = (lane & 1) ? y : theirs;
              bits = swiglu2(g, g, u, u, minus_alpha2, a.limit);
            } else {
              bits = pack_bf16x2(y, 0.0f);
            }
            if (mine && c + j < tl.n && !(kSwiglu && (lane & 1)))
              out[static_cast<long long>(c + j) * a.n_out] = static_cast<uint16_t>(bits & 0xFFFFu);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) grp_arrive<kPair>(acc_empty0 + 8 * b);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (kFp4 && threadIdx.x == 0) {
    // scales that nobody waited for (the last ones of an aborted run)
    for (int r = 0; r < S::kRawSlots && r < sb.raw_issued; ++r) {
      const int last = sb.raw_issued - 1 - ((sb.raw_issued - 1 - r) % S::kRawSlots);
      if (!mbar_wait(smem_u32(&sb.raw_full[r]), (last / S::kRawSlots) & 1, kDrainTimeoutNs))
        raise_status(a.status, kStatusTimeout);
    }
  }
  if constexpr (kPair) cluster_sync();
  if (threadIdx.x == 0 && rank == 0) {
    // Copies still in flight land before the shared memory is released.  A stage completes once
    // every producer warp has arrived; those that gave up earlier than others are less than
    // one round of the ring behind, and their arrivals are made up for here.
    auto peer = [&](const int* v, int cta) {
      int x;
      if constexpr (kPair)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(dsmem_addr(smem_u32(v), cta)) : "memory");
      else
        x = *const_cast<const volatile int*>(v);
      return x;
    };
    auto reports = [&](int w) { return w == 0 || (w <= kTurns ? !gather : kFp4 || gather); };
    int aborted = 0, most = 0;
    for (int c = 0; c < kCtas; ++c) {
      aborted |= peer(&sb.abort_flag, c);
      for (int w = 0; w < kProducers; ++w)
        if (reports(w)) most = max(most, peer(&sb.issued[w], c));
    }
    if (aborted) {
      for (int c = 0; c < kCtas; ++c)
        for (int w = 0; w < kProducers; ++w)
          for (int g = reports(w) ? peer(&sb.issued[w], c) : most; g < most; ++g)
            if (w == 0 || (w <= kTurns ? g % kTurns == w - 1 : g % kReportTurns == w - 1 - kTurns)) grp_arrive<kPair>(full0 + 8 * (g % stages));
      for (int s = 0; s < stages && s < most; ++s) {
        const int last = most - 1 - ((most - 1 - s) % stages);
        if (!mbar_wait(smem_u32(&sb.full[s]), (last / stages) & 1, kDrainTimeoutNs))
          raise_status(a.status, kStatusTimeout);
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
    grp_tmem_dealloc<kPair>(tmem, C::kTmemCols);
  }
}

template <bool kFp4, bool kSwiglu, bool kPair>
cudaError_t launch_grouped_t(const GroupedMaps& m, const GroupedArgs& a, int sms,
                             cudaStream_t stream) {
  auto kernel = grouped_kernel<kFp4, kSwiglu, kPair>;
  // the shared-memory opt-in, once per device (host threads may race here: atomic flags,
  // and setting the attribute twice is harmless)
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes<kFp4, kPair>()));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  constexpr int kCtas = kPair ? 2 : 1;
  GroupedArgs b = a;
  // x / tiles_f = x * magic >> shift for 0 <= x < 2^30: the excess of magic over 2^shift / tiles_f
  // is below 1, so the product is off by less than 2^30 / 2^shift <= 1 / tiles_f
  int bits = 0;
  while ((1LL << bits) < a.tiles_f) ++bits;
  b.f_shift = 30 + bits;
  b.f_magic = static_cast<uint32_t>((1ull << b.f_shift) / a.tiles_f + 1);
  b.stages = stage_count<kFp4, kPair>(kPair ? kFeat : a.width, a.cap / kCtas, kPair ? 1 : a.sub);
  if (b.stages < kTurns) return cudaErrorInvalidValue;  // not with any tile that grouped_plan makes
  // no more CTAs than tiles there can be
  const long long groups = a.num_experts < a.rows ? a.num_experts : a.rows;
  const long long most = (a.rows / a.cap + groups) * a.tiles_f;
  const int slots = sms / kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((most < slots ? most : slots) * kCtas));
  cfg.blockDim = dim3(GrpCfg<kFp4>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<kFp4, kPair>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, m.w, m.x, m.w_scales, m.x_scales, b);
}

template <bool kFp4>
cudaError_t launch_grouped_f(const GroupedMaps& m, const GroupedArgs& a, int sms,
                             cudaStream_t stream) {
  if (a.pair)
    return a.swiglu ? launch_grouped_t<kFp4, true, true>(m, a, sms, stream)
                    : launch_grouped_t<kFp4, false, true>(m, a, sms, stream);
  return a.swiglu ? launch_grouped_t<kFp4, true, false>(m, a, sms, stream)
                  : launch_grouped_t<kFp4, false, false>(m, a, sms, stream);
}

}  // namespace

void grouped_plan(GroupedArgs& a, bool mxfp4, int sms) {
  // More than 48 rows per expert on average: CTA pairs, which stage a tile's rows once for 256
  // features.  Fewer: single CTAs and small tiles, so that the ring's stages are small and many
  // and keep more weight bytes in flight.  (32 equal experts, 2880 -> 5760, us single / pair:
  // 40 rows bf16 162 / 167, MXFP4 55 / 54; 96 rows, two row tiles of single CTAs, 197 / 172 and
  // 89 / 57.  Groups of uneven size pass 64 rows, a single CTA's most, before their average does.)
  // The number of tiles is not part of the rule, so few experts leave SMs idle: one matrix of 2880 ->
  // 5120 in MXFP4 makes 20 pair tiles of 49 to 224 rows, 40 SMs' work (48 rows 9.3 us, 64 rows 10.9,
  // 224 rows 12.3, 1024 rows 17.6).
  a.pair = a.rows > 48LL * a.num_experts;
  a.cap = a.pair ? (mxfp4 ? GrpCfg<true>::kRows : GrpCfg<false>::kRows) : a.rows > 2LL * a.num_experts ? kMaxSingleRows : 16;
  a.width = kFeat;
  a.sub = 1;
  if (!a.pair) {
    // The width that lets the last round of tiles end soonest, were every group one row tile;
    // a tile costs about as much as 48 features more.  (One token, four experts, 2880 -> 5760:
    // 80 features, 288 tiles in two rounds, instead of 180 tiles of 128 in two.)
    const long long groups = a.num_experts < a.rows ? a.num_experts : a.rows;
    long long best = -1;
    for (int w = kFeat; w >= 64; w -= 16) {
      const long long tiles = groups * ((static_cast<long long>(a.N) + w - 1) / w);
      const long long cost = (tiles + sms - 1) / sms * (w + 48);
      if (best < 0 || cost < best) {
        best = cost;
        a.width = w;
      }
    }
    // as many blocks of K per stage as leave four stages: with few rows a stage costs its
    // barriers (about 0.1 us) more than its MMAs
    auto count = [&](int sub) {
      return mxfp4 ? stage_count<true, false>(a.width, a.cap, sub) : stage_count<false, false>(a.width, a.cap, sub);
    };
    for (const int most = mxfp4 ? 2 : 4; a.sub < most && count(2 * a.sub) >= 4;) a.sub *= 2;
  }
  const int features = a.pair ? 2 * kFeat : a.width;
  a.tiles_f = static_cast<int>((static_cast<long long>(a.N) + features - 1) / features);
}

cudaError_t launch_grouped(const GroupedMaps& m, const GroupedArgs& a, bool mxfp4, int sms, cudaStream_t stream) {
  return mxfp4 ? launch_grouped_f<true>(m, a, sms, stream) : launch_grouped_f<false>(m, a, sms, stream);
}

}  // namespace sa
