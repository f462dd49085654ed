// Matrix products grouped by expert, out[r, j] = sum_i x[row_token[r], i] w[e, j, i] + b[e, j]
// for the rows r of expert e, on the 5th-generation tensor cores, with operands in bf16 or
// MXFP4 and an optional clamped SwiGLU on interleaved gate / up features (the experts of the
// page "GPT-OSS on day 0": SwiGLU, bias terms; the models' own format is MXFP4).
//
// Orientation.  The group sizes are ragged and often tiny (a decode step gives an expert one
// or two rows), while the features are many and fixed, so the weights are the A operand (M =
// 128 features per MMA) and the rows the B operand, whose N is chosen per tile: a tile of n
// rows issues MMAs of N = n rounded up to 16 and loads only those rows.  Transposed this way
// no tensor work is padded beyond 16 rows, and one kernel serves one row and thousands.
//
// A tile is two 128-feature sub-tiles (the gate and the up features of the same 128 outputs
// with SwiGLU: a thread then holds both in its own TMEM lane) by up to kRows rows, so each
// staged row feeds 256 features.  Persistent kernel, one CTA per SM, 384 threads:
//   warp 0        producer: the sub-tiles' weight boxes (128 features x 128 bytes) and the
//                 rows, gathered four per TMA instruction by their indices (a lane keeps the
//                 four indices it issues) or in boxes of 16 consecutive rows; 128-byte
//                 swizzle, into a kStages-deep ring
//   warp 1        TMEM owner and MMA issuer (one elected thread): 32 bytes of K per MMA
//   warp 2        MXFP4: reads the scale bytes (16 per row: two stages), writes them into the
//                 ring in the layout that tcgen05.cp spreads over TMEM (row r of a block of
//                 128: 4 bytes at 16 (r % 32) + 4 (r / 32), 512 bytes per 128 values of K)
//   warps 4..11   epilogue: thread = one feature (TMEM lane), columns = rows; bias and
//                 activation in fp32, one rounding; a warp writes 64 consecutive bytes per row
// Two TMEM accumulators alternate, so the epilogue of a tile overlaps the next tile's MMAs.
//
// Tiles are numbered by expert, then feature tile, then row tile: the row tiles of one weight
// tile run at the same time and share it through L2, so weights come from memory once.  An
// expert's rows are split evenly among its row tiles.  Each CTA derives the numbering from
// the offsets in device memory (a prefix sum over at most 256 experts).
#include <atomic>
#include <cstdint>

#include "grouped_args.h"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr int kFeat = kGroupedFeatures;
constexpr int kStageKBytes = 128;  // bytes of K per ring stage: 64 bf16 or 256 E2M1 values
constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr unsigned long long kDrainTimeoutNs = 2000000000ull;

template <bool kFp4>
struct GrpCfg {
  // 4 accumulators of kRows columns (two buffers of two sub-tiles), MXFP4 scales beside them
  static constexpr int kRows = kFp4 ? 112 : 128;
  static constexpr int kSubBytes = kFeat * kStageKBytes;
  static constexpr int kWBytes = 2 * kSubBytes;
  static constexpr int kXBytes = kRows * kStageKBytes;
  static constexpr int kSfBlock = 512;                         // 128 rows x 4 scale bytes
  static constexpr int kSfBytes = kFp4 ? 2 * 3 * kSfBlock : 0;  // per 128 values of K: two weight blocks, one of rows
  static constexpr int kStageBytes = kWBytes + kXBytes + kSfBytes;
  static constexpr int kStages = 4;
  static constexpr int kStageK = kFp4 ? 256 : 64;
  static constexpr int kTmemCols = 512;
  static_assert(kStageBytes % 1024 == 0 && kXBytes % 1024 == 0, "stages keep the swizzle atom's alignment");
  static_assert(4 * kRows + (kFp4 ? 2 * 24 : 0) <= kTmemCols, "TMEM holds 512 columns");
};

struct GrpShared {
  uint64_t full[8], empty[8], sf_full[8], acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
  int issued;
  int total;                     // row tiles of all experts
  int cum[kMaxExperts + 32];     // row tiles of lower experts (a huge number from E + 1 on)
  int start[kMaxExperts];        // first row
  int rows[kMaxExperts];
};

template <bool kFp4>
constexpr size_t smem_bytes() {
  return 1024 /*alignment slack*/ + static_cast<size_t>(GrpCfg<kFp4>::kStages) * GrpCfg<kFp4>::kStageBytes +
         sizeof(GrpShared);
}

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

// kind::f16, bf16 operands, both K-major, fp32 accumulation.
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kFeat >> 4) << 24);
}
// kind::mxf4, E2M1 operands, E8M0 scales; `sf`: which scale bytes of a TMEM word (0 or 2).
__device__ __forceinline__ uint32_t idesc_mxf4(int n, int sf) {
  return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(kFeat >> 7) << 27) | (static_cast<uint32_t>(sf) << 29);
}

__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 512 bytes (32 rows x 16) to the same four columns of all four lane quarters.
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void tma_load_w(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int e,
                                           uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(e), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Four rows of 128 bytes by their indices (the map's box is one row high).
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&r)[4],
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                              volatile int* abort_flag) {
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

struct Tile {
  int e, f0;    // expert; first output feature
  int r0, n;    // first row, number of rows
  int subs;     // 128-feature sub-tiles with data
};

// Tile t of the numbering in `sb` (all 32 lanes of a warp call this together).
__device__ __forceinline__ Tile find_tile(const GrpShared& sb, const GroupedArgs& a, int t, int rows_per_tile,
                                          int lane) {
  const int q = t / a.tiles_f;  // row tiles before it are whole experts' and at most its own expert's
  const unsigned lt = __ballot_sync(0xffffffffu, sb.cum[8 * lane] <= q);
  const int base = 8 * (__popc(lt) - 1);
  const unsigned in = __ballot_sync(0xffffffffu, lane < 8 && sb.cum[base + (lane & 7)] <= q);
  Tile r;
  r.e = base + __popc(in) - 1;
  const int local = t - sb.cum[r.e] * a.tiles_f;
  const int rows = sb.rows[r.e];
  const int count = (rows + rows_per_tile - 1) / rows_per_tile;
  const int ft = local / count, rt = local - ft * count;
  const int per = ((rows + count - 1) / count + 15) & ~15;  // an even split, in multiples of 16
  r.r0 = sb.start[r.e] + rt * per;
  const int left = rows - rt * per;
  r.n = left < per ? left : per;
  r.f0 = ft * (a.swiglu ? kFeat : kFeat * a.subs);
  r.subs = a.swiglu || (a.subs == 2 && r.f0 + kFeat < a.n_out) ? 2 : 1;
  return r;
}

__device__ __forceinline__ float swiglu(float g, float u, float alpha, float limit) {
  g = g > limit ? limit : g;  // comparisons that let NaN through
  u = u > limit ? limit : (u < -limit ? -limit : u);
  return __fdividef(g, 1.0f + __expf(-alpha * g)) * (u + 1.0f);
}

template <bool kFp4>
__global__ void __launch_bounds__(kThreads, 1)
grouped_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
               const GroupedArgs a) {
  using C = GrpCfg<kFp4>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  GrpShared& sb = *reinterpret_cast<GrpShared*>(tiles + static_cast<size_t>(C::kStages) * C::kStageBytes);
  volatile int* abort_flag = &sb.abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int k_steps = (a.K + C::kStageK - 1) / C::kStageK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&sb.full[s]), 1);
      mbar_init(smem_u32(&sb.sf_full[s]), 1);
      mbar_init(smem_u32(&sb.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sb.acc_full[b]), 1);
      mbar_init(smem_u32(&sb.acc_empty[b]), kEpiWarps);
    }
    mbar_init(smem_u32(&sb.drain), 1);
    sb.abort_flag = 0;
    sb.issued = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sb.tmem_base), C::kTmemCols);
    tmem_relinquish();
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
      sb.start[e] = lo;
      sb.rows[e] = hi - lo;
      mine[j] = sum;
      sum += (hi - lo + C::kRows - 1) / C::kRows;
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
  tc_fence_after();
  const uint32_t tmem = sb.tmem_base;
  const int tiles_total = sb.total * a.tiles_f;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&wmap);
      tma_prefetch_desc(&xmap);
    }
    int g = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles_total && ok; t += gridDim.x) {
      const Tile tl = find_tile(sb, a, t, C::kRows, lane);
      const int n16 = (tl.n + 15) & ~15;
      int id[4];
      if (a.row_token) {
        // rows behind the tile's last one repeat its first: their columns are never stored
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 4 * lane + j;
          id[j] = __ldg(a.row_token + tl.r0 + (r < tl.n ? r : 0));
          if (id[j] < 0 || id[j] >= a.x_rows) {
            raise_status(a.status, kStatusBadLen);
            id[j] = 0;
          }
        }
      }
      for (int kb = 0; kb < k_steps; ++kb, ++g) {
        const int s = g % C::kStages;
        const uint32_t bar = smem_u32(&sb.full[s]);
        const uint32_t dst = smem_u32(tiles + static_cast<size_t>(s) * C::kStageBytes);
        const int x0 = kb * (kFp4 ? kStageKBytes : kStageKBytes / 2);  // in elements of the maps
        if (lane == 0) {
          ok = g < C::kStages ||
               wait_or_abort(smem_u32(&sb.empty[s]), ((g / C::kStages) - 1) & 1, a.timeout_ns, abort_flag);
          if (ok) {
            mbar_arrive_expect_tx(bar, tl.subs * C::kSubBytes + n16 * kStageKBytes);
            for (int sub = 0; sub < tl.subs; ++sub)  // features past N are zero-filled
              tma_load_w(dst + sub * C::kSubBytes, &wmap, x0, a.swiglu ? sub : 0,
                         a.swiglu ? tl.f0 : tl.f0 + sub * kFeat, tl.e, bar);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        if (a.row_token) {
          if (4 * lane < n16) tma_gather4(dst + C::kWBytes + lane * 4 * kStageKBytes, &xmap, x0, id, bar);
        } else {
          if (16 * lane < n16)
            tma_load_rows(dst + C::kWBytes + lane * 16 * kStageKBytes, &xmap, x0, tl.r0 + 16 * lane, bar);
        }
        __syncwarp();
        if (lane == 0) sb.issued = g + 1;
      }
    }
    if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
  } else if (warp == 1) {
    int g = 0, i = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles_total && ok; t += gridDim.x, ++i) {
      const Tile tl = find_tile(sb, a, t, C::kRows, lane);
      if (lane == 0) {
        const int n16 = (tl.n + 15) & ~15;
        const int b = i & 1;
        ok = i < 2 || wait_or_abort(smem_u32(&sb.acc_empty[b]), ((i >> 1) - 1) & 1, a.timeout_ns, abort_flag);
        tc_fence_after();
        const uint32_t d = tmem + b * 2 * C::kRows;
        for (int kb = 0; kb < k_steps && ok; ++kb) {
          const int s = (g + kb) % C::kStages;
          const uint32_t parity = ((g + kb) / C::kStages) & 1;
          ok = wait_or_abort(smem_u32(&sb.full[s]), parity, a.timeout_ns, abort_flag);
          if (kFp4 && ok) ok = wait_or_abort(smem_u32(&sb.sf_full[s]), parity, a.timeout_ns, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t w_addr = smem_u32(tiles + static_cast<size_t>(s) * C::kStageBytes);
          const uint32_t x_addr = w_addr + C::kWBytes;
          if constexpr (kFp4) {
            // this stage's scales: per 128 values of K the weight blocks and the rows' block
            const uint32_t sf = tmem + 4 * C::kRows + ((g + kb) & 1) * 24;
            const uint32_t sf_addr = x_addr + C::kXBytes;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int blk = 0; blk < 3; ++blk)
                tc_cp_scales(sf + 12 * c + 4 * blk, scale_desc(sf_addr + (3 * c + blk) * C::kSfBlock));
            const int left = (a.K - kb * C::kStageK + 63) / 64;  // 64-value steps with data
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk >= left) break;
              const uint32_t sfk = sf + 12 * (kk >> 1);
              const uint32_t idesc = idesc_mxf4(n16, 2 * (kk & 1));
              for (int sub = 0; sub < tl.subs; ++sub)
                tc_mma_mxf4(d + sub * C::kRows, sw128_kmajor_desc(w_addr + sub * C::kSubBytes + kk * 32),
                            sw128_kmajor_desc(x_addr + kk * 32), idesc, sfk + 4 * sub, sfk + 8, (kb | kk) != 0);
            }
          } else {
            const uint32_t idesc = idesc_bf16(n16);
            const int left = (a.K - kb * C::kStageK + 15) / 16;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk >= left) break;
              for (int sub = 0; sub < tl.subs; ++sub)
                tc_mma_ss(d + sub * C::kRows, sw128_kmajor_desc(w_addr + sub * C::kSubBytes + kk * 32),
                          sw128_kmajor_desc(x_addr + kk * 32), idesc, (kb | kk) != 0);
            }
          }
          tc_commit(smem_u32(&sb.empty[s]));
        }
        if (ok) tc_commit(smem_u32(&sb.acc_full[b]));
      }
      g += k_steps;
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    if (lane == 0) {
      if (!ok) raise_status(a.status, kStatusTimeout);
      // every MMA issued by this thread has finished before TMEM is released
      tc_commit(smem_u32(&sb.drain));
      if (!mbar_wait(smem_u32(&sb.drain), 0, kDrainTimeoutNs)) raise_status(a.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (kFp4 && warp == 2) {
    // Scale bytes: a lane keeps rows lane, lane + 32, lane + 64, lane + 96 of each block of
    // 128; 16 bytes of a row serve two stages, the next 16 are requested one pair ahead.
    const int blocks = (a.K + 31) / 32;  // scale bytes in use
    int g = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles_total && ok; t += gridDim.x) {
      const Tile tl = find_tile(sb, a, t, C::kRows, lane);
      const uint8_t* src[3][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 32 * j + lane;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const int f = a.swiglu ? tl.f0 + r : tl.f0 + sub * kFeat + r;  // output feature
          const bool in = sub < tl.subs && f < a.n_out;
          const long long row = static_cast<long long>(tl.e) * a.N + (a.swiglu ? 2 * f + sub : f);
          src[sub][j] = in ? a.w_scales + row * a.scale_stride : nullptr;
        }
        src[2][j] = nullptr;
        if (r < tl.n) {
          long long row = tl.r0 + r;
          if (a.row_token) {
            const int id = __ldg(a.row_token + tl.r0 + r);
            row = id < 0 || id >= a.x_rows ? 0 : id;  // reported by the producer
          }
          src[2][j] = a.x_scales + row * a.scale_stride;
        }
      }
      uint4 next[3][4];
      auto request = [&](int pair) {
#pragma unroll
        for (int blk = 0; blk < 3; ++blk)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            next[blk][j] = make_uint4(0, 0, 0, 0);
            if (src[blk][j]) next[blk][j] = __ldg(reinterpret_cast<const uint4*>(src[blk][j]) + pair);
          }
      };
      request(0);
      for (int kb = 0; kb < k_steps && ok; kb += 2) {
        uint4 cur[3][4];
        // bytes past K / 32 are padding, whatever they hold
        uint32_t mask[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int valid = blocks - 8 * kb - 4 * w;
          mask[w] = valid >= 4 ? 0xFFFFFFFFu : valid <= 0 ? 0u : (1u << (8 * valid)) - 1u;
        }
#pragma unroll
        for (int blk = 0; blk < 3; ++blk)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            cur[blk][j] = make_uint4(next[blk][j].x & mask[0], next[blk][j].y & mask[1], next[blk][j].z & mask[2],
                                     next[blk][j].w & mask[3]);
        if (kb + 2 < k_steps) request((kb + 2) / 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kb + h >= k_steps) break;
          const int gs = g + kb + h, s = gs % C::kStages;
          if (lane == 0)
            ok = gs < C::kStages ||
                 wait_or_abort(smem_u32(&sb.empty[s]), ((gs / C::kStages) - 1) & 1, a.timeout_ns, abort_flag);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          uint8_t* sf = tiles + static_cast<size_t>(s) * C::kStageBytes + C::kWBytes + C::kXBytes;
#pragma unroll
          for (int blk = 0; blk < 3; ++blk) {
            const uint4* c = cur[blk];
            reinterpret_cast<uint4*>(sf + blk * C::kSfBlock)[lane] =
                h == 0 ? make_uint4(c[0].x, c[1].x, c[2].x, c[3].x) : make_uint4(c[0].z, c[1].z, c[2].z, c[3].z);
            reinterpret_cast<uint4*>(sf + (3 + blk) * C::kSfBlock)[lane] =
                h == 0 ? make_uint4(c[0].y, c[1].y, c[2].y, c[3].y) : make_uint4(c[0].w, c[1].w, c[2].w, c[3].w);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sb.sf_full[s]));
        }
      }
      g += k_steps;
    }
    if (!ok && lane == 0) raise_status(a.status, kStatusTimeout);
  } else if (warp >= kEpiWarp0) {
    const int half = (warp - kEpiWarp0) >> 2;
    const int q = warp & 3;  // TMEM lane quarter (a warp reaches lanes 32 (warp % 4) ..)
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    int i = 0;
    for (int t = blockIdx.x; t < tiles_total; t += gridDim.x, ++i) {
      const Tile tl = find_tile(sb, a, t, C::kRows, lane);
      const int b = i & 1;
      // columns of this warp: with SwiGLU and with one sub-tile the halves take turns of
      // 16 columns, with two plain sub-tiles each half has one
      const bool split = a.swiglu || tl.subs == 1;
      const int sub = split ? 0 : half;
      const int f = tl.f0 + sub * kFeat + 32 * q + lane;
      const bool mine = f < a.n_out;
      float b0 = 0.0f, b1 = 0.0f;
      if (a.bias && mine) {
        const uint16_t* bias = a.bias + static_cast<long long>(tl.e) * a.N;
        if (a.swiglu) {
          b0 = __uint_as_float(static_cast<uint32_t>(__ldg(bias + 2 * f)) << 16);
          b1 = __uint_as_float(static_cast<uint32_t>(__ldg(bias + 2 * f + 1)) << 16);
        } else {
          b0 = __uint_as_float(static_cast<uint32_t>(__ldg(bias + f)) << 16);
        }
      }
      uint16_t* out = a.out + static_cast<long long>(tl.r0) * a.n_out + f;
      bool ok = true;
      if (lane == 0) ok = wait_or_abort(smem_u32(&sb.acc_full[b]), (i >> 1) & 1, a.timeout_ns, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + lane_base + b * 2 * C::kRows + sub * C::kRows;
#pragma unroll 1
      for (int c = split ? 16 * half : 0; c < tl.n; c += split ? 32 : 16) {
        uint32_t r[16], u[16];
        tmem_ld16(acc + c, r);
        if (a.swiglu) tmem_ld16(acc + C::kRows + c, u);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float y = __uint_as_float(r[j]) + b0;
          if (a.swiglu) y = swiglu(y, __uint_as_float(u[j]) + b1, a.alpha, a.limit);
          if (mine && c + j < tl.n)
            out[static_cast<long long>(c + j) * a.n_out] = static_cast<uint16_t>(pack_bf16x2(y, 0.0f) & 0xFFFFu);
        }
      }
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
    for (int s = 0; s < C::kStages && s < issued; ++s) {
      const int last = issued - 1 - ((issued - 1 - s) % C::kStages);
      if (!mbar_wait(smem_u32(&sb.full[s]), (last / C::kStages) & 1, kDrainTimeoutNs))
        raise_status(a.status, kStatusTimeout);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <bool kFp4>
cudaError_t launch_grouped_t(const CUtensorMap& wmap, const CUtensorMap& xmap, const GroupedArgs& a, int sms,
                             cudaStream_t stream) {
  // the shared-memory opt-in, once per device (host threads may race here: atomic flags,
  // and setting the attribute twice is harmless)
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(grouped_kernel<kFp4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes<kFp4>()));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  // no more CTAs than tiles there can be
  constexpr int kRows = GrpCfg<kFp4>::kRows;
  const long long groups = a.num_experts < a.rows ? a.num_experts : a.rows;
  const long long most = (a.rows / kRows + groups) * a.tiles_f;
  const int grid = static_cast<int>(most < sms ? most : sms);
  grouped_kernel<kFp4><<<grid, kThreads, smem_bytes<kFp4>(), stream>>>(wmap, xmap, a);
  return cudaGetLastError();
}

}  // namespace

int grouped_tile_rows(bool mxfp4) { return mxfp4 ? GrpCfg<true>::kRows : GrpCfg<false>::kRows; }

cudaError_t launch_grouped(const CUtensorMap& wmap, const CUtensorMap& xmap, const GroupedArgs& a, bool mxfp4,
                           int sms, cudaStream_t stream) {
  return mxfp4 ? launch_grouped_t<true>(wmap, xmap, a, sms, stream)
               : launch_grouped_t<false>(wmap, xmap, a, sms, stream);
}

}  // namespace sa
