// Grouping of (token, expert) pairs by expert and the weighted sum of the experts' outputs
// (the two ends of the expert layer; the page "GPT-OSS on day 0" names the router's indices
// and weights that they consume, and a combine by weighted accumulation).
#include <cstdint>

#include "experts_args.h"
#include "grouped_args.h"
#include "ptx.cuh"

namespace sa {
namespace {

// ----------------------------------------------------------------------------- grouping
// Stable counting sort in one launch.  A pair's row is (pairs of lower experts) + (pairs of its
// expert in earlier ranges, earlier warps, earlier steps of its warp, lower lanes): no counter
// is shared between warps that write rows, so the order never depends on timing.
//
// Few pairs: one CTA.  Many: 8 clusters of 8 CTAs.  The pairs are cut into 8 segments, one per
// cluster, and each segment into 8 ranges, one per CTA.  Every cluster counts all pairs (its
// CTA r counts segment r), so it knows what the segments before its own hold without waiting
// for another cluster; then each CTA counts its own range per warp, and the ranges' counts are
// exchanged through distributed shared memory.  131072 pairs take 10 us (20 on one cluster), bound
// by latency: 6.8 until the counts are exchanged (launch, two passes of counting in shared memory,
// the clusters' barrier), 3.1 for the rows, of which 0.3 are the scattered 4-byte writes of row_token
// and 0.6 the rounds of a batch that have no pairs (a warp has 64, a batch 256).  256 pairs take 4,
// most of it the launch.
constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kGroupCluster = 8;
constexpr int kBatch = 8;  // index loads in flight per lane

__global__ void __launch_bounds__(kGroupThreads, 1) group_rows_kernel(const GroupRowsArgs a, int cluster, int seg) {
  __shared__ int cnt[kGroupWarps][kMaxExperts];  // per warp: counts, then the next row of each expert
  __shared__ int seg_tot[kMaxExperts];           // counts of segment `rank` (read by the cluster)
  __shared__ int tot[kMaxExperts];               // counts of this CTA's range (read by the cluster)
  __shared__ int scan[kMaxExperts / 32];
  __shared__ int total_rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int mine = cluster > 1 ? blockIdx.x / kGroupCluster : 0;  // this cluster's segment
  const int E = a.num_experts;
  const long long range = static_cast<long long>(kGroupWarps) * seg, segment = range * kGroupCluster;

  bool bad = false;
  auto load = [&](int p0, int end, int (&e)[kBatch]) {  // -1: no pair, or a pair without expert
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = p0 + 32 * i + lane;
      e[i] = p < end ? __ldg(a.topk_idx + p) : -1;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (e[i] >= E) bad = true;
      if (e[i] < 0 || e[i] >= E) e[i] = -1;
    }
  };
  auto clip = [&](long long p) { return static_cast<int>(p < a.pairs ? p : a.pairs); };
  // counts of the pairs [begin, end) in this warp's row
  auto count = [&](int begin, int end) {
    for (int p0 = begin; p0 < end; p0 += 32 * kBatch) {
      int e[kBatch];
      load(p0, end, e);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (e[i] >= 0) atomicAdd(&cnt[warp][e[i]], 1);
    }
  };
  auto clear = [&]() {
    for (int i = threadIdx.x; i < kGroupWarps * kMaxExperts; i += kGroupThreads) (&cnt[0][0])[i] = 0;
  };
  // cnt -> exclusive prefix over the warps; returns the sum
  auto over_warps = [&]() {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < kGroupWarps; ++w) {
      const int c = cnt[w][threadIdx.x];
      cnt[w][threadIdx.x] = sum;
      sum += c;
    }
    return sum;
  };
  // v[threadIdx.x] of all CTAs of the cluster
  auto of_cluster = [&](const int* v, int (&c)[kGroupCluster]) {
    const uint32_t at = smem_u32(v + threadIdx.x);
#pragma unroll
    for (int r = 0; r < kGroupCluster; ++r)
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c[r]) : "r"(dsmem_addr(at, r)) : "memory");
  };

  const long long first = mine * segment + rank * range + static_cast<long long>(warp) * seg;
  const int begin = clip(first), end = clip(first + seg);
  clear();
  __syncthreads();
  int before = 0, all = 0;  // of expert threadIdx.x: pairs ahead of this CTA's range, and pairs in all
  if (cluster > 1) {
    const long long piece = segment / kGroupWarps;  // a multiple of 32
    count(clip(rank * segment + warp * piece), clip(rank * segment + (warp + 1) * piece));
    __syncthreads();
    if (threadIdx.x < kMaxExperts) seg_tot[threadIdx.x] = over_warps();
    __syncthreads();
    clear();
    __syncthreads();
  }
  count(begin, end);
  if (bad) raise_status(a.status, kStatusBadLen);
  __syncthreads();
  if (threadIdx.x < kMaxExperts) tot[threadIdx.x] = all = over_warps();
  if (cluster > 1) {
    cluster_sync();
    if (threadIdx.x < kMaxExperts) {
      int s[kGroupCluster], r[kGroupCluster];
      of_cluster(seg_tot, s);
      of_cluster(tot, r);
      all = 0;
#pragma unroll
      for (int i = 0; i < kGroupCluster; ++i) {
        all += s[i];
        before += (i < mine ? s[i] : 0) + (i < rank ? r[i] : 0);
      }
    }
  }
  // exclusive prefix over the experts
  int incl = all;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31 && warp < kMaxExperts / 32) scan[warp] = incl;
  __syncthreads();
  if (threadIdx.x < kMaxExperts) {
    int base = 0;
    for (int w = 0; w < warp; ++w) base += scan[w];
    const int off = base + incl - all;
    if (blockIdx.x == 0 && threadIdx.x < E) a.offsets[threadIdx.x] = off;
    if (threadIdx.x == kMaxExperts - 1) {
      total_rows = base + incl;
      if (blockIdx.x == 0) a.offsets[E] = base + incl;
    }
#pragma unroll 8
    for (int w = 0; w < kGroupWarps; ++w) cnt[w][threadIdx.x] += off + before;
  }
  __syncthreads();
  // Both sums of the other CTAs are in this one's shared memory now, so they have been read: no CTA
  // may leave before that is so of all.  (An arrival does not wait for loads under way; `before` has
  // its first use just above.)
  if (cluster > 1) cluster_arrive_relaxed();

  const unsigned below = (1u << lane) - 1u;
  for (int p0 = begin; p0 < end; p0 += 32 * kBatch) {
    int e[kBatch];
    load(p0, end, e);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = p0 + 32 * i + lane;
      const unsigned same = __match_any_sync(0xffffffffu, e[i]);
      int row = -1;
      if (e[i] >= 0) row = cnt[warp][e[i]] + __popc(same & below);
      __syncwarp();
      if (e[i] >= 0 && (same & below) == 0) cnt[warp][e[i]] += __popc(same);
      __syncwarp();
      if (p < end) a.pair_row[p] = row;
      if (row >= 0) a.row_token[row] = p / a.top_k;
    }
  }
  // rows that no pair has
  for (long long r = total_rows + static_cast<long long>(blockIdx.x) * kGroupThreads + threadIdx.x; r < a.pairs;
       r += static_cast<long long>(gridDim.x) * kGroupThreads)
    a.row_token[r] = -1;
  __syncwarp();
  if (cluster > 1) cluster_wait();
}

// ----------------------------------------------------------------------------- combine
// One thread per 8 columns of a token: its top_k row pieces are requested together (16 bytes
// each, coalesced along the row), summed in fp32 in slot order and rounded once.  Bound by memory:
// 32768 tokens, 4 rows of 2880 each, 140 us = 6.75 TB/s, the rate of a copy.
template <int K>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a) {
  const int vecs = a.hidden / 8;
  const long long total = static_cast<long long>(a.num_tokens) * vecs;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long step_t = step / vecs;
  const int step_c = static_cast<int>(step - step_t * vecs);
  long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (GridWalk at(i, vecs); i < total; i += step, at.advance(step_t, step_c, vecs)) {
    const long long t = at.row;
    const int c = at.col;
    int row[K];
    float w[K];
    uint4 v[K];
#pragma unroll
    for (int r = 0; r < K; ++r) {
      row[r] = __ldg(a.pair_row + t * K + r);
      w[r] = __uint_as_float(static_cast<uint32_t>(__ldg(a.weight + t * K + r)) << 16);
    }
#pragma unroll
    for (int r = 0; r < K; ++r) {
      if (row[r] < -1 || row[r] >= a.num_rows) {
        raise_status(a.status, kStatusBadLen);
        row[r] = -1;
      }
      if (row[r] >= 0)
        v[r] = __ldg(reinterpret_cast<const uint4*>(a.y + static_cast<long long>(row[r]) * a.hidden) + c);
    }
    float s[8] = {};
#pragma unroll
    for (int r = 0; r < K; ++r) {
      if (row[r] >= 0) {
        const uint32_t u[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[2 * j] = fmaf(w[r], __uint_as_float(u[j] << 16), s[2 * j]);
          s[2 * j + 1] = fmaf(w[r], __uint_as_float(u[j] & 0xFFFF0000u), s[2 * j + 1]);
        }
      }
    }
    reinterpret_cast<uint4*>(a.out)[i] = make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]),
                                                    pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
  }
}

template <int K>
cudaError_t launch_combine_k(const CombineArgs& a, int sms, cudaStream_t stream) {
  const long long total = static_cast<long long>(a.num_tokens) * (a.hidden / 8);
  // one wave of resident blocks: 5 per SM with the registers of up to five rows, else 4
  const long long blocks = (total + 255) / 256, most = (K <= 5 ? 5LL : 4LL) * sms;
  combine_kernel<K><<<static_cast<int>(blocks < most ? blocks : most), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_group_rows(const GroupRowsArgs& a, cudaStream_t stream) {
  // one CTA up to 128 pairs per warp
  const int cluster = a.pairs <= 128 * kGroupWarps ? 1 : kGroupCluster;
  const long long warps = static_cast<long long>(cluster) * cluster * kGroupWarps;
  const int seg = static_cast<int>(((a.pairs + warps - 1) / warps + 31) / 32 * 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster * cluster);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, group_rows_kernel, a, cluster, seg);
}

cudaError_t launch_combine(const CombineArgs& a, int sms, cudaStream_t stream) {
  switch (a.top_k) {
    case 1: return launch_combine_k<1>(a, sms, stream);
    case 2: return launch_combine_k<2>(a, sms, stream);
    case 3: return launch_combine_k<3>(a, sms, stream);
    case 4: return launch_combine_k<4>(a, sms, stream);
    case 5: return launch_combine_k<5>(a, sms, stream);
    case 6: return launch_combine_k<6>(a, sms, stream);
    case 7: return launch_combine_k<7>(a, sms, stream);
    default: return launch_combine_k<8>(a, sms, stream);
  }
}

}  // namespace sa
