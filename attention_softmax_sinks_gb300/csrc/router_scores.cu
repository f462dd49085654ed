// Router by scores: per token the scores of all experts, s = sigmoid(x) or softmax(x), of which
// the top_k largest s + bias are chosen, within the top_groups best groups of experts when there
// are groups (a group's merit is the sum of its two largest s + bias); the weights are the chosen
// experts' scores without the bias, optionally divided by their sum, times a scale.  (The page
// "GPT-OSS on day 0", section "Kernels for GPT-OSS / MoE", tells this family of routers, with a
// softmax over all experts, from its own.)
//
// Which experts are chosen is a question of order, and is answered as in exact arithmetic, equal
// values in favour of the lower index:
//  - Eight lanes per token; lane j holds experts 4 (j + 8 i) + c.  What is ordered becomes a
//    32-bit key: 24 bits of fixed point and 255 - expert.  The fixed point holds x - max x in
//    [-32, 0] where there is no bias (scores and logits have the same order), else s + bias over
//    its range.  Keys sort with one min and one max per comparison: sorting networks per lane,
//    then three rounds of merging between lanes.
//  - A key is off by a few units from what it stands for.  Where two neighbours among the chosen,
//    or the last chosen and the first not chosen, or the last group kept and the first dropped are
//    closer than that and not equal in logit and bias, the token is done once more in fp64, by
//    the whole warp (one token in some thousands for logits in 32 bits).
//
// What bounds it: at many tokens the instructions (about 1000 per four tokens), not the logits'
// way from memory; at few the latency of one pass.
#include <cstdint>

#include "ptx.cuh"
#include "router_scores_args.h"

namespace sa {
namespace {

constexpr int kLanes = 8;                    // per token
constexpr int kTokens = 32 / kLanes;         // per warp
constexpr int kVecs = 256 / (4 * kLanes);    // vectors of four experts per lane
constexpr int kOwn = 4 * kVecs;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr unsigned kFull = 0xffffffffu;
// Distance of two keys' 24-bit parts above which their order is certain.  Logits: x - max is
// rounded by at most 2^-20 (half a unit), to a unit by another half, for each of the two.  Scores:
// exp2 and reciprocal err by 2^-22 and 2^-23 relative, the exponent's rounding by 2^-24 |x| e^-|x|;
// with the sums' roundings at most 2^-21.5 of a range of at least 1, 6 units, for each of the two.
constexpr uint32_t kNear = 16;
// Merits are sums of two scores and biases in fp32: the same errors, relative to their sizes.
constexpr float kNearMerit = 1.0f / (1 << 19);

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int N>
__device__ __forceinline__ void compare_exchange(uint32_t (&x)[N], int i, int j) {  // afterwards x[i] >= x[j]
  const uint32_t hi = max(x[i], x[j]);
  x[j] = min(x[i], x[j]);
  x[i] = hi;
}

// Largest first.  K = 1, 2, 4: compare-exchange networks of minimal length; 8: two sorted halves
// and an odd-even merge.
template <int K>
__device__ __forceinline__ void sort_keys(uint32_t (&x)[K]) {
  if constexpr (K == 2) compare_exchange(x, 0, 1);
  if constexpr (K >= 4) {
#pragma unroll
    for (int h = 0; h < K; h += 4) {
      compare_exchange(x, h, h + 1);
      compare_exchange(x, h + 2, h + 3);
      compare_exchange(x, h, h + 2);
      compare_exchange(x, h + 1, h + 3);
      compare_exchange(x, h + 1, h + 2);
    }
  }
  if constexpr (K == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) compare_exchange(x, i, i + 4);
    compare_exchange(x, 2, 4);
    compare_exchange(x, 3, 5);
    compare_exchange(x, 1, 2);
    compare_exchange(x, 3, 4);
    compare_exchange(x, 5, 6);
  }
}

// best <- the K largest of best and other, both sorted: the elementwise maxima against the
// reversed other are a bitonic sequence.
template <int K>
__device__ __forceinline__ void merge_keys(uint32_t (&best)[K], const uint32_t (&other)[K]) {
#pragma unroll
  for (int r = 0; r < K; ++r) best[r] = max(best[r], other[K - 1 - r]);
#pragma unroll
  for (int stride = K / 2; stride > 0; stride >>= 1)
#pragma unroll
    for (int r = 0; r < K; ++r)
      if ((r & stride) == 0) compare_exchange(best, r, r + stride);
}

// A number as the sum of two doubles, the second at most half a step of the first: s + bias
// without any rounding, so that a huge bias does not hide the scores of the experts that share it.
struct Wide {
  double hi, lo;
};
__device__ __forceinline__ Wide wide_sum(double x, double y) {
  const double s = x + y, z = s - x;
  const double e = (x - (s - z)) + (y - z);
  if (s != s) return {-__builtin_huge_val(), 0.0};  // not a number: the least
  return {s, isinf(s) ? 0.0 : e};
}
__device__ __forceinline__ bool above(const Wide& v, const Wide& w) { return v.hi > w.hi || (v.hi == w.hi && v.lo > w.lo); }
__device__ __forceinline__ Wide least() { return {-__builtin_huge_val(), 0.0}; }

struct WarpScratch {
  union {
    uint32_t key[kTokens][256];
    Wide value[256];  // the whole warp's one token, done again
  };
  Wide merit[kRouterMaxGroups];
};

__device__ __forceinline__ float load_logit(const RouterScoresArgs& a, long long t, int e) {
  const long long i = t * a.num_experts + e;
  if (a.fp32) return __ldg(static_cast<const float*>(a.logits) + i);
  return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + i)) << 16);
}

__device__ __forceinline__ float bias_of(const RouterScoresArgs& a, int e) { return a.bias ? __ldg(a.bias + e) : 0.0f; }

// Are expert e's and f's logits and biases the same (so that their order is that of the indices)?
__device__ __forceinline__ bool same_inputs(const RouterScoresArgs& a, long long t, int e, int f) {
  return load_logit(a, t, e) == load_logit(a, t, f) && bias_of(a, e) == bias_of(a, f);
}

// Token t once more, in fp64, by the whole warp.  picked[r] on every lane: the experts (some in
// range, whatever the logits are: what is not a number counts as -inf).
__device__ __noinline__ void choose_exactly(const RouterScoresArgs& a, WarpScratch& ws, long long t, int (&picked)[8]) {
  const int lane = threadIdx.x & 31;
  const int E = a.num_experts;
  double top = -__builtin_huge_val(), sum = 0.0;
  for (int e = lane; e < E; e += 32) top = fmax(top, static_cast<double>(load_logit(a, t, e)));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, off));
  const bool grouped = a.num_groups > a.top_groups;
  const bool scored = a.bias != nullptr || grouped;  // else the logits' order is the answer
  if (!a.sigmoid && scored) {
    for (int e = lane; e < E; e += 32) sum += exp(static_cast<double>(load_logit(a, t, e)) - top);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  }
  __syncwarp();
  for (int e = lane; e < E; e += 32) {
    const double x = load_logit(a, t, e);
    if (scored) ws.value[e] = wide_sum(a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum, bias_of(a, e));
    else ws.value[e] = wide_sum(x, 0.0);
  }
  __syncwarp();
  unsigned kept = kFull;
  const int size = E / a.num_groups;
  if (grouped) {
    Wide mine = least();
    if (lane < a.num_groups) {
      Wide first = least(), second = first;
      for (int i = 0; i < size; ++i) {
        const Wide v = ws.value[lane * size + i];
        if (above(v, first)) {
          second = first;
          first = v;
        } else if (above(v, second)) {
          second = v;
        }
      }
      mine = first;
      if (size > 1) {
        const Wide s = wide_sum(first.hi, second.hi);
        mine = wide_sum(s.hi, s.lo + (first.lo + second.lo));
      }
      ws.merit[lane] = mine;
    }
    __syncwarp();
    int before = 0;
    if (lane < a.num_groups)
      for (int g = 0; g < a.num_groups; ++g) before += above(ws.merit[g], mine) || (g < lane && !above(mine, ws.merit[g]));
    kept = __ballot_sync(kFull, lane < a.num_groups && before < a.top_groups);
  }
  // without a bias the logits decide between experts (scores may round to the same number)
  if (scored && a.bias == nullptr) {
    __syncwarp();
    for (int e = lane; e < E; e += 32) ws.value[e] = wide_sum(load_logit(a, t, e), 0.0);
    __syncwarp();
  }
  unsigned taken = 0;  // which of this lane's experts (lane + 32 i)
  constexpr int kNone = 1 << 20;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (r >= a.top_k) break;
    Wide best = least();
    int at = kNone;
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(taken >> i & 1) && (kept >> (grouped ? e / size : 0) & 1)) {
        const Wide v = ws.value[e];
        if (at == kNone || above(v, best)) {
          best = v;
          at = e;
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const Wide v = {__shfl_xor_sync(kFull, best.hi, off), __shfl_xor_sync(kFull, best.lo, off)};
      const int f = __shfl_xor_sync(kFull, at, off);
      if (f != kNone && (at == kNone || above(v, best) || (!above(best, v) && f < at))) {
        best = v;
        at = f;
      }
    }
    picked[r] = at;
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
  }
  __syncwarp();
}

template <int K, bool kFp32, bool kSigmoid, bool kBias>
__global__ void __launch_bounds__(256, 2) router_scores_kernel(const RouterScoresArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ int hist[256];
  __shared__ float bias_range[2];  // least finite bias, keys per unit of score
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WarpScratch& ws = reinterpret_cast<WarpScratch*>(smem_raw)[warp];
  const int E = a.num_experts, k = a.top_k;
  const int j = lane % kLanes, tok = lane / kLanes;
  const bool grouped = a.top_groups < a.num_groups;
  const int size = E / a.num_groups;
  const int inv_size = (65536 + size - 1) / size;  // e / size == (e * inv_size) >> 16 for e < 256
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  if constexpr (kBias) {
    if (warp == 0) {
      float lo = __builtin_huge_valf(), hi = kNegInf;
      for (int e = lane; e < E; e += 32) {
        const float b = __ldg(a.bias + e);
        if (fabsf(b) <= 3.4e38f) {
          lo = fminf(lo, b);
          hi = fmaxf(hi, b);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(kFull, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, off));
      }
      if (lane == 0) {
        bias_range[0] = lo <= hi ? lo : 0.0f;
        bias_range[1] = lo <= hi ? 16777000.0f / (1.0f + (hi - lo)) : 16777000.0f;
      }
    }
  }
  __syncthreads();
  const float base = kBias ? bias_range[0] : 0.0f, per_unit = kBias ? bias_range[1] : 0.0f;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const long long passes = (a.num_tokens + kTokens - 1) / kTokens;
  for (long long p = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp; p < passes; p += warps) {
    const long long t = p * kTokens + tok;
    const bool live = t < a.num_tokens;  // the lanes of a token agree
    const long long tt = live ? t : a.num_tokens - 1;
    // ---- logits
    float x[kOwn];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = 4 * (j + kLanes * i);
      if (a.vec4) {
        if (kFp32) {
          const float4 v = e < E ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + tt * E + e))
                                 : make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
          x[4 * i] = v.x;
          x[4 * i + 1] = v.y;
          x[4 * i + 2] = v.z;
          x[4 * i + 3] = v.w;
        } else {
          const uint2 v = e < E ? __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + tt * E + e))
                                : make_uint2(0xFF80FF80u, 0xFF80FF80u);
          x[4 * i] = __uint_as_float(v.x << 16);
          x[4 * i + 1] = __uint_as_float(v.x & 0xFFFF0000u);
          x[4 * i + 2] = __uint_as_float(v.y << 16);
          x[4 * i + 3] = __uint_as_float(v.y & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[4 * i + c] = e + c < E ? load_logit(a, tt, e + c) : kNegInf;
      }
    }
    // ---- maximum, and for the softmax the sum
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kOwn; ++i) top = fmaxf(top, x[i]);
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    const float ref = top == kNegInf ? 0.0f : top;
    float inv_sum = 1.0f;
    if constexpr (!kSigmoid) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) sum += ex2((x[i] - ref) * kLog2e);
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
      inv_sum = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    auto score = [&](float v) { return kSigmoid ? rcp(1.0f + ex2(-v * kLog2e)) : ex2((v - ref) * kLog2e) * inv_sum; };
    // ---- keys
    uint32_t key[kOwn];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = 4 * (j + kLanes * i);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float f;
        if constexpr (kBias) f = (score(x[4 * i + c]) + ((e + c < E ? __ldg(a.bias + e + c) : 0.0f) - base)) * per_unit;
        else f = (x[4 * i + c] - ref + 32.0f) * 524287.0f;
        const uint32_t q = __float2uint_rn(fminf(fmaxf(f, 0.0f), 16777214.0f)) + 1;  // 1 .. 2^24 - 1
        key[4 * i + c] = e + c < E ? (q << 8) | (255u - static_cast<uint32_t>(e + c)) : 0u;
      }
    }
    bool doubt = false;  // the order of two groups or experts is not certain
    // ---- groups
    if (grouped) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        *reinterpret_cast<uint4*>(&ws.key[tok][4 * (j + kLanes * i)]) =
            make_uint4(key[4 * i], key[4 * i + 1], key[4 * i + 2], key[4 * i + 3]);
      __syncwarp();
      // lane j of a token takes groups j, j + 8, ..: their two largest keys, then their merits
      float merit[kRouterMaxGroups / kLanes];
#pragma unroll
      for (int n = 0; n < kRouterMaxGroups / kLanes; ++n) {
        const int g = j + kLanes * n;
        merit[n] = kNegInf;
        if (g < a.num_groups) {
          uint32_t first = 0, second = 0;
          int at = (4 * j + tok) % size;  // lanes begin in different banks
          for (int i = 0; i < size; ++i) {
            const uint32_t v = ws.key[tok][g * size + at];
            second = max(second, min(first, v));
            first = max(first, v);
            at = at + 1 == size ? 0 : at + 1;
          }
          const int e1 = 255 - static_cast<int>(first & 255u), e2 = 255 - static_cast<int>(second & 255u);
          merit[n] = score(load_logit(a, tt, e1)) + bias_of(a, e1);
          if (size > 1) merit[n] += score(load_logit(a, tt, e2)) + bias_of(a, e2);
        }
      }
      // a group is kept if fewer than top_groups come before it
      unsigned kept = 0;
      float last_kept = __builtin_huge_valf(), first_dropped = kNegInf;
#pragma unroll
      for (int n = 0; n < kRouterMaxGroups / kLanes; ++n) {
        int before = 0;
#pragma unroll
        for (int m = 0; m < kRouterMaxGroups / kLanes; ++m) {
          if (kLanes * m < a.num_groups) {
#pragma unroll
            for (int l = 0; l < kLanes; ++l) {
              const float other = __shfl_sync(kFull, merit[m], (lane & ~(kLanes - 1)) + l);
              before += other > merit[n] || (other == merit[n] && l + kLanes * m < j + kLanes * n);
            }
          }
        }
        if (j + kLanes * n < a.num_groups) {
          if (before < a.top_groups) {
            kept |= 1u << (j + kLanes * n);
            last_kept = fminf(last_kept, merit[n]);
          } else {
            first_dropped = fmaxf(first_dropped, merit[n]);
          }
        }
        if (kLanes * (n + 1) >= a.num_groups) break;
      }
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) {
        kept |= __shfl_xor_sync(kFull, kept, off);
        last_kept = fminf(last_kept, __shfl_xor_sync(kFull, last_kept, off));
        first_dropped = fmaxf(first_dropped, __shfl_xor_sync(kFull, first_dropped, off));
      }
      // (a tie in merit is settled in fp64 as well)
      float near = kNearMerit * (1.0f + fabsf(last_kept) + fabsf(first_dropped));
      if constexpr (kBias) near += 4.0f * static_cast<float>(kNear) / per_unit;
      doubt = !(last_kept - first_dropped > near);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int e = 4 * (j + kLanes * (i >> 2)) + (i & 3);
        if (!(kept >> ((e * inv_size) >> 16) & 1)) key[i] = 0;
      }
      __syncwarp();
    }
    // ---- the K largest keys
    uint32_t best[K];
#pragma unroll
    for (int r = 0; r < K; ++r) best[r] = key[r];
    sort_keys<K>(best);
#pragma unroll
    for (int i = K; i < kOwn; i += K) {
      uint32_t part[K];
#pragma unroll
      for (int r = 0; r < K; ++r) part[r] = key[i + r];
      sort_keys<K>(part);
      merge_keys<K>(best, part);
    }
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) {
      uint32_t other[K];
#pragma unroll
      for (int r = 0; r < K; ++r) other[r] = __shfl_xor_sync(kFull, best[r], off);
      merge_keys<K>(best, other);
    }
    uint32_t last = best[0];  // the k-th
#pragma unroll
    for (int r = 1; r < K; ++r)
      if (r < k) last = best[r];
    uint32_t next = 0;  // the largest key not chosen
#pragma unroll
    for (int i = 0; i < kOwn; ++i) next = max(next, key[i] < last ? key[i] : 0u);
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) next = max(next, __shfl_xor_sync(kFull, next, off));
    // ---- neighbours too close to be certain, unless logit and bias are the same
#pragma unroll
    for (int r = 0; r < K; ++r) {
      if (r < k) {
        uint32_t below = next;
        if constexpr (K > 1)
          if (r + 1 < K && r + 1 < k) below = best[r + 1 < K ? r + 1 : r];
        if (below != 0 && (best[r] >> 8) - (below >> 8) <= kNear &&
            !same_inputs(a, tt, 255 - static_cast<int>(best[r] & 255u), 255 - static_cast<int>(below & 255u)))
          doubt = true;
      }
    }
    // ---- experts of the token, on all of its lanes
    int picked[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) picked[r] = r < K ? 255 - static_cast<int>(best[r < K ? r : 0] & 255u) : 0;
    unsigned again = __ballot_sync(kFull, doubt && live && j == 0);
    while (again) {
      const int first = __ffs(again) - 1;  // lane 0 of the token
      again &= again - 1;
      int exact[8];
      choose_exactly(a, ws, p * kTokens + first / kLanes, exact);
      if (tok == first / kLanes) {
#pragma unroll
        for (int r = 0; r < 8; ++r) picked[r] = exact[r];
      }
    }
    // ---- weights: lane j writes the j-th
    float mine = 0.0f;
    int expert = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (j == r) expert = picked[r];
    if (j < k) {
      const float v = load_logit(a, tt, expert);
      mine = kSigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - ref) * inv_sum;
    }
    float sum = mine;
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
    if (live && j < k) {
      float w = a.scale * mine;
      if (a.renormalize) w = sum > 0.0f ? a.scale * (mine / sum) : 0.0f;
      a.topk_idx[t * k + j] = expert;
      a.topk_w[t * k + j] = static_cast<uint16_t>(pack_bf16x2(w, 0.0f) & 0xFFFFu);
      if (a.counts) atomicAdd(&hist[expert], 1);
    }
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
      if (hist[e]) atomicAdd(a.counts + e, hist[e]);
  }
}

template <int K, bool kFp32, bool kSigmoid>
cudaError_t launch_scores(const RouterScoresArgs& a, int sms, cudaStream_t stream) {
  // few tokens: a warp per block, so that they spread over the SMs; else eight
  const long long passes = (a.num_tokens + kTokens - 1) / kTokens;
  const int warps = passes <= 2LL * sms ? 1 : 8;
  const long long blocks = (passes + warps - 1) / warps;
  const long long most = 4LL * sms;  // resident ones
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  const size_t smem = warps * sizeof(WarpScratch);
  if (a.bias) router_scores_kernel<K, kFp32, kSigmoid, true><<<grid, 32 * warps, smem, stream>>>(a);
  else router_scores_kernel<K, kFp32, kSigmoid, false><<<grid, 32 * warps, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int K>
cudaError_t launch_scores_k(const RouterScoresArgs& a, int sms, cudaStream_t stream) {
  if (a.fp32) return a.sigmoid ? launch_scores<K, true, true>(a, sms, stream) : launch_scores<K, true, false>(a, sms, stream);
  return a.sigmoid ? launch_scores<K, false, true>(a, sms, stream) : launch_scores<K, false, false>(a, sms, stream);
}

}  // namespace

cudaError_t launch_router_scores(const RouterScoresArgs& a, int sms, cudaStream_t stream) {
  if (a.top_k == 1) return launch_scores_k<1>(a, sms, stream);
  if (a.top_k == 2) return launch_scores_k<2>(a, sms, stream);
  if (a.top_k <= 4) return launch_scores_k<4>(a, sms, stream);
  return launch_scores_k<8>(a, sms, stream);
}

}  // namespace sa
