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
//    32-bit key: 24 bits of fixed point and 255 - expert.  The fixed point holds s + bias over its
//    range, which leaves masked experts out (bias_range; their key is 0), and all ones for a bias of +inf;
//    without bias and groups x - max x in [-32, 0] (scores and logits have the same order).
//    Keys sort with one min and one max per comparison: sorting networks per lane, then three
//    rounds of merging between lanes.  (A lane's keys differ from each other without j, which is
//    added to the few that leave the lane.)
//  - A key is off by a few units from what it stands for.  Where the last group kept and the first
//    dropped, or two neighbours among the chosen, or the last chosen and the first not chosen are
//    closer than that, and not equal in logit and bias (or, behind an equal one not chosen, any other
//    is as close), the experts within reach of that border are compared once more, a lane for
//    each: scores by sigmoid in pairs of fp32, and where that does not settle it, or by softmax, in
//    fp64 (one token in a thousand of 256 experts in 8 groups with logits in 32 bits); more than 32 of
//    them by a walk over all experts in fp64.
//
// What bounds it: at many tokens the instructions, some 1700 for four tokens of 256 experts (issue slots
// are taken 56% of the time while an SM works), and behind them the latency of the doubtful tokens and
// the last, partial round, not the logits' way from memory: 32768 tokens of 256 experts in fp32, 8 of
// them from 4 of 8 groups, by sigmoid take 29.7 us, 5.2 for the bytes alone (with 32 lanes per token 90); in
// bf16 35.4, as more of them are near one another.  By softmax 47: more scores are small and near, and
// the doubtful go to fp64; without bias and groups, where keys hold logits, 24.6, and 20.2 in bf16.
// Masked experts (1 in 16 by -inf, the least fp32 number or -1e4): 31 and 47.
// At few tokens the latency of a launch and one pass: 64 tokens 6.1 us; 25.6 with a token that has more
// than 32 experts near its border.
#include <cstdint>

#include "ptx.cuh"
#include "router_scores_args.h"

namespace sa {
namespace {

constexpr int kLanes = 8;                    // per token
constexpr int kTokens = 32 / kLanes;         // per warp
constexpr int kVecs = 256 / (4 * kLanes);    // vectors of four experts per lane
constexpr int kOwn = 4 * kVecs;
constexpr int kBlock = 256;
constexpr int kMaxDoubtful = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr unsigned kFull = 0xffffffffu;
// Distance of two keys' 24-bit parts above which their order is certain.  Logits: the key never falls
// where the logit grows, only equal keys are uncertain.  Scores, with R the range of the biases, in steps
// of a key, 2^-24 (1 + R):
//  - the bias's part (none where R = 0): b - lo by R / (1 + R), its product and the 1 added by 1/2 each;
//    the sum with the score and the conversion by 1/2 each.  2 R / (1 + R) + 4 for two keys.
//  - sigmoid: the exponent by 0.3 (|x| s (1 - s) <= 0.224), exp2 (2^-22) by 1, 1 + e^-x by 1, the reciprocal
//    by 2.  8.6 / (1 + R) for two; with the above most near R = 0, 12.6.
//  - softmax: exp2 by 4 s, but not at the maximum, the exponent by 2.25 s |x - max| <= 0.63.  4 / (1 + R)
//    for two, whose scores are 1 together at most.  The sum's relative error counts with the difference of
//    the two scores, which is that of their biases: at most min(R, 1) times 10, for the 8 roundings of
//    exp_sum and between lanes, the reciprocal and a product; and for its terms 4.2 at most (1 of exp2;
//    3.2 of the exponents, for 255 of the same).  With the above most at R = 1, 14.1.
//    (Terms added one behind the other, 34 roundings, took it to 27.)
// A merit is the sum of two.
constexpr uint32_t kNear = 16;
constexpr float kKeyRange = 16777000.0f;  // keys are 1 .. 2^24 - 1, with room for what they are off by
// Biases that differ by more than this are looked over for masks, which would leave few keys to the scores.
constexpr float kWideBias = 32.0f;

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The key of an expert with a bias of +inf (as a 24-bit key: all ones).
constexpr uint32_t kPinned = 0xffffffffu;

// 24 bits of fixed point of what is ordered, 1 .. 2^24 - 1; 0 for what is not a number and for a
// masked expert, kPinned for one with a bias of +inf (conversion to unsigned saturates).  bias_key:
// 1 + the bias's part.
template <bool kSigmoid, bool kScored>
__device__ __forceinline__ uint32_t fixed_point(float x, float ref, float unit, float soft_unit, float bias_key) {
  if constexpr (!kScored) return __float2uint_rn(fmaxf((x - ref + 32.0f) * 524287.0f, 0.0f) + 1.0f);
  if constexpr (kSigmoid) return __float2uint_rn(fmaf(rcp(1.0f + ex2(-x * kLog2e)), unit, bias_key));
  return __float2uint_rn(fmaf(ex2((x - ref) * kLog2e), soft_unit, bias_key));
}

template <bool kSigmoid>
__device__ __forceinline__ float weight_of(float x, float ref, float inv_sum) {
  return kSigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - ref) * inv_sum;
}

// The chosen experts' scores (of logits x, a token's on kLanes neighbouring lanes; -inf behind the
// k-th) and their sum, for the weights.  Renormalised weights keep their ratios where scores fall below
// fp32's range, as a bias or groups can choose experts far below the largest: there they are taken
// relative to the largest chosen one, s_i / s_m = e^(x_i - x_m) (1 + e^x_m) / (1 + e^x_i) by sigmoid, without
// the fraction by softmax.  (A sum of 1/2 or more leaves nothing above 2^-126 out.)
struct Chosen {
  float score, sum;
};
template <bool kSigmoid>
__device__ __noinline__ Chosen vanishing_scores(float x, Chosen c) {
  float top = x;
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
  float r = expf(x - top);
  if (kSigmoid) r *= (1.0f + expf(top)) / (1.0f + expf(x));
  float sum = r;
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
  return c.sum < 0.5f && top > kNegInf ? Chosen{r, sum} : c;
}
template <bool kSigmoid>
__device__ __forceinline__ Chosen chosen_scores(float x, float ref, float inv_sum, bool renormalize) {
  Chosen c;
  c.score = c.sum = weight_of<kSigmoid>(x, ref, inv_sum);
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) c.sum += __shfl_xor_sync(kFull, c.sum, off);
  if (renormalize && __any_sync(kFull, x > kNegInf && c.score < 0x1p-100f && c.sum < 0.5f)) c = vanishing_scores<kSigmoid>(x, c);
  return c;
}

// sum exp(x - ref), added in pairs: a term is rounded log2(N) times.
template <int N>
__device__ __forceinline__ float exp_sum(const float* x, float ref) {
  if constexpr (N == 1) return ex2((x[0] - ref) * kLog2e);
  else return exp_sum<N / 2>(x, ref) + exp_sum<N / 2>(x + N / 2, ref);
}

// The r-th choice of token t: its score and the sum of the chosen ones'.
__device__ __forceinline__ void write_choice(const RouterScoresArgs& a, int* hist, long long t, int r, int expert, float score,
                                             float sum) {
  float w = a.scale * score;
  if (a.renormalize) w = sum > 0.0f ? a.scale * (score / sum) : 0.0f;
  a.topk_idx[t * a.top_k + r] = expert;
  a.topk_w[t * a.top_k + r] = static_cast<uint16_t>(pack_bf16x2(w, 0.0f) & 0xFFFFu);
  if (a.counts) atomicAdd(&hist[expert], 1);
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
// The same as two integers that sort like it: comparisons of doubles take tens of cycles here.
struct Order {
  long long hi, lo;
};
__device__ __forceinline__ long long order_of(double v) {
  const long long b = __double_as_longlong(v + 0.0);  // (-0 becomes 0)
  return b ^ (b >> 63 & 0x7fffffffffffffffll);
}
__device__ __forceinline__ Order order_of(const Wide& v) { return {order_of(v.hi), order_of(v.lo)}; }
__device__ __forceinline__ bool above(const Order& v, const Order& w) { return v.hi > w.hi || (v.hi == w.hi && v.lo > w.lo); }
__device__ __forceinline__ Order order_from(const Order& v, int lane) {
  return {__shfl_sync(kFull, v.hi, lane), __shfl_sync(kFull, v.lo, lane)};
}
__device__ __forceinline__ Wide least() { return {-__builtin_huge_val(), 0.0}; }
// Merit of a group from its two largest values.
__device__ __forceinline__ Wide merit_of(const Wide& first, const Wide& second) {
  const Wide s = wide_sum(first.hi, second.hi);
  return wide_sum(s.hi, s.lo + (first.lo + second.lo));
}

// ---- The same in pairs and triples of fp32 for scores by sigmoid: a step in fp64 takes some 100
// cycles here, so that exp, the division and the comparisons of one token took 20 us.  A pair holds
// a number to 2^-46 or so of its value (sum and product of two: Dekker 1971, Knuth's two-sum).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float x, float y) {
  const float s = __fadd_rn(x, y), z = __fsub_rn(s, x);
  return {s, __fadd_rn(__fsub_rn(x, __fsub_rn(s, z)), __fsub_rn(y, z))};
}
__device__ __forceinline__ Pair quick_sum(float x, float y) {  // |x| >= |y|
  const float s = __fadd_rn(x, y);
  return {s, __fsub_rn(y, __fsub_rn(s, x))};
}
// a b + c
__device__ __forceinline__ Pair multiply_add(const Pair& a, const Pair& b, const Pair& c) {
  const float p = __fmul_rn(a.hi, b.hi);
  const float e = __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.hi, b.hi, -p)));
  const Pair s = two_sum(p, c.hi);
  return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(e, c.lo)));
}
__host__ __device__ constexpr Pair pair_of(double v) { return {static_cast<float>(v), static_cast<float>(v - static_cast<float>(v))}; }

// 1 / (1 + e^-x), off by less than 2^-43: e^-x = 2^n e^r with n ln 2 + r = -x, |r| <= 0.35, and
// the power series of e^r up to r^12 / 12! (2^-47 is left out), from r^8 on in fp32 (2^-27 of the
// sum, so 2^-50).  Below x = -60 the result is off by its value, 2^-86.
__device__ __forceinline__ Pair sigmoid_pair(float x) {
  const float y = fminf(fmaxf(-x, -60.0f), 60.0f);
  const float n = rintf(y * kLog2e);
  constexpr double kLn2 = 0.69314718055994530942, kRough = 45426.0 / 65536.0;  // n kRough is exact
  constexpr Pair rest = pair_of(kLn2 - kRough);
  const float r0 = __fmaf_rn(-n, static_cast<float>(kRough), y);  // exact as well
  const float q = __fmul_rn(n, rest.hi);
  const Pair s = two_sum(r0, -q);
  const Pair r = quick_sum(s.hi, __fsub_rn(s.lo, __fmaf_rn(n, rest.lo, __fmaf_rn(n, rest.hi, -q))));
  constexpr double c3 = 0.5 / 3, c4 = c3 / 4, c5 = c4 / 5, c6 = c5 / 6, c7 = c6 / 7, c8 = c7 / 8, c9 = c8 / 9, c10 = c9 / 10,
                   c11 = c10 / 11, c12 = c11 / 12;
  float tail = __fmaf_rn(static_cast<float>(c12), r.hi, static_cast<float>(c11));
  tail = __fmaf_rn(tail, r.hi, static_cast<float>(c10));
  tail = __fmaf_rn(tail, r.hi, static_cast<float>(c9));
  tail = __fmaf_rn(tail, r.hi, static_cast<float>(c8));
  constexpr Pair p3 = pair_of(c3), p4 = pair_of(c4), p5 = pair_of(c5), p6 = pair_of(c6), p7 = pair_of(c7);
  Pair e = multiply_add({tail, 0.0f}, r, p7);
  e = multiply_add(e, r, p6);
  e = multiply_add(e, r, p5);
  e = multiply_add(e, r, p4);
  e = multiply_add(e, r, p3);
  e = multiply_add(e, r, {0.5f, 0.0f});
  e = multiply_add(e, r, {1.0f, 0.0f});
  e = multiply_add(e, r, {1.0f, 0.0f});
  const float scale = __int_as_float((static_cast<int>(n) + 127) << 23);
  const Pair u = two_sum(1.0f, e.hi * scale);
  const Pair d = quick_sum(u.hi, __fmaf_rn(e.lo, scale, u.lo));
  const float inv = __frcp_rn(d.hi);  // one step of Newton's
  return quick_sum(inv, __fmul_rn(inv, __fmaf_rn(-d.lo, inv, __fmaf_rn(-d.hi, inv, 1.0f))));
}

// A number as a sum of three, each at most half a step of the one before: s + bias, whatever the
// bias's size, and the sum of two such.
struct Triple {
  float v0, v1, v2;
};
__device__ __forceinline__ Triple triple_of(float x0, float x1, float x2) {
  const Pair a = two_sum(x1, x2), b = two_sum(x0, a.hi), c = two_sum(b.lo, a.lo);
  return {b.hi, c.hi, c.lo};
}
__device__ __forceinline__ Triple triple_of(const Pair& s, float bias) {
  const Pair a = two_sum(bias, s.hi);
  return triple_of(a.hi, a.lo, s.lo);
}
__device__ __forceinline__ Triple triple_sum(const Triple& a, const Triple& b) {
  const Pair s = two_sum(a.v0, b.v0), m = two_sum(a.v1, b.v1), n = two_sum(s.lo, m.hi);
  return triple_of(s.hi, n.hi, __fadd_rn(n.lo, __fadd_rn(m.lo, __fadd_rn(a.v2, b.v2))));
}
__device__ __forceinline__ Triple triple_from(const Triple& v, int lane) {
  return {__shfl_sync(kFull, v.v0, lane), __shfl_sync(kFull, v.v1, lane), __shfl_sync(kFull, v.v2, lane)};
}
// v - w, and whether its sign is certain: v and w are off by 2^-42 at most, the difference of the
// second terms by 2^-24 of itself (that of the first ones is exact where they are near).
__device__ __forceinline__ float difference(const Triple& v, const Triple& w, bool& certain) {
  const float d1 = __fsub_rn(v.v1, w.v1);
  const float d = __fadd_rn(__fadd_rn(__fsub_rn(v.v0, w.v0), d1), __fsub_rn(v.v2, w.v2));
  certain = fabsf(d) > fmaf(fabsf(d1), 0x1p-20f, 0x1p-40f);  // (not where something is not a number)
  return d;
}

struct WarpScratch {
  union {
    uint32_t key[kTokens][256];
    Wide value[256];  // the whole warp's one token, done again
  };
  uint32_t second[kRouterMaxGroups];
  int list[32];
  uint32_t kept[kTokens][kRouterMaxGroups];  // first experts of the groups kept
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

// Expert e's s + bias of token t in fp64 (its logit where that has the same order).
template <bool kSigmoid>
__device__ __noinline__ Wide exact_value(const RouterScoresArgs& a, long long t, int e, double top, double sum, bool scored) {
  const double x = load_logit(a, t, e);
  if (!scored) return wide_sum(x, 0.0);
  return wide_sum(kSigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum, bias_of(a, e));
}

// The token's largest logit and, for scores by softmax, the sum below it (0 and 1 where every logit is
// -inf, so that the scores are 0).
template <bool kSigmoid>
__device__ __forceinline__ void exact_sum(const RouterScoresArgs& a, long long t, bool scored, double& top, double& sum) {
  const int lane = threadIdx.x & 31;
  top = 0.0;
  sum = 1.0;
  if (kSigmoid || !scored) return;
  float most = kNegInf;
  for (int e = lane; e < a.num_experts; e += 32) most = fmaxf(most, load_logit(a, t, e));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, off));
  if (most == kNegInf) return;
  top = most;
  sum = 0.0;
#pragma unroll 2
  for (int e = lane; e < a.num_experts; e += 32) sum += exp(static_cast<double>(load_logit(a, t, e)) - top);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
}

// Token t in fp64 over all experts, by the whole warp.  picked[r] on every lane: the experts (some
// in range, whatever the logits are: what is not a number counts as -inf).
template <bool kSigmoid>
__device__ __noinline__ void choose_among_all(const RouterScoresArgs& a, WarpScratch& ws, long long t, int (&picked)[8]) {
  const int lane = threadIdx.x & 31;
  const int E = a.num_experts, size = E / a.num_groups;
  const bool grouped = a.num_groups > a.top_groups;
  const bool scored = a.bias != nullptr || grouped;  // else the logits' order is the answer
  double top, sum;
  exact_sum<kSigmoid>(a, t, scored, top, sum);
  __syncwarp();
  for (int e = lane; e < E; e += 32) ws.value[e] = exact_value<kSigmoid>(a, t, e, top, sum, scored);
  __syncwarp();
  unsigned kept = kFull;
  if (grouped) {
    Wide first = least(), second = least();
    if (lane < a.num_groups) {
      for (int i = 0; i < size; ++i) {
        const Wide v = ws.value[lane * size + i];
        if (above(order_of(v), order_of(first))) {
          second = first;
          first = v;
        } else if (above(order_of(v), order_of(second))) {
          second = v;
        }
      }
    }
    const Order merit = order_of(size > 1 ? merit_of(first, second) : first);
    int before = 0;
    for (int g = 0; g < a.num_groups; ++g) {
      const Order w = order_from(merit, g);
      before += above(w, merit) || (g < lane && !above(merit, w));
    }
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
#pragma unroll 1
  for (int r = 0; r < a.top_k; ++r) {
    Order best = order_of(least());
    int at = kNone;
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(taken >> i & 1) && (kept >> (grouped ? e / size : 0) & 1)) {
        const Order v = order_of(ws.value[e]);
        if (at == kNone || above(v, best)) {
          best = v;
          at = e;
        }
      }
    }
#pragma unroll 1
    for (int off = 16; off > 0; off >>= 1) {
      const Order v = {__shfl_xor_sync(kFull, best.hi, off), __shfl_xor_sync(kFull, best.lo, off)};
      const int f = __shfl_xor_sync(kFull, at, off);
      if (f != kNone && (at == kNone || above(v, best) || (!above(best, v) && f < at))) {
        best = v;
        at = f;
      }
    }
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s == r) picked[s] = at;
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
  }
  __syncwarp();
}

// (not NaN)
__device__ __forceinline__ float warp_min(float v) {
  auto swap = [](int b) { return b ^ (b >> 31 & 0x7fffffff); };  // sorts like the float, and back
  return __int_as_float(swap(__reduce_min_sync(kFull, swap(__float_as_int(v)))));
}
__device__ __forceinline__ float warp_max(float v) { return -warp_min(-v); }

// The biases' range [lo, hi] for the keys (a warp; a lane's biases, NaN behind the last expert).  With
// R = hi - lo, a finite bias is left out, as masked, only below lo - R - 2.  A score adds 0 to 1.  So
// a masked expert's value is below every other's, and the merit of a group with fewer than two
// others is below hi + 1 + (lo - R - 2) + 1 = 2 lo, which no group with two others is below: the order
// of keys with 0 for masked experts and for such groups is certain.  The highest range that leaves
// at least `need` experts in it is taken, if there is one; it doubles with every second step.
__device__ __forceinline__ void bias_range(const float (&b)[8], int need, float& lo, float& hi) {
  constexpr float kMost = 3.402823466e38f;
  float least = __builtin_huge_valf(), most = kNegInf;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (fabsf(b[i]) <= kMost) {
      least = fminf(least, b[i]);
      most = fmaxf(most, b[i]);
    }
  }
  lo = warp_min(least);
  hi = warp_max(most);
  if (!(lo <= hi)) lo = hi = 0.0f;  // no finite one
  if (hi - lo <= kWideBias) return;
  lo = hi;
  for (;;) {
    // in fp64, rounded down: exact enough beside the steps of fp32 at any size
    const float reach = __double2float_rd(static_cast<double>(lo) - (static_cast<double>(hi) - lo) - 2.0);
    float within = lo, below = kNegInf;
    int n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(b[i]) <= kMost) {
        if (b[i] >= reach) within = fminf(within, b[i]);
        else below = fmaxf(below, b[i]);
        n += b[i] >= lo;
      }
    }
    within = warp_min(within);
    if (within < lo) {
      lo = within;
      continue;
    }
    below = warp_max(below);
    if (__reduce_add_sync(kFull, n) >= need || below == kNegInf) return;
    lo = below;  // too few: with the next ones below
  }
}

// Experts whose key (24 bits, in ws.key[0]; 0: not to be chosen) is at least that of their place
// `floor`, listed in expert order in ws.list.  Returns their number.
template <typename Floor>
__device__ __forceinline__ int list_candidates(WarpScratch& ws, int E, Floor floor) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const bool in = e < E && ws.key[0][e] != 0 && ws.key[0][e] >= floor(e);
    const unsigned m = __ballot_sync(kFull, in);
    const int at = n + __popc(m & ((1u << lane) - 1));
    if (in && at < 32) ws.list[at] = e;
    n += __popc(m);
  }
  __syncwarp();
  return n;
}

__device__ __forceinline__ uint32_t below_by(uint32_t q, uint32_t d) { return q > d ? q - d : 0u; }

// Token t by the whole warp, with the comparisons that keys cannot settle made in fp64; writes its
// results.  bias_key, unit, keyless: as in the kernel.
template <bool kSigmoid, bool kScored>
__device__ __noinline__ void settle(const RouterScoresArgs& a, WarpScratch& ws, int* hist, const float* bias_key, float unit,
                                    bool keyless, long long t) {
  const int lane = threadIdx.x & 31;
  const int E = a.num_experts, k = a.top_k, size = E / a.num_groups;
  const bool grouped = kScored && a.top_groups < a.num_groups;
  // ---- the keys once more, in expert order, without the experts' codes
  float x[8], ref = kNegInf;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = lane + 32 * i < E ? load_logit(a, t, lane + 32 * i) : kNegInf;
    ref = fmaxf(ref, x[i]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ref = fmaxf(ref, __shfl_xor_sync(kFull, ref, off));
  if (ref == kNegInf) ref = 0.0f;
  float total = exp_sum<8>(x, ref);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kFull, total, off);
  const float inv_sum = total > 0.0f ? 1.0f / total : 0.0f;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    if (e < E) ws.key[1][e] = __float_as_uint(x[i]);
    if (e < E)  // 0 stands for experts of other groups here (masked ones: below or at the others' least)
      ws.key[0][e] = max(fixed_point<kSigmoid, kScored>(x[i], ref, unit, unit * inv_sum, kScored ? bias_key[e] : 0.0f), 1u);
  }
  __syncwarp();
  int picked[8];
  bool walk = keyless;
  // ---- groups: the candidates for the two largest of each
  if (grouped && !walk) {
    if (lane < a.num_groups) {
      uint32_t first = 0, second = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t v = ws.key[0][lane * size + i];
        second = max(second, min(first, v));
        first = max(first, v);
      }
      ws.second[lane] = size > 1 ? second : first;
    }
    __syncwarp();
    const int n = list_candidates(ws, E, [&](int e) { return below_by(ws.second[e / size], kNear); });
    walk = n > 32;
    if (!walk) {
      const int e = lane < n ? ws.list[lane] : 0;
      unsigned kept = 0;
      // scores by sigmoid, two candidates in every group: lanes 2 g and 2 g + 1
      bool sure = kSigmoid && size > 1 && n == 2 * a.num_groups;
      if (sure) {
        const Triple v = triple_of(sigmoid_pair(__uint_as_float(ws.key[1][e])), bias_of(a, e));
        const Triple merit = triple_sum(triple_from(v, 2 * lane & 31), triple_from(v, (2 * lane & 31) + 1));
        int before = 0;
        for (int g = 0; g < a.num_groups; ++g) {
          bool certain;
          const float d = difference(triple_from(merit, g), merit, certain);
          before += d > 0.0f;
          if (!certain && g != lane && lane < a.num_groups) sure = false;
        }
        kept = __ballot_sync(kFull, lane < a.num_groups && before < a.top_groups);
        sure = __all_sync(kFull, sure);
      }
      if (!sure) {
        double top, sum;
        exact_sum<kSigmoid>(a, t, true, top, sum);
        const Wide v = exact_value<kSigmoid>(a, t, e, top, sum, true);
        const Order mine = order_of(v);
        const int group = lane < n ? e / size : -1;
        int first = -1, second = -1;  // the lanes with the two largest of group `lane`
        Order of_first = order_of(least()), of_second = of_first;
        for (int i = 0; i < n; ++i) {
          const Order w = order_from(mine, i);
          if (__shfl_sync(kFull, group, i) == lane) {
            if (first < 0 || above(w, of_first)) {
              second = first;
              of_second = of_first;
              first = i;
              of_first = w;
            } else if (second < 0 || above(w, of_second)) {
              second = i;
              of_second = w;
            }
          }
        }
        const Wide v1 = {__shfl_sync(kFull, v.hi, max(first, 0)), __shfl_sync(kFull, v.lo, max(first, 0))};
        const Wide v2 = {__shfl_sync(kFull, v.hi, max(second, 0)), __shfl_sync(kFull, v.lo, max(second, 0))};
        const Order merit = order_of(size > 1 ? merit_of(v1, v2) : v1);
        int before = 0;
        for (int g = 0; g < a.num_groups; ++g) {
          const Order w = order_from(merit, g);
          before += above(w, merit) || (g < lane && !above(merit, w));
        }
        kept = __ballot_sync(kFull, lane < a.num_groups && before < a.top_groups);
      }
      for (int e2 = lane; e2 < E; e2 += 32)
        if (!(kept >> (e2 / size) & 1)) ws.key[0][e2] = 0;
      __syncwarp();
    }
  }
  // ---- the k-th largest key, and in fp64 all that are near it or above
  if (!walk) {
    uint32_t last = 0xffffffffu;
    for (int r = 0; r < k; ++r) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = lane + 32 * i;
        const uint32_t v = e < E && ws.key[0][e] != 0 ? ws.key[0][e] << 8 | (255 - e) : 0u;
        if (v < last) most = max(most, v);
      }
      last = __reduce_max_sync(kFull, most);
    }
    const uint32_t floor = below_by(last >> 8, kNear);
    const int n = list_candidates(ws, E, [&](int) { return floor; });
    walk = n > 32;
    if (!walk) {
      const bool scored = a.bias != nullptr;  // else the logits' order is the answer
      const int e = lane < n ? ws.list[lane] : 0;
      int rank = 0;
      bool sure = kSigmoid && scored;
      if (sure) {
        const float logit = __uint_as_float(ws.key[1][e]), bias = bias_of(a, e);
        const Triple mine = triple_of(sigmoid_pair(logit), bias);
        for (int i = 0; i < n; ++i) {
          bool certain;
          const float d = difference(triple_from(mine, i), mine, certain);
          const float its_logit = __shfl_sync(kFull, logit, i), its_bias = __shfl_sync(kFull, bias, i);
          const bool same = its_logit == logit && its_bias == bias;
          rank += same ? i < lane : d > 0.0f;
          if (!certain && !same && lane < n) sure = false;
        }
        sure = __all_sync(kFull, sure);
      }
      if (!sure) {
        double top, sum;
        exact_sum<kSigmoid>(a, t, scored, top, sum);
        const Order mine = order_of(exact_value<kSigmoid>(a, t, e, top, sum, scored));
        rank = 0;
        for (int i = 0; i < n; ++i) {
          const Order w = order_from(mine, i);
          rank += above(w, mine) || (i < lane && !above(mine, w));  // candidates are in expert order
        }
      }
      if (lane >= n) rank = 32;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const unsigned m = __ballot_sync(kFull, rank == r);
        picked[r] = __shfl_sync(kFull, e, m ? __ffs(m) - 1 : 0);
      }
    }
  }
  if (walk) choose_among_all<kSigmoid>(a, ws, t, picked);
  int expert = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (lane == r) expert = picked[r];
  const Chosen c = chosen_scores<kSigmoid>(lane < k ? load_logit(a, t, expert) : kNegInf, ref, inv_sum, a.renormalize);
  if (lane < k) write_choice(a, hist, t, lane, expert, c.score, c.sum);
  __syncwarp();
}

// kScored: keys hold s + bias (0 without one), else x - max x.
// The sorting runs over the keys in shared memory, eight at a time in a loop: unrolled over a
// lane's 32 keys the pass is 27 KB of code, and warps wait for instructions a third of the time.
template <int K, bool kFp32, bool kSigmoid, bool kScored>
__global__ void __launch_bounds__(kBlock, 3) router_scores_kernel(const RouterScoresArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ int hist[256];
  __shared__ __align__(16) float bias_key[256];  // 1 + the bias's part of a key
  __shared__ float key_unit;                     // keys per unit of score
  __shared__ int bias_kind;                      // 1: masked experts have an order of their own
                                                 // 2: biases too far apart for keys, every token in fp64
  __shared__ long long doubtful[kMaxDoubtful];   // tokens left for the end
  __shared__ int num_doubtful;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WarpScratch& ws = reinterpret_cast<WarpScratch*>(smem_raw)[warp];
  const int E = a.num_experts, k = a.top_k;
  const int j = lane % kLanes, tok = lane / kLanes;
  const bool grouped = kScored && a.top_groups < a.num_groups;
  const int size = E / a.num_groups;
  const int inv_size = (65536 + size - 1) / size;  // e / size == (e * inv_size) >> 16 for e < 256
  int vecs = (E + 4 * kLanes - 1) / (4 * kLanes);  // vectors of a lane that hold experts
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const long long passes = (a.num_tokens + kTokens - 1) / kTokens;
  // (the last, partial round by few blocks: the others settle their doubtful tokens meanwhile; spread
  // over all blocks, 32768 tokens took 33.3 us instead of 30.8)
  long long p = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;
  auto token_of = [&](long long pass) { return min(pass * kTokens + tok, a.num_tokens - 1); };  // lanes behind: the last one
  float x[kOwn];
  auto load = [&](long long t) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = 4 * (j + kLanes * i);
      if (a.vec4) {
        if (kFp32) {
          const float4 v = e < E ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + t * E + e))
                                 : make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
          x[4 * i] = v.x;
          x[4 * i + 1] = v.y;
          x[4 * i + 2] = v.z;
          x[4 * i + 3] = v.w;
        } else {
          const uint2 v = e < E ? __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + t * E + e))
                                : make_uint2(0xFF80FF80u, 0xFF80FF80u);
          x[4 * i] = __uint_as_float(v.x << 16);
          x[4 * i + 1] = __uint_as_float(v.x & 0xFFFF0000u);
          x[4 * i + 2] = __uint_as_float(v.y << 16);
          x[4 * i + 3] = __uint_as_float(v.y & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[4 * i + c] = e + c < E ? load_logit(a, t, e + c) : kNegInf;
      }
    }
  };
  if (p < passes) load(token_of(p));  // on their way during the set-up
  for (int e = threadIdx.x; e < 256; e += blockDim.x) hist[e] = 0;
  if (threadIdx.x == 0) num_doubtful = 0;
  if constexpr (kScored) {
    if (warp == 0) {
      float b[8], lo, hi;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = lane + 32 * i < E ? bias_of(a, lane + 32 * i) : __int_as_float(0x7fffffff);
      bias_range(b, grouped ? max(k, 2 * a.top_groups) : k, lo, hi);
      const float unit = kKeyRange / (1.0f + (hi - lo));
      bool differ = false;
      // b - lo first: what is rounded is small beside the range
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = b[i] >= lo;  // (not a NaN, which counts as -inf)
        bias_key[lane + 32 * i] = in ? (b[i] - lo) * unit + 1.0f : -4e7f;
        if (b[i] < lo && b[i] != kNegInf) differ = true;
      }
      differ = __any_sync(kFull, differ);
      if (lane == 0) {
        key_unit = unit;
        bias_kind = (differ ? 1 : 0) | (hi - lo <= 1e30f ? 0 : 2);
      }
    }
  }
  __syncthreads();
  const float unit = kScored ? key_unit : 0.0f;
  const bool masks_differ = kScored && (bias_kind & 1), keyless = kScored && (bias_kind & 2);
  for (; p < passes; p += warps) {
    const long long t = p * kTokens + tok, tt = token_of(p);
    const bool live = t < a.num_tokens;  // the lanes of a token agree
    // ---- maximum, and for the softmax the sum
    float ref = 0.0f, inv_sum = 1.0f;
    if constexpr (!kSigmoid || !kScored) {
      float top = x[0];
#pragma unroll
      for (int i = 1; i < kOwn; ++i) top = fmaxf(top, x[i]);
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      ref = top == kNegInf ? 0.0f : top;
    }
    if constexpr (!kSigmoid) {
      float sum = exp_sum<kOwn>(x, ref);
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
      inv_sum = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    // ---- 24-bit keys into the scratch, by expert (0 behind the last)
    const float soft_unit = unit * inv_sum;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = 4 * (j + kLanes * i);
      float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
      if constexpr (kScored) b = *reinterpret_cast<const float4*>(&bias_key[e]);
      const float bc[4] = {b.x, b.y, b.z, b.w};
      uint32_t q[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) q[c] = fixed_point<kSigmoid, kScored>(x[4 * i + c], ref, unit, soft_unit, bc[c]);
      if (e + 4 > E) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e + c >= E) q[c] = 0;
      }
      *reinterpret_cast<uint4*>(&ws.key[tok][e]) = make_uint4(q[0], q[1], q[2], q[3]);
    }
    if (p + warps < passes) load(token_of(p + warps));
    auto expert_of = [](uint32_t full_key) { return 255 - static_cast<int>(full_key & 255u); };
    bool doubt = keyless;  // some comparison is not certain
    unsigned kept = kFull;
    // ---- groups
    if (grouped) {
      __syncwarp();
      // lane j of a token takes groups j, j + 8, ..: the sum of their two largest keys
      constexpr int kMine = kRouterMaxGroups / kLanes;
      uint32_t merit[kMine];
#pragma unroll
      for (int n = 0; n < kMine; ++n) {
        const int g = j + kLanes * n;
        merit[n] = 0;
        if (kLanes * n < a.num_groups && g < a.num_groups) {
          uint32_t first = 0, second = 0;
          auto take = [&](uint32_t v) {
            second = max(second, min(first, v));
            first = max(first, v);
          };
          const uint32_t* from = &ws.key[tok][g * size];
          if (size % 4 == 0) {
            int at = 4 * j % size;  // the lanes of a token begin in different banks
#pragma unroll 2
            for (int i = 0; i < size; i += 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(from + at);
              take(v.x);
              take(v.y);
              take(v.z);
              take(v.w);
              at = at + 4 == size ? 0 : at + 4;
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < size; ++i) take(from[i]);
          }
          merit[n] = first;  // 0: masked, or one left
          if (size > 1) {
            merit[n] = second == 0 ? 0 : first == kPinned ? kPinned : first + second;
            if (second == 0 && first == kPinned) doubt = true;
          }
        }
      }
      // a group is kept if fewer than top_groups come before it
      uint32_t last_kept = 0xffffffffu, first_dropped = 0;
      kept = 0;
#pragma unroll
      for (int n = 0; n < kMine; ++n) {
        if (kLanes * n < a.num_groups) {
          int before = 0;
#pragma unroll
          for (int m = 0; m < kMine; ++m) {
            if (kLanes * m < a.num_groups) {
#pragma unroll
              for (int l = 0; l < kLanes; ++l) {
                const uint32_t other = __shfl_sync(kFull, merit[m], (lane & ~(kLanes - 1)) + l);
                before += other > merit[n] || (other == merit[n] && l + kLanes * m < j + kLanes * n);
              }
            }
          }
          if (j + kLanes * n < a.num_groups) {
            if (before < a.top_groups) {
              kept |= 1u << (j + kLanes * n);
              last_kept = min(last_kept, merit[n]);
            } else {
              first_dropped = max(first_dropped, merit[n]);
            }
          }
        }
      }
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) {
        kept |= __shfl_xor_sync(kFull, kept, off);
        last_kept = min(last_kept, __shfl_xor_sync(kFull, last_kept, off));
        first_dropped = max(first_dropped, __shfl_xor_sync(kFull, first_dropped, off));
      }
      // a tie in merit as well; not of +inf, and of 0 only if the masks make a difference
      doubt |= last_kept - first_dropped <= 2 * kNear && last_kept != kPinned && (last_kept != 0 || masks_differ);
      if (size % 4 == 0) {  // the kept groups' first experts, in order
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
          const int g = j + kLanes * n;
          if (kept >> g & 1) ws.kept[tok][__popc(kept & ((1u << g) - 1))] = g * size;
        }
        vecs = (a.top_groups * size + 4 * kLanes - 1) / (4 * kLanes);
      }
    }
    __syncwarp();
    // this lane's i-th vector of experts that may be chosen, as full keys (0: none)
    auto load_keys = [&](int i, uint32_t* key) {
      int e = 4 * (j + kLanes * i);
      bool in = true;
      if (grouped && size % 4 == 0) {  // of the kept groups, one behind the other
        const int nth = (e * inv_size) >> 16;
        in = nth < a.top_groups;
        if (in) e += static_cast<int>(ws.kept[tok][nth]) - nth * size;
      } else {
        in = i < kVecs;
      }
      const uint4 v = in ? *reinterpret_cast<const uint4*>(&ws.key[tok][e]) : make_uint4(0, 0, 0, 0);
      const uint32_t code = in ? 255u - e : 3u;
      key[0] = (v.x << 8) + code;
      key[1] = (v.y << 8) + code - 1;
      key[2] = (v.z << 8) + code - 2;
      key[3] = (v.w << 8) + code - 3;
      if (!in) key[0] = key[1] = key[2] = key[3] = 0;
      if (grouped && size % 4 != 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!(kept >> (((e + c) * inv_size) >> 16) & 1)) key[c] = 0;
      }
    };
    // ---- the K largest keys
    uint32_t best[K], local[K];
#pragma unroll
    for (int r = 0; r < K; ++r) best[r] = 0;
#pragma unroll 1
    for (int i = 0; i < vecs; i += 2) {
      uint32_t key[8];
      load_keys(i, key);
      load_keys(i + 1, key + 4);
#pragma unroll
      for (int h = 0; h < 8; h += K) {
        uint32_t part[K];
#pragma unroll
        for (int r = 0; r < K; ++r) part[r] = key[h + r];
        sort_keys<K>(part);
        merge_keys<K>(best, part);
      }
    }
#pragma unroll
    for (int r = 0; r < K; ++r) local[r] = best[r];
#pragma unroll 1
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
    // the largest key not chosen: the first of a lane's list below the last chosen
    uint32_t next = 0;
#pragma unroll
    for (int r = 0; r < K; ++r) next = max(next, local[r] < last ? local[r] : 0u);
    if (__any_sync(kFull, local[K - 1] >= last)) {  // a lane whose whole list was chosen: its other keys
#pragma unroll 1
      for (int i = 0; i < vecs; ++i) {
        uint32_t key[4];
        load_keys(i, key);
#pragma unroll
        for (int c = 0; c < 4; ++c) next = max(next, key[c] < last ? key[c] : 0u);
      }
    }
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) next = max(next, __shfl_xor_sync(kFull, next, off));
    // ---- neighbours too close to be certain, unless logit and bias are the same; and lane j of a
    // token: its j-th expert
    int expert = 0;
    uint32_t below = next;  // the neighbour of this lane's
#pragma unroll
    for (int r = 0; r < K; ++r) {
      if (j == r) expert = expert_of(best[r]);
      if (r > 0 && r < k && j == r - 1) below = best[r];
    }
    uint32_t own = 0;
#pragma unroll
    for (int r = 0; r < K; ++r)
      if (j == r) own = best[r];
    constexpr uint32_t kDistance = kScored ? kNear : 0;
    const bool near = j < k && below >= 256 && (own >> 8) - (below >> 8) <= kDistance && below >> 8 != kPinned >> 8;
    const bool same = near && same_inputs(a, tt, expert, expert_of(below));
    if (near && !same) doubt = true;
    // At the border only the first behind it has been looked at.  Where it is the last one's equal, others
    // as near may be above both.
    const unsigned equal = __ballot_sync(kFull, same && j == k - 1);
    if (equal) {
      bool mine = (equal >> (lane & ~(kLanes - 1)) & ((1u << kLanes) - 1)) != 0;
      if (!kFp32 && mine && a.bias == nullptr) {
        // Equal logits are common in bf16, where another logit is |x| 2^-8 away at least: mostly more than
        // the 31 steps of keys (4 for logits) within which it could be one of those (32768 x 256 in bf16, no
        // bias: 18.6 us, 22.9 if every token with equals at its border looks)
        const float x = fabsf(load_logit(a, tt, expert_of(last))), q = static_cast<float>(last >> 8);
        if (kScored ? (kSigmoid ? x >= 0x1p-8f && x <= 8.0f : x <= 64.0f && q * x >= 16384.0f) : x >= 0x1p-8f && q > 1.0f)
          mine = false;
      }
#pragma unroll 1
      for (int i = 0; i < vecs && mine && !doubt; ++i) {
        uint32_t key[4];
        load_keys(i, key);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (key[c] < last && key[c] >= 256 && (last >> 8) - (key[c] >> 8) <= kDistance &&
              !same_inputs(a, tt, expert_of(last), expert_of(key[c])))
            doubt = true;
      }
      __syncwarp();
    }
    if (kScored && j < k && own < 256 && masks_differ) doubt = true;  // a masked expert among the chosen
    const unsigned doubts = __ballot_sync(kFull, doubt && live);
    doubt = (doubts >> (lane & ~(kLanes - 1)) & ((1u << kLanes) - 1)) != 0;
    // ---- weights
    const Chosen c = chosen_scores<kSigmoid>(j < k ? load_logit(a, tt, expert) : kNegInf, ref, inv_sum, a.renormalize);
    if (live && !doubt && j < k) write_choice(a, hist, t, j, expert, c.score, c.sum);
    __syncwarp();  // the keys have been read
    if (doubt && live && j == 0) {  // left for the end: in the list, or marked where it is full
      const int at = atomicAdd(&num_doubtful, 1);
      if (at < kMaxDoubtful) doubtful[at] = t;
      else a.topk_idx[t * k] = -1;
    }
  }
  // the block's doubtful tokens, shared among its warps
  __syncthreads();
  const int left = min(num_doubtful, kMaxDoubtful);
  for (int i = warp; i < left; i += blockDim.x >> 5)
    settle<kSigmoid, kScored>(a, ws, hist, bias_key, unit, keyless, doubtful[i]);
  if (num_doubtful > kMaxDoubtful) {  // the marked ones, by the warps that met them
    p = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;
    for (; p < passes; p += warps) {
      for (long long t = p * kTokens; t < min((p + 1) * kTokens, a.num_tokens); ++t) {
        const int first = *const_cast<volatile int32_t*>(a.topk_idx + t * k);
        if (__shfl_sync(kFull, first, 0) < 0) settle<kSigmoid, kScored>(a, ws, hist, bias_key, unit, keyless, t);
      }
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
  const int warps = passes <= 2LL * sms ? 1 : kBlock / 32;
  const long long blocks = (passes + warps - 1) / warps;
  const long long most = 3LL * sms;  // resident ones
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  const size_t smem = warps * sizeof(WarpScratch);
  if (a.bias || a.top_groups < a.num_groups)
    router_scores_kernel<K, kFp32, kSigmoid, true><<<grid, 32 * warps, smem, stream>>>(a);
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
  if (a.top_k <= 2) return launch_scores_k<2>(a, sms, stream);
  if (a.top_k <= 4) return launch_scores_k<4>(a, sms, stream);
  return launch_scores_k<8>(a, sms, stream);
}

}  // namespace sa
