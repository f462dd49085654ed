/*
 * moe_experts.h -- the expert layer behind the router: grouping of the
 * (token, expert) pairs, the experts' matrix products over ragged groups of
 * rows, and the weighted sum back to the tokens (libsinkattn.so, sm_103a).
 *
 * The page "GPT-OSS on day 0" (Perplexity, 2025) lists in its model overview
 * a SwiGLU activation and bias terms in the experts, and the router whose
 * indices and weights these calls consume (moe_router.h).  A layer is
 *
 *     moe_router            -> topk_idx, topk_weight          [T, K]
 *     moe_group_rows        -> expert_offsets, row_token, pair_row
 *     grouped_linear_swiglu -> h [T * K, I]    (gate and up projection, x gathered)
 *     grouped_linear_bias   -> y [T * K, H]    (down projection)
 *     moe_combine           -> out [T, H]
 *
 * (mxfp4.h has the same products on 4-bit operands.)  The conventions of
 * sink_attn.h apply: device pointers owned by the caller, asynchronous on
 * `stream`, no allocation, no synchronisation, CUDA-graph capturable.  Arrays
 * lie at multiples of their element's size, or of 16 bytes where stated
 * (SA_ERR_ALIGNMENT otherwise); outputs overlap no input.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "sink_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Stable counting sort of the pairs p = t * top_k + r by their expert:
 *
 *     expert_offsets[e] = number of pairs of experts below e
 *     row(p)            = expert_offsets[e_p] + number of pairs q < p with e_q = e_p
 *     row_token[row(p)] = t,   pair_row[p] = row(p)
 *
 *  topk_idx       int32 [num_tokens, top_k].  A negative index is a pair
 *                 without expert (a padded token): its pair_row is -1.  An
 *                 index >= num_experts is treated the same way and sets
 *                 SA_ERR_BOUNDS in the device status word.  A token may name
 *                 the same expert twice: that makes two rows.
 *  expert_offsets int32 [num_experts + 1]; the last entry is the row count R
 *  row_token      int32 [num_tokens * top_k]: entries from R on are -1
 *  pair_row       int32 [num_tokens, top_k]
 *  1 <= num_experts <= 256, 1 <= top_k <= 8, num_tokens * top_k <= 2^30.
 *  The order is that of the pairs, whatever the schedule: the result is a
 *  function of the indices alone.  num_tokens == 0 still writes the offsets.
 */
sa_status moe_group_rows(const int32_t* topk_idx, int num_tokens, int top_k, int num_experts,
                         int32_t* expert_offsets, int32_t* row_token, int32_t* pair_row,
                         cudaStream_t stream);

/*
 * One product per expert over its rows r in [offsets[e], offsets[e + 1]):
 *
 *     out[r, j] = sum_i x[row_token[r], i] * w[e, j, i] + bias[e, j]
 *
 * bf16 operands, fp32 accumulation on the tcgen05 tensor cores, the bias
 * added in fp32, one rounding to bf16.
 *
 *  x              bf16 [x_rows, k];  w bf16 [num_experts, n, k] (one row per
 *                 output feature);  bias bf16 [num_experts, n] or NULL
 *  expert_offsets int32 [num_experts + 1], device, non-decreasing, within
 *                 [0, rows].  A group that starts below an earlier offset or
 *                 ends below its start or beyond rows is skipped and sets
 *                 SA_ERR_BOUNDS in the device status word.  Empty groups cost
 *                 nothing; rows outside every group are left as they were.
 *  row_token      int32 [rows] or NULL: which row of x each row reads (NULL:
 *                 its own, x_rows == rows).  Read inside the groups only.  An
 *                 entry outside [0, x_rows) sets SA_ERR_BOUNDS; that row's
 *                 result is unspecified, the others are not affected.
 *  out            bf16 [rows, n]
 *  k a multiple of 8, x and w 16-byte aligned, 1 <= num_experts <= 256, any
 *  n >= 1, rows >= 0 (0 launches nothing), rows, n and k <= 2^30,
 *  num_experts * n <= 2^31 - 1024, (rows / 16 + num_experts) * (n / 64 + 1) < 2^30.
 *  A device wait that runs out of time (sink_attn_set_wait_timeout_ns) ends
 *  the kernel cleanly and sets SA_ERR_TIMEOUT in the device status word.
 */
sa_status grouped_linear_bias(const void* x, const void* w, const void* bias,
                              const int32_t* expert_offsets, const int32_t* row_token, int x_rows,
                              int rows, int num_experts, int n, int k, void* out,
                              cudaStream_t stream);

/*
 * The same product followed by the clamped SwiGLU of GPT-OSS on interleaved
 * gate and up features (rows 2i and 2i + 1 of w), before the one rounding:
 *
 *     g = min(y[r, 2i], limit),  u = min(max(y[r, 2i + 1], -limit), limit)
 *     out[r, i] = g * sigmoid(alpha * g) * (u + 1)
 *
 *  out bf16 [rows, n / 2]; n even; alpha finite; limit > 0 (+infinity: no
 *  clamp).  A sigmoid below 2^-126 counts as 0 (with alpha = 1.702 that of
 *  gates below -51); otherwise infinities and NaN are those of the formula.
 *  Everything else as for grouped_linear_bias.
 */
sa_status grouped_linear_swiglu(const void* x, const void* w, const void* bias,
                                const int32_t* expert_offsets, const int32_t* row_token,
                                int x_rows, int rows, int num_experts, int n, int k, float alpha,
                                float limit, void* out, cudaStream_t stream);

/*
 * out[t, :] = sum_r topk_weight[t, r] * y[pair_row[t, r], :], summed in fp32
 * in the order of r and rounded once to bf16.  A pair_row of -1 adds nothing
 * (a token without experts becomes 0); one outside [-1, num_rows) adds
 * nothing and sets SA_ERR_BOUNDS.
 *
 *  y           bf16 [num_rows, hidden], 16-byte aligned, hidden a multiple of 8
 *  pair_row    int32 [num_tokens, top_k];  topk_weight bf16 [num_tokens, top_k]
 *  out         bf16 [num_tokens, hidden], 16-byte aligned
 *  1 <= top_k <= 8, num_tokens * hidden < 2^40.
 */
sa_status moe_combine(const void* y, const int32_t* pair_row, const void* topk_weight,
                      int num_rows, int num_tokens, int top_k, int hidden, void* out,
                      cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
