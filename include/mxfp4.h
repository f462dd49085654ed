/*
 * mxfp4.h -- microscaled 4-bit floating point (OCP MX, MXFP4: E2M1 values in
 * blocks of 32 with one E8M0 scale each): quantisation and matrix products
 * (libsinkattn.so, sm_103a).
 *
 * The page "GPT-OSS on day 0" (Perplexity, 2025) states that the models ship
 * in MXFP4 and were served in FP8 only because Hopper has no FP4 tensor
 * cores; the block-scaled tcgen05 products here take that format directly.
 *
 * A matrix [rows, k] (k a multiple of 32) is held as
 *   codes  uint8 [rows, k / 2]: value 2i in the low half of byte i, value
 *          2i + 1 in the high half.  E2M1: sign, two exponent bits, one
 *          mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.
 *   scales uint8 [rows, s], s = k / 32 rounded up to a multiple of 16: byte b
 *          stands for 2^(b - 127), 255 for NaN.  Bytes from k / 32 on are
 *          padding: written as 0, never used.
 * (A checkpoint's [rows, k / 32] scales need only that padding.)
 *
 * The conventions of sink_attn.h apply.  Codes, scales and 16-bit matrices
 * are 16-byte aligned (SA_ERR_ALIGNMENT otherwise).
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "sink_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantise x to MXFP4, each block of 32 on its own:
 *
 *     scale = 2^(floor(log2 max|x|) - 2), at least 2^-127
 *     code  = x / scale rounded to the nearest E2M1 value (ties to even),
 *             magnitudes above 6 to 6
 *
 * (the conversion of the OCP MX specification).  A block of zeros has scale
 * byte 0; a block that holds an infinity or a NaN has scale byte 255 and codes 0.
 *
 *  x [rows, k] bf16 (is_fp32 == 0) or fp32 (is_fp32 != 0), 16-byte aligned
 *  k > 0, a multiple of 32 (SA_ERR_UNSUPPORTED otherwise); rows * k < 2^40;
 *  rows == 0 launches nothing.
 */
sa_status mxfp4_quantize(const void* x, int is_fp32, long long rows, int k, void* codes,
                         void* scales, cudaStream_t stream);

/* The values that codes and scales stand for, as bf16 [rows, k]: exact, except
 * that values beyond the largest bf16 number become infinite.  A block with
 * scale byte 255 is NaN. */
sa_status mxfp4_dequantize(const void* codes, const void* scales, long long rows, int k,
                           void* out, cudaStream_t stream);

/*
 * out[r, j] = sum_i x[r, i] * w[j, i] + bias[j] with both operands in MXFP4:
 * block-scaled tensor-core products, fp32 accumulation, the bias added in
 * fp32, one rounding to bf16.
 *
 *  x [m, k] and w [n, k] as above;  bias bf16 [n] or NULL;  out bf16 [m, n]
 *  k a multiple of 32; any n >= 1, m >= 0; limits as for grouped_linear_bias.
 */
sa_status mxfp4_linear_bias(const void* x_codes, const void* x_scales, const void* w_codes,
                            const void* w_scales, const void* bias, int m, int n, int k, void* out,
                            cudaStream_t stream);

/* grouped_linear_bias and grouped_linear_swiglu (moe_experts.h) with both
 * operands in MXFP4: x [x_rows, k], w [num_experts, n, k]; row_token gathers
 * rows of codes and of scales alike.  Everything else as stated there. */
sa_status grouped_mxfp4_linear_bias(const void* x_codes, const void* x_scales, const void* w_codes,
                                    const void* w_scales, const void* bias,
                                    const int32_t* expert_offsets, const int32_t* row_token,
                                    int x_rows, int rows, int num_experts, int n, int k, void* out,
                                    cudaStream_t stream);
sa_status grouped_mxfp4_linear_swiglu(const void* x_codes, const void* x_scales,
                                      const void* w_codes, const void* w_scales, const void* bias,
                                      const int32_t* expert_offsets, const int32_t* row_token,
                                      int x_rows, int rows, int num_experts, int n, int k,
                                      float alpha, float limit, void* out, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
