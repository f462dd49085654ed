/*
 * linear_bias.h -- bias-seeded linear layer of libsinkattn.so (sm_103a), the
 * GEMM shape that follows sink attention (the output projection) and runs the
 * experts.
 *
 * The page "GPT-OSS on day 0" (Perplexity, 2025) states in its model overview
 * that the output projection and the experts carry bias terms, and in section
 * "Kernels for GPT-OSS / MoE" that bias support was added to the GEMM kernels
 * by initialising the accumulator from the bias values, once per output tile.
 * This call computes
 *
 *     out[m, n] = sum_k x[m, k] * w[n, k] + bias[n]
 *
 * on the tcgen05 tensor cores: bf16 inputs, fp32 accumulation in tensor
 * memory that starts from the bias (no separate bias add), bf16 output
 * (round to nearest even).
 *
 *  x    bf16 [m, k] row-major;   w bf16 [n, k] row-major (one row per output
 *       feature, the layout of a PyTorch Linear weight);  bias bf16 [n] or NULL
 *  out  bf16 [m, n] row-major
 *  n and k must be multiples of 8 (16-byte rows for the tensor-memory copies);
 *  any m >= 0.  x, w, out 16-byte aligned.
 *
 * Conventions of sink_attn.h apply (device pointers, asynchronous on
 * `stream`, no allocation).  Status: SA_ERR_SHAPE (m < 0, n or k <= 0 or > 2^30,
 * more than 2^31 - 1 output tiles),
 * SA_ERR_UNSUPPORTED (n or k not a multiple of 8), SA_ERR_NULL,
 * SA_ERR_ALIGNMENT, SA_ERR_CUDA / SA_ERR_LAUNCH; m == 0 launches nothing.
 * A device wait that runs out of time (sink_attn_set_wait_timeout_ns) stops
 * the kernel cleanly and sets SA_ERR_TIMEOUT in the device status word.
 */
#ifndef LINEAR_BIAS_H
#define LINEAR_BIAS_H

#include "sink_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

sa_status linear_bias(const void* x, const void* w, const void* bias, int m, int n, int k,
                      void* out, cudaStream_t stream);

/*
 * The same layer with the low-rank adapters of many requests at once beside it:
 *
 *     out[m] = x[m] W^T + bias + s_a (x[m] A_a^T) B_a^T,    a = adapter_idx[m]
 *
 * and without the last term where adapter_idx[m] is negative.  x A^T is summed in fp32, times
 * s_a rounded once to bf16 for the second product; everything adds up in the fp32 accumulator
 * that starts from the bias, and the result rounds once to bf16.  Rows stand alone: a NaN or an infinity
 * in one token's x or adapter does not reach others (outputs of theirs that it would have reached
 * are computed once more, which takes longer the more of them there are).
 *
 *  x, w, bias, out, m, n, k: as for linear_bias
 *  lora_a       bf16 [num_adapters, rank, k], lora_b bf16 [num_adapters, n, rank], 16-byte
 *               aligned; rank a multiple of 8, at most 128 (adapters of lower rank are padded
 *               with zeros); num_adapters 1..1024
 *  lora_scale   fp32 [num_adapters] or NULL (1)
 *  adapter_idx  int32 [m], device, in any order.  An index >= num_adapters counts as none and
 *               sets SA_ERR_BOUNDS in the device status word.
 *  workspace    as many bytes of device memory as lora_workspace_bytes says, 16-byte aligned,
 *               overwritten; calls that overlap on the GPU, captured graphs among them, need
 *               workspaces of their own
 * Status codes as for linear_bias (SA_ERR_SHAPE also for rank <= 0, num_adapters out of range and
 * more than 65535 * 128 tokens; SA_ERR_UNSUPPORTED for other ranks).
 */
sa_status lora_linear_bias(const void* x, const void* w, const void* bias, const void* lora_a,
                           const void* lora_b, const float* lora_scale, const int32_t* adapter_idx,
                           int m, int n, int k, int rank, int num_adapters, void* workspace,
                           void* out, cudaStream_t stream);

/* Bytes of workspace for lora_linear_bias into *bytes (0 for sizes that it refuses or does
 * nothing for).  No CUDA call. */
void lora_workspace_bytes(int m, int k, int rank, long long* bytes);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_BIAS_H */
