/*
 * attn_prompt.h -- C ABI of the attention over packed prompts (same library
 * as gemm.h).
 *
 * Sequences of different lengths stand one after the other: queries of
 * sequence b are rows cu_q[b] .. cu_q[b+1] - 1 of Q, its keys and values rows
 * cu_k[b] .. cu_k[b+1] - 1 of K and V.  For query i of nq and key j of nk,
 *   out[i][h] = softmax over visible j of (Q[i][h] . K[j][h / group] * scale), times V[j][h / group],
 * group = q_heads / k_heads; key j is visible when causal = 0 or
 * j <= i + nk - nq: the last query sees the last key, so a later piece of a
 * prompt attends to all keys before it, and a single new query to all keys.
 * A query with no visible key (no keys, or nk < nq) gives zeros.  Nothing of
 * another sequence's rows reaches a result.
 *
 * Logits, softmax and sums in fp32; the weights are rounded to the input type
 * for the second product (an fp16 one below 2^-14 of the row's largest so far
 * to 2^-25 of that); one rounding of the result.
 *
 * Errors are status codes (gemm_status_t); nothing aborts or prints.
 */
#ifndef LGT_ATTN_PROMPT_H
#define LGT_ATTN_PROMPT_H

#include <stddef.h>
#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct attn_prompt_desc {
  int32_t q_heads;   /* a multiple of k_heads, at most 128 times it */
  int32_t k_heads;   /* >= 1 */
  int32_t head_dim;  /* 64 or 128 */
  int32_t dtype;     /* GEMM_F16 or GEMM_BF16, for Q, K, V and out */
  int32_t causal;    /* 0 or 1 */
  float scale;       /* > 0; 0 = 1 / sqrt(head_dim) */
} attn_prompt_desc_t;

typedef struct attn_prompt_plan attn_prompt_plan_t;

/* Validate `desc` and make a plan (host state and a 16-byte device status
 * word on the current device).  GEMM_ERR_INVALID_ARG, or GEMM_ERR_CUDA when
 * no device is usable. */
gemm_status_t attn_prompt_create(const attn_prompt_desc_t* desc, attn_prompt_plan_t** plan);

/* Enqueue the pass on `stream` (a cudaStream_t; NULL = legacy default
 * stream).
 *   Q, out: total_q rows, K, V: total_k rows; head h of row t at
 *      [t * stride + h * head_dim], strides in elements (0 = heads *
 *      head_dim; a multiple of 8), so each may be a slice of a projection's
 *      output; device pointers, 16-byte aligned; out overlaps no input.
 *   cu_q, cu_k: batch + 1 int32 in device memory, not decreasing, from 0 to
 *      at most total_q, total_k (values beyond are cut to those); rows of out
 *      that belong to no sequence are left as they are.
 * batch = 0 or total_q = 0 does nothing.  The plan's device must be current.
 * GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT, GEMM_ERR_UNSUPPORTED (more than
 * 2^30 rows or 2^20 sequences, or 2^31 or more work units), GEMM_ERR_CUDA (launch failure).  A kernel whose bounded wait ran out
 * records GEMM_ERR_TIMEOUT in the plan's status word
 * (attn_prompt_sync_status); out is then invalid. */
gemm_status_t attn_prompt_run(attn_prompt_plan_t* plan, const void* Q, int64_t q_stride, const void* K,
                              int64_t k_stride, const void* V, int64_t v_stride, const int32_t* cu_q,
                              const int32_t* cu_k, int32_t batch, int64_t total_q, int64_t total_k, void* out,
                              int64_t out_stride, void* stream);

/* Synchronise `stream`, read and clear the plan's status word: GEMM_OK or
 * GEMM_ERR_TIMEOUT. */
gemm_status_t attn_prompt_sync_status(attn_prompt_plan_t* plan, void* stream);

/* Test aid for failure detection, without a fault: the plan's next run leaves
 * out the first load of keys of one CTA, so the CTA's waits run out after the
 * plan's limit (LGT_GEMM_WAIT_LIMIT_MS at attn_prompt_create, 2 s by default).
 * It winds down -- the copies that it did make land first -- and the run's
 * status is GEMM_ERR_TIMEOUT; runs after it are normal. */
gemm_status_t attn_prompt_withhold_load(attn_prompt_plan_t* plan);

gemm_status_t attn_prompt_destroy(attn_prompt_plan_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* LGT_ATTN_PROMPT_H */
