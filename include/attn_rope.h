/*
 * attn_rope.h -- C ABI of the query / key preparation of an attention layer
 * (same library as gemm.h): the RMS norm of every query and key head and the
 * rotation by its position, in one pass.
 *
 * For every token t and head (q_heads of Q, k_heads of K), on its head_dim
 * values x, in fp32, rounded once at the end:
 *   y = x * rsqrt(mean(x^2) + eps) * w        (norm; w: one vector for Q, one for K)
 *   y = x                                     (norm = 0)
 *   for i < rot_dim / 2, with (a, b) = (y[i], y[i + rot_dim/2]) in the half
 *   layout, (y[2i], y[2i+1]) in the interleaved one:
 *   (a, b) <- magnitude * (a cos p - b sin p, b cos p + a sin p),  p = position[t] * f_i
 * The values from rot_dim on are normed and not turned.
 *
 * Frequencies, radians a position: f_i = base^(-2i / rot_dim), or the
 * caller's own.  For contexts longer than the trained one (factor > 1): with
 * r_i = context * f_i / (2 pi), the turns of pair i in the trained context, a
 * pair with r_i <= low_turns is slowed to f_i / factor, one with r_i >=
 * high_turns is kept, and between them f_i * (t + (1 - t) / factor), t =
 * (r_i - low_turns) / (high_turns - low_turns).  low_turns = high_turns
 * = 0 with factor > 1 slows every pair.
 *
 * Errors are status codes (gemm_status_t); nothing aborts or prints.
 */
#ifndef LGT_ATTN_ROPE_H
#define LGT_ATTN_ROPE_H

#include <stddef.h>
#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { ATTN_ROPE_HALF = 0, ATTN_ROPE_INTERLEAVED = 1 };

typedef struct attn_rope_desc {
  int32_t q_heads;    /* >= 1 */
  int32_t k_heads;    /* >= 1 */
  int32_t head_dim;   /* a multiple of 8, at most 256 */
  int32_t rot_dim;    /* a multiple of 8, 0 .. head_dim */
  int32_t layout;     /* ATTN_ROPE_HALF or ATTN_ROPE_INTERLEAVED */
  int32_t dtype;      /* GEMM_F16 or GEMM_BF16, for Q, K, the weights and the results */
  float eps;          /* >= 0 */
  float magnitude;    /* of the rotated values; 0 = 1 */
  double base;        /* > 0 (not read when the caller gives the frequencies) */
  double factor;      /* >= 1; 0 = 1 */
  double context;     /* trained context in positions, > 0 when factor > 1 and high_turns > 0 */
  double low_turns;   /* 0 <= low_turns <= high_turns */
  double high_turns;
} attn_rope_desc_t;

typedef struct attn_rope_plan attn_rope_plan_t;

/* The frequencies `desc` stands for: rot_dim / 2 doubles (host memory). */
gemm_status_t attn_rope_frequencies(const attn_rope_desc_t* desc, double* frequencies);

/* Validate `desc` and make a plan (host state only).  `frequencies`:
 * rot_dim / 2 finite doubles in host memory, copied, or NULL for those of
 * attn_rope_frequencies. */
gemm_status_t attn_rope_create(const attn_rope_desc_t* desc, const double* frequencies, attn_rope_plan_t** plan);

/* Enqueue the pass on `stream` (a cudaStream_t; NULL = legacy default
 * stream), for the current device.
 *   Q, K: head h of token t at [t * stride + h * head_dim], strides in
 *      elements (0 = heads * head_dim; a multiple of 8, >= heads * head_dim),
 *      so both may be slices of one projection's output.
 *   q_weight, k_weight: head_dim values each; NULL for no norm of Q / of K.
 *   positions: tokens int32 (any value).
 *   q_out, k_out: as Q and K; each may be its input (same pointer and
 *      stride) and must not overlap anything else.
 * All device pointers, 16-byte aligned (positions 4).  tokens = 0 does
 * nothing.  GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT, GEMM_ERR_UNSUPPORTED
 * (2^31 or more heads in all), GEMM_ERR_CUDA (launch failure). */
gemm_status_t attn_rope_run(const attn_rope_plan_t* plan, const void* Q, int64_t q_stride, const void* K,
                            int64_t k_stride, const void* q_weight, const void* k_weight, const int32_t* positions,
                            int64_t tokens, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                            void* stream);

gemm_status_t attn_rope_destroy(attn_rope_plan_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* LGT_ATTN_ROPE_H */
