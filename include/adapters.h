/*
 * adapters.h -- C ABI of low-rank adapters beside a shared projection (same
 * library as gemm.h): many requests in one batch, each with an adapter of its
 * own or with none.
 *
 *   out[r] = base[r] + scale[g] * (x[r] A[g]^T) B[g]^T,   r in group g,
 *   out[r] = base[r],                                     r in no group.
 *
 * base is what the shared projection (gemm_run, in any of its forms) gave for x.
 * The rows of group g are order[offsets[g]] .. order[offsets[g + 1] - 1]
 * (row_groups.h makes both from the rows' adapter numbers), or, where order is
 * NULL, offsets[g] .. offsets[g + 1] - 1 themselves.
 *
 * fp16 or bf16, all of one type; sums in fp32.  The first product's result u
 * goes into the second one as two values of the type, u = (hi + lo) * 2^p with p
 * the row's, so that it loses no more than 2^-16 (bf16) or 2^-21 (fp16) of the
 * row's largest and cannot overflow; one rounding of out.  A row reaches no
 * other row's result, whatever it holds.  Repeated calls give the same bits.
 *
 * Errors are status codes (gemm_status_t); nothing aborts or prints.
 */
#ifndef LGT_ADAPTERS_H
#define LGT_ADAPTERS_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_adapters_desc {
  int32_t groups;  /* 1 to 1024 */
  int32_t rank;    /* a multiple of 8, at most 128 */
  int64_t N;       /* columns of base and out */
  int64_t K;       /* columns of x; both multiples of 8 below 2^30 */
  int32_t dtype;   /* GEMM_F16 or GEMM_BF16 */
} gemm_adapters_desc_t;

/* Enqueue the pass on `stream` (a cudaStream_t; NULL = legacy default stream).
 *   x, base, out: `rows` rows of pitch x_stride, base_stride, out_stride, in
 *      elements (0 = dense; multiples of 8).  out may be base itself, with its
 *      pitch; else it overlaps no input.
 *   A: [groups][rank][K], B: [groups][N][rank], dense (an adapter of a smaller
 *      rank ends in zeros).
 *   scales: fp32 [groups], or NULL for 1.
 *   offsets: groups + 1 int32, not decreasing, from 0 or more to at most `rows`
 *      (as in gemm_grouped.h).  order: `rows` int32, all different; one that is no
 *      row's number is left out.  Both in device memory.
 * Device pointers, 16-byte aligned (scales, offsets and order: 4).
 * rows = 0 does nothing.
 * GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT, GEMM_ERR_UNSUPPORTED (more than 2^30
 * rows), GEMM_ERR_CUDA (launch failure). */
gemm_status_t gemm_adapters_run(const gemm_adapters_desc_t* desc, const void* x, int64_t x_stride, const void* A,
                                const void* B, const float* scales, const int32_t* offsets, const int32_t* order,
                                int64_t rows, const void* base, int64_t base_stride, void* out, int64_t out_stride,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LGT_ADAPTERS_H */
