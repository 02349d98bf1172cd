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
 * row's largest finite one and cannot overflow, with the scale neither; one rounding
 * of out.  An infinite value of x, A or B gives the infinity, or the NaN, that the
 * formula gives.  A row reaches no other row's result, whatever it holds.  Repeated
 * calls give the same bits; with another number of rows, or an order where there was
 * none, K may be summed in other parts.
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

typedef struct gemm_adapters_plan gemm_adapters_plan_t;

/* Validate `desc` and make a plan (host state and a 16-byte device status word
 * on the current device; without a device the plan's runs are refused).
 * LGT_GEMM_ADAPTERS_FORM in the environment, for tests and measurements: the form
 * that the plan's runs take where the sizes allow it, 0 the one for few rows, 1, 2,
 * 4, 8 the one for many rows with so many CTAs a tile.
 * LGT_GEMM_ADAPTERS_ROWS, likewise: 8, 16 or 32 rows a tile of the form for few rows
 * (16 for ranks up to 64, 32 up to 32 and from 72).
 * GEMM_ERR_INVALID_ARG, GEMM_ERR_CUDA. */
gemm_status_t gemm_adapters_create(const gemm_adapters_desc_t* desc, gemm_adapters_plan_t** plan);

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
 * rows = 0 does nothing.  The plan's device must be current.  A plan holds no
 * workspace: runs of it may be under way at the same time.
 * GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT, GEMM_ERR_UNSUPPORTED (more than 2^30
 * rows), GEMM_ERR_CUDA (launch failure).  A kernel whose bounded wait ran out
 * records GEMM_ERR_TIMEOUT in the plan's status word
 * (gemm_adapters_sync_status); out is then invalid. */
gemm_status_t gemm_adapters_run(gemm_adapters_plan_t* plan, const void* x, int64_t x_stride, const void* A, const void* B,
                                const float* scales, const int32_t* offsets, const int32_t* order, int64_t rows,
                                const void* base, int64_t base_stride, void* out, int64_t out_stride, void* stream);

/* Synchronise `stream`, read and clear the plan's status word: GEMM_OK or
 * GEMM_ERR_TIMEOUT. */
gemm_status_t gemm_adapters_sync_status(gemm_adapters_plan_t* plan, void* stream);

/* Test aid for failure detection, without a fault: the plan's next run on the
 * form for many rows leaves out one CTA's first load of A, so
 * waits run out after the plan's limit (LGT_GEMM_WAIT_LIMIT_MS at
 * gemm_adapters_create, 2 s by default), the kernel winds down and the run's
 * status is GEMM_ERR_TIMEOUT; runs after it are normal. */
gemm_status_t gemm_adapters_withhold_load(gemm_adapters_plan_t* plan);

gemm_status_t gemm_adapters_destroy(gemm_adapters_plan_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* LGT_ADAPTERS_H */
