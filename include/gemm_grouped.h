/*
 * gemm_grouped.h -- C ABI of products over groups of rows (same library as
 * gemm.h): every group has a matrix of its own, as the experts of a layer do.
 * The rows of group g are offsets[g] .. offsets[g + 1] - 1; the sizes are known
 * on the device only (row_groups.h makes them) and any of them may be 0.
 *
 * GEMM_GROUPED_M, groups along M:
 *   C[r][n] = sum over k of A[r][k] * B[g][k, n],  r in group g.
 * B as b_layout says: GEMM_K_CONTIG [g][n][k], GEMM_MN_CONTIG [g][k][n].  The
 * gradient to A is the same product with the other layout.
 *
 * GEMM_GROUPED_K, groups along K: the gradient to the matrices,
 *   C[g][m][n] = sum over r in group g of A[r][m] * B[r][n],
 * zeros for a group without rows.
 *
 * fp16 or bf16, all of one type; sums in fp32, one rounding of the result.  A
 * row or value of another group, or behind the last, reaches no result,
 * infinities and NaN included.  Repeated calls give the same bits; with another number
 * of rows or groups K may be summed in parts, and so in another order.
 *
 * Errors are status codes (gemm_status_t); nothing aborts or prints.
 */
#ifndef LGT_GEMM_GROUPED_H
#define LGT_GEMM_GROUPED_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_GROUPED_M 0
#define GEMM_GROUPED_K 1

typedef struct gemm_grouped_desc {
  int32_t groups;    /* 1 to 1024 */
  int32_t form;      /* GEMM_GROUPED_M or GEMM_GROUPED_K */
  int64_t M;         /* GEMM_GROUPED_K: rows of each C[g]; else 0 */
  int64_t N;         /* columns of C */
  int64_t K;         /* GEMM_GROUPED_M: columns of A; else 0 */
  int32_t b_layout;  /* GEMM_GROUPED_M: GEMM_K_CONTIG or GEMM_MN_CONTIG; else GEMM_MN_CONTIG */
  int32_t dtype;     /* GEMM_F16 or GEMM_BF16, for A, B and C */
} gemm_grouped_desc_t;

typedef struct gemm_grouped_plan gemm_grouped_plan_t;

/* Validate `desc` and make a plan (host state and a 16-byte device status word
 * on the current device; without a device the plan's runs are refused).  M, N
 * and K are multiples of 8 below 2^30.  GEMM_ERR_INVALID_ARG, GEMM_ERR_CUDA. */
gemm_status_t gemm_grouped_create(const gemm_grouped_desc_t* desc, gemm_grouped_plan_t** plan);

/* Enqueue the products on `stream` (a cudaStream_t; NULL = legacy default
 * stream).
 *   A: `rows` rows of pitch lda; GEMM_GROUPED_K: B too, of pitch ldb.
 *   GEMM_GROUPED_M: B is `groups` matrices of row pitch ldb, b_stride apart, and
 *      C `rows` rows of pitch ldc (b_stride is of no meaning for
 *      GEMM_GROUPED_K, c_stride for GEMM_GROUPED_M).
 *   GEMM_GROUPED_K: C is `groups` matrices of row pitch ldc, c_stride apart.
 *   Pitches and strides in elements, multiples of 8, no less than the row (or
 *   the matrix) that they lead over; 0 = dense.  Device pointers, 16-byte
 *   aligned; C overlaps no input.
 *   offsets: groups + 1 int32 in device memory, not decreasing, from 0 or more to
 *      at most `rows` (values beyond are cut to it, one that is less than an
 *      earlier one counts as that one).  Rows of C that belong to no group are
 *      left as they are.
 * rows = 0 does nothing for GEMM_GROUPED_M.  The plan's device must be current.
 * A plan holds no workspace: runs of it may be under way at the same time.
 * GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT, GEMM_ERR_UNSUPPORTED (more than 2^30
 * rows, or 2^31 or more tiles), GEMM_ERR_CUDA (launch failure).  A kernel whose
 * bounded wait ran out records GEMM_ERR_TIMEOUT in the plan's status word
 * (gemm_grouped_sync_status); C is then invalid. */
gemm_status_t gemm_grouped_run(gemm_grouped_plan_t* plan, const void* A, int64_t lda, const void* B, int64_t ldb,
                               int64_t b_stride, const int32_t* offsets, int64_t rows, void* C, int64_t ldc,
                               int64_t c_stride, void* stream);

/* Synchronise `stream`, read and clear the plan's status word: GEMM_OK or
 * GEMM_ERR_TIMEOUT. */
gemm_status_t gemm_grouped_sync_status(gemm_grouped_plan_t* plan, void* stream);

/* Test aid for failure detection, without a fault: the plan's next run leaves
 * out one CTA's first load of A's rows, so waits run out after the plan's limit
 * (LGT_GEMM_WAIT_LIMIT_MS at gemm_grouped_create, 2 s by default), the kernel
 * winds down and the run's status is GEMM_ERR_TIMEOUT; runs after it are
 * normal. */
gemm_status_t gemm_grouped_withhold_load(gemm_grouped_plan_t* plan);

gemm_status_t gemm_grouped_destroy(gemm_grouped_plan_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* LGT_GEMM_GROUPED_H */
