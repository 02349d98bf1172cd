/*
 * row_groups.h -- C ABI that puts rows in order by the group that each belongs
 * to (same library as gemm.h): what products with weights of their own for each
 * group of rows (gemm_grouped.h) and adapters (adapters.h) start from.
 *
 * Errors are status codes (gemm_status_t); nothing aborts or prints.
 */
#ifndef LGT_ROW_GROUPS_H
#define LGT_ROW_GROUPS_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Enqueue on `stream`, from ids[r], the group of row r (device memory):
 *   offsets[g] = the number of rows of groups before g, for g = 0 .. groups;
 *   order: the rows of group 0, of group 1, ..., then those of no group (an id
 *      below 0 or from `groups` on), ascending within each;
 *   places: the reverse, order[places[r]] = r; may be NULL.
 * offsets holds groups + 1 values, the others `rows`, all int32 in device memory
 * and apart from each other.  Whole numbers from counts alone: the same ids give
 * the same results.  No workspace, one launch.
 * groups: 1 to 1024.  rows: 0 to 2^30.
 * GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT, GEMM_ERR_UNSUPPORTED (more rows),
 * GEMM_ERR_CUDA (launch failure). */
gemm_status_t gemm_row_groups(const int32_t* ids, int64_t rows, int32_t groups, int32_t* offsets, int32_t* order,
                              int32_t* places, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LGT_ROW_GROUPS_H */
