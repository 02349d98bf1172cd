/*
 * attn_cache.h -- C ABI of the paged 8-bit cache of keys and values (same
 * library as gemm.h): written token by token, read back, and attended to by
 * one new query a sequence.
 *
 * The cache.  Keys and values are kept in pages of page_size tokens; a slot
 * is page * page_size + place in the page.  The head_dim values of one token
 * and key head are e4m3 codes times a power of two of their own, the least
 * one that keeps them in e4m3's range:
 *   k, v:         uint8 codes     [pages][k_heads][page_size][head_dim]
 *   k_exp, v_exp: uint8 exponents [pages][k_heads][page_size], power + 127
 * A value is code * 2^(exponent - 127).  With amax the largest finite
 * magnitude of the row, power = ceil(log2(amax / 448)), at least -126; a row
 * without finite values other than 0 has power 0.  The division by a power of
 * two is exact, so a code is one rounding (to nearest even) of the value; an
 * infinity becomes the largest code of its sign, a NaN the NaN code.
 *
 * Errors are status codes (gemm_status_t); nothing aborts or prints.
 */
#ifndef LGT_ATTN_CACHE_H
#define LGT_ATTN_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct attn_cache {
  void* k;            /* device pointers: 16-byte aligned codes */
  void* v;
  void* k_exp;        /* any alignment */
  void* v_exp;
  int64_t pages;      /* >= 1 */
  int32_t page_size;  /* a multiple of 16, at most 1024 */
  int32_t k_heads;    /* >= 1 */
  int32_t head_dim;   /* 64 or 128 */
} attn_cache_t;

/* Enqueue the quantisation of `tokens` tokens of K and V (dtype GEMM_F16 or
 * GEMM_BF16; head h of token t at [t * stride + h * head_dim], strides in
 * elements, 0 = k_heads * head_dim, a multiple of 8) into their slots (int32,
 * device memory).  A token whose slot is negative or past the last page is
 * left out, which is the way to pad a call.  The other slots of a call are
 * distinct: where two tokens have the same one, what is left in it is
 * unspecified (codes of one with the exponent of the other, even), and no
 * other slot is touched. */
gemm_status_t attn_cache_write(const attn_cache_t* cache, const void* K, int64_t k_stride, const void* V,
                               int64_t v_stride, const int32_t* slots, int64_t tokens, int32_t dtype, void* stream);

/* Enqueue the reverse: the values of `tokens` slots into K and V, rounded
 * once to dtype (finite values beyond its range become its largest).  A slot
 * that is negative or past the last page gives zeros. */
gemm_status_t attn_cache_read(const attn_cache_t* cache, const int32_t* slots, int64_t tokens, void* K,
                              int64_t k_stride, void* V, int64_t v_stride, int32_t dtype, void* stream);

/* Bytes of device workspace attn_cache_attend needs on the current device for
 * `batch` sequences of q_heads query heads (at most 8192 sequences).  It must
 * be zero-filled before its first use and every run leaves it usable by the
 * next, of whatever heads, head_dim, type and batch it is large enough for;
 * concurrent runs need distinct workspaces. */
gemm_status_t attn_cache_attend_workspace_size(int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t batch,
                                               size_t* bytes);

/* Enqueue, for every sequence b and query head h, with n = lengths[b],
 *   out[b][h] = softmax(Q[b][h] K[b][h / (q_heads / k_heads)]^T * scale) V[b][...]
 * over the n tokens whose keys and values lie in the pages page_table[b][0],
 * [1], ...; zeros where n <= 0.
 *   Q, out: head h of sequence b at [b * stride + h * head_dim], dtype
 *      GEMM_F16 or GEMM_BF16, strides in elements (0 = q_heads * head_dim; a
 *      multiple of 8), 16-byte aligned; out must not overlap Q.
 *   q_heads: a multiple of the cache's k_heads.
 *   page_table: batch rows of max_pages int32, pitch table_stride (0 =
 *      max_pages).  A length is cut to max_pages * page_size, and a page that
 *      is not one of the cache's counts as no keys.
 *   scale > 0; 0 = 1 / sqrt(head_dim).
 * Logits, softmax and sums are fp32; the products take the codes' values as
 * they are and the queries and weights in fp16 (a query's head times a power
 * of two), which loses of a bf16 query only what is below 2^-25 of its largest
 * value and holds a weight to 2^-11.
 * The other sequences of the batch decide where a sequence's keys are cut into
 * shares, and a share's weights are rounded against a reference of its own.  So
 * the same sequence in another batch gives other bits: its fp32 sums have
 * another order, and every weight is rounded anew, each time to within 2^-11 of
 * it (below 2^-14 of the largest contribution, to within 2^-24 of that).  In the
 * same batch it gives the same bits. */
gemm_status_t attn_cache_attend(const attn_cache_t* cache, const void* Q, int64_t q_stride, int32_t q_heads,
                                const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                const int32_t* lengths, int32_t batch, float scale, int32_t dtype, void* out,
                                int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LGT_ATTN_CACHE_H */
