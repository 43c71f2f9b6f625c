/*
 * msa_cache4.h -- C ABI of libmsa's 4-bit KV cache, and of reading either
 * cache back.
 *
 * The 4-bit cache holds a token in half the bytes of the 8-bit one
 * (msa_cache.h), whose pages, block tables and lengths it shares; the element
 * and scale types are those of the OCP Microscaling format MXFP4.  A page
 * holds one block of `block` token slots (32, 64, 128 or 256) of one sequence,
 * for all KV heads:
 *   k_codes, v_codes [n_pages, Hkv, block, d / 2]   two e2m1 codes a byte, the
 *                    even dim in the low four bits (S.EE.M: 0, 0.5, 1, 1.5, 2,
 *                    3, 4, 6 and their negatives)
 *   k_scale, v_scale [n_pages, Hkv, block, d / 32]  e8m0: the byte x stands
 *                    for 2^(x - 127), 255 for NaN
 * Dim i of a slot stands for its code times the scale i / 32.  Every slot has
 * scales of its own: what an append writes does not depend on what the block
 * holds, and nothing is rounded twice.
 *   The scale msa_cache4_append gives 32 values is 2^e, e the least exponent
 * (>= -126) with amax <= 7 * 2^e; values are rounded to the nearest code, ties
 * to the even one, those above 6 * 2^e to it (where amax lies between 6 and 7
 * times 2^e, twice the scale would bring the largest value no nearer, and the
 * others further off).  32 zeros beside other values have the largest scale of
 * the slot and head (so that heads held with zeros behind them cost an attention
 * nothing), a slot of zeros the least.  Where a slot's key (or value) of one head holds a NaN,
 * an infinity or a magnitude above 1.75 * 2^127, which no code stands for, all
 * its scales are 255 and its codes 0.
 * Conventions of every entry point, and what is checked on the device: as in
 * msa_cache.h; besides, n_pages * Hkv * block >= 2^32 - 1 is UNSUPPORTED.
 */
#ifndef MSA_CACHE4_H_
#define MSA_CACHE4_H_

#include "msa_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct msa_kv_cache4 {
    void *k_codes, *v_codes; /* 16-byte aligned */
    void *k_scale, *v_scale; /* 16-byte aligned */
    int64_t n_pages;
    int Hkv;
    int d;     /* 64 or 128 */
    int block; /* slots a page: 32, 64, 128 or 256 */
} msa_kv_cache4;

/*
 * msa_cache_append for the 4-bit cache: the same arguments, the same checks
 * and errors.  Only the new slots are written (not the others of their
 * blocks).
 */
msa_status msa_cache4_append(const msa_kv_cache4 *cache, const void *k,
                             const void *v, const int32_t *cu, int64_t total,
                             int64_t max_new, const int32_t *table,
                             int max_blocks, const int32_t *lens, int batch,
                             msa_dtype in_dt, msa_stream_t stream);

/* Bytes of workspace msa_cache4_attn needs (0 for invalid sizes); the pointers
 * in `cache` are not looked at. */
size_t msa_cache4_attn_workspace_size(const msa_kv_cache4 *cache,
                                      int max_blocks, int batch, int n_q,
                                      int Hq, msa_dtype in_dt);

/*
 * msa_cache_attn for the 4-bit cache, without weights: attention of n_q query
 * tokens of each sequence over its cached slots, the query tokens' own among
 * them; the same arguments, checks and errors.  A row that attends a slot
 * whose key has a scale of 255 gets NaN and an lse of NaN; one that attends a
 * slot whose value has one gets NaN in every dim, its lse stays.
 * All rows run on the tensor cores.  Codes times scales are halves, exactly
 * where a scale is no less than 2^-27 of the largest of the same slot, head and
 * side (a smaller one counts as 0).  bf16 queries and softmax weights are one
 * half each (11 bits), fp32 ones two (22 bits); a weight below 2^-23 of the
 * row's largest is off by 2^-33 of that one (its product with the value by at most
 * 2^-20 of the row's largest product, where values lie far apart).  Sums are fp32.
 * As with the 8-bit cache the result does not depend on the run, but its rounding
 * does on the whole batch's lengths; here also on max_blocks and window (and the
 * sizes), which choose the rows and chunks taken together: a wider table can give
 * other last bits.
 */
msa_status msa_cache4_attn(const msa_kv_cache4 *cache, const void *q,
                           const int32_t *table, int max_blocks,
                           const int32_t *lens, int batch, int n_q, int Hq,
                           int64_t window, float scale, void *out, float *lse,
                           msa_dtype in_dt, msa_dtype out_dt, void *workspace,
                           size_t workspace_bytes, msa_stream_t stream);

/*
 * Reads a cache back as rows of keys and values: of sequence b the last
 * cu[b+1] - cu[b] of its lens[b] slots go to the rows cu[b] .. cu[b+1]-1 of k
 * and v, as msa_cache_append takes them (any range of a sequence is read with
 * lens[b] lowered to its end).  A value is code * scale, rounded once to
 * `out_dt`.
 *   k, v    [total, Hkv, d] in `out_dt`; rows of no sequence are left as they
 *           were
 *   cu      [batch + 1] device int32, ascending
 *   max_rows  at least the largest cu[b+1] - cu[b] (it sizes the launch; 0
 *           does nothing)
 * A slot whose page is not in [0, n_pages) reads as zeros and
 * MSA_ERR_INVALID_ARG is recorded in the device status word; a sequence that
 * an append would skip is skipped likewise.
 * Errors: as msa_cache_append.
 */
msa_status msa_cache_read(const msa_kv_cache *cache, const int32_t *cu,
                          int64_t total, int64_t max_rows,
                          const int32_t *table, int max_blocks,
                          const int32_t *lens, int batch, void *k, void *v,
                          msa_dtype out_dt, msa_stream_t stream);
msa_status msa_cache4_read(const msa_kv_cache4 *cache, const int32_t *cu,
                           int64_t total, int64_t max_rows,
                           const int32_t *table, int max_blocks,
                           const int32_t *lens, int batch, void *k, void *v,
                           msa_dtype out_dt, msa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_CACHE4_H_ */
