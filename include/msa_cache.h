/*
 * msa_cache.h -- C ABI of libmsa's 8-bit KV cache.
 *
 * An 8-bit KV cache, and what a serving loop does with it: append the new
 * tokens' keys and values, attend to it (in full, over a window, or over a
 * window and the blocks each query selects), and evict slots by the
 * attention they drew.  ("Million Token Context Window Optimization: What
 * Actually Works", section "The indexing game", attends a history window and
 * the top-k chunks of an index; "Training at 1M+ Token Context" sizes the
 * 70B layer's KV cache at 2 GB in bf16 for a million tokens.  The pages
 * define no format: it is fixed here.)
 *
 * The cache is a pool of pages.  A page holds one block of `block` token
 * slots (32, 64, 128 or 256) of one sequence, for all KV heads:
 *   k_codes, v_codes [n_pages, Hkv, block, d]  e4m3 (S.EEEE.MMM, no infinity)
 *   k_scale, v_scale [n_pages, Hkv]            fp32
 *   k_mean           [n_pages, Hkv, d]         bf16: mean of the block's keys
 * A slot stands for code * scale.  Block j of sequence b is page
 * table[b * max_blocks + j]; sequence b holds lens[b] slots, in order, in its
 * first ceil(lens[b] / block) blocks.  table [batch, max_blocks] and lens
 * [batch] are device int32 arrays; a table entry past a sequence's last block
 * is never read.  A sequence of length 0 (a padded batch) is allowed
 * everywhere.
 *   The scale msa_cache_append gives a block is 2^e, e the least exponent
 * (>= -126) with amax <= 448 * 2^e over the block's slots; 0 for a block of
 * zeros; NaN, with codes of 0, for a block that holds a NaN or an infinity
 * (every row that attends a slot of such a block gets NaN; its lse and weights
 * too where the block's keys hold it).  The attention
 * takes any finite scale >= 0 and finite codes; an append to a block that holds
 * slots and an eviction take the powers of two that these two write.  k_mean
 * is written when a block becomes full: the mean of its keys code * scale,
 * rounded once.
 *   The pages of one sequence are distinct.  Pages of full blocks may be
 * shared between sequences (a common prefix): the attention and the
 * selection only read, an append writes only the blocks that take new slots
 * (which must not be shared), an eviction writes only dst_table's pages.  A
 * sequence's last slots (rejected drafts) are dropped by lowering its length;
 * the block that then ends it keeps its scale.
 * Device data is checked by the kernels: a length outside [0, max_blocks *
 * block] is clamped (an append skips the sequence), a slot whose page is not in
 * [0, n_pages) is left out (not written, not attended; an eviction that keeps it
 * gathers zeros), and MSA_ERR_INVALID_ARG is recorded in the device status word
 * (msa_device_status).
 * Conventions of every entry point: as in msa.h.
 */
#ifndef MSA_CACHE_H_
#define MSA_CACHE_H_

#include "msa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct msa_kv_cache {
    void *k_codes, *v_codes;  /* 16-byte aligned */
    float *k_scale, *v_scale; /* 4-byte aligned */
    void *k_mean;             /* 16-byte aligned */
    int64_t n_pages;
    int Hkv;
    int d;     /* 64 or 128 */
    int block; /* slots a page: 32, 64, 128 or 256 */
} msa_kv_cache;

/*
 * Appends tokens: sequence b's new keys and values are the rows cu[b] ..
 * cu[b+1]-1 of k and v, and become its last slots, lens[b] being the length
 * AFTER the append (so slot lens[b] - (cu[b+1] - cu[b]) is the first new
 * one).  Works for a whole prompt and for single tokens.
 *   k, v   [total, Hkv, d] in `in_dt`
 *   cu     [batch + 1] device int32, ascending
 *   max_new  at least the largest cu[b+1] - cu[b] (it sizes the launch;
 *            0 does nothing)
 *   table  must name a page for every block that takes a new slot.
 * A block that already held slots keeps the larger of its scale and the one
 * the new slots need; if that grew, the old codes are rounded to it (exact
 * above e4m3's subnormals).  Slots past lens[b] are left as they were.
 * Appending the same tokens again (same lens) changes nothing.
 * Errors: INVALID_ARG for null or misaligned pointers, sizes below 1 or out
 * of range, max_new > total; UNSUPPORTED if d is not 64 or 128 or block not
 * one of the four.  A sequence whose rows do not lie in [0, total], number
 * more than max_new or exceed lens[b], or whose length cannot be, is skipped
 * and MSA_ERR_INVALID_ARG recorded in the device status word.
 */
msa_status msa_cache_append(const msa_kv_cache *cache, const void *k,
                            const void *v, const int32_t *cu, int64_t total,
                            int64_t max_new, const int32_t *table,
                            int max_blocks, const int32_t *lens, int batch,
                            msa_dtype in_dt, msa_stream_t stream);

/* Bytes of workspace msa_cache_attn needs (0 for invalid sizes); the pointers
 * in `cache` are not looked at.  With weights it holds every row's scores:
 * 4 * batch * n_q * Hq * max_blocks * block bytes more. */
size_t msa_cache_attn_workspace_size(const msa_kv_cache *cache, int max_blocks,
                                     int batch, int n_q, int Hq,
                                     int with_weights, msa_dtype in_dt);

/*
 * Attention of n_q query tokens of each sequence over its cached slots, the
 * query tokens' own among them: row t of sequence b is at position p =
 * lens[b] - n_q + t and attends the slots j with p - window < j <= p; one
 * softmax, scores scale * <q, k>.
 *   q        [batch, n_q, Hq, d] in `in_dt`
 *   window   >= 1; max_blocks * block or more: every slot up to p
 *   out      [batch, n_q, Hq, d] in `out_dt`, written
 *   lse      [batch, Hq, n_q] fp32, written
 *   weights  NULL, or [batch, Hkv, weights_ld] fp32, weights_ld >= max_blocks
 *            * block: the softmax weight that slot j drew, summed over the n_q
 *            rows and the query heads of KV head c, is added to
 *            weights[(b * Hkv + c) * weights_ld + j]
 * A row with nothing to attend (p < 0) gets out = 0 and lse = -inf.
 * bf16 queries run on the tensor cores (halves of 11 bits for the softmax
 * weights, fp32 sums), fp32 ones on the CUDA cores in fp32.  The result does
 * not depend on the run (no atomics), but its rounding does on the whole
 * batch's lengths, which decide where long sequences are cut.
 * Errors: INVALID_ARG for null or misaligned pointers or sizes out of range,
 * Hq % Hkv != 0, window < 1, scale not finite and > 0, a null, misaligned
 * (256 bytes) or too small workspace; UNSUPPORTED for d, block as above, n_q *
 * Hq / Hkv > 4096, or batch * Hkv > 65535 with weights.
 */
msa_status msa_cache_attn(const msa_kv_cache *cache, const void *q,
                          const int32_t *table, int max_blocks,
                          const int32_t *lens, int batch, int n_q, int Hq,
                          int64_t window, float scale, void *out, float *lse,
                          float *weights, int64_t weights_ld, msa_dtype in_dt,
                          msa_dtype out_dt, void *workspace,
                          size_t workspace_bytes, msa_stream_t stream);

/* Bytes of workspace msa_cache_select needs (0 for invalid sizes): about
 * 16 * batch * n_q * Hkv * max_blocks. */
size_t msa_cache_select_workspace_size(const msa_kv_cache *cache,
                                       int max_blocks, int batch, int n_q);

/*
 * Block selection for single query tokens (msa_block_select takes 128 rows
 * together): for query token t of sequence b at position p = lens[b] - n_q +
 * t, and KV head c, block l scores
 *   score(l) = sum over query heads h of c's group of <q_h, k_mean_l>,
 * for the blocks wholly before the window, (l+1) * block <= p - window + 1.
 * The min(top_k, #candidates) best are chosen, ties to the lower index, as
 * the scores are in 64-bit arithmetic (a head sum's own rounding 2^-48 * Hq /
 * Hkv of its magnitudes at most); NaN ranks last.
 *   sel  [batch, n_q, Hkv, top_k] int32, written: chosen blocks ascending,
 *        then -1
 *   cnt  [batch, n_q, Hkv] int32, written: how many were chosen
 * Errors: as msa_cache_attn, plus INVALID_ARG unless 1 <= top_k <= max_blocks.
 */
msa_status msa_cache_select(const msa_kv_cache *cache, const void *q,
                            const int32_t *table, int max_blocks,
                            const int32_t *lens, int batch, int n_q, int Hq,
                            int64_t window, int top_k, int32_t *sel,
                            int32_t *cnt, msa_dtype in_dt, void *workspace,
                            size_t workspace_bytes, msa_stream_t stream);

/* Bytes of workspace msa_cache_attn_select needs (0 for invalid sizes). */
size_t msa_cache_attn_select_workspace_size(const msa_kv_cache *cache,
                                            int max_blocks, int batch, int n_q,
                                            int Hq, msa_dtype in_dt);

/*
 * msa_cache_attn over each row's window plus every slot of the first
 * cnt[b, t, c] blocks of sel[b, t, c, :] (as msa_cache_select wrote them for
 * the same sizes; a shorter list is allowed, a block must not appear twice).
 * Errors: as msa_cache_attn and msa_cache_select.  A count or block that
 * cannot be (see msa_attn_fwd_select) is clamped and MSA_ERR_INVALID_ARG
 * recorded in the device status word.
 */
msa_status msa_cache_attn_select(const msa_kv_cache *cache, const void *q,
                                 const int32_t *table, int max_blocks,
                                 const int32_t *lens, int batch, int n_q,
                                 int Hq, int64_t window, const int32_t *sel,
                                 const int32_t *cnt, int top_k, float scale,
                                 void *out, float *lse, msa_dtype in_dt,
                                 msa_dtype out_dt, void *workspace,
                                 size_t workspace_bytes, msa_stream_t stream);

/* Bytes of workspace msa_cache_attn_topk needs (0 for invalid sizes). */
size_t msa_cache_attn_topk_workspace_size(const msa_kv_cache *cache,
                                          int max_blocks, int batch, int n_q,
                                          int Hq, int top_k, msa_dtype in_dt);

/* msa_cache_select and msa_cache_attn_select in one call, the selection kept
 * in the workspace.  Errors: as the two. */
msa_status msa_cache_attn_topk(const msa_kv_cache *cache, const void *q,
                               const int32_t *table, int max_blocks,
                               const int32_t *lens, int batch, int n_q, int Hq,
                               int64_t window, int top_k, float scale,
                               void *out, float *lse, msa_dtype in_dt,
                               msa_dtype out_dt, void *workspace,
                               size_t workspace_bytes, msa_stream_t stream);

/*
 * Eviction by accumulated attention weight: of each sequence and KV head the
 * last min(recent, K) slots are kept and, of the others, those of the
 * greatest weight, K = min(lens[b], budget) in all, ties to the lower slot
 * (NaN counts as the greatest).  The kept slots, in their order, become slots
 * 0 .. K-1 of the pages dst_table[b, 0 .. ceil(K / block)), which get scales
 * (and k_mean) as an append of the values code * scale would give them.
 * Different heads keep different tokens.
 *   weights     [batch, Hkv, weights_ld] fp32, weights_ld >= max_blocks *
 *               block, as msa_cache_attn accumulated them
 *   dst_table   [batch, dst_blocks] device int32; its pages must not be among
 *               those being read, nor repeat; budget <= dst_blocks * block
 *   new_lens    [batch] int32, written: K
 *   kept        [batch, Hkv, budget] int32, written: kept slots ascending,
 *               then -1
 *   new_weights [batch, Hkv, new_weights_ld] fp32, new_weights_ld >= budget,
 *               written: the kept slots' weights, then 0
 * Errors: INVALID_ARG for null or misaligned pointers, sizes out of range,
 * recent > budget, new_lens == lens or new_weights == weights; UNSUPPORTED as
 * above.
 */
msa_status msa_cache_evict(const msa_kv_cache *cache, const int32_t *table,
                           int max_blocks, const int32_t *lens, int batch,
                           const float *weights, int64_t weights_ld,
                           int64_t budget, int64_t recent,
                           const int32_t *dst_table, int dst_blocks,
                           int32_t *new_lens, int32_t *kept,
                           float *new_weights, int64_t new_weights_ld,
                           msa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_CACHE_H_ */
