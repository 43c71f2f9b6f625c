/*
 * msa_rope.h -- C ABI of libmsa's norms of queries and keys for each head,
 * with the rotary position embedding in the same pass, and their gradients.
 *
 * What stands between a layer's projections and its attention or its cache.
 * Of each row x (one token and head, d values):
 *   z = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)   (z = x without a weight w)
 * and every pair (a, b) of z is turned by the angle t = position * f_i:
 *   (a cos t - b sin t, a sin t + b cos t) * mscale
 * pair i being dims (i, i + d/2), or (2i, 2i + 1) if `interleaved`.  ("Training
 * at 1M+ Token Context: Ring Attention, YaRN, NTK-Aware Scaling" extends the
 * context by other frequencies f and, in YaRN, by an mscale: both are given.)
 *
 * Frequencies are turns a position as 64-bit fixed-point numbers, 2^64 to the
 * turn: position * f in integers that wrap around is the angle of any position
 * to 2^-64 of a turn for each position, where a product of floats loses the
 * angle of a far one.
 * Conventions of every entry point: as in msa.h.
 */
#ifndef MSA_ROPE_H_
#define MSA_ROPE_H_

#include "msa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   q          [n, Hq, d], k [n, Hkv, d] in `dt`, tokens q_stride (k_stride)
 *              elements apart, the heads of a token next to each other: a
 *              slice of the projections' common output is taken as it is
 *   positions  [n] device int64 (any value)
 *   freqs      [d / 2] device int64
 *   q_weight, k_weight  [d] in `w_dt`; NULL: that side is rotated only
 *   q_out, k_out  [n, Hq, d], [n, Hkv, d] in `dt`, written
 * Sums of squares are fp32: values above 2^60 pass its range (the row's norm
 * gives zeros), and with an eps below 2^-120 those below 2^-64 lose bits of r.
 * Hkv may be 0 (k and k_out are not looked at), and
 * so may n (nothing is done).
 * Errors: INVALID_ARG for null or misaligned pointers (16 bytes; positions and
 * freqs 8, weights 4), sizes out of range, strides below heads * d or not a
 * multiple of 16 bytes, eps < 0 or not finite, mscale not finite; UNSUPPORTED
 * if d is not 64 or 128.
 */
msa_status msa_qk_norm_rope(const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, int64_t n, int Hq, int Hkv,
                            int d, const int64_t *positions,
                            const int64_t *freqs, const void *q_weight,
                            const void *k_weight, float eps, float mscale,
                            int interleaved, void *q_out, void *k_out,
                            msa_dtype dt, msa_dtype w_dt, msa_stream_t stream);

/* Bytes of workspace msa_qk_norm_rope_bwd needs (0 for invalid sizes). */
size_t msa_qk_norm_rope_bwd_workspace_size(int64_t n, int Hq, int Hkv, int d);

/*
 * The gradients: dq, dk of sum <dq_out, q_out> + sum <dk_out, k_out>, and those
 * of the weights.
 *   dq_out, dk_out  [n, Hq, d], [n, Hkv, d] in `dt`, tokens dq_out_stride,
 *                   dk_out_stride elements apart
 *   q, k, ...       what the forward took
 *   dq, dk          [n, Hq, d], [n, Hkv, d] in `dt`, written
 *   dq_weight, dk_weight  [d] in `w_dt`, written; NULL where the weight is
 * The weights' gradients are summed in an order that the sizes fix: few terms
 * (a thread's 8 rows, 8 lanes) in fp32, beyond that in two floats each, so that
 * their bits do not go with the number of rows.
 * n = 0 writes zeros to them.
 * Errors: as msa_qk_norm_rope, and a null, misaligned (256 bytes) or too small
 * workspace where there is a weight.
 */
msa_status msa_qk_norm_rope_bwd(
    const void *dq_out, int64_t dq_out_stride, const void *dk_out,
    int64_t dk_out_stride, const void *q, int64_t q_stride, const void *k,
    int64_t k_stride, int64_t n, int Hq, int Hkv, int d,
    const int64_t *positions, const int64_t *freqs, const void *q_weight,
    const void *k_weight, float eps, float mscale, int interleaved, void *dq,
    void *dk, void *dq_weight, void *dk_weight, msa_dtype dt, msa_dtype w_dt,
    void *workspace, size_t workspace_bytes, msa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_ROPE_H_ */
