/*
 * qsa_rope.h -- C ABI of libqsa: what happens to a layer's new queries and
 * keys between their projection and the paged cache (qsa_cache.h): a norm of
 * each head and the rotation by its token's position, in one pass.
 *
 * Conventions (device pointers, fail-closed validation, no allocation,
 * asynchronous launch on the caller's stream, any host thread) are those of
 * qsa.h.
 */
#ifndef QSA_ROPE_H
#define QSA_ROPE_H

#include "qsa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QSA_ROPE_MAX_DIM 256
#define QSA_ROPE_MAX_HEADS 65536

/*
 * qsa_qk_norm_rope -- for every token t with positions[t] >= 0 and every head
 * x = q[t, h, :] (with q_weight) or k[t, h, :] (with k_weight):
 *
 *   y_i = x_i * w_i / sqrt(eps + (sum_j x_j^2) / head_dim)
 *   z   = y with pair i < rot_dim / 2 of its first rot_dim elements,
 *         (y_a, y_b), turned by angle_i = positions[t] * inv_freq[i]:
 *           z_a = y_a cos - y_b sin,   z_b = y_b cos + y_a sin
 *         a = i, b = i + rot_dim / 2, or with interleaved != 0
 *         a = 2 i, b = 2 i + 1
 *
 * z goes to q_out or k_out, rounded once; everything before is binary32:
 * sum_j x_j^2 has to be finite there (as it is for elements up to 2^59), eps +
 * (sum_j x_j^2) / head_dim 2^-120 at least, and w_i over its root a normal number
 * or 0.  (FP16 rows are within the first two whatever numbers they hold, but for
 * zeros with eps 0, which give NaN.)  A token with a negative position (the
 * metadata builder's padding) is left as it was in both.  The product of position
 * and frequency is reduced to one turn in 64 bits before it is rounded, so an
 * angle is off by at most 2^-24 of a half turn wherever positions[t] * (1 +
 * |inv_freq[i]|) is below 2^37.
 *
 * Arguments
 *   q, k           [num_tokens, q_heads, head_dim], [num_tokens, k_heads,
 *                  head_dim], both of dtype QSA_DT_F16 or QSA_DT_BF16; strides
 *                  in elements, the last 1, the others multiples of 16 bytes;
 *                  16-byte aligned.  Either may have no heads (and be NULL)
 *   head_dim       a multiple of 8 up to QSA_ROPE_MAX_DIM
 *   q_weight, k_weight  [head_dim], weight_dtype QSA_DT_F32 or dtype, or NULL
 *                  (all 1); aligned to their element
 *   eps            >= 0, finite
 *   positions      int64 [num_tokens]
 *   inv_freq       fp32 [rot_dim / 2], finite; NULL with rot_dim 0
 *   rot_dim        a multiple of 16 up to head_dim; 0 rotates nothing
 *   q_out, k_out   as q and k, strides of their own.  q_out may be q (same
 *                  address and strides), k_out may be k; they overlap nothing
 *                  else.  Views of one tensor whose tokens lie side by side
 *                  (a projection's q, k and v) do not overlap
 */
QSA_API qsa_status qsa_qk_norm_rope(
    const void* q, const void* k, qsa_dtype dtype, int64_t num_tokens, int64_t q_heads,
    int64_t k_heads, int64_t head_dim, const int64_t q_strides[3], const int64_t k_strides[3],
    const void* q_weight, const void* k_weight, qsa_dtype weight_dtype, float eps,
    const int64_t* positions, const float* inv_freq, int64_t rot_dim, int interleaved,
    void* q_out, void* k_out, const int64_t q_out_strides[3], const int64_t k_out_strides[3],
    qsa_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QSA_ROPE_H */
