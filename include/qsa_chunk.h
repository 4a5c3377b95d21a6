/*
 * qsa_chunk.h -- C ABI of libqsa: attention of ragged chunks of new tokens
 * over the paged K/V cache of qsa_cache.h.  A chunk is a request's single new
 * token, a draft, a part of its prompt or all of it; a batch may hold all of
 * these at once.
 *
 *   qsa_chunk_attention    each request's own cached entries, with a sliding
 *                          window and first entries that stay visible
 *   qsa_prefix_attention   the same, behind a prefix that all requests share
 *
 * Conventions (device pointers, fail-closed validation, no allocation,
 * asynchronous launch on the caller's stream, device-side data errors
 * reported in *error_word, any host thread) are those of qsa.h, caches and
 * entries those of qsa_cache.h.  A call clobbers its workspace; calls that
 * share one must not overlap on the GPU.  No call keeps anything from another.
 */
#ifndef QSA_CHUNK_H
#define QSA_CHUNK_H

#include "qsa_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QSA_CHUNK_MAX_TOKENS 16777216  /* new tokens in one call; times the query
                                          heads at most 2^31 - 1 */

/*
 * Workspace for qsa_chunk_attention and qsa_prefix_attention (prefix_cols: the
 * columns of the prefix's table; -1 for qsa_chunk_attention): bytes for up to
 * num_tokens new tokens with num_heads query heads over this cache.  What the
 * cache's pointers hold does not matter.  0 for a call that needs none and for
 * one that is refused.  Alignment 256 bytes.
 *
 * qsa_chunk_attention needs head_dim * 0.33 MB at most for the pieces of row tiles
 * that runs cut, and 48 bytes for each token and request besides.
 * qsa_prefix_attention needs twice that and 8 bytes for each element of q, 16 for
 * each of its rows and heads: what a row sees of the prefix and what of its
 * request's entries, both in binary32 (30000 tokens of 32 heads of 128: 1 GB).
 */
QSA_API size_t qsa_chunk_attention_workspace_bytes(const qsa_paged_cache* cache,
                                                   int64_t num_tokens, int64_t num_heads,
                                                   int64_t prefix_cols);

/*
 * qsa_chunk_attention -- request b's new tokens are the rows
 * [query_start_loc[b], query_start_loc[b+1]) of q, n of them; its cache holds
 * context_lens[b] entries, the last n of them the new tokens' own (written
 * before, by qsa_paged_append).  Token j of the n sees the entries e with
 *
 *   e < hi,  hi = context_lens[b] - n + j + 1,  and
 *   e >= hi - window  or  e < num_sink           (window 0: all below hi)
 *
 * (entries that are absent, or past the table, do not count).  Query head h
 * reads K/V head h / (num_heads / cache->num_heads):
 *
 *   z_e = scale * (q[t,h,:] . K_e),  p_e = e^{z_e} / sum e^{z_e}
 *   out[t,h,:] = sum_e p_e V_e,      lse[t,h] = log sum_e e^{z_e}
 *
 * A row that sees no entry gets zeros and an lse of -inf.  Rows of no request
 * (before query_start_loc[0], from query_start_loc[num_reqs] on) are left as
 * they were.  What an entry holds (infinities and NaN too) does not matter to a
 * row that does not see it.  The softmax's statistics and sums are binary32, so
 * q . K_e, z_e and the sum of |V_e| over the entries that a row sees have to be
 * finite there; over an E4M3 cache also q . K_e without K's scale, and scale *
 * log2(e) * k_scale[h] from 2^-126 to 2^127.  The results are the same bit for bit
 * each time a call is repeated on one kind of GPU.
 *
 * The weights multiply V rounded to one value of 16 bits: each is off by at most
 * 2^-11 of itself, or 2^-33 of its row's sum of weights where that is more (FP16,
 * and any E4M3 cache), 2^-8 or 2^-118 (BF16).  lse does not carry that rounding.
 * (qsa_paged_attention rounds few rows' weights less.)
 *
 * Arguments
 *   q             [num_tokens, num_heads, head_dim], dtype QSA_DT_F16 or
 *                 QSA_DT_BF16, the cache's own unless it is E4M3; strides in
 *                 elements, the last 1, the others multiples of 16 bytes;
 *                 16-byte aligned.  num_heads: a multiple of the cache's,
 *                 65535 at most
 *   query_start_loc  int32 [num_reqs + 1], non-decreasing, from 0 to num_tokens
 *                 (device data: what lies outside is cut, and of rows that two
 *                 requests claim the results are undefined)
 *   context_lens  int32 [num_reqs]: cached entries, the new ones included
 *   scale         > 0, scale * log2(e) finite in binary32
 *   window        >= 0
 *   num_sink      >= 0 (nothing without a window)
 *   out           as q (strides out_strides, no two elements at one address);
 *                 overlaps no input
 *   lse           fp32 [num_tokens, num_heads] contiguous, or NULL
 *   workspace     >= qsa_chunk_attention_workspace_bytes(...) bytes, 256-byte
 *                 aligned; may be NULL where that is 0
 */
QSA_API qsa_status qsa_chunk_attention(
    const qsa_paged_cache* cache,
    const void* q, qsa_dtype dtype, int64_t num_tokens, int64_t num_heads,
    const int64_t q_strides[3],
    const int32_t* query_start_loc, const int32_t* context_lens, float scale, int64_t window,
    int64_t num_sink,
    void* out, const int64_t out_strides[3], float* lse,
    void* workspace, size_t workspace_bytes,
    uint32_t* error_word, qsa_stream_t stream);

/*
 * qsa_prefix_attention -- qsa_chunk_attention (window 0) where every row sees
 * besides its request's entries all entries [0, prefix_len) of one more table,
 * the prefix that the batch shares; those are read once for the batch.  A
 * request's own table, context_lens[b] and the rule above count what lies
 * behind the prefix.
 *
 *   prefix_table  int32 [prefix_cols], prefix_cols >= 0: pages of the same cache
 *   prefix_len    int32 [1], on the device; 0 or less: no prefix
 */
QSA_API qsa_status qsa_prefix_attention(
    const qsa_paged_cache* cache, const int32_t* prefix_table, int64_t prefix_cols,
    const int32_t* prefix_len,
    const void* q, qsa_dtype dtype, int64_t num_tokens, int64_t num_heads,
    const int64_t q_strides[3],
    const int32_t* query_start_loc, const int32_t* context_lens, float scale,
    void* out, const int64_t out_strides[3], float* lse,
    void* workspace, size_t workspace_bytes,
    uint32_t* error_word, qsa_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QSA_CHUNK_H */
