/*
 * qsa_cache.h -- C ABI of libqsa: a paged K/V cache and the operators of a
 * decode step that work on all of it: writing new tokens' keys and values
 * (qsa_paged_append), dense attention of the new tokens over the cached
 * entries (qsa_paged_attention, next to the sparse attention over chosen
 * indices of qsa.h), and bounding the cache by evicting the entries that
 * received the least attention weight (qsa_evict_entries).
 *
 * Conventions (device pointers, fail-closed validation, no allocation,
 * asynchronous launch on the caller's stream, device-side data errors
 * reported in *error_word, any host thread) are those of qsa.h.  The
 * attention clobbers its workspace (the others need none); calls that share
 * one must not overlap on the GPU.  No call keeps anything from another.
 *
 * A request's cached tokens are its ENTRIES 0, 1, 2, ...: entry e of request
 * b is slot e % page_size of page block_tables[b, e / page_size].  Without
 * evictions an entry's number is the token's position; an eviction renumbers
 * the entries that stay (attention does not depend on their order), and
 * entry_positions says which token an entry holds.
 */
#ifndef QSA_CACHE_H
#define QSA_CACHE_H

#include "qsa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QSA_DERR_CONTEXT 32u  /* a context length, or an entry to append, past
                                 what the block table (and the per-entry
                                 arrays, where given) can hold: what lies
                                 past it counts as absent */

#define QSA_CACHE_MIN_PAGE 8       /* page sizes: powers of two from 8 */
#define QSA_CACHE_MAX_PAGE 65536   /* to 65536 */
#define QSA_CACHE_MAX_HEADS 1024   /* K/V heads; query heads x next_n <= 65536 */
#define QSA_CACHE_MAX_REQS 65535   /* requests in one call */
#define QSA_CACHE_MAX_ENTRIES 1073741824 /* entries of a request that count; a
                                            table that holds more is past it */
#define QSA_CACHE_MAX_NEXT 8       /* new tokens per request in one call */

/*
 * A paged K/V cache.  K and V are views [num_pages, page_size, num_heads,
 * head_dim]; strides in elements, the last one 1, the others multiples of 16
 * bytes and such that no two elements of a view share an address (the stride of
 * a dimension of size 1 is not looked at).  So K and V may be two tensors, or lie side by side in one (the
 * exact-packed cache of qsa.h is strides {262144, 512, any, 1} with v = k +
 * 256), tokens or heads outermost within a page; the two views must not
 * share an element (qsa_paged_append refuses one view given as both).
 *
 *   dtype         QSA_DT_F16, QSA_DT_BF16 or QSA_DT_F8E4M3
 *   head_dim      64, 128 or 256
 *   k_scale, v_scale  fp32 [num_heads] or NULL (all 1), each from 2^-64 to
 *                 2^64: an element stands for its value times its head's
 *                 scale; QSA_DT_F8E4M3 only
 *   block_tables  int32 [num_reqs, table_cols] (num_reqs <=
 *                 QSA_CACHE_MAX_REQS), row stride table_stride0,
 *                 column stride 1; a page id outside [0, num_pages) makes its
 *                 entries absent (QSA_DERR_KV_PAGE when one is looked up)
 */
typedef struct qsa_paged_cache {
  void* k;
  void* v;
  int64_t num_pages, page_size, num_heads, head_dim;
  int64_t k_strides[4], v_strides[4];
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  int64_t num_reqs, table_cols, table_stride0;
  int64_t dtype;                /* a qsa_dtype */
} qsa_paged_cache;

/*
 * qsa_paged_append -- write num_tokens tokens' keys and values into the
 * cache: token t becomes entry e = entries[t] of request r =
 * token_to_request[t] (the metadata builder's token_to_req and
 * logical_positions are these two for a cache without evictions; its padding
 * tokens have entry -1):
 *
 *   e < 0: nothing.  Otherwise, for every K/V head h,
 *   K[page, slot, h, :] = k[t, h, :], V likewise; into an E4M3 cache
 *   k[t, h, :] * (1 / k_scale[h]) (both in binary32), rounded to nearest
 *   even, magnitudes above 448 to 448, NaN to NaN;
 *   entry_positions[r, e] = positions[t] (e itself when positions is NULL), as
 *   32 bits;
 *   weight_sums[r, e] = 0.
 *
 * A request outside [0, num_reqs) (QSA_DERR_REQUEST), an entry past the table
 * or past entry_cols (QSA_DERR_CONTEXT) or an absent page (QSA_DERR_KV_PAGE)
 * writes nothing for that token.  Two tokens of one call with the same
 * request and entry (or requests sharing a page that both write) leave that
 * entry with a mixture of the two.
 *
 * Arguments
 *   k, v             [num_tokens, num_heads, head_dim], dtype QSA_DT_F16 or
 *                    QSA_DT_BF16, the cache's own unless it is E4M3; strides
 *                    in elements, the last 1, the others multiples of 16
 *                    bytes; 16-byte aligned
 *   token_to_request int32 [num_tokens]
 *   entries          int64 [num_tokens]
 *   positions        int64 [num_tokens] or NULL
 *   entry_positions  int32 [num_reqs, entry_cols], row stride
 *                    entry_positions_stride0, or NULL
 *   weight_sums      fp32 [num_reqs, entry_cols], row stride
 *                    weight_sums_stride0, or NULL
 */
QSA_API qsa_status qsa_paged_append(
    const qsa_paged_cache* cache,
    const void* k, const void* v, qsa_dtype dtype, int64_t num_tokens,
    const int64_t k_strides[3], const int64_t v_strides[3],
    const int32_t* token_to_request, const int64_t* entries, const int64_t* positions,
    int32_t* entry_positions, int64_t entry_positions_stride0,
    float* weight_sums, int64_t weight_sums_stride0, int64_t entry_cols,
    uint32_t* error_word, qsa_stream_t stream);

/*
 * Workspace for qsa_paged_attention: bytes for next_n new tokens a request
 * with num_heads query heads over this cache, with_weights != 0 when weight
 * sums are asked for.  What the cache's pointers hold does not matter.  0 for a
 * call that needs none (short tables, no weight sums) and for one that is
 * refused.  Alignment 256 bytes.
 */
QSA_API size_t qsa_paged_attention_workspace_bytes(const qsa_paged_cache* cache, int64_t next_n,
                                                   int64_t num_heads, int with_weights);

/*
 * qsa_paged_attention -- dense attention of next_n new tokens per request.
 * Row r = b*next_n + j is token j of request b; it sees the entries
 *
 *   [max(0, hi - window), hi),  hi = context_lens[b] - next_n + j + 1
 *
 * (window 0: all below hi; entries that are absent, or past the table, do not
 * count).  Query head h reads K/V head h / (num_heads / cache->num_heads):
 *
 *   z_e = scale * (q[r,h,:] . K_e),  p_e = e^{z_e} / sum e^{z_e}
 *   out[r,h,:] = sum_e p_e V_e,      lse[r,h] = log sum_e e^{z_e}
 *   weight_sums_out[b,e] = weight_sums[b,e] + sum_{j,h} p_e   for every entry
 *                          e < min(context_lens[b], table's entries); the rest of
 *                          weight_sums_out is left as it was
 *
 * A row that sees no entry gets zeros and an lse of -inf; rows of requests
 * with a context length of 0 or less are such rows.  What a masked or absent
 * entry holds (infinities and NaN too) does not matter.  The softmax's
 * statistics and sums are binary32, so q . K_e, z_e and the sum of |V_e| over the
 * entries that a row sees have to be finite there; the results are the same bit
 * for bit each time a call is repeated on one kind of GPU.
 *
 * The weights enter the product with V rounded, relative to themselves, by 2^-22
 * (FP16) or 2^-16 (BF16) where next_n * num_heads / cache->num_heads is 32 or less
 * and the cache is not E4M3; by 2^-11 (FP16, and any E4M3 cache) or 2^-8 (BF16)
 * elsewhere; or by 2^-39 of the row's sum of weights (FP16; logits past 2^19:
 * 2^-25), 2^-126 (BF16), where that is more.  lse and weight sums do not carry that
 * rounding.
 *
 * Weight sums need every logit until its row is complete: num_reqs * next_n *
 * num_heads * table_cols * page_size * 4 bytes of workspace, whatever the
 * contexts and the window (64 requests, 32 heads, a table of 131072 entries: 1.1
 * GB).  A table cut to the columns that the longest context needs keeps it small.
 *
 * Arguments
 *   q             [num_reqs*next_n, num_heads, head_dim], dtype QSA_DT_F16 or
 *                 QSA_DT_BF16, the cache's own unless it is E4M3; strides in
 *                 elements, the last 1, the others multiples of 16 bytes;
 *                 16-byte aligned.  num_heads: a multiple of the cache's
 *   context_lens  int32 [num_reqs]: cached tokens, the new ones included
 *   next_n        1 .. QSA_CACHE_MAX_NEXT
 *   scale         > 0, scale * log2(e) finite in binary32
 *   window        >= 0
 *   out           as q (strides out_strides, no two elements at one address);
 *                 overlaps no input
 *   lse           fp32 [num_reqs*next_n, num_heads] contiguous, or NULL
 *   weight_sums, weight_sums_out  fp32 [num_reqs, entry_cols], row strides
 *                 weight_sums_stride0 and weight_sums_out_stride0, both NULL or
 *                 neither; they may be one buffer (the sums then grow in
 *                 place), or must not overlap.  entry_cols >= table_cols *
 *                 page_size
 *   workspace     >= qsa_paged_attention_workspace_bytes(...) bytes, 256-byte
 *                 aligned; may be NULL where that is 0
 */
QSA_API qsa_status qsa_paged_attention(
    const qsa_paged_cache* cache,
    const void* q, qsa_dtype dtype, int64_t next_n, int64_t num_heads,
    const int64_t q_strides[3],
    const int32_t* context_lens, float scale, int64_t window,
    void* out, const int64_t out_strides[3], float* lse,
    const float* weight_sums, int64_t weight_sums_stride0,
    float* weight_sums_out, int64_t weight_sums_out_stride0, int64_t entry_cols,
    void* workspace, size_t workspace_bytes,
    uint32_t* error_word, qsa_stream_t stream);

/*
 * qsa_evict_entries -- cut every request down to at most `budget` entries.
 * Request b has n = min(context_lens[b], table_cols*page_size, entry_cols)
 * entries.  If n > budget, the budget first ones stay in the order
 *
 *   protected ones: position < num_sink, or position > newest - num_recent,
 *     newest the largest position of the request's entries;
 *   then by weight_sums, largest first (-0 equals +0, NaN below -inf);
 *   equal ones: the lower entry first.
 *
 * Those that stay and are below `budget` keep their place; those at or above
 * it move, in order, into the places of the ones that go: K and V are copied
 * within the cache, and the pages past entry budget-1 are free afterwards.
 *
 *   kept[b, i]     the entry that is now entry i (i itself if it did not
 *                  move); -1 for i >= new_lens[b]
 *   new_lens[b]    min(n, budget) (0 if context_lens[b] < 0)
 *   weight_sums_out[b, i], entry_positions_out[b, i]
 *                  of that entry; 0 and -1 for i >= new_lens[b]
 *
 * The inputs are not written.  (A next step that appends and attends needs room
 * behind the budget in its per-entry arrays: qsa_evict_entries_strided.)  A page
 * that holds entries below `budget` must belong to one request alone.  An entry
 * whose page is absent still counts; its K and V are not moved
 * (QSA_DERR_KV_PAGE).
 *
 * An eviction renumbers entries.  What holds token numbers of its own stays as it
 * was: a cache that qsa_sparse_attention reads through selected token numbers, or
 * whose compressed keys the selection scores, must not be evicted from.
 *
 * Arguments
 *   weight_sums       fp32 [num_reqs, entry_cols], row stride weight_sums_stride0
 *   entry_positions   int32 [num_reqs, entry_cols], row stride
 *                     entry_positions_stride0
 *   budget            1 .. QSA_CACHE_MAX_ENTRIES; num_sink, num_recent >= 0, num_sink + num_recent
 *                     <= budget (positions are distinct, so that many entries
 *                     are protected at most; of more, the first stay)
 *   kept, weight_sums_out, entry_positions_out
 *                     int32, fp32, int32 [num_reqs, budget], contiguous
 *   new_lens          int32 [num_reqs]
 */
QSA_API qsa_status qsa_evict_entries(
    const qsa_paged_cache* cache,
    const float* weight_sums, int64_t weight_sums_stride0,
    const int32_t* entry_positions, int64_t entry_positions_stride0, int64_t entry_cols,
    const int32_t* context_lens, int64_t budget, int64_t num_sink, int64_t num_recent,
    int32_t* kept, int32_t* new_lens, float* weight_sums_out, int32_t* entry_positions_out,
    uint32_t* error_word, qsa_stream_t stream);

/*
 * qsa_evict_entries_strided -- qsa_evict_entries with weight_sums_out and
 * entry_positions_out as rows of wider arrays: row b starts at b * the array's
 * stride0 (>= budget); columns from budget on are left as they were.  With two
 * arrays [num_reqs, entry_cols] of each kind, entry_cols >= the table's entries,
 * used as input and output in turn, the outputs and new_lens are what the next
 * step's append (whose tokens become the entries from new_lens[b] on), attention
 * and eviction take.
 */
QSA_API qsa_status qsa_evict_entries_strided(
    const qsa_paged_cache* cache,
    const float* weight_sums, int64_t weight_sums_stride0,
    const int32_t* entry_positions, int64_t entry_positions_stride0, int64_t entry_cols,
    const int32_t* context_lens, int64_t budget, int64_t num_sink, int64_t num_recent,
    int32_t* kept, int32_t* new_lens,
    float* weight_sums_out, int64_t weight_sums_out_stride0,
    int32_t* entry_positions_out, int64_t entry_positions_out_stride0,
    uint32_t* error_word, qsa_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QSA_CACHE_H */
