// qsa_chunk.cu -- attention of ragged chunks of new tokens over the paged K/V
// cache, declared in include/qsa_chunk.h.
#include "qsa_chunk_attn.h"
#include "qsa_cache_host.h"
#include "qsa_cache_map.h"
#include "qsa_host.h"
#include "qsa_chunk.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

namespace qsa {
namespace {

#ifdef QSA_WAIT_TEST
int32_t g_test_withhold = -1;
#endif

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// The workspace: the plan of a call's row tiles, the pieces of those that runs
// cut (at most two a run), and with a prefix the results of both lists.
struct Layout {
  int64_t max_tiles, max_own, part_rows;
  size_t tiles, pos, first, cuts, owners, part_ml, part_o, res_ml[2], res_o[2], total;
};
Layout layout_of(const qsa_paged_cache& c, int64_t tokens, int64_t heads, bool prefix) {
  const int sub = chunk_heads((int)(heads / c.num_heads)), accs = chunk_accs((int)c.head_dim);
  const int64_t acc_toks = 128 / sub, per = accs * acc_toks, tiles = (tokens + per - 1) / per;
  Layout l;
  l.max_own = tiles + std::min(c.num_reqs, tokens);
  l.max_tiles = l.max_own + (prefix ? tiles : 0);
  l.part_rows = tokens > acc_toks ? accs * 128 : tokens * sub;
  size_t at = round256(sizeof(ChunkPlan));
  const auto take = [&](size_t bytes) {
    const size_t x = at;
    at += round256(bytes);
    return x;
  };
  l.tiles = take((size_t)l.max_tiles * sizeof(ChunkTile));
  l.pos = take((size_t)(l.max_tiles + 1) * 8);
  l.first = take((size_t)c.num_reqs * 4);
  l.cuts = take(kChunkMaxCtas * sizeof(ChunkCut));
  l.owners = take(prefix ? (size_t)l.max_tiles * sizeof(ChunkOwner) : 0);
  const int64_t pieces = (prefix ? 4 : 2) * kChunkMaxCtas;
  l.part_ml = take((size_t)(pieces * l.part_rows) * 8);
  l.part_o = take((size_t)(pieces * l.part_rows * c.head_dim) * 4);
  for (int i = 0; i < 2; ++i) {
    l.res_ml[i] = prefix ? take((size_t)(tokens * heads) * 8) : 0;
    l.res_o[i] = prefix ? take((size_t)(tokens * heads * c.head_dim) * 4) : 0;
  }
  l.total = at;
  return l;
}

// q as (dim, head, token); a box is 64 dims (128 bytes) of a set's heads and of an
// accumulator's tokens.
bool encode_queries(CUtensorMap* map, const ChunkParams& p) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)p.c.dim, (cuuint64_t)p.heads, (cuuint64_t)p.tokens};
  // a dimension of size 1 has any stride; the encoder wants a legal one
  const cuuint64_t row = (cuuint64_t)p.c.dim * 2;
  const cuuint64_t strides[2] = {p.q_head ? (cuuint64_t)p.q_head : row, p.q_row ? (cuuint64_t)p.q_row : row};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.sub, (cuuint32_t)p.acc_toks};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<unsigned char*>(p.q), dims, strides, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool sizes_ok(const qsa_paged_cache& c, int64_t tokens, int64_t heads) {
  return tokens >= 0 && tokens <= QSA_CHUNK_MAX_TOKENS && heads >= 1 && heads <= 65535 &&
         heads % c.num_heads == 0 && tokens * heads <= INT32_MAX;
}

qsa_status attend(const qsa_paged_cache* cache, bool prefix, const int32_t* prefix_table,
                  int64_t prefix_cols, const int32_t* prefix_len, const void* q, qsa_dtype dtype,
                  int64_t tokens, int64_t heads, const int64_t* q_strides, const int32_t* starts,
                  const int32_t* ctx, float scale, int64_t window, int64_t sink, void* out,
                  const int64_t* out_strides, float* lse, void* workspace, size_t workspace_bytes,
                  uint32_t* error_word, qsa_stream_t stream) {
  using namespace cache_host;
  ChunkParams p{};
  CacheSpans cs{};
  const qsa_status st = check_cache(cache, &p.c, &cs);
  if (st != QSA_OK) return st;
  if (dtype != QSA_DT_F16 && dtype != QSA_DT_BF16) return QSA_ERR_DTYPE;
  if (cache->dtype != QSA_DT_F8E4M3 && cache->dtype != dtype) return QSA_ERR_DTYPE;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!(std::isfinite(scale_log2) && scale > 0.f) || window < 0 || sink < 0) return QSA_ERR_CONTRACT;
  const int64_t R = cache->num_reqs;
  if (!sizes_ok(*cache, tokens, heads)) return QSA_ERR_SHAPE;
  if (prefix && (prefix_cols < 0 || prefix_cols > INT32_MAX)) return QSA_ERR_SHAPE;
  if (!q_strides || !out_strides) return QSA_ERR_NULL;
  const int64_t shape[3] = {tokens, heads, cache->head_dim};
  if (!strides_ok(shape, q_strides, 3, 2) || !strides_ok(shape, out_strides, 3, 2) ||
      !separate(shape, out_strides, 3))
    return QSA_ERR_STRIDE;
  if (R == 0 || tokens == 0) return QSA_OK;
  const int64_t qx = extent(shape, q_strides, 3, 2), ox = extent(shape, out_strides, 3, 2);
  if (qx < 0 || ox < 0) return QSA_ERR_STRIDE;
  if (!q || !out || !starts || !ctx) return QSA_ERR_NULL;
  if (prefix && (!prefix_len || (prefix_cols > 0 && !prefix_table))) return QSA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(starts, 4) || !aligned(ctx, 4) ||
      !aligned(lse, 4) || !aligned(error_word, 4) ||
      (prefix && (!aligned(prefix_table, 4) || !aligned(prefix_len, 4))))
    return QSA_ERR_ALIGN;
  const bool fp8 = cache->dtype == QSA_DT_F8E4M3;
  const Layout l = layout_of(*cache, tokens, heads, prefix);
  const size_t need = l.total;
  const Span outs[4] = {span(out, ox), span(lse, tokens * heads * 4), span(error_word, 4),
                        span(workspace, (int64_t)need)};
  const Span ins[10] = {span(q, qx), cs.k, cs.v, cs.tables, cs.k_scale, cs.v_scale,
                        span(starts, (R + 1) * 4), span(ctx, R * 4),
                        prefix ? span(prefix_table, prefix_cols * 4) : Span{},
                        prefix ? span(prefix_len, 4) : Span{}};
  if (any_overlap(outs, 4, ins, 10)) return QSA_ERR_ALIAS;
  if (need > 0 && (!workspace || workspace_bytes < need)) return QSA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QSA_ERR_ALIGN;
  const int64_t pcap = prefix ? prefix_cols << p.c.page_log2 : 0;
  p.prefix_table = prefix && prefix_cols > 0 ? prefix_table : nullptr;
  p.prefix_cap = (int32_t)std::min<int64_t>(pcap, kMaxEntries);
  p.prefix_len = prefix ? prefix_len : nullptr;
  p.q = static_cast<const unsigned char*>(q);
  p.q_row = tokens > 1 ? q_strides[0] * 2 : 0;
  p.q_head = heads > 1 ? q_strides[1] * 2 : 0;
  p.out = static_cast<unsigned char*>(out);
  p.out_row = tokens > 1 ? out_strides[0] * 2 : 0;
  p.out_head = heads > 1 ? out_strides[1] * 2 : 0;
  p.starts = starts;
  p.ctx = ctx;
  p.tokens = (int32_t)tokens;
  p.heads = (int32_t)heads;
  const int group = (int)(heads / cache->num_heads);
  p.sub = chunk_heads(group);
  p.sets = (int32_t)(heads / p.sub);
  p.per_kv = group / p.sub;
  p.acc_toks = 128 / p.sub;
  p.heavy_rows = chunk_accs(p.c.dim) == 2 ? p.acc_toks * p.sub : 32;
  p.heavy_extra = fp8 ? kHeavyExtraE4M3 : kHeavyExtra;
  p.scale_log2 = scale_log2;
  // (a context is 2^31 - 1 at most: a window as wide hides nothing)
  p.window = (int32_t)std::min<int64_t>(window, INT32_MAX);
  p.sink = window > 0 ? (int32_t)std::min<int64_t>(sink, kMaxEntries) : 0;
  p.lse = lse;
  p.err = error_word;
  bind_calling_thread();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == QSA_DT_BF16;
  unsigned char* w = static_cast<unsigned char*>(workspace);
  p.max_tiles = (int32_t)l.max_tiles;
  p.plan = reinterpret_cast<ChunkPlan*>(w);
  p.tiles = reinterpret_cast<ChunkTile*>(w + l.tiles);
  p.pos = reinterpret_cast<int64_t*>(w + l.pos);
  p.first = reinterpret_cast<int32_t*>(w + l.first);
  p.cuts = reinterpret_cast<ChunkCut*>(w + l.cuts);
  p.owners = reinterpret_cast<ChunkOwner*>(w + l.owners);
  p.max_own = (int32_t)l.max_own;
  p.part_rows = (int32_t)l.part_rows;
  p.part_ml = reinterpret_cast<float*>(w + l.part_ml);
  p.part_o = reinterpret_cast<float*>(w + l.part_o);
  for (int i = 0; i < 2 && prefix; ++i) {
    p.res_ml[i] = reinterpret_cast<float*>(w + l.res_ml[i]);
    p.res_o[i] = reinterpret_cast<float*>(w + l.res_o[i]);
  }
  const int box = (int)std::min<int64_t>(cache->page_size, chunk_tile(p.c.dim));
  CUtensorMap kmap, vmap, qmap;
  if (!encode_view(&kmap, p.c.k, p.c, fp8 ? 1 : 2, p.c.k_page, p.c.k_token, p.c.k_head, box) ||
      !encode_view(&vmap, p.c.v, p.c, fp8 ? 1 : 2, p.c.v_page, p.c.v_token, p.c.v_head, box) ||
      !encode_queries(&qmap, p))
    return QSA_ERR_CUDA;
#ifdef QSA_WAIT_TEST
  p.test_withhold = g_test_withhold;                       // heads of 64 alone are built
  const cudaError_t e = p.c.dim == 64 ? launch_chunk_64(p, bf16, fp8, kmap, vmap, qmap, s)
                                      : cudaErrorNotSupported;
#else
  const cudaError_t e = p.c.dim == 64    ? launch_chunk_64(p, bf16, fp8, kmap, vmap, qmap, s)
                        : p.c.dim == 128 ? launch_chunk_128(p, bf16, fp8, kmap, vmap, qmap, s)
                                         : launch_chunk_256(p, bf16, fp8, kmap, vmap, qmap, s);
#endif
  return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

}  // namespace
}  // namespace qsa

extern "C" size_t qsa_chunk_attention_workspace_bytes(const qsa_paged_cache* cache,
                                                      int64_t num_tokens, int64_t num_heads,
                                                      int64_t prefix_cols) {
  using namespace qsa;
  CacheView view{};
  cache_host::CacheSpans spans{};
  if (cache_host::check_cache(cache, &view, &spans) != QSA_OK || cache->num_reqs == 0 ||
      num_tokens == 0 || !sizes_ok(*cache, num_tokens, num_heads))
    return 0;
  return layout_of(*cache, num_tokens, num_heads, prefix_cols >= 0).total;
}

extern "C" qsa_status qsa_chunk_attention(
    const qsa_paged_cache* cache, const void* q, qsa_dtype dtype, int64_t num_tokens,
    int64_t num_heads, const int64_t q_strides[3], const int32_t* query_start_loc,
    const int32_t* context_lens, float scale, int64_t window, int64_t num_sink, void* out,
    const int64_t out_strides[3], float* lse, void* workspace, size_t workspace_bytes,
    uint32_t* error_word, qsa_stream_t stream) {
  return qsa::attend(cache, false, nullptr, 0, nullptr, q, dtype, num_tokens, num_heads, q_strides,
                     query_start_loc, context_lens, scale, window, num_sink, out, out_strides, lse,
                     workspace, workspace_bytes, error_word, stream);
}

extern "C" qsa_status qsa_prefix_attention(
    const qsa_paged_cache* cache, const int32_t* prefix_table, int64_t prefix_cols,
    const int32_t* prefix_len, const void* q, qsa_dtype dtype, int64_t num_tokens,
    int64_t num_heads, const int64_t q_strides[3], const int32_t* query_start_loc,
    const int32_t* context_lens, float scale, void* out, const int64_t out_strides[3], float* lse,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, qsa_stream_t stream) {
  return qsa::attend(cache, true, prefix_table, prefix_cols, prefix_len, q, dtype, num_tokens,
                     num_heads, q_strides, query_start_loc, context_lens, scale, 0, 0, out,
                     out_strides, lse, workspace, workspace_bytes, error_word, stream);
}

#ifdef QSA_WAIT_TEST
// Test build only, declared in no public header: the next chunk attention launches
// leave slot fill `issue` (K's and V's tiles counted in turn) of the walk's CTA 0
// without a copy (-1: none).
extern "C" __attribute__((visibility("default"))) void qsa_test_withhold_chunk_fill(int32_t issue) {
  qsa::g_test_withhold = issue;
}
#endif
