// qsa_cache_host.h -- host-side checks and the device view of a paged K/V
// cache (include/qsa_cache.h), shared by the operators that take one.
#pragma once

#include "qsa.h"
#include "qsa_cache.h"

#include <cstdint>
#include <cuda_runtime.h>

namespace qsa {

// What the kernels see of a cache.  Strides in bytes.
struct CacheView {
  unsigned char* k;
  unsigned char* v;
  int64_t num_pages;
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;
  const int32_t* bt;
  int64_t bt_s0;
  const float* k_scale;       // nullable: 1
  const float* v_scale;
  int32_t num_reqs, cols;
  int32_t page_log2, heads, dim;
  int32_t cap;                // entries a table row can hold, at most kMaxEntries
};

// Entries of a request that the operators count (more bytes than a GPU has).
constexpr int32_t kMaxEntries = QSA_CACHE_MAX_ENTRIES;

namespace cache_host {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

struct Span {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Span span(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + (uintptr_t)(p != nullptr && bytes > 0 ? bytes : 0)};
}
inline bool overlaps(Span a, Span b) {
  return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}
inline bool any_overlap(const Span* outs, int n_outs, const Span* ins, int n_ins) {
  for (int a = 0; a < n_outs; ++a) {
    for (int b = a + 1; b < n_outs; ++b)
      if (overlaps(outs[a], outs[b])) return true;
    for (int b = 0; b < n_ins; ++b)
      if (overlaps(outs[a], ins[b])) return true;
  }
  return false;
}
// rows of cols 4-byte elements, stride0 elements apart
inline Span rows_span(const void* p, int64_t rows, int64_t cols, int64_t stride0) {
  if (rows <= 0 || cols <= 0) return span(p, 0);
  const __int128 bytes = ((__int128)(rows - 1) * stride0 + cols) * 4, most = (__int128)1 << 62;
  return span(p, (int64_t)(bytes < most ? bytes : most));
}

constexpr int64_t kMaxStride = (int64_t)1 << 38;   // elements; bytes stay below 2^40

inline bool row_stride_ok(int64_t stride0, int64_t cols) {
  return stride0 >= cols && stride0 <= kMaxStride;
}

// Strides of an [n0, ..., D] tensor of 16-bit or smaller elements, the last
// one 1: each one that is used is a multiple of 16 bytes and at least D.
inline bool strides_ok(const int64_t* shape, const int64_t* strides, int rank, int64_t esize) {
  if (strides[rank - 1] != 1) return false;
  for (int i = 0; i + 1 < rank; ++i) {
    if (shape[i] <= 1) continue;
    if (strides[i] < shape[rank - 1] || strides[i] > kMaxStride || strides[i] * esize % 16 != 0)
      return false;
  }
  return true;
}

// Whether no two elements share an address: the strides in ascending order, each
// passes what the smaller ones reach.  (All are at least the last dimension's
// extent: strides_ok.)
inline bool separate(const int64_t* shape, const int64_t* strides, int rank) {
  __int128 reach = shape[rank - 1];      // elements that the dimensions taken so far span
  bool taken[4] = {false, false, false, false};
  for (int step = 0; step + 1 < rank; ++step) {
    int next = -1;
    for (int i = 0; i + 1 < rank; ++i)
      if (!taken[i] && (next < 0 || strides[i] < strides[next])) next = i;
    taken[next] = true;
    if (shape[next] <= 1) continue;
    if (strides[next] < reach) return false;
    reach += (__int128)(shape[next] - 1) * strides[next];
  }
  return true;
}

// Bytes from the first to the last element, or -1 where that passes 2^62.
inline int64_t extent(const int64_t* shape, const int64_t* strides, int rank, int64_t esize) {
  __int128 last = 0;
  for (int i = 0; i < rank; ++i) {
    if (shape[i] <= 0) return 0;
    if (shape[i] > 1) last += (__int128)(shape[i] - 1) * strides[i];
  }
  const __int128 bytes = (last + 1) * esize;
  return bytes < ((__int128)1 << 62) ? (int64_t)bytes : -1;
}

struct CacheSpans {
  Span k, v, tables, k_scale, v_scale;
};

inline int64_t dtype_size(int64_t dt) { return dt == QSA_DT_F8E4M3 ? 1 : 2; }

// Checks a cache descriptor; fills *view and *spans.
inline qsa_status check_cache(const qsa_paged_cache* c, CacheView* view, CacheSpans* spans) {
  if (!c) return QSA_ERR_NULL;
  if (c->dtype != QSA_DT_F16 && c->dtype != QSA_DT_BF16 && c->dtype != QSA_DT_F8E4M3)
    return QSA_ERR_DTYPE;
  if (c->dtype != QSA_DT_F8E4M3 && (c->k_scale || c->v_scale)) return QSA_ERR_CONTRACT;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QSA_ERR_SHAPE;
  if (c->num_heads < 1 || c->num_heads > QSA_CACHE_MAX_HEADS) return QSA_ERR_SHAPE;
  if (c->page_size < QSA_CACHE_MIN_PAGE || c->page_size > QSA_CACHE_MAX_PAGE ||
      (c->page_size & (c->page_size - 1)) != 0)
    return QSA_ERR_SHAPE;
  if (c->num_pages < 0 || c->num_pages > INT32_MAX) return QSA_ERR_SHAPE;
  if (c->num_reqs < 0 || c->num_reqs > QSA_CACHE_MAX_REQS || c->table_cols < 0 ||
      c->table_cols > INT32_MAX)
    return QSA_ERR_SHAPE;
  const int64_t es = dtype_size(c->dtype);
  const int64_t shape[4] = {c->num_pages, c->page_size, c->num_heads, c->head_dim};
  if (!strides_ok(shape, c->k_strides, 4, es) || !strides_ok(shape, c->v_strides, 4, es) ||
      !separate(shape, c->k_strides, 4) || !separate(shape, c->v_strides, 4))
    return QSA_ERR_STRIDE;
  if (!row_stride_ok(c->table_stride0, c->table_cols)) return QSA_ERR_STRIDE;
  const int64_t kx = extent(shape, c->k_strides, 4, es), vx = extent(shape, c->v_strides, 4, es);
  if (kx < 0 || vx < 0) return QSA_ERR_STRIDE;
  if (c->num_pages > 0 && (!c->k || !c->v)) return QSA_ERR_NULL;
  if (c->num_reqs > 0 && c->table_cols > 0 && !c->block_tables) return QSA_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->block_tables, 4) ||
      !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return QSA_ERR_ALIGN;
  int lg = 0;
  while (((int64_t)1 << lg) < c->page_size) ++lg;
  const int64_t cap = c->table_cols << lg;
  const auto used = [&](const int64_t* st, int i) { return shape[i] > 1 ? st[i] * es : 0; };
  view->k = static_cast<unsigned char*>(c->k);
  view->v = static_cast<unsigned char*>(c->v);
  view->num_pages = c->num_pages;
  view->k_page = used(c->k_strides, 0);
  view->k_token = used(c->k_strides, 1);
  view->k_head = used(c->k_strides, 2);
  view->v_page = used(c->v_strides, 0);
  view->v_token = used(c->v_strides, 1);
  view->v_head = used(c->v_strides, 2);
  view->bt = c->block_tables;
  view->bt_s0 = c->table_stride0;
  view->k_scale = c->k_scale;
  view->v_scale = c->v_scale;
  view->num_reqs = (int32_t)c->num_reqs;
  view->cols = (int32_t)c->table_cols;
  view->page_log2 = lg;
  view->heads = (int32_t)c->num_heads;
  view->dim = (int32_t)c->head_dim;
  view->cap = cap > kMaxEntries ? kMaxEntries : (int32_t)cap;
  spans->k = span(c->k, kx);
  spans->v = span(c->v, vx);
  spans->tables = rows_span(c->block_tables, c->num_reqs, c->table_cols, c->table_stride0);
  spans->k_scale = span(c->k_scale, c->num_heads * 4);
  spans->v_scale = span(c->v_scale, c->num_heads * 4);
  return QSA_OK;
}

}  // namespace cache_host
}  // namespace qsa
