// qsa_append.cu -- writing new tokens into a paged K/V cache, declared in
// include/qsa_cache.h (qsa_paged_append).
//
// A pure move of num_tokens * 2 * heads * dim elements, so it is bound by
// memory (and, for the few tokens of a decode step, by one chain of
// dependent loads: request and entry, then the page id, then the store).  A
// token's K and V rows are cut into 16-byte pieces of the cache, dealt out to
// a power of two of threads, a few each: the chain is walked once for them,
// and their source loads do not wait for it.
#include "qsa_cache.h"
#include "qsa_cache_host.h"
#include "qsa_device.cuh"
#include "qsa_host.h"
#include "qsa_internal.h"

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

namespace qsa {
namespace {

constexpr int kAppendThreads = 256;

struct AppendParams {
  CacheView c;
  const unsigned char* k;
  const unsigned char* v;
  int64_t k_token, k_head, v_token, v_head;   // source strides in bytes
  const int32_t* t2r;
  const int64_t* entries;
  const int64_t* positions;                   // nullable: the entry itself
  int32_t* entry_pos;                         // nullable
  int64_t entry_pos_s0;
  float* sums;                                // nullable
  int64_t sums_s0;
  int32_t cap;                                // entries a request can hold here
  int64_t num_tokens;
  uint32_t* err;
};

// Eight 16-bit values of type T to eight E4M3 bytes: value * inverse in
// binary32, then to nearest even, saturating.  (The product and the inverse
// are off by 2^-23 together, E4M3's own rounding by 2^-4: the quotient itself
// took twice the instructions and made the kernel bound by them.)
template <typename T>
__device__ __forceinline__ uint2 to_e4m3(uint4 x, float inverse) {
  const T* h = reinterpret_cast<const T*>(&x);
  uint16_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2((float)h[2 * i] * inverse, (float)h[2 * i + 1] * inverse);
    o[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
}

// 64 bytes of source a thread, six CTAs an SM (16384 tokens of 8 heads of 128:
// into E4M3 20.1 us with two pieces and 23.6 with four, at whatever occupancy
// 26 and up; 16-bit 22.6 with four, 26.5 with two).
template <bool kFp8>
constexpr int kPiecesOf = kFp8 ? 2 : 4;

// kFp8: an E4M3 cache; T: the new tokens' type.  2^lt_log2 threads a token;
// 2^dim_log2 pieces a head.
template <typename T, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads, 6)
append_kernel(const AppendParams p, int lt_log2, int dim_log2) {
  constexpr int kPieces = kPiecesOf<kFp8>;
  const int part = threadIdx.x & ((1 << lt_log2) - 1);
  const int64_t t = ((int64_t)blockIdx.x << (8 - lt_log2)) + (threadIdx.x >> lt_log2);
  static_assert(kAppendThreads == 256, "8 bits of thread index");
  pdl_wait();          // on every path: the grid's end must mean its predecessor's
  if (t >= p.num_tokens) return;
  const int row = p.c.heads << dim_log2;                // pieces of a token's K
  const unsigned char* k_src = p.k + t * p.k_token;
  const unsigned char* v_src = p.v + t * p.v_token;
  const int64_t e = p.entries[t];
  const int32_t r = p.t2r[t];
  int32_t page = -1;
  int64_t k_dst = 0, v_dst = 0;
  for (int i0 = part; i0 < 2 * row; i0 += kPieces << lt_log2) {
    uint4 x[kPieces][kFp8 ? 2 : 1];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int i = i0 + (j << lt_log2);
      if (i < 2 * row) {
        const bool is_v = i >= row;
        const int u = is_v ? i - row : i, h = u >> dim_log2, o = u & ((1 << dim_log2) - 1);
        const unsigned char* src = is_v ? v_src + h * p.v_head : k_src + h * p.k_head;
#pragma unroll
        for (int q = 0; q < (kFp8 ? 2 : 1); ++q)
          x[j][q] = ld_stream16(src + o * (kFp8 ? 32 : 16) + q * 16);
      }
    }
    if (i0 == part) {                                   // where the token goes
      if (e < 0) return;                                // padding
      uint32_t bad = 0;
      if (r < 0 || r >= p.c.num_reqs) {
        bad = QSA_DERR_REQUEST;
      } else if (e >= p.cap) {
        bad = QSA_DERR_CONTEXT;
      } else {
        page = p.c.bt[(int64_t)r * p.c.bt_s0 + (e >> p.c.page_log2)];
        if (page < 0 || page >= p.c.num_pages) bad = QSA_DERR_KV_PAGE;
      }
      if (bad) {
        if (part == 0) report(p.err, bad);
        return;
      }
      const int64_t slot = e & (((int64_t)1 << p.c.page_log2) - 1);
      k_dst = page * p.c.k_page + slot * p.c.k_token;
      v_dst = page * p.c.v_page + slot * p.c.v_token;
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int i = i0 + (j << lt_log2);
      if (i < 2 * row) {
        const bool is_v = i >= row;
        const int u = is_v ? i - row : i, h = u >> dim_log2, o = u & ((1 << dim_log2) - 1);
        unsigned char* dst = is_v ? p.c.v + v_dst + h * p.c.v_head : p.c.k + k_dst + h * p.c.k_head;
        uint4 y = x[j][0];
        if constexpr (kFp8) {
          const float* sc = is_v ? p.c.v_scale : p.c.k_scale;
          const float inv = sc ? 1.f / sc[h] : 1.f;
          const uint2 lo = to_e4m3<T>(x[j][0], inv), hi = to_e4m3<T>(x[j][1], inv);
          y = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        *reinterpret_cast<uint4*>(dst + o * 16) = y;
      }
    }
  }
  if (part == 0) {
    if (p.entry_pos)
      p.entry_pos[(int64_t)r * p.entry_pos_s0 + e] = (int32_t)(p.positions ? p.positions[t] : e);
    if (p.sums) p.sums[(int64_t)r * p.sums_s0 + e] = 0.f;
  }
}

template <typename T, bool kFp8>
cudaError_t launch_append(const AppendParams& p, cudaStream_t st) {
  const int head_pieces = p.c.dim / (kFp8 ? 16 : 8);
  int dim_log2 = 0, lt_log2 = 0;
  while ((1 << dim_log2) < head_pieces) ++dim_log2;
  while ((kPiecesOf<kFp8> << lt_log2) < 2 * p.c.heads * head_pieces && lt_log2 < 8) ++lt_log2;
  const int64_t per_cta = kAppendThreads >> lt_log2;
  const int64_t grid = (p.num_tokens + per_cta - 1) / per_cta;
  return launch_after(append_kernel<T, kFp8>, dim3((unsigned)grid), dim3(kAppendThreads), 0, st, p,
                      lt_log2, dim_log2);
}

}  // namespace
}  // namespace qsa

extern "C" qsa_status qsa_paged_append(
    const qsa_paged_cache* cache, const void* k, const void* v, qsa_dtype dtype,
    int64_t num_tokens, const int64_t k_strides[3], const int64_t v_strides[3],
    const int32_t* token_to_request, const int64_t* entries, const int64_t* positions,
    int32_t* entry_positions, int64_t entry_positions_stride0, float* weight_sums,
    int64_t weight_sums_stride0, int64_t entry_cols, uint32_t* error_word, qsa_stream_t stream) {
  using namespace qsa;
  using namespace qsa::cache_host;
  AppendParams p{};
  CacheSpans cs{};
  const qsa_status st = check_cache(cache, &p.c, &cs);
  if (st != QSA_OK) return st;
  if (dtype != QSA_DT_F16 && dtype != QSA_DT_BF16) return QSA_ERR_DTYPE;
  if (cache->dtype != QSA_DT_F8E4M3 && cache->dtype != dtype) return QSA_ERR_DTYPE;
  if (!k_strides || !v_strides) return QSA_ERR_NULL;
  if (num_tokens < 0 || num_tokens > (int64_t)1 << 24) return QSA_ERR_SHAPE;
  const bool book = entry_positions || weight_sums;
  if (book && (entry_cols < 0 || entry_cols > INT32_MAX)) return QSA_ERR_SHAPE;
  const int64_t shape[3] = {num_tokens, p.c.heads, p.c.dim};
  if (num_tokens > 0 && (!strides_ok(shape, k_strides, 3, 2) || !strides_ok(shape, v_strides, 3, 2)))
    return QSA_ERR_STRIDE;
  if ((entry_positions && !row_stride_ok(entry_positions_stride0, entry_cols)) ||
      (weight_sums && !row_stride_ok(weight_sums_stride0, entry_cols)))
    return QSA_ERR_STRIDE;
  if (num_tokens == 0) return QSA_OK;
  const int64_t kx = extent(shape, k_strides, 3, 2), vx = extent(shape, v_strides, 3, 2);
  if (kx < 0 || vx < 0) return QSA_ERR_STRIDE;
  if (!k || !v || !token_to_request || !entries) return QSA_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(token_to_request, 4) ||
      !aligned(entries, 8) || !aligned(positions, 8) || !aligned(entry_positions, 4) ||
      !aligned(weight_sums, 4) || !aligned(error_word, 4))
    return QSA_ERR_ALIGN;
  if (p.c.k == p.c.v && p.c.num_pages > 0) return QSA_ERR_ALIAS;   // one tensor given twice
  // the cache's K and V may interleave in one buffer, so their spans are
  // outputs that may overlap each other
  const Span book_outs[3] = {
      rows_span(entry_positions, p.c.num_reqs, entry_cols, entry_positions_stride0),
      rows_span(weight_sums, p.c.num_reqs, entry_cols, weight_sums_stride0),
      span(error_word, 4)};
  const Span ins[8] = {span(k, kx), span(v, vx), span(token_to_request, num_tokens * 4),
                       span(entries, num_tokens * 8), span(positions, num_tokens * 8),
                       cs.tables, cs.k_scale, cs.v_scale};
  if (any_overlap(book_outs, 3, ins, 8)) return QSA_ERR_ALIAS;
  for (const Span& o : {cs.k, cs.v}) {
    if (any_overlap(&o, 1, ins, 8) || any_overlap(&o, 1, book_outs, 3)) return QSA_ERR_ALIAS;
  }
  p.k = static_cast<const unsigned char*>(k);
  p.v = static_cast<const unsigned char*>(v);
  p.k_token = num_tokens > 1 ? k_strides[0] * 2 : 0;
  p.k_head = p.c.heads > 1 ? k_strides[1] * 2 : 0;
  p.v_token = num_tokens > 1 ? v_strides[0] * 2 : 0;
  p.v_head = p.c.heads > 1 ? v_strides[1] * 2 : 0;
  p.t2r = token_to_request;
  p.entries = entries;
  p.positions = positions;
  p.entry_pos = entry_positions;
  p.entry_pos_s0 = entry_positions_stride0;
  p.sums = weight_sums;
  p.sums_s0 = weight_sums_stride0;
  p.cap = book && entry_cols < p.c.cap ? (int32_t)entry_cols : p.c.cap;
  p.num_tokens = num_tokens;
  p.err = error_word;
  bind_calling_thread();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype != QSA_DT_F8E4M3) e = launch_append<__half, false>(p, s);   // a copy of 16-bit values
  else if (dtype == QSA_DT_F16) e = launch_append<__half, true>(p, s);
  else e = launch_append<__nv_bfloat16, true>(p, s);
  return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}
