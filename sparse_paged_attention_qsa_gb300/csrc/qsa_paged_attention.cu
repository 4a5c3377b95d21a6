// qsa_paged_attention.cu -- dense attention of a request's new tokens over
// its paged K/V cache, declared in include/qsa_cache.h: the entry point and
// the kernel that adds up the weights entries received.  The attention's own
// kernels are in qsa_paged_attn_impl.cuh.
//
// Weights: an entry's weight is known only once its row's sum is, so the walk
// leaves the logits (binary32, base 2) in the workspace and weights_kernel
// reads them back, 8 bytes a head beside the 2 * dim * esize * kv_heads that
// K and V take: 6 % for four heads of 128 on a 16-bit K/V head.  (Reading K
// again instead would be half of the whole.)  Up to eight warps each add a part of
// an entry's (row, head) pairs in order, and the parts are added in warp order, so
// the sum does not change from run to run.
#include "qsa_cache.h"
#include "qsa_cache_host.h"
#include "qsa_device.cuh"
#include "qsa_host.h"
#include "qsa_internal.h"
#include "qsa_paged_attn.h"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

namespace qsa {
namespace {

// Warps of a CTA of weights_kernel, at most; a lane has four loads of each in flight
// (39 requests of 5081 entries and 128 pairs of row and head, a call: 172 us; 16
// warps with eight loads 184, 8 with two 176, 4 with four 176).
constexpr int kWeightParts = 8;

#ifdef QSA_WAIT_TEST
int32_t g_test_withhold = -1;
#endif

struct WeightParams {
  const int32_t* ctx;
  const float* z;             // [rows][heads][pitch] logits (base 2)
  const float2* stats;        // [rows][heads] reference and log2 of the sum
  int64_t pitch;
  int32_t window;
  int32_t cap, next_n, heads;
  const float* sums;
  int64_t sums_s0;
  float* sums_out;
  int64_t sums_out_s0;
};

// A lane holds four entries of one request (the table's entries are a multiple
// of 8), a warp a part of the (row, head) pairs, so that their logits are all in
// flight at once; the parts are added in warp order.
__global__ void __launch_bounds__(kWeightParts * 32) weights_kernel(const WeightParams p) {
  __shared__ float4 s_part[kWeightParts][32];
  const int b = blockIdx.y, lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int parts = blockDim.x >> 5;
  const int e = ((int)blockIdx.x * 32 + lane) * 4;
  pdl_wait();          // on every path: the grid's end must mean the walk's and the join's
  const int64_t ctx = p.ctx[b];
  const int n = (int)min(ctx, (int64_t)p.cap);
  if ((int)blockIdx.x * 128 >= n) return;
  const int pairs = p.next_n * p.heads, per = (pairs + parts - 1) / parts;
  const int x0 = part * per, x1 = min(pairs, x0 + per);
  const int64_t first = (int64_t)b * pairs;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  int j = x0 / p.heads, left = (j + 1) * p.heads - x0;     // pairs of token j still to come
  for (int x = x0; x < x1;) {
    const int64_t hi = ctx - p.next_n + j + 1;
    const int64_t lo = p.window > 0 ? max((int64_t)0, hi - p.window) : 0;
    const int end = min(x1, x + left);
    if (e + 3 >= lo && e < min(hi, (int64_t)n)) {
      const bool in[4] = {e >= lo, e + 1 >= lo && e + 1 < hi, e + 2 >= lo && e + 2 < hi,
                          e + 3 >= lo && e + 3 < hi};
#pragma unroll 4
      for (int y = x; y < end; ++y) {
        const float4 z = *reinterpret_cast<const float4*>(p.z + (first + y) * p.pitch + e);
        const float2 r = p.stats[first + y];
        // -inf (an absent entry): 0, also where the row saw nothing and r.x is -inf
        s.x += in[0] && z.x != -INFINITY ? exp2f(z.x - r.x - r.y) : 0.f;
        s.y += in[1] && z.y != -INFINITY ? exp2f(z.y - r.x - r.y) : 0.f;
        s.z += in[2] && z.z != -INFINITY ? exp2f(z.z - r.x - r.y) : 0.f;
        s.w += in[3] && z.w != -INFINITY ? exp2f(z.w - r.x - r.y) : 0.f;
      }
    }
    x = end;
    ++j;
    left = p.heads;
  }
  s_part[part][lane] = s;
  __syncthreads();
  if (part < 4 && e + part < n) {        // warp i: the i-th entry of each four
    float v = 0.f;
    for (int k = 0; k < parts; ++k) v += reinterpret_cast<const float*>(&s_part[k][lane])[part];
    p.sums_out[b * p.sums_out_s0 + e + part] = p.sums[b * p.sums_s0 + e + part] + v;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// One of the cache's views as (dim, head, slot, page); a box is one head's
// `rows` slots of up to 128 bytes, so that a row is one line of the swizzle.
bool encode_view(CUtensorMap* map, const unsigned char* p, const CacheView& c, int esize,
                 int64_t page, int64_t token, int64_t head, int rows) {
  memset(map, 0, sizeof(*map));
  if (c.num_pages == 0) return true;                       // no copy is ever issued
  const auto fn = encode_fn();
  if (!fn) return false;
  const int row_bytes = c.dim * esize, inner = std::min(row_bytes, 128);
  const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.heads,
                              (cuuint64_t)1 << c.page_log2, (cuuint64_t)c.num_pages};
  // a dimension of size 1 has any stride; the encoder wants a legal one
  const cuuint64_t strides[3] = {(cuuint64_t)(head ? head : row_bytes), (cuuint64_t)token,
                                 (cuuint64_t)(page ? page : token)};
  const cuuint32_t box[4] = {(cuuint32_t)(inner / esize), 1, (cuuint32_t)rows, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
            const_cast<unsigned char*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            // no wider than a row: what follows it is another head's
            row_bytes >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                             : CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

bool sizes_ok(const qsa_paged_cache& c, int64_t next_n, int64_t heads) {
  return next_n >= 1 && next_n <= QSA_CACHE_MAX_NEXT && heads >= 1 && heads <= 65536 &&
         heads % c.num_heads == 0 && heads * next_n <= 65536;
}

// The workspace: where each run starts, the pieces of K/V heads that the
// runs cut (at most two a run), neither in the modes without a second kernel;
// then, when weights are asked for, the rows' sums and logits.
struct Layout {
  PagedMode mode;
  size_t ml, o, stats, z, total;
};

// 0 as the total where it cannot be addressed.
Layout layout_of(const qsa_paged_cache& c, const CacheView& v, int64_t next_n, int64_t heads,
                 bool weights) {
  const size_t rows = (size_t)std::min<int64_t>(next_n * (heads / c.num_heads), kPagedMaxRows);
  const int64_t all = c.num_reqs * next_n * heads, entries = weights ? v.cap : 0;
  Layout l;
  const int64_t request = (int64_t)v.cap * 2 * c.head_dim * cache_host::dtype_size(c.dtype);
  l.mode = request <= kPagedWholeBytes ? kPagedWhole
           : rows <= 16 && c.num_reqs * request <= kPagedCluster8 * kPagedWholeBytes ? kPagedCluster
                                                                                     : kPagedCut;
  const bool pieces = l.mode == kPagedCut;
  l.ml = pieces ? round256(kPagedMaxCtas * sizeof(int4)) : 0;
  l.o = l.ml + (pieces ? round256(2 * kPagedMaxCtas * rows * 2 * sizeof(float)) : 0);
  l.stats = l.o + (pieces ? round256(2 * kPagedMaxCtas * rows * (size_t)c.head_dim * sizeof(float)) : 0);
  l.z = l.stats + (entries > 0 ? round256((size_t)all * sizeof(float2)) : 0);
  const __int128 total = (__int128)l.z + (__int128)all * entries * 4;
  l.total = total < ((__int128)1 << 60) ? (size_t)total : 0;
  if (l.total == 0) l.total = total == 0 ? 0 : SIZE_MAX;
  return l;
}

}  // namespace
}  // namespace qsa

extern "C" size_t qsa_paged_attention_workspace_bytes(const qsa_paged_cache* cache, int64_t next_n,
                                                      int64_t num_heads, int with_weights) {
  using namespace qsa;
  CacheView view{};
  cache_host::CacheSpans spans{};
  if (cache_host::check_cache(cache, &view, &spans) != QSA_OK || cache->num_reqs == 0 ||
      !sizes_ok(*cache, next_n, num_heads))
    return 0;
  const size_t n = layout_of(*cache, view, next_n, num_heads, with_weights != 0).total;
  return n == SIZE_MAX ? 0 : n;
}

extern "C" qsa_status qsa_paged_attention(
    const qsa_paged_cache* cache, const void* q, qsa_dtype dtype, int64_t next_n,
    int64_t num_heads, const int64_t q_strides[3], const int32_t* context_lens, float scale,
    int64_t window, void* out, const int64_t out_strides[3], float* lse, const float* weight_sums,
    int64_t weight_sums_stride0, float* weight_sums_out, int64_t weight_sums_out_stride0,
    int64_t entry_cols, void* workspace, size_t workspace_bytes, uint32_t* error_word,
    qsa_stream_t stream) {
  using namespace qsa;
  using namespace qsa::cache_host;
  PagedParams p{};
  CacheSpans cs{};
  const qsa_status st = check_cache(cache, &p.c, &cs);
  if (st != QSA_OK) return st;
  if (dtype != QSA_DT_F16 && dtype != QSA_DT_BF16) return QSA_ERR_DTYPE;
  if (cache->dtype != QSA_DT_F8E4M3 && cache->dtype != dtype) return QSA_ERR_DTYPE;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!(std::isfinite(scale_log2) && scale > 0.f) || window < 0) return QSA_ERR_CONTRACT;
  const int64_t R = cache->num_reqs;
  if (!sizes_ok(*cache, next_n, num_heads)) return QSA_ERR_SHAPE;
  if (!q_strides || !out_strides) return QSA_ERR_NULL;
  const int64_t shape[3] = {R * next_n, num_heads, cache->head_dim};
  if (!strides_ok(shape, q_strides, 3, 2) || !strides_ok(shape, out_strides, 3, 2) ||
      !separate(shape, out_strides, 3))
    return QSA_ERR_STRIDE;
  const bool weights = weight_sums || weight_sums_out;
  const int64_t entries = cache->table_cols * cache->page_size;
  if (weights) {
    if (!weight_sums || !weight_sums_out) return QSA_ERR_NULL;
    if (entries > kMaxEntries || entry_cols < entries || entry_cols > INT32_MAX) return QSA_ERR_SHAPE;
    if (!row_stride_ok(weight_sums_stride0, entry_cols) ||
        !row_stride_ok(weight_sums_out_stride0, entry_cols))
      return QSA_ERR_STRIDE;
  }
  if (R == 0) return QSA_OK;
  const int64_t qx = extent(shape, q_strides, 3, 2), ox = extent(shape, out_strides, 3, 2);
  if (qx < 0 || ox < 0) return QSA_ERR_STRIDE;
  if (!q || !out || !context_lens) return QSA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(context_lens, 4) || !aligned(lse, 4) ||
      !aligned(weight_sums, 4) || !aligned(weight_sums_out, 4) || !aligned(error_word, 4))
    return QSA_ERR_ALIGN;
  const Layout l = layout_of(*cache, p.c, next_n, num_heads, weights);
  const size_t need = l.total;
  if (need == SIZE_MAX) return QSA_ERR_SHAPE;
  const Span ws = span(workspace, (int64_t)need);
  const Span sums_in = weights ? rows_span(weight_sums, R, entry_cols, weight_sums_stride0) : Span{};
  const Span outs[5] = {span(out, ox), span(lse, R * next_n * num_heads * 4),
                        weights ? rows_span(weight_sums_out, R, entry_cols, weight_sums_out_stride0)
                                : Span{},
                        span(error_word, 4), ws};
  const Span ins[7] = {span(q, qx), cs.k, cs.v, cs.tables, cs.k_scale, cs.v_scale,
                       span(context_lens, R * 4)};
  if (any_overlap(outs, 5, ins, 7)) return QSA_ERR_ALIAS;
  const bool in_place = weights && weight_sums == weight_sums_out &&
                        weight_sums_stride0 == weight_sums_out_stride0;
  for (int i = 0; i < 5; ++i)
    if (!(i == 2 && in_place) && overlaps(outs[i], sums_in)) return QSA_ERR_ALIAS;
  if (need > 0 && (!workspace || workspace_bytes < need)) return QSA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QSA_ERR_ALIGN;
  p.q = static_cast<const unsigned char*>(q);
  p.q_row = R * next_n > 1 ? q_strides[0] * 2 : 0;
  p.q_head = num_heads > 1 ? q_strides[1] * 2 : 0;
  p.out = static_cast<unsigned char*>(out);
  p.out_row = R * next_n > 1 ? out_strides[0] * 2 : 0;
  p.out_head = num_heads > 1 ? out_strides[1] * 2 : 0;
  p.ctx = context_lens;
  p.next_n = (int)next_n;
  p.heads = (int)num_heads;
  p.group = (int)(num_heads / cache->num_heads);
  p.rows = p.next_n * p.group;
  p.chunks = (p.rows + kPagedMaxRows - 1) / kPagedMaxRows;
  p.chunk_rows = std::min(p.rows, kPagedMaxRows);
  p.scale_log2 = scale_log2;
  // a window past every capacity (2^30 at most) hides nothing, whatever it is
  p.window = (int32_t)std::min<int64_t>(window, INT32_MAX - 16);
  p.lse = lse;
  unsigned char* w = static_cast<unsigned char*>(workspace);
  p.mode = l.mode;
  p.starts = reinterpret_cast<int4*>(w);
  p.part_ml = reinterpret_cast<float*>(w + l.ml);
  p.part_o = reinterpret_cast<float*>(w + l.o);
  if (weights && entries > 0) {
    p.stats = reinterpret_cast<float2*>(w + l.stats);
    p.z = reinterpret_cast<float*>(w + l.z);
    p.z_pitch = entries;
  }
  p.err = error_word;
  bind_calling_thread();
  const bool bf16 = dtype == QSA_DT_BF16, fp8 = cache->dtype == QSA_DT_F8E4M3;
  const int esize = fp8 ? 1 : 2;
  const int tile = paged_tile(p.c.dim, p.c.dim * esize, paged_sets(p.chunk_rows));
  const int rows = (int)std::min<int64_t>(cache->page_size, tile);
  CUtensorMap kmap, vmap;
  if (!encode_view(&kmap, p.c.k, p.c, esize, p.c.k_page, p.c.k_token, p.c.k_head, rows) ||
      !encode_view(&vmap, p.c.v, p.c, esize, p.c.v_page, p.c.v_token, p.c.v_head, rows))
    return QSA_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // a launch's tiles are counted in 31 bits
  const int64_t per_row = std::max<int64_t>(1, ((int64_t)p.c.cap + tile - 1) / tile);
  const int64_t step = std::max<int64_t>(1, std::min<int64_t>(kPagedBatch, INT32_MAX / per_row));
  for (int64_t b0 = 0; b0 < R; b0 += step) {
    p.b0 = (int32_t)b0;
    p.batch = (int32_t)std::min<int64_t>(step, R - b0);
#ifdef QSA_WAIT_TEST
    p.test_withhold = b0 == 0 ? g_test_withhold : -1;      // heads of 64 alone are built
    const cudaError_t e = p.c.dim == 64 ? launch_paged_64(p, bf16, fp8, kmap, vmap, s)
                                        : cudaErrorNotSupported;
#else
    const cudaError_t e = p.c.dim == 64    ? launch_paged_64(p, bf16, fp8, kmap, vmap, s)
                          : p.c.dim == 128 ? launch_paged_128(p, bf16, fp8, kmap, vmap, s)
                                           : launch_paged_256(p, bf16, fp8, kmap, vmap, s);
#endif
    if (e != cudaSuccess) return QSA_ERR_CUDA;
  }
  if (p.z) {
    WeightParams wp{};
    wp.ctx = context_lens;
    wp.z = p.z;
    wp.stats = p.stats;
    wp.pitch = p.z_pitch;
    wp.window = p.window;
    wp.cap = p.c.cap;
    wp.next_n = p.next_n;
    wp.heads = p.heads;
    wp.sums = weight_sums;
    wp.sums_s0 = weight_sums_stride0;
    wp.sums_out = weight_sums_out;
    wp.sums_out_s0 = weight_sums_out_stride0;
    const int64_t per_cta = 128;
    const dim3 grid((unsigned)((entries + per_cta - 1) / per_cta), (unsigned)R);
    // eight pairs a warp; four warps at least, one for each entry of a lane's
    const int pairs = p.next_n * p.heads;
    const int parts = std::max(4, std::min(kWeightParts, (pairs + 7) / 8));
    if (launch_after(weights_kernel, grid, dim3(parts * 32), 0, s, wp) != cudaSuccess)
      return QSA_ERR_CUDA;
  }
  return QSA_OK;
}

#ifdef QSA_WAIT_TEST
// Test build only, declared in no public header: the next attention launches
// leave slot fill `issue` of the walk's CTA 0 without a copy (-1: none).
extern "C" __attribute__((visibility("default"))) void qsa_test_withhold_paged_fill(
    int32_t issue) {
  qsa::g_test_withhold = issue;
}
#endif
