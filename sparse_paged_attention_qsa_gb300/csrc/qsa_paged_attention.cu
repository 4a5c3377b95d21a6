// qsa_paged_attention.cu -- dense attention of a request's new tokens over
// its paged K/V cache, declared in include/qsa_cache.h.
//
// One CTA per (row, query head) walks the row's entries, a warp an entry at a
// time, with the running maximum and sum of a softmax in binary32; the warps
// merge through shared memory.  A second kernel adds up the weights from the
// logits that the first one leaves in the workspace.
#include "qsa_cache.h"
#include "qsa_cache_host.h"
#include "qsa_device.cuh"
#include "qsa_host.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

namespace qsa {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxDim = 256;

struct DenseParams {
  CacheView c;
  const unsigned char* q;
  int64_t q_row, q_head;      // bytes
  unsigned char* out;
  int64_t out_row, out_head;  // bytes
  const int32_t* ctx;
  int next_n, heads, group;
  float scale;
  int64_t window;
  float* lse;                 // nullable
  float* ml;                  // workspace: [rows*heads][2] maximum and sum
  float* z;                   // workspace: [rows*heads][cap] logits, or null
  const float* sums;
  int64_t sums_s0;
  float* sums_out;
  int64_t sums_out_s0;
  uint32_t* err;
};

template <typename T> __device__ __forceinline__ float to_f(T x) { return (float)x; }

template <typename T, typename KV>
__global__ void __launch_bounds__(kWarps * 32)
row_kernel(const DenseParams p) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_acc[kWarps][kMaxDim];
  const int rh = blockIdx.x, h = rh % p.heads, row = rh / p.heads;
  const int b = row / p.next_n, j = row % p.next_n, kvh = h / p.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.c.dim, per = D / 32;
  const int64_t ctx = p.ctx[b];
  const int64_t hi0 = ctx - p.next_n + j + 1;
  const int64_t lo = p.window > 0 ? max((int64_t)0, hi0 - p.window) : 0;
  const int64_t hi = min(hi0, (int64_t)p.c.cap);
  if (ctx > p.c.cap && threadIdx.x == 0) report(p.err, QSA_DERR_CONTEXT);
  const T* q = reinterpret_cast<const T*>(p.q + row * p.q_row + h * p.q_head);
  const float ks = p.c.k_scale ? p.c.k_scale[kvh] : 1.f, vs = p.c.v_scale ? p.c.v_scale[kvh] : 1.f;
  float qf[kMaxDim / 32], acc[kMaxDim / 32];
  for (int i = 0; i < per; ++i) {
    qf[i] = to_f(q[lane * per + i]);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t e = lo + warp; e < hi; e += kWarps) {
    const int32_t page = p.c.bt[(int64_t)b * p.c.bt_s0 + (e >> p.c.page_log2)];
    float z = -INFINITY;
    if (page < 0 || page >= p.c.num_pages) {
      if (lane == 0) report(p.err, QSA_DERR_KV_PAGE);
    } else {
      const int64_t slot = e & (((int64_t)1 << p.c.page_log2) - 1);
      const KV* k = reinterpret_cast<const KV*>(p.c.k + page * p.c.k_page + slot * p.c.k_token + kvh * p.c.k_head);
      const KV* v = reinterpret_cast<const KV*>(p.c.v + page * p.c.v_page + slot * p.c.v_token + kvh * p.c.v_head);
      float s = 0.f;
      for (int i = 0; i < per; ++i) s = fmaf(qf[i], to_f(k[lane * per + i]), s);
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      z = s * ks * p.scale;
      const float mn = fmaxf(m, z);
      const float c = m == -INFINITY ? 0.f : expf(m - mn), w = expf(z - mn);
      l = l * c + w;
      for (int i = 0; i < per; ++i) acc[i] = acc[i] * c + w * to_f(v[lane * per + i]);
      m = mn;
    }
    if (p.z && lane == 0) p.z[(int64_t)rh * p.c.cap + e] = z;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int i = 0; i < per; ++i) s_acc[warp][lane * per + i] = acc[i];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  for (int w = 0; w < kWarps; ++w) L += s_m[w] == -INFINITY ? 0.f : s_l[w] * expf(s_m[w] - M);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (s_m[w] != -INFINITY) o += s_acc[w][d] * expf(s_m[w] - M);
    T* out = reinterpret_cast<T*>(p.out + row * p.out_row + h * p.out_head);
    out[d] = (T)(M == -INFINITY ? 0.f : o / L * vs);
  }
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[rh] = M == -INFINITY ? -INFINITY : M + logf(L);
    p.ml[2 * rh] = M;
    p.ml[2 * rh + 1] = L;
  }
}

__global__ void __launch_bounds__(256) weights_kernel(const DenseParams p) {
  const int b = blockIdx.y;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t ctx = p.ctx[b];
  if (e >= min(ctx, (int64_t)p.c.cap)) return;
  float s = 0.f;
  for (int j = 0; j < p.next_n; ++j) {
    const int64_t hi = ctx - p.next_n + j + 1;
    const int64_t lo = p.window > 0 ? max((int64_t)0, hi - p.window) : 0;
    if (e < lo || e >= hi) continue;
    for (int h = 0; h < p.heads; ++h) {
      const int64_t rh = ((int64_t)b * p.next_n + j) * p.heads + h;
      const float z = p.z[rh * p.c.cap + e];
      if (z != -INFINITY) s += expf(z - p.ml[2 * rh]) / p.ml[2 * rh + 1];
    }
  }
  p.sums_out[b * p.sums_out_s0 + e] = p.sums[b * p.sums_s0 + e] + s;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

bool sizes_ok(int64_t reqs, int64_t next_n, int64_t heads, int64_t kv_heads, int64_t dim) {
  return reqs >= 0 && reqs <= QSA_CACHE_MAX_REQS && next_n >= 1 && next_n <= QSA_CACHE_MAX_NEXT &&
         kv_heads >= 1 && kv_heads <= QSA_CACHE_MAX_HEADS && heads >= 1 && heads % kv_heads == 0 &&
         heads * next_n <= 65536 && (dim == 64 || dim == 128 || dim == 256);
}

}  // namespace
}  // namespace qsa

extern "C" size_t qsa_paged_attention_workspace_bytes(
    int64_t num_reqs, int64_t next_n, int64_t num_heads, int64_t kv_heads, int64_t head_dim,
    int64_t weight_cols) {
  if (!qsa::sizes_ok(num_reqs, next_n, num_heads, kv_heads, head_dim) || num_reqs == 0 ||
      weight_cols < 0 || weight_cols > INT32_MAX)
    return 0;
  const __int128 rows = (__int128)num_reqs * next_n * num_heads;
  const __int128 n = rows * 8 + 256 + rows * weight_cols * 4 + 256;
  return n > ((__int128)1 << 60) ? 0 : (size_t)n;
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
  DenseParams p{};
  CacheSpans cs{};
  const qsa_status st = check_cache(cache, &p.c, &cs);
  if (st != QSA_OK) return st;
  if (dtype != QSA_DT_F16 && dtype != QSA_DT_BF16) return QSA_ERR_DTYPE;
  if (cache->dtype != QSA_DT_F8E4M3 && cache->dtype != dtype) return QSA_ERR_DTYPE;
  if (!(std::isfinite(scale) && scale > 0.f) || window < 0) return QSA_ERR_CONTRACT;
  const int64_t R = cache->num_reqs;
  if (!sizes_ok(R, next_n, num_heads, cache->num_heads, cache->head_dim)) return QSA_ERR_SHAPE;
  if (!q_strides || !out_strides) return QSA_ERR_NULL;
  const int64_t shape[3] = {R * next_n, num_heads, cache->head_dim};
  if (!strides_ok(shape, q_strides, 3, 2) || !strides_ok(shape, out_strides, 3, 2))
    return QSA_ERR_STRIDE;
  const bool weights = weight_sums || weight_sums_out;
  const int64_t entries = cache->table_cols * cache->page_size;
  if (weights) {
    if (!weight_sums || !weight_sums_out) return QSA_ERR_NULL;
    if (entries > INT32_MAX || entry_cols < entries || entry_cols > INT32_MAX) return QSA_ERR_SHAPE;
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
  const size_t need = qsa_paged_attention_workspace_bytes(R, next_n, num_heads, cache->num_heads,
                                                          cache->head_dim, weights ? entries : 0);
  if (need == 0) return QSA_ERR_SHAPE;
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
  if (!workspace || workspace_bytes < need) return QSA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QSA_ERR_ALIGN;
  p.q = static_cast<const unsigned char*>(q);
  p.q_row = q_strides[0] * 2;
  p.q_head = q_strides[1] * 2;
  p.out = static_cast<unsigned char*>(out);
  p.out_row = out_strides[0] * 2;
  p.out_head = out_strides[1] * 2;
  p.ctx = context_lens;
  p.next_n = (int)next_n;
  p.heads = (int)num_heads;
  p.group = (int)(num_heads / cache->num_heads);
  p.scale = scale;
  p.window = window;
  p.lse = lse;
  p.ml = static_cast<float*>(workspace);
  const int64_t rows = R * next_n * num_heads;
  if (weights) p.z = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + round256(rows * 8));
  p.sums = weight_sums;
  p.sums_s0 = weight_sums_stride0;
  p.sums_out = weight_sums_out;
  p.sums_out_s0 = weight_sums_out_stride0;
  p.err = error_word;
  bind_calling_thread();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool half = dtype == QSA_DT_F16, fp8 = cache->dtype == QSA_DT_F8E4M3;
  auto kernel = half ? (fp8 ? row_kernel<__half, __nv_fp8_e4m3> : row_kernel<__half, __half>)
                     : (fp8 ? row_kernel<__nv_bfloat16, __nv_fp8_e4m3>
                            : row_kernel<__nv_bfloat16, __nv_bfloat16>);
  kernel<<<(unsigned)rows, kWarps * 32, 0, s>>>(p);
  if (weights && entries > 0)
    weights_kernel<<<dim3((unsigned)((entries + 255) / 256), (unsigned)R), 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}
