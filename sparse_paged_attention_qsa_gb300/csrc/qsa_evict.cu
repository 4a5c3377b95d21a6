// qsa_evict.cu -- evicting the entries of a paged K/V cache that received
// the least attention weight, declared in include/qsa_cache.h
// (qsa_evict_entries).
//
// rank_kernel  per request: the budget-th largest key (protected entries, then
//              the weight sums' order-preserving bits) by radix select; in
//              entry order, which entries of equal key stay, which places
//              below the budget fall free (holes) and which kept entries lie
//              above it (movers).  As many of one as of the other, so the i-th
//              mover goes to the i-th hole: no entry is written that is read,
//              and only what has to move moves.
// move_kernel  copies the movers' K and V.
#include "qsa_cache.h"
#include "qsa_cache_host.h"
#include "qsa_device.cuh"
#include "qsa_host.h"

#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

namespace qsa {
namespace {

constexpr int kRankThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

struct EvictParams {
  CacheView c;
  const float* sums;
  int64_t sums_s0;
  const int32_t* pos;
  int64_t pos_s0;
  const int32_t* ctx;
  int32_t cap;                // entries a request can have here
  int32_t budget, sink, recent;
  int32_t* kept;              // [reqs, budget]
  int32_t* new_lens;
  float* sums_out;
  int32_t* pos_out;
  int32_t* moves;             // workspace: [reqs, budget, 2] (from, to)
  int32_t* count;             // workspace: [reqs] moves of a request
  uint32_t* err;
};

// Order-preserving bits of a weight sum: NaN 0, -inf next, +0 and -0 equal;
// +inf stays below kProtected.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Sum of v over the threads before this one; *total over all of them.
__device__ __forceinline__ int block_prefix(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                       // s_warp free again
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kRankThreads / 32; ++i) {
    const int c = s_warp[i];
    if (i < warp) before += c;
    all += c;
  }
  *total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kRankThreads)
rank_kernel(const EvictParams p) {
  __shared__ int s_hist[2048];
  __shared__ int s_warp[kRankThreads / 32];
  __shared__ int s_newest, s_digit, s_need;
  const int b = blockIdx.x, tid = threadIdx.x;
  const float* w = p.sums + b * p.sums_s0;
  const int32_t* pos = p.pos + b * p.pos_s0;
  const int32_t ctx = p.ctx[b];
  const int n = max(0, min(ctx, p.cap));
  const int len = min(n, p.budget);
  int32_t* kept = p.kept + (int64_t)b * p.budget;
  int32_t* moves = p.moves + (int64_t)b * p.budget * 2;
  if (tid == 0) {
    if (ctx > p.cap) report(p.err, QSA_DERR_CONTEXT);
    p.new_lens[b] = len;
    s_newest = INT32_MIN;
  }
  int moved = 0;
  if (n > p.budget) {
    __syncthreads();
    int newest = INT32_MIN;
    for (int e = tid; e < n; e += kRankThreads) newest = max(newest, pos[e]);
    atomicMax(&s_newest, newest);
    __syncthreads();
    // position > newest - recent, in 64 bits: neither may wrap
    const int64_t after = (int64_t)s_newest - p.recent;
    const auto key_of = [&](int e) {
      const int32_t q = pos[e];
      return q < p.sink || q > after ? kProtected : weight_key(w[e]);
    };
    // the budget-th largest key, 11 + 11 + 10 bits at a time
    uint32_t prefix = 0, mask = 0;
    int need = p.budget;                   // entries still to take below the digits found
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bins = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < bins; i += kRankThreads) s_hist[i] = 0;
      __syncthreads();
      for (int e = tid; e < n; e += kRankThreads) {
        const uint32_t k = key_of(e);
        if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // bins from the top: the one in which the count reaches `need`
      int total = 0;
      const int per = bins / kRankThreads;              // 2, 2, 1
      int mine = 0;
      const int top = bins - 1 - tid * per;
      for (int i = 0; i < per; ++i) mine += s_hist[top - i];
      int before = block_prefix(mine, s_warp, &total);
      for (int i = 0; i < per; ++i) {
        const int c = s_hist[top - i];
        if (before < need && before + c >= need) {
          s_digit = top - i;
          s_need = need - before;
        }
        before += c;
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      need = s_need;
      __syncthreads();
    }
    // in entry order: ties by entry, then holes and movers
    int ties = 0, holes = 0;
    for (int e0 = 0; e0 < n; e0 += kRankThreads) {
      const int e = e0 + tid;
      const bool there = e < n;
      const uint32_t k = there ? key_of(e) : 0u;
      const bool tie = there && k == prefix;
      int total = 0;
      const int rank = ties + block_prefix(tie, s_warp, &total);
      ties += total;
      const bool keep = there && (k > prefix || (tie && rank < need));
      const bool hole = there && e < p.budget && !keep;
      const bool mover = keep && e >= p.budget;
      // both counts in one prefix sum: neither passes 2^10 in a step
      const int both = block_prefix((int)hole | (int)mover << 16, s_warp, &total);
      if (hole) moves[2 * (holes + (both & 0xffff)) + 1] = e;
      if (mover) moves[2 * (moved + (both >> 16))] = e;
      if (there && e < p.budget && keep) kept[e] = e;
      holes += total & 0xffff;
      moved += total >> 16;
    }
    __syncthreads();
    for (int i = tid; i < moved; i += kRankThreads) kept[moves[2 * i + 1]] = moves[2 * i];
    __syncthreads();
  } else {
    for (int i = tid; i < p.budget; i += kRankThreads) kept[i] = i < len ? i : -1;
    __syncthreads();
  }
  if (tid == 0) p.count[b] = moved;
  for (int i = tid; i < p.budget; i += kRankThreads) {
    const int e = kept[i];
    p.sums_out[(int64_t)b * p.budget + i] = i < len ? w[e] : 0.f;
    p.pos_out[(int64_t)b * p.budget + i] = i < len ? pos[e] : -1;
  }
}

// CTA (x, b) takes the moves x, x + gridDim.x, ... of request b; the threads
// share a move's 16-byte pieces of K and V.
__global__ void __launch_bounds__(kMoveThreads)
move_kernel(const EvictParams p, int head_bytes) {
  const int b = blockIdx.y;
  const int count = p.count[b];
  const int32_t* moves = p.moves + (int64_t)b * p.budget * 2;
  const int32_t* bt = p.c.bt + (int64_t)b * p.c.bt_s0;
  const int slot_mask = (1 << p.c.page_log2) - 1;
  const int head_pieces = head_bytes / 16, row = p.c.heads * head_pieces;
  for (int m = blockIdx.x; m < count; m += gridDim.x) {
    const int from = moves[2 * m], to = moves[2 * m + 1];
    const int32_t pf = bt[from >> p.c.page_log2], pt = bt[to >> p.c.page_log2];
    if (pf < 0 || pf >= p.c.num_pages || pt < 0 || pt >= p.c.num_pages) {
      if (threadIdx.x == 0) report(p.err, QSA_DERR_KV_PAGE);
      continue;
    }
    const int sf = from & slot_mask, st = to & slot_mask;
    for (int i = threadIdx.x; i < 2 * row; i += kMoveThreads) {
      const bool is_v = i >= row;
      const int u = is_v ? i - row : i;
      const int h = u / head_pieces, o = u - h * head_pieces;
      unsigned char* base = is_v ? p.c.v : p.c.k;
      const int64_t ps = is_v ? p.c.v_page : p.c.k_page, ts = is_v ? p.c.v_token : p.c.k_token;
      unsigned char* at = base + h * (is_v ? p.c.v_head : p.c.k_head) + o * 16;
      *reinterpret_cast<uint4*>(at + pt * ps + st * ts) =
          *reinterpret_cast<const uint4*>(at + pf * ps + sf * ts);
    }
  }
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace
}  // namespace qsa

extern "C" size_t qsa_evict_workspace_bytes(int64_t num_reqs, int64_t budget) {
  if (num_reqs <= 0 || num_reqs > QSA_CACHE_MAX_REQS || budget <= 0 || budget > INT32_MAX) return 0;
  const __int128 n = (__int128)num_reqs * budget * 8;
  if (n > ((__int128)1 << 60)) return 0;
  return qsa::round256((size_t)n) + qsa::round256((size_t)num_reqs * 4);
}

extern "C" qsa_status qsa_evict_entries(
    const qsa_paged_cache* cache, const float* weight_sums, int64_t weight_sums_stride0,
    const int32_t* entry_positions, int64_t entry_positions_stride0, int64_t entry_cols,
    const int32_t* context_lens, int64_t budget, int64_t num_sink, int64_t num_recent,
    int32_t* kept, int32_t* new_lens, float* weight_sums_out, int32_t* entry_positions_out,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, qsa_stream_t stream) {
  using namespace qsa;
  using namespace qsa::cache_host;
  EvictParams p{};
  CacheSpans cs{};
  const qsa_status st = check_cache(cache, &p.c, &cs);
  if (st != QSA_OK) return st;
  if (budget < 1 || budget > INT32_MAX || num_sink < 0 || num_recent < 0 || num_sink > budget ||
      num_recent > budget - num_sink)
    return QSA_ERR_CONTRACT;
  if (entry_cols < 0 || entry_cols > INT32_MAX) return QSA_ERR_SHAPE;
  if (!row_stride_ok(weight_sums_stride0, entry_cols) ||
      !row_stride_ok(entry_positions_stride0, entry_cols))
    return QSA_ERR_STRIDE;
  const int64_t R = cache->num_reqs;
  if (R == 0) return QSA_OK;
  const size_t need = qsa_evict_workspace_bytes(R, budget);
  if (need == 0) return QSA_ERR_SHAPE;
  if (!context_lens || !kept || !new_lens || !weight_sums_out || !entry_positions_out)
    return QSA_ERR_NULL;
  if (entry_cols > 0 && (!weight_sums || !entry_positions)) return QSA_ERR_NULL;
  if (!aligned(weight_sums, 4) || !aligned(entry_positions, 4) || !aligned(context_lens, 4) ||
      !aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(weight_sums_out, 4) ||
      !aligned(entry_positions_out, 4) || !aligned(error_word, 4))
    return QSA_ERR_ALIGN;
  const Span ws = span(workspace, (int64_t)need);
  const Span outs[6] = {rows_span(kept, R, budget, budget), span(new_lens, R * 4),
                        rows_span(weight_sums_out, R, budget, budget),
                        rows_span(entry_positions_out, R, budget, budget),
                        span(error_word, 4), ws};
  const Span ins[6] = {rows_span(weight_sums, R, entry_cols, weight_sums_stride0),
                       rows_span(entry_positions, R, entry_cols, entry_positions_stride0),
                       span(context_lens, R * 4), cs.tables, cs.k_scale, cs.v_scale};
  if (any_overlap(outs, 6, ins, 6)) return QSA_ERR_ALIAS;
  for (const Span& o : {cs.k, cs.v}) {
    if (any_overlap(&o, 1, ins, 6) || any_overlap(&o, 1, outs, 6)) return QSA_ERR_ALIAS;
  }
  if (!workspace || workspace_bytes < need) return QSA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return QSA_ERR_ALIGN;
  p.sums = weight_sums;
  p.sums_s0 = weight_sums_stride0;
  p.pos = entry_positions;
  p.pos_s0 = entry_positions_stride0;
  p.ctx = context_lens;
  p.cap = entry_cols < p.c.cap ? (int32_t)entry_cols : p.c.cap;
  p.budget = (int32_t)budget;
  p.sink = (int32_t)num_sink;
  p.recent = (int32_t)num_recent;
  p.kept = kept;
  p.new_lens = new_lens;
  p.sums_out = weight_sums_out;
  p.pos_out = entry_positions_out;
  p.moves = static_cast<int32_t*>(workspace);
  p.count = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(workspace) +
                                       round256((size_t)R * budget * 8));
  p.err = error_word;
  bind_calling_thread();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  rank_kernel<<<(unsigned)R, kRankThreads, 0, s>>>(p);
  const int64_t most = std::min<int64_t>(budget, std::max<int64_t>(0, p.cap - budget));
  if (most > 0) {
    const dim3 grid((unsigned)std::min<int64_t>(most, std::max<int64_t>(1, 8192 / R)), (unsigned)R);
    move_kernel<<<grid, kMoveThreads, 0, s>>>(p, (int)(cache->head_dim * dtype_size(cache->dtype)));
  }
  return cudaGetLastError() == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}
