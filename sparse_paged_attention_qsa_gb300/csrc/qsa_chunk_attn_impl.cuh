// qsa_chunk_attn_impl.cuh -- the kernels of the chunk attention
// (include/qsa_chunk.h).
//
// For one K/V head, rows i (a request's tokens by the group's heads) and entries
// e:  s_ie = q_i . k_e,  o_i = sum_e w_ie v_e,  l_i = sum_e w_ie,
// w_ie = 2^(c (s_ie - m_i) + shift); out = o / l.
//
// chunk_plan_kernel  cuts each request's rows into row tiles (and, where there is
//   a prefix, all requests' rows once more) and lays their K/V tiles end to end.
// chunk_walk_kernel  one CTA an SM walks an equal run of them.
//   Three producer warps load the queries and, by way of the page tables, K and V
//   tiles into a ring, all by TMA; one warp issues the products, S = Q K^T with Q
//   and K in shared memory into tensor memory, then O += P V with P in tensor
//   memory: 128 rows a product, two products' S and O beside each other, so that
//   one is in the softmax while the other is in the tensor pipe.  Two warpgroups
//   form the softmax, a thread a row: no reduction crosses threads.  The two hold
//   two halves of 256 rows over the same K/V tiles.  Of 128 rows and fewer they take
//   one row tile each in turn, so that one's output leaves while the other is at work,
//   or (heads of 64, many K/V tiles) every other K/V tile each and merge at the end.
//   (Heads of 256 hold one O of 256 columns: one warpgroup, two S.)  Four more warps
//   widen E4M3 tiles to FP16 on their way to the ring.
// chunk_join_kernel, chunk_join_all_kernel  join the pieces of row tiles that runs
//   cut; with a prefix, the prefix's and the requests' own.
//
// The reference m_i is a product that occurred, the row's maximum when it was
// taken, subtracted before the scaling: logits of any size keep the differences
// that binary32 products have.  It moves only when weights would pass 2^15 (FP16)
// or 1 (BF16, the reference's own 2^-8), and O in tensor memory is rescaled at such
// moves alone.
//
// What bounds it.  Long prompts: shared memory, which Q K^T reads at its whole rate
// (8 KB a product of 128 x 128 x 16, 64 cycles), and the chain softmax (1400 cycles a
// tile), issuing warp, products, of which two row halves hide each other's but in
// part.  4096 tokens behind 4096 others, 16 heads: of 128 150 us, 1.35 PFLOP/s, 0.69 of
// the measured cuBLAS rate; of 256 (2048 behind 8192, 8 heads) 129 us, 1.18 PFLOP/s; of
// 64 118 us, 0.85 PFLOP/s.  A row tile's end (output, next queries, first S) is 5600
// cycles, a sixth of prompts of 2000 tokens.  Single tokens: HBM (64 requests of 8192
// entries, 8 K/V heads of 128: 310 us, 6.9 TB/s); over E4M3 caches the widening and the
// slots that it waits for (257 us, 0.6 of HBM).
//
// Rounding: q, K and V enter the products as they are (E4M3 as FP16, exactly; BF16
// queries of an E4M3 cache as FP16 after a power-of-two scaling of the row, where
// only bits 2^-25 below the row's largest element can be lost), weights rounded to
// the products' type.
#pragma once

#include "qsa_chunk_attn.h"
#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_tcgen05.cuh"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <mutex>

namespace qsa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kChunkJoinThreads = 256;
constexpr int64_t kJoinFew = 1 << 16;   // threads: rows up to here are joined by four times as many
constexpr int kTileFlags = 16;      // tiles whose page masks are kept
constexpr int kSegments = 4;        // segments known ahead

// A weight is at most 2^(shift + slack), the reference's own 2^shift.  FP16 weights
// stay normal down to 2^-22 of the reference's.  BF16 has binary32's exponents, for V
// as well: weights of 1 at most keep the sums of w V within those of |V|.
constexpr float chunk_shift(bool bf16) { return bf16 ? -8.f : 8.f; }
constexpr float chunk_slack(bool bf16) { return bf16 ? 8.f : 7.f; }

__device__ __forceinline__ float cex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t cpack2(float lo, float hi) {
  uint32_t r;
  if constexpr (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// A row's lse: the weights are 2^(mult (s - m) + shift), l their sum.
template <bool kBf16>
__device__ __forceinline__ float row_lse(float m, float l, float mult) {
  return l == 0.f ? -INFINITY : fmaf(m, mult, log2f(l) - chunk_shift(kBf16)) * 0.693147180559945309f;
}
// What the logits of a set of heads are multiplied by, base 2.
__device__ __forceinline__ float set_mult(const ChunkParams& p, int set) {
  return p.scale_log2 * (p.c.k_scale ? p.c.k_scale[set / p.per_kv] : 1.f);
}
// --- geometry ---------------------------------------------------------------------

// The rows of request b, cut to what q holds.
__device__ __forceinline__ void request_rows(const ChunkParams& p, int b, int32_t* t0, int32_t* n) {
  const int32_t s = min(max(p.starts[b], 0), p.tokens);
  *t0 = s;
  *n = min(max(p.starts[b + 1], s), p.tokens) - s;
}

// What the rows of a row tile see: token j of a request sees the entries e below
// hi(j) with e >= lo(j) or e < sink.
struct Sight {
  int32_t base;            // hi(j) = base + j before it is cut to [0, cap]
  int32_t cap, window, sink;
  bool prefix;             // all rows see [0, cap)
  int32_t ns, w0, tiles;   // K/V tiles: ns from 0 on, then from w0 on
  __device__ __forceinline__ int32_t hi(int j) const {
    return prefix ? cap : min(max(base + j, 0), cap);
  }
  __device__ __forceinline__ int32_t lo(int j) const {
    return window > 0 ? (int32_t)min(max((int64_t)base + j - window, (int64_t)0), (int64_t)cap) : 0;
  }
  __device__ __forceinline__ int32_t at(int t) const { return t < ns ? t : t - ns + w0; }
};
__device__ __forceinline__ int32_t prefix_entries(const ChunkParams& p) {
  return p.prefix_table ? min(max(*p.prefix_len, 0), p.prefix_cap) : 0;
}
// Both warpgroups share a row tile of one accumulator.  Heads of 64, whose K/V tiles
// come faster than one warpgroup takes them: 64 requests of 16384 entries, 4 rows a
// K/V head, 328 us (by one 358), E4M3 356 (416), with two buffers of S.  Wider heads wait for K and V, and
// their joint row tile is only begun and ended later: E4M3 heads of 128 with 128 rows a
// K/V head, 8 x 32768 entries, 107 (98).
template <int D>
__device__ __forceinline__ bool splits(bool dual, int tiles) {
  return D == 64 && !dual && tiles >= kChunkSplit;
}
template <int TT>
__device__ __forceinline__ Sight prefix_sight(const ChunkParams& p) {
  Sight s;
  s.cap = prefix_entries(p);
  s.prefix = true;
  s.base = s.window = s.sink = s.ns = s.w0 = 0;
  s.tiles = (s.cap + TT - 1) / TT;
  return s;
}
// of the tokens [j0, j1] of a request with ctx entries, n of them new
template <int TT>
__device__ __forceinline__ Sight request_sight(const ChunkParams& p, int32_t ctx, int32_t n, int j0,
                                               int j1) {
  Sight s;
  s.prefix = false;
  s.base = max(ctx, 0) - n + 1;
  s.cap = p.c.cap;
  s.window = p.window;
  s.sink = p.sink;
  const int32_t hi = s.hi(j1), lo = s.lo(j0);
  const int32_t sink = p.window > 0 ? min(p.sink, hi) : 0;
  s.w0 = lo / TT;
  s.ns = (sink + TT - 1) / TT;
  if (s.ns >= s.w0 && s.ns > 0) s.ns = s.w0 = 0;
  s.tiles = hi > 0 ? s.ns + (hi + TT - 1) / TT - s.w0 : 0;
  return s;
}
// The first row of a CTA's piece: its first segment of a list, or a later one.
__device__ __forceinline__ int64_t piece_at(const ChunkParams& p, int list, int cta, int second) {
  return (int64_t)((list ? 0 : 2 * kChunkMaxCtas) + 2 * cta + second) * p.part_rows;
}
// What a row tile costs beside its K/V tiles (kTileCost each): its queries' way in
// and its output's way out.  (One that sees nothing costs 1 in all.)
__device__ __forceinline__ int32_t extra_cost(const ChunkParams& p, int32_t toks) {
  return toks * p.sub > p.heavy_rows ? p.heavy_extra : kLightExtra;
}

// Not negative; 64-bit divisions take several times as long.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Equal runs of all sets' row tiles, of the prefix's and of the requests' own: a CTA
// walks one of each, so that it does not matter what the one costs beside the other,
// and half of the CTAs begin with either, products and memory side by side.  Where
// the sets divide the CTAs evenly enough every set has the same runs, so that the K/V
// heads of the same entries, whose elements lie side by side, are read at the same
// time.  Where a CTA's two runs would be short, the lists get CTAs of their own.
struct ChunkRuns {
  int64_t total, each, more;    // of one set of heads, or of all
  int n;                        // runs of it
  bool by_head;
};
__device__ __forceinline__ ChunkRuns chunk_runs(const ChunkList& list, int heads) {
  ChunkRuns r;
  const int64_t total = list.total;
  // a row tile in more than kChunkPieces pieces: longer runs, while they are short,
  // cost the walk less than its pieces the join
  // (and no run without a tile's end: kTileCost at least)
  const int least = max(kTileCost, min(kChunkMinRun, list.longest / kChunkPieces + 1));
  const int ctas = (int)max((int64_t)1, min((int64_t)list.ctas, total * heads / least));
  const int per = ctas / heads;
  r.by_head = per > 0 && per * heads * 16 >= ctas * 15;
  r.n = r.by_head ? per : ctas;
  r.total = r.by_head ? total : total * heads;
  r.each = divide(r.total, r.n);
  r.more = r.total - r.each * r.n;
  return r;
}
__device__ __forceinline__ int64_t chunk_run_start(const ChunkRuns& r, int c) {
  return r.each * c + min((int64_t)c, r.more);
}
__device__ __forceinline__ int chunk_run_of(const ChunkRuns& r, int64_t x) {
  const int64_t big = (r.each + 1) * r.more;
  return (int)(x < big ? divide(x, r.each + 1) : r.more + divide(x - big, r.each));
}
// the runs [*c0, *c1] that hold K/V tiles of row tile k of a head, and where it begins
__device__ __forceinline__ int64_t chunk_owners(const ChunkParams& p, const ChunkRuns& r,
                                                const ChunkList& list, int head, int k, int* c0, int* c1) {
  const int64_t at = p.pos[list.k0], a = p.pos[k] - at, b = p.pos[k + 1] - at;
  const int64_t base = r.by_head ? 0 : list.total * head;
  // the first tile is the run's that holds its end
  *c0 = chunk_run_of(r, base + (b - a > 1 ? a + extra_cost(p, p.tiles[k].toks) + kTileCost - 1 : a));
  *c1 = chunk_run_of(r, base + b - 1);
  return base + a;
}

// The segments of a CTA: K/V tiles [t0, t1) of a row tile of one set of heads.
struct Segment {
  Sight sight;
  int32_t k, set, t0, t1;
  int32_t req, token, tok0, toks;   // token: the row of q that tok0 counts from
  int32_t which, whole, list;
};
struct Walk {
  int64_t x, x1, total, base;    // position, end; cost of a set; what p.pos[k] is past it
  int32_t k, k0, k1, set, token0, list;
  bool first;
};
// Where this CTA's run of a list begins.
__device__ __forceinline__ Walk walk_start(const ChunkParams& p, const ChunkPlan& plan, int list) {
  Walk w;
  const ChunkList l = plan.list[list];
  w.total = l.total;
  w.k0 = l.k0;
  w.k1 = l.k1;
  w.token0 = plan.token0;
  w.list = list;
  w.first = true;
  w.x = w.x1 = w.base = 0;
  w.k = l.k0;
  w.set = 0;
  if (l.total == 0) return w;
  const ChunkRuns r = chunk_runs(l, p.sets);
  const int cta = (int)blockIdx.x - l.cta0, run = r.by_head ? cta / p.sets : cta;
  if (cta < 0 || run >= r.n) return w;
  w.x = chunk_run_start(r, run);
  w.x1 = chunk_run_start(r, run + 1);
  w.set = r.by_head ? cta % p.sets : (int)divide(w.x, l.total);
  const int64_t base = r.by_head ? 0 : l.total * w.set, at0 = p.pos[l.k0];
  const int64_t at = w.x - base + at0;
  int lo = l.k0, hi = l.k1 - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.pos[mid] <= at) lo = mid; else hi = mid - 1;
  }
  w.k = lo;
  w.base = base - at0;
  return w;
}
// The CTA's two runs, one after the other.
struct Runs2 {
  Walk w;
  int32_t left;                  // lists not begun
};
__device__ __forceinline__ Runs2 walk_begin() {
  Runs2 r;
  r.w.x = r.w.x1 = 0;
  r.left = 2;
  return r;
}
// The next segment with something to do; false where there is none.
template <int TT>
__device__ __forceinline__ bool walk_next(const ChunkParams& p, Runs2& runs, Segment* s) {
  for (;;) {
    Walk& w = runs.w;
    if (w.x >= w.x1) {
      if (runs.left == 0) return false;
      const ChunkPlan plan = *p.plan;
      // every other run, the same for all sets, begins with the requests' own
      const int order = plan.list[1].cta0 > 0 ? 0 : (blockIdx.x / p.sets) & 1;
      w = walk_start(p, plan, runs.left == 2 ? order : order ^ 1);
      --runs.left;
      continue;
    }
    if (w.k == w.k1) {
      w.k = w.k0;
      ++w.set;
      w.base += w.total;
    }
    const int64_t a = w.base + p.pos[w.k], b = w.base + p.pos[w.k + 1];
    const ChunkTile t = p.tiles[w.k];
    const int64_t end = b < w.x1 ? b : w.x1;
    const int extra = extra_cost(p, t.toks);
    s->k = w.k;
    s->set = w.set;
    s->t0 = t.tiles > 0 ? (int)(max((int64_t)0, w.x - a - extra) >> kTileCostLog2) : 0;
    s->t1 = t.tiles > 0 ? (int)(max((int64_t)0, end - a - extra) >> kTileCostLog2) : 0;
    s->whole = s->t0 == 0 && s->t1 == t.tiles;
    s->which = w.first ? 0 : 1;
    s->list = w.list;
    w.first = false;
    w.x = end;
    ++w.k;
    if (s->t1 <= s->t0 && t.tiles > 0) continue;
    s->req = t.req;
    s->tok0 = t.tok0;
    s->toks = t.toks;
    if (t.req < 0) {
      s->token = w.token0;
      s->sight = prefix_sight<TT>(p);
    } else {
      int32_t n;
      request_rows(p, t.req, &s->token, &n);
      s->sight = request_sight<TT>(p, p.ctx[t.req], n, t.tok0, t.tok0 + t.toks - 1);
    }
    return true;
  }
}

// --- plan -------------------------------------------------------------------------

__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, k);
    if (lane >= k) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t y = warp_sums[lane];
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, k);
      if (lane >= k) y += z;
    }
    warp_sums[lane] = y;
  }
  __syncthreads();
  *all = warp_sums[31];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

// One CTA: row tiles of each request, then the cost of each row tile, both summed
// up.  Row tiles past what the workspace holds (starts that are not in order) are
// left out.
template <int TT, int kAccs>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p, int ctas) {
  __shared__ int64_t s_sums[32];
  __shared__ int32_t s_longest[2];
  __shared__ int64_t s_own;
  __shared__ int32_t s_first[kPlanThreads];  // of up to as many requests
  const int tid = threadIdx.x, R = p.c.num_reqs, RT = kAccs * p.acc_toks;   // tokens of a row tile
  pdl_wait();
  const int32_t token0 = min(max(p.starts[0], 0), p.tokens);
  const int32_t tokens = min(max(p.starts[R], token0), p.tokens) - token0;
  const Sight pre = prefix_sight<TT>(p);
  if (tid == 0 && p.prefix_len && *p.prefix_len > p.prefix_cap) report(p.err, QSA_DERR_CONTEXT);
  const int n_prefix = pre.tiles > 0 ? (tokens + RT - 1) / RT : 0;
  int64_t before = n_prefix, all;
  for (int b0 = 0; b0 < R; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int64_t k = 0;
    if (b < R) {
      int32_t t0, n;
      request_rows(p, b, &t0, &n);
      k = (n + RT - 1) / RT;
      if (n > 0 && p.ctx[b] > p.c.cap) report(p.err, QSA_DERR_CONTEXT);
    }
    const int64_t at = before + block_scan(k, s_sums, &all);
    if (b < R) p.first[b] = s_first[tid] = (int)min(at, (int64_t)p.max_tiles);
    before += all;
  }
  const int n = (int)min(before, (int64_t)p.max_tiles);
  __syncthreads();
  int64_t cost = 0;
  if (tid < 2) s_longest[tid] = 0;
  for (int k0 = 0; k0 < n; k0 += kPlanThreads) {
    const int k = k0 + tid;
    int64_t c = 0;
    if (k < n) {
      ChunkTile t;
      if (k < n_prefix) {
        t.req = -1;
        t.tok0 = k * RT;
        t.toks = min(RT, tokens - t.tok0);
        t.tiles = pre.tiles;
      } else {
        const int32_t* first = R <= kPlanThreads ? s_first : p.first;
        int lo = 0, hi = R - 1;              // the last request that begins at or before k
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (first[mid] <= k) lo = mid; else hi = mid - 1;
        }
        int32_t t0, m;
        request_rows(p, lo, &t0, &m);
        t.req = lo;
        t.tok0 = (k - first[lo]) * RT;
        t.toks = min(RT, m - t.tok0);
        t.tiles = request_sight<TT>(p, p.ctx[lo], m, t.tok0, t.tok0 + t.toks - 1).tiles;
      }
      p.tiles[k] = t;
      c = t.tiles > 0 ? (int64_t)t.tiles * kTileCost + extra_cost(p, t.toks) : 1;
    }
    const int64_t at = cost + block_scan(c, s_sums, &all);
    if (k < n) {
      p.pos[k] = at;
      atomicMax(&s_longest[k >= n_prefix], (int32_t)min(c, (int64_t)INT32_MAX));
      if (k == n_prefix) s_own = at;
    }
    cost += all;
  }
  if (tid == 0 && n_prefix >= n) s_own = cost;
  __syncthreads();
  // CTAs of their own where a CTA's two runs would be short
  const int64_t t0 = s_own, t1 = cost - s_own;
  int shares = ctas, cut = 0;                // CTAs of the first list; of both to the second
  if (t0 > 0 && t1 > 0 && (t0 + t1) * p.sets < (int64_t)ctas * kChunkShare) {
    const int unit = ctas >= 2 * p.sets ? p.sets : 1, units = ctas / unit;
    cut = (int)min(max((units * t0 + (t0 + t1) / 2) / (t0 + t1), (int64_t)1), (int64_t)units - 1);
    cut *= unit;
    shares = cut;
  }
  const ChunkPlan plan{{{t0, 0, min(n_prefix, n), s_longest[0], 0, shares},
                        {t1, min(n_prefix, n), n, s_longest[1], cut, ctas - cut}},
                       token0, tokens};
  if (tid == 0) {
    p.pos[n] = cost;
    *p.plan = plan;
  }
  // with a prefix every row tile is joined: which runs hold it, where that is the
  // same for all sets
  if (p.res_o[0]) {
    __syncthreads();
    for (int x = 0; x < 2; ++x) {
      const ChunkRuns r = chunk_runs(plan.list[x], p.sets);
      for (int k = plan.list[x].k0 + tid; k < plan.list[x].k1; k += kPlanThreads) {
        ChunkOwner o;
        o.c0 = -1;                           // to be found for each set
        if (r.by_head) {
          const int64_t x0 = chunk_owners(p, r, plan.list[x], 0, k, &o.c0, &o.c1);
          o.second = chunk_run_start(r, o.c0) < x0;
        }
        const ChunkTile t = p.tiles[k];
        int32_t begin = token0, m;
        if (t.req >= 0) request_rows(p, t.req, &begin, &m);
        o.token = begin + t.tok0;
        o.toks = t.toks;
        p.owners[k] = o;
      }
    }
  }
  if (tid < kChunkMaxCtas) p.cuts[tid].set = -1;
}

// --- walk -------------------------------------------------------------------------

struct ChunkTables {
  uint64_t full[16], empty[16];            // ring: K's slots, then V's; E4M3: both in turn
  uint64_t in_full[8], in_empty[8];        // E4M3: tiles as they came, K's and V's in turn
  uint64_t s_full[2][3];                   // of a warpgroup's S in each buffer
  uint64_t p_half[3][2], o_done[2], scanned[2];
  uint64_t q_full, q_ready, q_free, pv_done[2], drain;   // products of even and odd steps
  uint64_t seg_full[kSegments], seg_empty[kSegments], pair[4];
  uint32_t boxes[kTileFlags];              // a bit per copy of a tile, 0: it had no page
  uint32_t bad[8][4];                      // entries of a V slot that hold what is not finite
  float ml[128][2];
  float q_mul[2][256];                     // E4M3: what a row's queries were divided by
  Segment seg[kSegments];                  // the next ones; k < 0: no more
  uint32_t tmem;
  int32_t abort;
  int32_t pad[3];
};

template <int D, bool kFp8>
struct ChunkShape {
  static constexpr int TT = chunk_tile(D);
  static constexpr int kGroups = chunk_accs(D);            // softmax warpgroups
  static constexpr int kSoft = kGroups * 128;              // softmax threads
  static constexpr int kConvert = kFp8 ? 128 : 0;          // and those that widen E4M3 tiles
  static constexpr int kThreads = kSoft + kConvert + 128;  // + K's, V's, Q's producer, the issuer
  static constexpr int kBlocks = D / 64;                   // of 64 dims: a line of 128 bytes
  static constexpr int kSlot = TT * D * 2;
  static constexpr int kQTile = 128 * D * 2;
  // Slots: K's and V's of their own, two each (heads of 64 four).  E4M3 tiles come in
  // as they are and are widened into a ring that K and V share: its third slot is
  // filled while the products read two.
  static constexpr int NS = kFp8 ? (D == 64 ? 6 : 3) : (D == 64 ? 4 : 2);
  static constexpr int kIn = TT * D, NI = kFp8 ? (D == 64 ? 8 : 3) : 0;
  // columns of O that a warp's rows leave through shared memory at a time
  static constexpr int kOutCols = kFp8 && D == 128 ? 8 : 16;
  static constexpr int kQ = (kFp8 ? NS : 2 * NS) * kSlot;  // offsets: ring, queries, E4M3, output, tables
  static constexpr int kStaged = kQ + kGroups * kQTile;
  static constexpr int kOut = kStaged + NI * kIn;
  // Rows of a row tile whose ends leave without the stages: those that one warp holds.
  static constexpr int kFew = kGroups == 1 ? 16 : 4 * 32 * kOutCols / D;
  // Where both warpgroups share a row tile of so few, the second's columns of them, in
  // bytes of their own: the stages of its other warps, which hold none of the rows, may
  // be in use for its next row tile by the time that the first warpgroup reads.
  static constexpr int kHand = kOut + kGroups * 4 * 32 * kOutCols * 4;
  static constexpr int kTables = kHand + (D == 64 ? kFew * D * 4 : 0);
  static constexpr size_t kSmem = 1024 + kTables + sizeof(ChunkTables);
  // Tensor memory columns.  S in turn in kBufs buffers: two, a warpgroup's own where it
  // has half of the rows.  Heads of 64 leave room for a third: a warpgroup finds its
  // next S formed while it was in the softmax, where two buffers make it wait for the
  // product with its weights first (one prompt of 32768 tokens, window 4096, 16 heads:
  // 582 us for 647; heads of 256, one warpgroup on all rows, gain nothing, 130 for 129 in
  // 2048 behind 8192).  Weights take the place of half of their S (heads of
  // 256: beside it).
  static constexpr int kBufs = D == 64 ? 3 : 2;
  static constexpr int kS = TT, kP = D == 256 ? 2 * TT : 64, kPs = D == 256 ? TT / 2 : kS;
  static constexpr int kO = D == 64 ? 384 : 256;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kHand >= kOut + kSoft / 32 * (32 * kOutCols * 4), "apart from every warp's stage");
  // Registers: 384 threads of 168 at launch, dealt out as 208, 208 and 88 a thread
  // of a warpgroup; over an E4M3 cache 512 of 128 as 192, 192, 64, 64.  A row of S
  // stays in registers whole.  (The compiler allots by the launch's share: over an
  // E4M3 cache 40 to 64 bytes a thread lie on the stack, elsewhere none.)
  static constexpr int kRegs = kGroups == 1 ? 0 : kFp8 ? 128 : 168;
  static constexpr int kMore = kFp8 ? 192 : 208, kFewer = kFp8 ? 64 : 88;
  static_assert(2 * kMore + (kThreads / 128 - 2) * kFewer <= kThreads / 128 * kRegs || kGroups == 1,
                "no more registers than the launch has");
  static __device__ __forceinline__ void more_registers() {
    if constexpr (kGroups == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMore));
  }
  static __device__ __forceinline__ void fewer_registers() {
    if constexpr (kGroups == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewer));
  }
  // the ring's slot of tile f's K (V), and the phase in which it is full
  static __device__ __forceinline__ int slot(int f, int kv) {
    return kFp8 ? (2 * f + kv) % NS : kv * NS + f % NS;
  }
  static __device__ __forceinline__ uint32_t phase(int f, int kv) {
    return (uint32_t)((kFp8 ? (2 * f + kv) / NS : f / NS) & 1);
  }
};

// A slot of the ring and the phase in which it is full, for K or V in turn.
template <int NS, bool kFp8>
struct Ring {
  int slot;                                                // V's of its own: NS on
  uint32_t phase;
  __device__ __forceinline__ void next() {
    if constexpr (kFp8) {
      slot += 2;
      if (slot >= NS) slot -= NS, phase ^= 1;
    } else {
      ++slot;
      if (slot % NS == 0) slot -= NS, phase ^= 1;
    }
  }
};

// Two E4M3 values (the low, the high half of x) as FP16, exactly.
__device__ __forceinline__ uint32_t widen_lo(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
  return r;
}

// Row r of a query tile, BF16, as FP16 in its place: divided by the power of two,
// returned, that brings its largest magnitude to [2^14, 2^15), or by 2^-120 where that
// takes less (1 where the magnitude is not finite).
template <int D>
__device__ __forceinline__ float row_to_fp16(unsigned char* tile, int r) {
  const auto at = [&](int x) {
    return reinterpret_cast<uint4*>(tile + (x >> 3) * (128 * 128) + r * 128 + (((x & 7) ^ (r & 7)) << 4));
  };
  float a = 0.f;
#pragma unroll 4
  for (int x = 0; x < D / 8; ++x) {
    const uint4 v = *at(x);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      a = fmaxf(a, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u))));
  }
  const int e = (int)(__float_as_uint(a) >> 23);
  float mul = 1.f, by = 1.f;
  if (e < 255) {
    const int up = min(14 + 127 - e, 120);
    mul = __uint_as_float((uint32_t)(127 - up) << 23);
    by = __uint_as_float((uint32_t)(127 + up) << 23);
  }
#pragma unroll 4
  for (int x = 0; x < D / 8; ++x) {
    const uint4 v = *at(x);
    const auto half = [&](uint32_t u) {
      return cpack2<false>(__uint_as_float(u << 16) * by, __uint_as_float(u & 0xffff0000u) * by);
    };
    *at(x) = make_uint4(half(v.x), half(v.y), half(v.z), half(v.w));
  }
  return mul;
}

// T: the type of q and out; the products' is T, or FP16 over an E4M3 cache.
template <typename T, int D, bool kFp8>
__global__ void __launch_bounds__((ChunkShape<D, kFp8>::kThreads), 1)
chunk_walk_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using C = ChunkShape<D, kFp8>;
  constexpr bool kOutBf16 = __is_same(T, __nv_bfloat16), kBf16 = kOutBf16 && !kFp8;
  constexpr bool kQToFp16 = kOutBf16 && kFp8;
  constexpr int TT = C::TT, NS = C::NS;
  constexpr int kWords = TT / 32;                          // of 32 columns of S
  extern __shared__ unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  unsigned char* base = smem_raw + pad;
  const uint32_t ring = raw + pad;
  ChunkTables& tb = *reinterpret_cast<ChunkTables*>(base + C::kTables);
  const auto bar = [&](uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };
  volatile int32_t* s_abort = &tb.abort;

  if (tid == 0) {
    for (int i = 0; i < (kFp8 ? NS : 2 * NS); ++i) {
      mbar_init(bar(tb.full[i]), kFp8 ? 4 : 1);
      mbar_init(bar(tb.empty[i]), 1);
    }
    for (int i = 0; i < C::NI; ++i) {
      mbar_init(bar(tb.in_full[i]), 1);
      mbar_init(bar(tb.in_empty[i]), 4);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(bar(tb.pv_done[u]), 1);
      for (int b = 0; b < C::kBufs; ++b) {
        mbar_init(bar(tb.s_full[u][b]), 1);
        mbar_init(bar(tb.p_half[b][u]), 4);
      }
      mbar_init(bar(tb.o_done[u]), 1);
      mbar_init(bar(tb.scanned[u]), 4);
    }
    mbar_init(bar(tb.q_full), 1);
    mbar_init(bar(tb.q_ready), 4);
    mbar_init(bar(tb.q_free), 1);
    mbar_init(bar(tb.drain), 1);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(bar(tb.seg_full[i]), 1);
      mbar_init(bar(tb.seg_empty[i]), (C::kSoft + C::kConvert) / 32 + 3);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar(tb.pair[i]), 2);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  constexpr int kProducer = (C::kSoft + C::kConvert) / 32, kIssuer = kProducer + 2, kQueries = kProducer + 3;
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&tb.tmem)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = tb.tmem;
  pdl_wait();
  pdl_trigger();

  // No wait is without an end, and after a time-out nothing waits any more: roles
  // leave at their next segment.
  const auto wait_for = [&](uint32_t b, uint32_t phase, uint64_t limit = kWaitLimitNs) {
    if (!mbar_try_wait(b, phase) && *s_abort == 0 && !mbar_wait(b, phase, limit)) {
      *s_abort = 1;
      report(p.err, QSA_DERR_TIMEOUT);
    }
  };
  // The n-th segment, as the queries' producer has made it known; null: no more.
  const auto segment = [&](int n) -> const Segment* {
    wait_for(bar(tb.seg_full[n % kSegments]), (uint32_t)((n / kSegments) & 1));
    const Segment* s = &tb.seg[n % kSegments];
    return __any_sync(0xffffffffu, *s_abort != 0) || s->k < 0 ? nullptr : s;
  };
  const auto segment_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(tb.seg_empty[n % kSegments]));
  };
  int issued = 0;                                          // a producer's fills
  bool used = false;                                       // the issuer's products
  int withheld = -1;                                       // test build: a slot fill left out
  if (warp < C::kSoft / 32) {
    C::more_registers();
    // ---------------- softmax ----------------
    const int g = warp >> 2, wl = warp & 3, r = wl * 32 + lane;   // warpgroup; row of 128
    const uint32_t lanes = tmem + ((uint32_t)(wl * 32) << 16);
    const int box_log2 = min(p.c.page_log2, TT == 128 ? 7 : 6);
    const int rj = r / p.sub, rh = r - rj * p.sub;         // the row's token and head in its accumulator
    unsigned char* out_stage = base + C::kOut + warp * (32 * C::kOutCols * 4);
    int fill = 0, units = 0;
    uint32_t pvs[2] = {0, 0};                              // products with weights, of even and odd steps
    uint32_t got = 0;                                      // phases of S, a bit a buffer
    int outs = 0, scans = 0;                               // O taken, V searched so far
    int turn = 0;                                          // whose the next row tile of one O is
    int pairs = 0;                                         // meetings of two warps that hold the same rows
    for (int sn = 0;; ++sn) {
      const Segment* next = segment(sn);
      if (!next) break;
      const Segment& seg = *next;
      const Sight& s = seg.sight;
      const int tiles = seg.t1 - seg.t0;
      const bool dual = seg.toks > p.acc_toks, split = splits<D>(dual, tiles), two = dual || split;
      const bool own = C::kGroups == 1 || two || g == turn;
      // this thread's row, and what all rows see
      const int jt = (dual ? g * p.acc_toks : 0) + rj;     // of the row tile's tokens
      const bool mine = own && rj < p.acc_toks && jt < seg.toks;
      const int j = seg.tok0 + min(jt, seg.toks - 1), jl = seg.tok0 + seg.toks - 1;
      const int32_t hi = s.hi(j), lo = s.lo(j), sink = s.window > 0 ? min(s.sink, hi) : 0;
      const int32_t in_hi = s.hi(seg.tok0), in_lo = s.lo(jl);
      const int32_t in_sink = s.window > 0 ? min(s.sink, in_hi) : 0;
      const int kv_head = seg.set / p.per_kv;
      float mult = kFp8 ? set_mult(p, seg.set) : p.scale_log2, q_mul = 1.f;
      float m = -INFINITY, l = 0.f;
      const int steps = dual ? 2 * tiles : tiles;
      // K/V tile t of the segment: from 0 on up to the sinks' end, then the window's
      const int first_tile = seg.t0, first_gap = s.ns - seg.t0, rest_tile = seg.t0 - s.ns + s.w0;
      const int stride = two ? 2 : 1;
      int u = two ? g : 0;                                 // the buffer of S: st modulo kBufs
      const auto next_buffer = [&]() {
        u += stride;
        if (u >= C::kBufs) u -= C::kBufs;
      };
      for (int st = two ? g : own ? 0 : steps; st < steps; st += stride, next_buffer()) {
        const int t = dual ? st >> 1 : st, f = fill + t;
        const int32_t e0 = (t < first_gap ? t + first_tile : t + rest_tile) * TT;
        wait_for(bar(tb.s_full[g][0]) + u * 8, got >> u & 1);
        got ^= 1u << u;
        tc5_fence_after();
        if constexpr (kQToFp16) {
          if (st < stride) {                               // the row's first
            q_mul = tb.q_mul[units & 1][(dual ? g * 128 : 0) + r];
            // where it leaves binary32's normal numbers, logits are either the same to
            // 2^-90 or apart by 2^90: its ends do as well, and keep infinities from zeros
            mult = fminf(fmaxf(mult * q_mul, FLT_MIN), FLT_MAX);
          }
        }
        const uint32_t boxes = tb.boxes[f % kTileFlags];
        const bool edge = e0 + TT > in_hi || (e0 < in_lo && e0 + TT > in_sink) ||
                          boxes != (1u << (TT >> box_log2)) - 1;
        const uint32_t zs = lanes + u * C::kS;
        uint32_t vis[kWords];
        if (edge) {                                        // hidden entries: -inf
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            const int32_t b = e0 + w * 32;
            const auto upto = [&](int32_t x) -> uint32_t {   // entries below x
              const int32_t n = min(max(x - b, 0), 32);
              return n == 32 ? 0xffffffffu : (1u << n) - 1;
            };
            uint32_t there = 0;
            if (box_log2 >= 5) {
              there = (boxes >> ((w * 32) >> box_log2)) & 1u ? 0xffffffffu : 0u;
            } else {
              const uint32_t one = (1u << (1 << box_log2)) - 1;
              for (int x = 0; x < 32 >> box_log2; ++x)
                if ((boxes >> (((w * 32) >> box_log2) + x)) & 1u) there |= one << (x << box_log2);
            }
            vis[w] = ((upto(hi) & ~upto(lo)) | upto(sink)) & there;
            uint32_t x[32];
            tc5_ld32(zs + w * 32, x);
            tc5_wait_ld();
            tc5_hold(x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((vis[w] >> i) & 1u)) x[i] = 0xff800000u;
            tc5_st(zs + w * 32, x);
          }
          tc5_wait_st();
        } else {
#pragma unroll
          for (int w = 0; w < kWords; ++w) vis[w] = 0xffffffffu;
        }
        uint32_t z[kWords][32];
        float mx[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w) tc5_ld32_max(zs + w * 32, z[w], mx[w]);
        tc5_wait_ld();
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          tc5_hold(z[w]);
          tc5_hold(mx[w]);
        }
        float top = fmaxf(mx[0], mx[1]);
        if constexpr (TT == 128) top = max3(top, mx[2], mx[3]);
        const float old = m;
        const bool move = (top - m) * mult > chunk_slack(kBf16);
        if (move) m = top;
        if (__any_sync(0xffffffffu, move)) {
          const float a = !move ? 1.f : old == -INFINITY ? 0.f : cex2((old - m) * mult);
          l *= a;
          if (st >= stride) {
            // the product before this one into the same O: done where S of this step
            // came behind it, else to be waited for (the one before that is done, so
            // that its phase is not taken for this one's)
            const int last = st - stride;
            if (C::kBufs > stride)
              wait_for(bar(tb.pv_done[last & 1]), ((last & 1 ? pvs[1] : pvs[0]) + (last >> 1)) & 1);
            tc5_fence_after();
            const uint32_t o = lanes + C::kO + g * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t x[32];
              tc5_ld32(o + c, x);
              tc5_wait_ld();
              tc5_hold(x);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * a);
              tc5_st(o + c, x);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 mult2 = make_float2(mult, mult), ref2 = make_float2(-ref, -ref);
        const float2 shift2 = make_float2(chunk_shift(kBf16), chunk_shift(kBf16));
        const uint32_t pa = lanes + C::kP + u * C::kPs;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const auto weights = [&](int w, uint32_t(&x)[32]) {
          uint32_t h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 y = ffma2(
                fadd2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), ref2), mult2,
                shift2);
            const float2 e = make_float2(cex2(y.x), cex2(y.y));
            sum[i & 1] = fadd2(sum[i & 1], e);
            h[i] = cpack2<kBf16>(e.x, e.y);
          }
          tc5_st(pa + w * 16, h);
        };
        const auto ready = [&](int half) {                 // the half's product may begin
          tc5_wait_st();
          tc5_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(tb.p_half[0][half]) + u * 16);
        };
#pragma unroll
        for (int w = 0; w < kWords / 2; ++w) weights(w, z[w]);
        // V is there too before its first product is asked for
        if (wl == 0) wait_for(bar(tb.full[C::slot(f, 1)]), C::phase(f, 1));
        if (!edge) ready(0);
#pragma unroll
        for (int w = kWords / 2; w < kWords; ++w) weights(w, z[w]);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (edge) {
          // 0 times what a hidden entry holds may be NaN: whatever is not finite in
          // V leaves the tile, and rows that see it get NaN
          const int slot = C::slot(f, 1), i = kFp8 ? slot : slot - NS;
          wait_for(bar(tb.full[slot]), C::phase(f, 1));
          constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u;
          constexpr uint32_t kUp = kBf16 ? 0x00800080u : 0x04000400u;
          uint4* v = reinterpret_cast<uint4*>(base + slot * C::kSlot);
          for (int x = r; x < C::kSlot / 16; x += 128) {
            const uint4 y = v[x];
            const uint32_t e = ((y.x & kExp) + kUp) | ((y.y & kExp) + kUp) | ((y.z & kExp) + kUp) |
                               ((y.w & kExp) + kUp);
            if (e & 0x80008000u) {
              const int token = x >> 3 & (TT - 1);         // lines of 8 pieces, blocks of TT lines
              atomicOr(&tb.bad[i][token >> 5], 1u << (token & 31));
              __threadfence_block();
              v[x] = make_uint4(0, 0, 0, 0);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          // (an mbarrier: which tiles are edges is not sure to be the same in all warps
          // after a time-out, and waits on it end)
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(tb.scanned[g]));
          wait_for(bar(tb.scanned[g]), (uint32_t)(scans & 1));
          ++scans;
#pragma unroll
          for (int w = 0; w < kWords; ++w)
            if (vis[w] & *reinterpret_cast<volatile uint32_t*>(&tb.bad[i][w])) l = NAN;
          ready(0);
        }
        ready(1);
      }
      if (C::kBufs == 3 || !two) {
        pvs[0] += (steps + 1) >> 1;
        pvs[1] += steps >> 1;
      }
      fill += tiles;
      if (tiles > 0) ++units;
      if (!two) turn ^= 1;
      // ---- the row tile's end
      if (own && steps > 0) {
        wait_for(bar(tb.o_done[g]), (uint32_t)(outs & 1));
        ++outs;
        tc5_fence_after();
      }
      if (__any_sync(0xffffffffu, mine)) {                 // the same in both warps of a pair
        // rows go out by way of shared memory, kOutCols columns at a time, so that
        // stores are whole sectors; of a pair of warps that hold the same rows the
        // second hands its columns to the first
        const auto pair_sync = [&]() {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(tb.pair[wl]));
          wait_for(bar(tb.pair[wl]), (uint32_t)(pairs & 1));
          ++pairs;
        };
        float f0 = 1.f, f1 = 0.f;
        if (split) {
          if (g == 1) {
            tb.ml[r][0] = m;
            tb.ml[r][1] = l;
          }
          pair_sync();
          if (g == 0) {
            const float m1 = tb.ml[r][0], l1 = tb.ml[r][1], M = fmaxf(m, m1);
            f0 = m == -INFINITY ? 0.f : cex2((m - M) * mult);
            f1 = m1 == -INFINITY ? 0.f : cex2((m1 - M) * mult);
            l = l * f0 + l1 * f1;
            m = M;
          }
        }
        const bool first = g == 0 || !split;               // writes
        const bool few = !dual && seg.toks * p.sub <= C::kFew;
        const bool direct = seg.whole && !p.res_o[0];
        const int64_t token = seg.token + seg.tok0 + jt;
        const int head = seg.set * p.sub + rh;
        const int64_t at = token * p.heads + head;
        const int64_t piece = piece_at(p, seg.list, blockIdx.x, seg.which) + (dual ? g * 128 : 0) + r;
        uint64_t dst = 0;                                  // the row's first element
        float inv = 1.f;
        if (mine && first) {
          if (direct) {
            dst = reinterpret_cast<uint64_t>(p.out + token * p.out_row + head * p.out_head);
            inv = l == 0.f ? 0.f : (kFp8 && p.c.v_scale ? p.c.v_scale[kv_head] : 1.f) / l;
            if (p.lse) p.lse[at] = row_lse<kBf16>(m * q_mul, l, kFp8 ? set_mult(p, seg.set) : mult);
          } else {
            dst = reinterpret_cast<uint64_t>(seg.whole ? p.res_o[seg.list] + at * D : p.part_o + piece * D);
            *reinterpret_cast<float2*>(seg.whole ? p.res_ml[seg.list] + at * 2 : p.part_ml + piece * 2) =
                make_float2(m * q_mul, l);                 // as the products of q itself
          }
        }
        if (inv != 1.f) f0 *= inv, f1 *= inv;
        constexpr int kQuads = C::kOutCols / 4;            // 16-byte pieces of a staged row
        uint4* stage = reinterpret_cast<uint4*>(out_stage);
        const auto place = [&](int row, int q) {           // eight rows' pieces on all banks
          return row * kQuads + (kQuads == 4 ? q ^ ((row >> 1) & 3) : q ^ ((row >> 2) & 1));
        };
        const uint4* other = stage + 4 * 32 * kQuads;      // the second warpgroup's
        // Few rows (one warp's): the second warpgroup's go over at once.  The first one
        // has read the last ones when it comes to this row tile's first meeting.
        uint4* whole = reinterpret_cast<uint4*>(base + C::kHand);
        const auto spot = [&](int q) { return lane * (D / 4) + (q ^ (lane & 7)); };
        if (few && split && g == 0) pair_sync();
        uint64_t to[kQuads];                               // the rows that this lane stores pieces of
#pragma unroll
        for (int k = 0; k < kQuads; ++k)
          to[k] = __shfl_sync(0xffffffffu, dst, k * (32 / kQuads) + lane / kQuads);
        const auto store = [&](uint64_t offset) {          // the staged rows, `offset` bytes into them
          __syncwarp();
          uint4 v[kQuads];
#pragma unroll
          for (int k = 0; k < kQuads; ++k)
            v[k] = stage[place(k * (32 / kQuads) + lane / kQuads, lane % kQuads)];
#pragma unroll
          for (int k = 0; k < kQuads; ++k)
            if (to[k]) *reinterpret_cast<uint4*>(to[k] + offset + lane % kQuads * 16) = v[k];
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t x[32];
          if (tiles > 0) {
            tc5_ld32(lanes + C::kO + g * D + c, x);
            tc5_wait_ld();
            tc5_hold(x);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0;
          }
          const auto f = [&](int i) { return __uint_as_float(x[i]); };
          if (!first && few) {
            if (mine) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                whole[spot(c / 4 + q)] = make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            }
            if (c + 32 == D) pair_sync();
            continue;
          }
          if (!first) {
#pragma unroll
            for (int h = 0; h < 32; h += C::kOutCols) {
#pragma unroll
              for (int q = 0; q < kQuads; ++q)
                stage[place(lane, q)] =
                    make_uint4(x[h + 4 * q], x[h + 4 * q + 1], x[h + 4 * q + 2], x[h + 4 * q + 3]);
              pair_sync();                                 // there
              pair_sync();                                 // taken
            }
            continue;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(f(i) * f0);
          if (split && few) {
            if (mine) {
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const uint4 y = whole[spot(c / 4 + q)];
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  x[4 * q + i] = __float_as_uint(fmaf(__uint_as_float(w[i]), f1, f(4 * q + i)));
              }
            }
          } else if (split) {
#pragma unroll
            for (int h = 0; h < 32; h += C::kOutCols) {
              pair_sync();
#pragma unroll
              for (int q = 0; q < kQuads; ++q) {
                const uint4 y = other[place(lane, q)];
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  x[h + 4 * q + i] = __float_as_uint(fmaf(__uint_as_float(w[i]), f1, f(h + 4 * q + i)));
              }
              pair_sync();
            }
          }
          if (few) {
            if (dst && direct) {
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4*>(dst + (uint64_t)(c + i) * 2) =
                    make_uint4(cpack2<kOutBf16>(f(i), f(i + 1)), cpack2<kOutBf16>(f(i + 2), f(i + 3)),
                               cpack2<kOutBf16>(f(i + 4), f(i + 5)), cpack2<kOutBf16>(f(i + 6), f(i + 7)));
            } else if (dst) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4*>(dst + (uint64_t)(c + i) * 4) =
                    make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
          } else if (direct) {
#pragma unroll
            for (int h = 0; h < 32; h += 2 * C::kOutCols) {
#pragma unroll
              for (int q = 0; q < kQuads; ++q) {
                const int i = h + 8 * q;
                stage[place(lane, q)] =
                    make_uint4(cpack2<kOutBf16>(f(i), f(i + 1)), cpack2<kOutBf16>(f(i + 2), f(i + 3)),
                               cpack2<kOutBf16>(f(i + 4), f(i + 5)), cpack2<kOutBf16>(f(i + 6), f(i + 7)));
              }
              store((uint64_t)(c + h) * 2);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 32; h += C::kOutCols) {
#pragma unroll
              for (int q = 0; q < kQuads; ++q)
                stage[place(lane, q)] =
                    make_uint4(x[h + 4 * q], x[h + 4 * q + 1], x[h + 4 * q + 2], x[h + 4 * q + 3]);
              store((uint64_t)(c + h) * 4);
            }
          }
        }
        // a run's first row tile, where it is not its beginning: for the join
        if (!p.res_o[0] && seg.which == 0 && seg.t0 > 0 && r == 0 && (g == 0 || !two)) {
          const ChunkPlan plan = *p.plan;
          const ChunkRuns runs = chunk_runs(plan.list[1], p.sets);
          ChunkCut cut;
          const int64_t x0 = chunk_owners(p, runs, plan.list[1], seg.set, seg.k, &cut.c0, &cut.c1);
          if ((int)(runs.by_head ? blockIdx.x / p.sets : blockIdx.x) == cut.c0 + 1) {
            cut.set = seg.set;
            cut.second = chunk_run_start(runs, cut.c0) < x0;
            cut.by_head = runs.by_head;
            cut.token = seg.token + seg.tok0;
            cut.toks = seg.toks;
            p.cuts[blockIdx.x] = cut;
          }
        }
      }
      tc5_fence_before();
      segment_done(sn);
    }
  } else {
    C::fewer_registers();
    if (warp == kProducer || warp == kProducer + 1) {
      // ---------------- producers of K and V ----------------
      const int kv = warp - kProducer;
      const int lg = p.c.page_log2;
      const int box_rows = min(TT, 1 << lg), n_boxes = TT / box_rows;
      const uint64_t policy = evict_normal_policy();
      bool stop = false;
      for (int sn = 0; !stop; ++sn) {
        const Segment* next = segment(sn);
        if (!next) break;
        const Segment& seg = *next;
        const Sight& s = seg.sight;
        const int32_t* table = s.prefix ? p.prefix_table : p.c.bt + (int64_t)seg.req * p.c.bt_s0;
        const int kv_head = seg.set / p.per_kv;
        // the entries that some row sees: [0, sink) and [lo, end)
        const int32_t end = s.hi(seg.tok0 + seg.toks - 1), lo = s.lo(seg.tok0);
        const int32_t sink = s.window > 0 ? min(s.sink, end) : 0;
        int col0 = -64;                                    // 32 page ids from this column on
        int32_t ids = -1;
        for (int t = seg.t0; t < seg.t1; ++t) {
          const int32_t e0 = s.at(t) * TT;
          const int col = e0 >> lg, cols = max(1, TT >> lg);
          if (col < col0 || col + cols > col0 + 32) {
            col0 = col;
            // the columns of entries below `end` are inside the table
            ids = ((int64_t)(col + lane) << lg) < end ? __ldg(table + col + lane) : -1;
          }
          const int32_t id =
              __shfl_sync(0xffffffffu, ids, col - col0 + (lane < n_boxes ? (lane * box_rows) >> lg : 0));
          const int32_t be = e0 + lane * box_rows;
          const bool want = lane < n_boxes && be < end && (be + box_rows > lo || be < sink);
          const bool good = want && id >= 0 && id < p.c.num_pages;
          const uint32_t mask = __ballot_sync(0xffffffffu, good);
          if (__any_sync(0xffffffffu, want && !good) && lane == 0) report(p.err, QSA_DERR_KV_PAGE);
          // the slot that this fill takes: of the ring, or of the tiles as they come
          const int n = kFp8 ? 2 * issued + kv : issued;
          const int slot = kFp8 ? n % C::NI : C::slot(issued, kv), fills = kFp8 ? n / C::NI : issued / NS;
          const uint32_t full = kFp8 ? bar(tb.in_full[slot]) : bar(tb.full[slot]);
          const uint32_t empty = kFp8 ? bar(tb.in_empty[slot]) : bar(tb.empty[slot]);
          if (fills > 0) {
            bool ok = *s_abort == 0 && mbar_wait(empty, (uint32_t)((fills - 1) & 1));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
              if (lane == 0 && *s_abort == 0) {
                *s_abort = 1;
                report(p.err, QSA_DERR_TIMEOUT);
              }
              stop = true;
              break;
            }
          }
          if (kv == 0) {
            if (lane == 0) tb.boxes[issued % kTileFlags] = mask;
          } else if (!kFp8 && lane < 4) {
            tb.bad[slot - NS][lane] = 0;
          }
          __syncwarp();
#ifdef QSA_WAIT_TEST
          // test build: leave this fill without a copy, so that the waits on it run out
          // (the failure-detection test)
          const bool withhold = blockIdx.x == 0 && 2 * issued + kv == p.test_withhold;
          if (withhold) withheld = issued;
          if (!withhold)
#endif
          {
            if (lane == 0) mbar_expect_tx(full, (uint32_t)(__popc(mask) * box_rows * D * (kFp8 ? 1 : 2)));
            __syncwarp();
            if (good) {
              constexpr int kLine = kFp8 && D == 64 ? 64 : 128, kLines = D * (kFp8 ? 1 : 2) / kLine;
              const uint32_t dst = ring + (kFp8 ? C::kStaged + slot * C::kIn : slot * C::kSlot);
#pragma unroll
              for (int c = 0; c < kLines; ++c)
                tma_load_4d(dst + c * (TT * kLine) + lane * box_rows * kLine, kv ? &vmap : &kmap,
                            c * (kFp8 ? kLine : 64), kv_head, be & ((1 << lg) - 1), id, full, policy);
            }
          }
          ++issued;
        }
        segment_done(sn);
      }
    } else if (warp == kQueries) {
      // ---------------- producer of the segments and the queries ----------------
      // waits here are for row tiles of any length: 20 us a K/V tile more
      Runs2 runs = walk_begin();
      int64_t recent = 0;                                  // K/V tiles of the last segments
      for (int sn = 0;; ++sn) {
        Segment seg;
        seg.t0 = seg.t1 = 0;
        const bool more = walk_next<TT>(p, runs, &seg);
        if (!more) seg.k = -1;
        if (sn >= kSegments)
          wait_for(bar(tb.seg_empty[sn % kSegments]), (uint32_t)((sn / kSegments - 1) & 1),
                   kWaitLimitNs + (uint64_t)recent * 20000);
        if (__any_sync(0xffffffffu, *s_abort != 0)) break;
        if (lane == 0) {
          tb.seg[sn % kSegments] = seg;
          mbar_arrive(bar(tb.seg_full[sn % kSegments]));
        }
        __syncwarp();
        if (!more) break;
        if (seg.t1 <= seg.t0) continue;
        if (issued > 0)
          wait_for(bar(tb.q_free), (uint32_t)((issued - 1) & 1), kWaitLimitNs + (uint64_t)recent * 20000);
        recent = (recent * 7 >> 3) + (seg.t1 - seg.t0);
        if (__any_sync(0xffffffffu, *s_abort != 0)) break;
        if (lane == 0) {
          // a line of 64 dims for each head of the set and each token
          const int accs = seg.toks > p.acc_toks ? 2 : 1;
          mbar_expect_tx(bar(tb.q_full), (uint32_t)(accs * p.sub * p.acc_toks * D * 2));
          for (int u = 0; u < accs; ++u)
            for (int c = 0; c < C::kBlocks; ++c)
              tma_load_3d(ring + C::kQ + u * C::kQTile + c * (128 * 128), &qmap, c * 64, seg.set * p.sub,
                          seg.token + seg.tok0 + u * p.acc_toks, bar(tb.q_full));
        }
        __syncwarp();
        ++issued;
      }
    } else if (warp == kIssuer) {
      // ---------------- issuer ----------------
      constexpr uint32_t kQk = tc5_idesc(kBf16, 128, TT, false), kPv = tc5_idesc(kBf16, 128, D, true);
      const uint64_t q0 = tc5_desc(ring + C::kQ, 16), k0 = tc5_desc(ring, 16), v0 = tc5_desc(ring, TT * 128);
      const bool leader = tc5_elect();
      Ring<NS, kFp8> ks{0, 0}, vs{kFp8 ? 1 : NS, 0};       // the next K's and V's slot
      uint32_t ready[2] = {0, 0};                          // phases of P (of three buffers a bit each)
      int units = 0, turn = 0;                             // row tiles; whose the next of one O is
      for (int sn = 0;; ++sn) {
        const Segment* next = segment(sn);
        if (!next) break;
        // the same in every lane, and said so
        const int tiles = __shfl_sync(0xffffffffu, next->t1 - next->t0, 0);
        const bool dual = __shfl_sync(0xffffffffu, next->toks, 0) > p.acc_toks;
        const bool two = dual || splits<D>(dual, tiles);
        segment_done(sn);
        if (tiles <= 0) {
          if (!two) turn ^= 1;
          continue;
        }
        const int steps = dual ? 2 * tiles : tiles;
        wait_for(kQToFp16 ? bar(tb.q_ready) : bar(tb.q_full), (uint32_t)(units & 1));
        ++units;
        // Few instructions: this warp's own time is on the way of every product.  Which
        // buffer and which mode are constants in each use, slots go round by adding
        // (4096 tokens behind 4096 others, 16 heads of 128: 169 -> 150 us).
        const auto run = [&](auto dual_) {
          constexpr bool kDual = decltype(dual_)::value;
          const int which = C::kGroups == 1 ? 0 : turn;    // of !two: whose row tile it is
          // S of step s; its buffer (with two a constant), and whose it is
          const auto qk = [&](int s, int turn_b, auto u_, bool there) {
            constexpr int u = decltype(u_)::value;
            const int b = C::kBufs == 2 ? u : turn_b;
            if (!there) wait_for(bar(tb.full[0]) + ks.slot * 8, ks.phase);
            tc5_fence_after();
            // 16 dims a product: 32 bytes on in a line of 64, then the next block of lines
            const uint64_t q = q0 + (kDual ? u * (C::kQTile >> 4) : 0), k = k0 + ks.slot * (C::kSlot >> 4);
            if (leader) {
#pragma unroll
              for (int x = 0; x < D / 16; ++x)
                tc5_mma_ss(tmem + b * C::kS, q + (x >> 2) * (128 * 128 / 16) + (x & 3) * 2,
                           k + (x >> 2) * (TT * 128 / 16) + (x & 3) * 2, kQk, x > 0);
              tc5_commit(bar(tb.s_full[0][0]) + b * 8 + (kDual || two ? u : which) * 24);
              if (!kDual || u == 1) tc5_commit(bar(tb.empty[0]) + ks.slot * 8);
              if (s + 1 == steps) tc5_commit(bar(tb.q_free));
            }
            __syncwarp();
            if (!kDual || u == 1) ks.next();
            used = true;
          };
          // (after a time-out without waits, on whatever the buffers hold)
          const auto step = [&](int s, int turn_b, auto u_) {
            constexpr int u = decltype(u_)::value, un = (u + C::kBufs) & 1;
            const int b = C::kBufs == 2 ? u : turn_b;
            // what is there already costs no wait behind the softmax's
            const bool k_there =
                (kDual && un == 1) || mbar_test_wait(bar(tb.full[0]) + ks.slot * 8, ks.phase);
            const uint64_t v = v0 + vs.slot * (C::kSlot >> 4);
            const uint32_t o = tmem + C::kO + (kDual || two ? u * D : which * D);
            const uint32_t pa = tmem + C::kP + b * C::kPs;
            const auto phase = [&]() { return C::kBufs == 2 ? ready[u] : ready[0] >> b & 1; };
            const bool add = s > (kDual || two ? 1 : 0);
            const auto half = [&](int h) {
#pragma unroll
              for (int y = 0; y < TT / 32; ++y) {
                const int x = h * (TT / 32) + y;
                tc5_mma_ts(o, pa + x * 8, v + x * (16 * 128 / 16), kPv, add || x > 0);
              }
            };
            wait_for(bar(tb.p_half[b][0]), phase());
            tc5_fence_after();
            if (leader) half(0);
            __syncwarp();
            wait_for(bar(tb.p_half[b][1]), phase());
            if constexpr (C::kBufs == 2) ready[u] ^= 1;
            else ready[0] ^= 1u << b;
            tc5_fence_after();
            if (leader) {
              half(1);
              if (!kDual || u == 1) tc5_commit(bar(tb.empty[0]) + vs.slot * 8);
              if (C::kBufs == 3 || (!kDual && !two)) tc5_commit(bar(tb.pv_done[u]));
              if (s + (kDual || two ? 2 : 1) >= steps)
                tc5_commit(bar(tb.o_done[0]) + (kDual || two ? u : which) * 8);
            }
            __syncwarp();
            if (!kDual || u == 1) vs.next();
            if (s + C::kBufs < steps)
              qk(s + C::kBufs, b, std::integral_constant<int, un>(), __all_sync(0xffffffffu, k_there));
          };
          using Zero = std::integral_constant<int, 0>;
          using One = std::integral_constant<int, 1>;
          qk(0, 0, Zero(), false);
          if (kDual || steps > 1) qk(1, 1, One(), kDual);
          if (C::kBufs == 3 && steps > 2) qk(2, 2, Zero(), false);
          if constexpr (C::kBufs == 2) {
            for (int s = 0; s < steps; s += 2) {
              step(s, 0, Zero());
              if (kDual || s + 1 < steps) step(s + 1, 1, One());
            }
          } else {
            int b = 0;
            for (int s = 0; s < steps; s += 2) {
              step(s, b, Zero());
              b = b == 2 ? 0 : b + 1;
              if (kDual || s + 1 < steps) step(s + 1, b, One());
              b = b == 2 ? 0 : b + 1;
            }
          }
        };
        if (C::kGroups == 2 && dual) run(std::bool_constant<C::kGroups == 2>());
        else run(std::false_type());
        if (!two) turn ^= 1;
      }
    } else if constexpr (kFp8) {
      // ---------------- E4M3 tiles to FP16 ----------------
      const int ct = tid - C::kSoft;
      int n = 0, units = 0;                                // K's and V's tiles in turn
      for (int sn = 0;; ++sn) {
        const Segment* next = segment(sn);
        if (!next) break;
        const Segment& seg = *next;
        if (kQToFp16 && seg.t1 > seg.t0) {
          wait_for(bar(tb.q_full), (uint32_t)(units & 1));
          for (int u = 0; u < (seg.toks > p.acc_toks ? 2 : 1); ++u)
            if (ct < p.sub * p.acc_toks)
              tb.q_mul[units & 1][u * 128 + ct] = row_to_fp16<D>(base + C::kQ + u * C::kQTile, ct);
          ++units;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(tb.q_ready));
        }
        for (int end = n + 2 * (seg.t1 - seg.t0); n < end; ++n) {
          const int in = n % C::NI, out = n % NS;
          wait_for(bar(tb.in_full[in]), (uint32_t)((n / C::NI) & 1));
          if (n >= NS) wait_for(bar(tb.empty[out]), (uint32_t)((n / NS - 1) & 1));
          if ((n & 1) && ct < 4) tb.bad[out][ct] = 0;
          // 16 values a thread and step, 8 and 8: of a line, pieces of a line of FP16.
          // Lanes that would meet in a bank take their halves in the other order.
          constexpr int kLine = D == 64 ? 64 : 128, kPieces = D / 16;
          constexpr int kSteps = TT * kPieces / 128, kRows = 128 / kPieces;
          static_assert(kRows % 8 == 0, "the same place in each line");
          const int row = ct / kPieces, x = ct % kPieces;  // dims [16 x, 16 x + 16)
          const int sw = D == 64 ? (row >> 1) & 3 : row & 7, y = 2 * (x & 3);
          const int turned = (D == 64 ? row >> 1 : D == 128 ? x >> 2 ^ row : x >> 2 ^ x >> 3) & 1;
          const unsigned char* src = base + C::kStaged + in * C::kIn + (x * 16 / kLine) * (TT * kLine) +
                                     row * kLine + (((x % (kLine / 16)) ^ sw) << 4);
          unsigned char* line = base + out * C::kSlot + (x >> 2) * (TT * 128) + row * 128;
          unsigned char* dst[2] = {line + (((y + turned) ^ (row & 7)) << 4),
                                   line + (((y + 1 - turned) ^ (row & 7)) << 4)};
          uint2 v[kSteps][2];
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              v[i][h] = *reinterpret_cast<const uint2*>(src + i * (kRows * kLine) + (h ^ turned) * 8);
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<uint4*>(dst[h] + i * (kRows * 128)) =
                  make_uint4(widen_lo(v[i][h].x), widen_hi(v[i][h].x), widen_lo(v[i][h].y),
                             widen_hi(v[i][h].y));
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(tb.full[out]));
            mbar_arrive(bar(tb.in_empty[in]));
          }
        }
        segment_done(sn);
      }
    }
  }
  __syncthreads();
  // after a time-out, what this CTA issued lands before it exits
  if (*s_abort != 0) {
    if ((warp == kProducer || warp == kProducer + 1) && lane == 0) {
      const int kv = warp - kProducer;
      for (int i = max(0, issued - 8); i < issued; ++i) {
        const int n = kFp8 ? 2 * i + kv : i, slots = kFp8 ? C::NI : NS;
        const int last = kFp8 ? 2 * issued - 2 + kv : issued - 1;
        if (n + slots <= last || i == withheld) continue;  // refilled since, or never begun
        mbar_wait(kFp8 ? bar(tb.in_full[n % slots]) : bar(tb.full[C::slot(i, kv)]),
                  (uint32_t)((n / slots) & 1), kDrainLimitNs);
      }
    }
    if (warp == kQueries && lane == 0 && issued > 0)
      mbar_wait(bar(tb.q_full), (uint32_t)((issued - 1) & 1), kDrainLimitNs);
    if (warp == kIssuer && __any_sync(0xffffffffu, used)) {
      if (tc5_elect()) tc5_commit(bar(tb.drain));
      mbar_wait(bar(tb.drain), 0, kDrainLimitNs);
    }
    __syncthreads();
  }
  if (warp == kIssuer) {
    tc5_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

// --- join -------------------------------------------------------------------------

// A row's sums so far, four elements a thread.
struct Acc {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float2 ml, float4 v, float mult) {
    const float mn = fmaxf(m, ml.x);
    const float a = mn == m ? 1.f : cex2((m - mn) * mult);
    const float f = ml.x == -INFINITY ? 0.f : cex2((ml.x - mn) * mult);
    l = l * a + ml.y * f;
    o.x = o.x * a + v.x * f;
    o.y = o.y * a + v.y * f;
    o.z = o.z * a + v.z * f;
    o.w = o.w * a + v.w * f;
    m = mn;
  }
};

// Where row (token j of a row tile, head g of the set) lies among its rows.
__device__ __forceinline__ int tile_row(const ChunkParams& p, int j, int g) {
  return j < p.acc_toks ? j * p.sub + g : 128 + (j - p.acc_toks) * p.sub + g;
}

// Adds what the runs [c0, c1] left of row i of a row tile, in c0 as its second
// segment or its first; of them this thread's: k0, k0 + dk, ...
template <int D>
__device__ __forceinline__ void add_pieces(const ChunkParams& p, int list, int cta0, bool by_head,
                                           int set, int c0, int c1,
                                           int second, int i, int ln, int k0, int dk, float mult, Acc& acc) {
#pragma unroll 4
  for (int c = c0 + k0; c <= c1; c += dk) {
    const int cta = cta0 + (by_head ? c * p.sets + set : c);
    const int64_t at = piece_at(p, list, cta, c == c0 ? second : 0) + i;
    acc.add(*reinterpret_cast<const float2*>(p.part_ml + at * 2),
            *reinterpret_cast<const float4*>(p.part_o + at * D + ln * 4), mult);
  }
}

// kBf16: of out; kBf16W: of the weights, whose shift l holds.
template <bool kBf16, bool kBf16W, int D>
__device__ __forceinline__ void store_row(const ChunkParams& p, int64_t token, int set, int g, int ln,
                                          float mult, const Acc& a) {
  const float inv = a.l == 0.f ? 0.f : (p.c.v_scale ? p.c.v_scale[set / p.per_kv] : 1.f) / a.l;
  const int head = set * p.sub + g;
  *reinterpret_cast<uint2*>(p.out + token * p.out_row + head * p.out_head + ln * 8) =
      make_uint2(cpack2<kBf16>(a.o.x * inv, a.o.y * inv), cpack2<kBf16>(a.o.z * inv, a.o.w * inv));
  if (ln == 0 && p.lse)
    p.lse[token * p.heads + head] = row_lse<kBf16W>(a.m, a.l, mult);
}

// CTA (c, y): rows of the row tile that the start of CTA c's run cuts, if that is
// its first cut.  D/4 threads a row; where it has many pieces, all threads one row.
template <bool kBf16, bool kBf16W, int D>
__global__ void __launch_bounds__(kChunkJoinThreads) chunk_join_kernel(const ChunkParams p) {
  constexpr int L = D / 4, kG = kChunkJoinThreads / L, kFew = 12;
  __shared__ __align__(16) float4 s_o[kChunkJoinThreads];
  __shared__ float2 s_ml[kG];
  const int tid = threadIdx.x, grp = tid / L, ln = tid % L;
  pdl_wait();
  const ChunkCut cut = p.cuts[blockIdx.x];
  if (cut.set < 0) return;
  const bool few = cut.c1 - cut.c0 < kFew;
  const float mult = set_mult(p, cut.set);
  const int rows = cut.toks * p.sub;
  for (int i0 = blockIdx.y * (few ? kG : 1); i0 < rows; i0 += gridDim.y * (few ? kG : 1)) {
    const int i = few ? i0 + grp : i0, j = i / p.sub, g = i - j * p.sub;
    Acc a{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (i < rows)
      add_pieces<D>(p, 1, 0, cut.by_head, cut.set, cut.c0, cut.c1, cut.second, tile_row(p, j, g), ln,
                    few ? 0 : grp, few ? 1 : kG, mult, a);
    if (!few) {
      __syncthreads();
      s_o[tid] = a.o;
      if (ln == 0) s_ml[grp] = make_float2(a.m, a.l);
      __syncthreads();
      if (grp > 0) continue;
      for (int k = 1; k < kG; ++k) a.add(s_ml[k], s_o[k * L + ln], mult);
    }
    if (i < rows) store_row<kBf16, kBf16W, D>(p, cut.token + j, cut.set, g, ln, mult, a);
  }
}

// With a prefix: CTA (row tile of a request, set of heads, some of its rows); D/4
// threads a row, or `ways` times as many, which share its pieces.
template <bool kBf16, bool kBf16W, int D>
__global__ void __launch_bounds__(kChunkJoinThreads) chunk_join_all_kernel(const ChunkParams p, int ways) {
  constexpr int L = D / 4, kG = kChunkJoinThreads / L;
  __shared__ __align__(16) float4 s_o[kChunkJoinThreads];
  __shared__ float2 s_ml[kG];
  const int tid = threadIdx.x, grp = tid / L, ln = tid % L, set = blockIdx.y;
  const int RT = chunk_accs(D) * p.acc_toks;
  pdl_wait();
  const ChunkPlan plan = *p.plan;
  const int k1 = plan.list[1].k0 + blockIdx.x;
  if (k1 >= plan.list[1].k1) return;
  const auto owner = [&](int list, int k) {
    ChunkOwner o = p.owners[k];
    if (o.c0 < 0) {                                        // not the same for all sets
      const ChunkRuns r = chunk_runs(plan.list[list], p.sets);
      const int64_t x0 = chunk_owners(p, r, plan.list[list], set, k, &o.c0, &o.c1);
      o.second = chunk_run_start(r, o.c0) < x0;
      o.c0 |= kBySet;
    }
    return o;
  };
  const ChunkOwner own = owner(1, k1);
  const float mult = set_mult(p, set);
  const int all = own.toks * p.sub;
  const int way = grp % ways, rows = kG / ways;
  for (int i0 = blockIdx.z * rows; i0 < all; i0 += gridDim.z * rows) {
    const int i = i0 + grp / ways, j = i / p.sub, g = i - j * p.sub;
    const int32_t token = own.token + j;
    Acc a{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (i < all) {
      const int64_t rh = (int64_t)token * p.heads + set * p.sub + g;
      for (int list = 0; list < 2; ++list) {
        const int32_t at = token - plan.token0;
        const int k = list ? k1 : at / RT;
        if (!list && (at < 0 || k >= plan.list[0].k1)) continue;
        const ChunkOwner o = list ? own : owner(0, k);
        const int c0 = o.c0 & ~kBySet;
        if (c0 < o.c1)
          add_pieces<D>(p, list, plan.list[list].cta0, !(o.c0 & kBySet), set, c0, o.c1, o.second,
                        tile_row(p, list ? j : at % RT, g), ln, way, ways, mult, a);
        else if (way == 0)
          a.add(*reinterpret_cast<const float2*>(p.res_ml[list] + rh * 2),
                *reinterpret_cast<const float4*>(p.res_o[list] + rh * D + ln * 4), mult);
      }
    }
    if (ways > 1) {
      __syncthreads();
      s_o[tid] = a.o;
      if (ln == 0) s_ml[grp] = make_float2(a.m, a.l);
      __syncthreads();
      if (way == 0)
        for (int k = 1; k < ways; ++k) a.add(s_ml[grp + k], s_o[(grp + k) * L + ln], mult);
    }
    if (i < all && way == 0) store_row<kBf16, kBf16W, D>(p, token, set, g, ln, mult, a);
  }
}

// --- launch -----------------------------------------------------------------------

// The SMs of the current device; the kernel's set-up once per device.
template <typename T, int D, bool kFp8>
cudaError_t chunk_device(int* n_sms) {
  static std::mutex mu;
  static int sms[64];                                      // 0: not set up on that device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (sms[dev] == 0) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // the registers that warpgroups deal out among themselves are those of the launch:
    // with fewer, one would wait for its share without end
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, chunk_walk_kernel<T, D, kFp8>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < ChunkShape<D, kFp8>::kRegs) return cudaErrorInvalidKernelImage;
    e = cudaFuncSetAttribute(chunk_walk_kernel<T, D, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)ChunkShape<D, kFp8>::kSmem);
    if (e != cudaSuccess) return e;
    sms[dev] = std::min(n, kChunkMaxCtas);
  }
  *n_sms = sms[dev];
  return cudaSuccess;
}

template <typename T, int D, bool kFp8>
cudaError_t launch_chunk_typed(const ChunkParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const CUtensorMap& qmap, cudaStream_t st) {
  using C = ChunkShape<D, kFp8>;
  constexpr bool kBf16 = __is_same(T, __nv_bfloat16), kBf16W = kBf16 && !kFp8;
  int ctas = 0;
  cudaError_t e = chunk_device<T, D, kFp8>(&ctas);
  if (e != cudaSuccess) return e;
  e = launch_after(chunk_plan_kernel<C::TT, C::kGroups>, dim3(1), dim3(kPlanThreads), 0, st, p,
                   ctas);
  if (e != cudaSuccess) return e;
  e = launch_after(chunk_walk_kernel<T, D, kFp8>, dim3((unsigned)ctas), dim3(C::kThreads), C::kSmem, st, p,
                   kmap, vmap, qmap);
  if (e != cudaSuccess) return e;
  if (p.res_o[0]) {
    // few rows: four times the threads a row, for the prefix's pieces
    constexpr int kG = kChunkJoinThreads / (D / 4);
    const int ways = (int64_t)p.tokens * p.heads * (D / 4) <= kJoinFew ? std::min(4, kG) : 1;
    const int64_t rows = std::min<int64_t>((int64_t)p.tokens * p.sub / std::min(p.c.num_reqs, p.tokens) + 1,
                                           C::kGroups * 128);
    const int64_t z = std::min<int64_t>((rows * ways + kG - 1) / kG, 32);
    return launch_after(chunk_join_all_kernel<kBf16, kBf16W, D>,
                        dim3((unsigned)p.max_own, (unsigned)p.sets, (unsigned)z),
                        dim3(kChunkJoinThreads), 0, st, p, ways);
  }
  const int64_t rows = std::min<int64_t>((int64_t)p.tokens * p.sub, C::kGroups * 128);
  return launch_after(chunk_join_kernel<kBf16, kBf16W, D>,
                      dim3((unsigned)ctas, (unsigned)std::min<int64_t>(rows, 8)),
                      dim3(kChunkJoinThreads), 0, st, p);
}

template <int D>
cudaError_t launch_chunk(const ChunkParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, const CUtensorMap& qmap, cudaStream_t st) {
  if (fp8) return bf16 ? launch_chunk_typed<__nv_bfloat16, D, true>(p, kmap, vmap, qmap, st)
                       : launch_chunk_typed<__half, D, true>(p, kmap, vmap, qmap, st);
  return bf16 ? launch_chunk_typed<__nv_bfloat16, D, false>(p, kmap, vmap, qmap, st)
              : launch_chunk_typed<__half, D, false>(p, kmap, vmap, qmap, st);
}

}  // namespace
}  // namespace qsa
