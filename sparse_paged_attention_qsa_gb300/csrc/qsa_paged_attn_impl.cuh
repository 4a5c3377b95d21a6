// qsa_paged_attn_impl.cuh -- the kernels of the dense paged attention
// (include/qsa_cache.h, qsa_paged_attention).
//
// For one K/V head of one request, its M = next_n * group query rows and its
// entries e:  z_ie = c_i (q_i . k_e),  o_i = sum_e 2^(z_ie - m_i) v_e,
// l_i = sum_e 2^(z_ie - m_i); out = o / l.  The reference m_i is the running
// maximum less a shift, rounded up: its own binary32 value is what every sum,
// merge and lse uses, so logits of any size subtract from it without a weight
// passing 2^shift (the maximum less the shift, rounded to nearest, is off by up to
// half a unit of a logit past 2^24, and weights of 2^16 are infinite in FP16).  4 M flops
// for every K/V element of 1 or 2 bytes: for M <= 64 the bytes set the time, so
// everything here serves one thing, that K and V stream through once at the
// rate of the memory.
//
// paged_walk_kernel  The requests' tiles (TT entries), laid end to end, are cut
//   into equal runs; a CTA walks one run for one K/V head (and up to 64 of its
//   query rows), all CTAs in a single wave: every SM streams the same bytes
//   whatever the lengths.
//   Two producer warps look pages up and load K and V tiles into a ring by
//   TMA (swizzled, completion on mbarriers); four or eight consumer warps share a
//   tile: WM sets of 16 query rows by WK slices of its tokens.
//   Each warp keeps its rows' reference, sum and output in registers: S = Q K^T
//   and P V by mma.sync.m16n8k16 (binary32 accumulation) on fragments that
//   ldmatrix reads from the ring.  (With at most 16 rows as a rule mma.sync is
//   a third busy at the memory's rate.  From 17 rows on it is not: every set of 16
//   reads, and for E4M3 converts, the tile again, 64 rows at 0.56 to 0.68 of the
//   copy rate, 0.25 to 0.30 for E4M3.  tcgen05 with the tokens, then the head's
//   dims, as M and the query rows as N could share the tile; it has not been
//   built, so what its softmax by columns and the staging of the weights cost is not
//   known.)  At a request's end,
//   or the run's, the slices merge through shared memory into the output, or
//   into a piece in the workspace when the K/V head's entries are cut.
// paged_join_kernel  joins a cut K/V head's pieces.
// Short work needs no second kernel: its runs end where requests do, or are one
// cluster a K/V head, whose CTAs keep their pieces in shared memory and join
// them there (PagedMode).
//
// Rounding: q, K and V enter the products as they are (E4M3 as FP16, exactly;
// BF16 queries of an E4M3 cache as FP16 after a power-of-two scaling of the
// row, where only bits 2^-25 below the row's largest element can be lost).
// The weights multiply V as a pair of 16-bit values (a value and what its
// rounding left), 2^-16 (BF16) or 2^-22 (FP16) relative, for up to 32 rows
// over a 16-bit cache, where the second product is free; above that, and for
// E4M3 caches (whose elements carry 4 bits), as one value.
#pragma once

#include "qsa_paged_attn.h"
#include "qsa_device.cuh"
#include "qsa_internal.h"

#include <algorithm>
#include <cmath>
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <mutex>

namespace qsa {
namespace {

// The largest weight is about 2^shift: 15 where weights are FP16, so that small ones
// stay normal; BF16 has binary32's exponents and needs none, and 2^15 times a value
// past 2^113 would leave them.
constexpr float paged_shift(bool bf16) { return bf16 ? 0.f : 15.f; }
constexpr int kJoinThreads = 256;
constexpr int kMaxSlots = 16;
constexpr int kSmemPerSm = 233472, kSmemReserved = 1024;   // 228 KB, 1 KB of it a CTA's own

// Small tables of a CTA, behind the ring, the queries and the merge buffer.
struct WalkTables {
  uint64_t full[kMaxSlots], empty[kMaxSlots];   // mbarriers of the ring
  uint64_t q_full[2], q_empty[2];               // and of the two query slots
  uint32_t boxes[kMaxSlots];                    // a bit per copy, 0: it had no page
  float ml[8][16][2];                            // reference and sum of the warps' rows
  float qs[kPagedMaxRows];                      // what the queries were divided by
  int32_t scan[12];                             // tiles of the requests of each warp
  uint8_t token[kPagedMaxRows];                 // the row's token of the draft
  int32_t ctx[kPagedBatch];                     // cached tokens of each request
  int32_t pre[kPagedBatch + 1];                 // tiles before each
  int32_t abort;
  int32_t pad[2];
};
static_assert(sizeof(WalkTables) % 16 == 0, "a whole number of 16-byte pieces");

template <bool kFp8, int D, int WM, bool kCluster>
struct WalkShape {
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);        // a token's K (or V) of one head
  static constexpr int NW = paged_warps(D, WM);           // consumer warps
  static constexpr int kRows = 16 * WM;                       // query rows they hold
  static constexpr int kConsumers = NW * 32;
  static constexpr int kThreads = kConsumers + 64;            // + K's and V's producer
  static constexpr int TT = paged_tile(D, kRowBytes, WM);
  static constexpr int WK = NW / WM;
  static constexpr int kSlice = TT / WK;                      // tokens of a warp
  static constexpr int NS = kSlice / 16;                      // in steps of 16
  static constexpr int kChunkBytes = kRowBytes < 128 ? kRowBytes : 128;   // TMA inner extent
  static constexpr int kChunks = kRowBytes / kChunkBytes;     // copies that fill a slot
  static constexpr int kSlot = TT * kRowBytes;                // K (or V) of a tile
  static constexpr int kQPitch = D + 8;                       // halves; + 16 B against conflicts
  static constexpr int kQBytes = kRows * kQPitch * 2;         // a query slot
  static constexpr int kQSlots = kFp8 ? 3 : 2;                // the third: as FP16, reordered
  static constexpr int kMergeBytes = NW == 8 ? 128 * 40 * 4 : 17408;   // at least 32 columns
  // of the first and the last segment: 16 rows and their reference and sum
  static constexpr int kPieceBytes = kCluster ? 2 * 16 * (D + 4) * 4 : 0;
  static constexpr int kFixed =
      1024 + kQSlots * kQBytes + kMergeBytes + kPieceBytes + (int)sizeof(WalkTables);
  static constexpr int kCtas = kCluster ? 1 : paged_ctas(D, WM);
  static constexpr int kFit = (kSmemPerSm / kCtas - kSmemReserved - kFixed) / kSlot;
  // two CTAs keep four tiles each on their way; a fifth was slower (FP16 heads of
  // 64 236 us against 229, E4M3 128 against 121, heads of 128 with weights 241
  // against 228) and three no better (234, 126, 227); one CTA takes what fits
  // (heads of 256 602 us with four, 597 with five)
  static constexpr int kMost = kCtas == 2 ? 4 : kMaxSlots;
  static constexpr int S = kFit < kMost ? kFit : kMost;
  static constexpr size_t kSmem = (size_t)kFixed + (size_t)S * kSlot;
  static_assert(S >= 3, "the ring needs K, V and one slot ahead");
  static_assert(NS >= 1 && NS <= 4, "logits of a tile stay in registers");
  static constexpr bool kPair = !kFp8 && kRows <= 32;         // weights as value + remainder
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (lo, hi) rounded to 16 bits each, lo in the low half
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t r) {
  if constexpr (kBf16)
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  else
    return h2f2(r);
}
// the two E4M3 values in the low (high) half of x, as FP16
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r) : "r"(x));
  return r;
}
template <int kThreads>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

// Visible entries [lo, hi) of token j of a request with ctx cached tokens,
// cut to what the table holds.
__device__ __forceinline__ void visible(const PagedParams& p, int32_t ctx, int j, int32_t* lo,
                                        int32_t* hi) {
  // 32 bits hold it all: h >= -7, and the window is at most INT32_MAX - 16
  const int32_t cap = (int32_t)p.c.cap;
  const int32_t h = max(ctx, 0) - p.next_n + j + 1;
  *hi = min(max(h, 0), cap);
  *lo = p.window > 0 ? min(max(h - p.window, 0), cap) : 0;
}

// What a row's reference m and sum l (0: it saw nothing) leave: its lse, and for the
// weights the two apart, since their sum is off by half a unit of a large logit.
__device__ __forceinline__ void store_stats(const PagedParams& p, int64_t rh, float m, float l) {
  const float log_l = log2f(l);
  if (p.lse) p.lse[rh] = l == 0.f ? -INFINITY : (m + log_l) * 0.693147180559945309f;
  if (p.stats) p.stats[rh] = make_float2(m, log_l);
}

// The tiles a request's entries span, [*first, *first + count).
template <int TT>
__device__ __forceinline__ int32_t tiles_of(const PagedParams& p, int32_t ctx, int32_t* first) {
  int32_t lo, hi, x;
  visible(p, ctx, 0, &lo, &x);
  visible(p, ctx, p.next_n - 1, &x, &hi);
  *first = lo / TT;
  return hi > lo ? (hi + TT - 1) / TT - lo / TT : 0;
}

// The requests' tiles laid end to end and cut into n runs: the first `more`
// runs take each + 1 tiles.
struct Runs {
  int32_t total, each, more;
};
__device__ __forceinline__ Runs cut_runs(int32_t total, int n) {
  Runs r;
  r.total = total;
  r.each = total / n;
  r.more = total - r.each * n;
  return r;
}
__device__ __forceinline__ int32_t run_start(const Runs& r, int c) {
  return r.each * c + min(c, r.more);
}
__device__ __forceinline__ int run_of(const Runs& r, int32_t x) {
  const int32_t big = (r.each + 1) * r.more;
  return x < big ? x / (r.each + 1) : r.more + (x - big) / r.each;
}

// Where tile w lies: the request, the tile within it and how many it has;
// pre[] holds the tiles before each request.
struct TileAt {
  int b, tile, count;
};
__device__ __forceinline__ TileAt tile_at(const int32_t* pre, int batch, int32_t w) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= w) lo = mid; else hi = mid - 1;
  }
  return TileAt{lo, w - pre[lo], pre[lo + 1] - pre[lo]};
}

// Where the tile behind the last one of at's request lies (there is one): in the
// next request as a rule.
__device__ __forceinline__ TileAt tile_behind(const int32_t* pre, int batch, const TileAt& at) {
  const int32_t w = pre[at.b + 1], n = pre[min(at.b + 2, batch)] - w;
  return n > 0 ? TileAt{at.b + 1, 0, n} : tile_at(pre, batch, w);
}

template <typename T, bool kFp8, int D, int WM, bool kCluster>
__global__ void __launch_bounds__((WalkShape<kFp8, D, WM, kCluster>::kThreads),
                                  (WalkShape<kFp8, D, WM, kCluster>::kCtas))
paged_walk_kernel(const PagedParams p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using W = WalkShape<kFp8, D, WM, kCluster>;
  constexpr bool kBf16 = sizeof(T) == 2 && !kFp8 && __is_same(T, __nv_bfloat16);   // product type
  constexpr int TT = W::TT, WK = W::WK, NS = W::NS, S = W::S;
  extern __shared__ unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  unsigned char* base = smem_raw + pad;
  const uint32_t ring = raw + pad;
  const uint32_t queries = ring + S * W::kSlot;            // query slots, then the merge buffer
  constexpr int kBehind = S * W::kSlot + W::kQSlots * W::kQBytes;
  float* merge = reinterpret_cast<float*>(base + kBehind);
  constexpr int kTables = kBehind + W::kMergeBytes + W::kPieceBytes;
  float* pieces = reinterpret_cast<float*>(base + kBehind + W::kMergeBytes);   // [2][16][D + 4]
  WalkTables& tb = *reinterpret_cast<WalkTables*>(base + kTables);
  const uint32_t bar_full = ring + kTables, bar_empty = bar_full + 8 * kMaxSlots;
  const uint32_t bar_qfull = bar_empty + 8 * kMaxSlots, bar_qempty = bar_qfull + 16;
  volatile int32_t* s_abort = &tb.abort;
  int32_t* pre = tb.pre;

  // CTA: run * units + unit, so that the K/V heads of the same tokens, whose
  // elements lie side by side, are read at the same time; a cluster's are the
  // runs of one unit
  const int units = p.c.heads * p.chunks, n_runs = gridDim.x / units;
  const int run = kCluster ? blockIdx.x % n_runs : blockIdx.x / units;
  const int unit = kCluster ? blockIdx.x / n_runs : blockIdx.x % units;
  const int head = unit / p.chunks, chunk = unit - head * p.chunks;
  const int row0 = chunk * kPagedMaxRows;
  const int n_rows = min(kPagedMaxRows, p.rows - row0);    // query rows of this unit

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, W::NW);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_qfull + 8 * s, 1);
      mbar_init(bar_qempty + 8 * s, W::NW);
    }
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows past the last query stay zero in every slot
  for (int i = tid; i < W::kQSlots * W::kQBytes / 16; i += W::kThreads)
    reinterpret_cast<uint4*>(base + S * W::kSlot)[i] = make_uint4(0, 0, 0, 0);
  // launched while the kernel before it on the stream may still run: what that
  // one wrote, and what it read and this one writes, is touched from here on
  pdl_wait();
  // tiles before each request
  {
    const int per = (p.batch + W::kThreads - 1) / W::kThreads;
    const int lo = min(p.batch, tid * per), hi = min(p.batch, lo + per);
    int32_t sum = 0, x;
    for (int b = lo; b < hi; ++b) {
      const int32_t ctx = p.ctx[p.b0 + b];
      const int32_t n = tiles_of<TT>(p, ctx, &x);
      tb.ctx[b] = ctx;
      pre[b + 1] = n;
      sum += n;
    }
    int32_t upto = sum;                                    // of this warp's threads to here
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += v;
    }
    if (lane == 31) tb.scan[warp] = upto;
    for (int i = tid; i < kPagedMaxRows; i += W::kThreads)
      tb.token[i] = (uint8_t)(min(row0 + i, p.rows - 1) / p.group);
    // the zeros above were written through the generic proxy, copies follow
    // through the async one
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    int32_t before = upto - sum;
    for (int i = 0; i < warp; ++i) before += tb.scan[i];
    for (int b = lo; b < hi; ++b) {
      before += pre[b + 1];
      pre[b + 1] = before;
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
  }
  const Runs runs = cut_runs(pre[p.batch], n_runs);
  int32_t w_begin = run_start(runs, run), w_end = run_start(runs, run + 1);
  if (!kCluster && p.mode == kPagedWhole) {   // on to the next request's first tile
    const auto snap = [&](int32_t w) {
      if (w >= runs.total) return runs.total;
      const TileAt at = tile_at(pre, p.batch, w);
      return at.tile > 0 ? w - at.tile + at.count : w;
    };
    w_begin = snap(w_begin);
    w_end = snap(w_end);
  }
  pdl_trigger();     // every CTA is resident: the join may be put in place (it waits)
  // where the run starts, for the join; run 0 always says how many tiles there are
  if (!kCluster && p.mode == kPagedCut && unit == 0 && tid == 0 && (run == 0 || w_begin < w_end)) {
    TileAt at = {0, 0, 0};
    if (w_begin < w_end) at = tile_at(pre, p.batch, w_begin);
    p.starts[run] = make_int4(at.b, at.tile, at.count, runs.total);
  }

  const auto row_ptr = [&](const unsigned char* t, int64_t rs, int64_t hs, int b, int i) {
    const int r = row0 + i, j = tb.token[i];
    return t + ((int64_t)(p.b0 + b) * p.next_n + j) * rs +
           (int64_t)(head * p.group + r - j * p.group) * hs;
  };

  // the request that starts in this run and is cut: its place, and its pieces
  int own_b = -1, own_piece = 0, own_runs = 0;
  int withheld = -1;                                       // test build: a slot fill left out
  int issued = 0, segments = 0;                            // producers: slots, queries loaded
  if (warp >= W::NW) {
    // ---------------- producers ----------------
    // Tile t's K is slot fill 2t, its V 2t + 1; a warp each, since a copy takes its
    // warp 80 to 100 cycles to issue and small pages need many (one warp for both:
    // pages of 8, FP16 heads of 256 244 us against 155, E4M3 heads of 64 137 against
    // 96; pages of 16 157 against 142 and 92 against 75; of 64 no difference).
    const int kv = warp - W::NW;
    const int lg = p.c.page_log2;
    const int box_rows = min(TT, 1 << lg);
    const int n_boxes = TT / box_rows;
    const int tile_cols = max(1, TT >> lg);
    int32_t w = w_begin;
    int s = kv, round = 0;                                 // ring position of the next fill
    // Narrow rows, and K and V beside logits that are read again, give way in L2
    // first (E4M3 heads of 128: 292 us against 296, FP16 heads of 64: 45 against
    // 48); wide rows go through as anything does (heads of 256: 635 against 656).
    const uint64_t policy = p.chunks == 1 && (p.z != nullptr || W::kRowBytes <= 128)
                                ? evict_first_policy() : evict_normal_policy();
    bool stop = false;
    // a slot free again; false (and the walk stopped) after the limit
    const auto wait_empty = [&](uint32_t bar, uint32_t phase) {
      bool ok = *s_abort == 0 && mbar_wait(bar, phase);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) {
          *s_abort = 1;
          report(p.err, QSA_DERR_TIMEOUT);
        }
        stop = true;
      }
      return ok;
    };
    // 32 page ids of a request, one a lane; the next segment's are on their way
    // while this one's tiles are issued
    const auto first_col = [&](const TileAt& at) {
      int32_t first;
      tiles_of<TT>(p, tb.ctx[at.b], &first);
      return ((first + at.tile) * TT) >> lg;
    };
    const auto page_ids = [&](int b, int col) {
      return col + lane < p.c.cols ? __ldg(p.c.bt + (int64_t)(p.b0 + b) * p.c.bt_s0 + col + lane)
                                   : -1;
    };
    TileAt at = {0, 0, 0};
    int chunk_col = 0;
    int32_t chunk_id = -1;
    if (w < w_end) {
      at = tile_at(pre, p.batch, w);
      chunk_col = first_col(at);
      chunk_id = page_ids(at.b, chunk_col);
    }
    while (w < w_end && !stop) {
      const int32_t ctx = tb.ctx[at.b];
      int32_t first, lo, hi, x;
      tiles_of<TT>(p, ctx, &first);
      visible(p, ctx, 0, &lo, &x);
      visible(p, ctx, p.next_n - 1, &x, &hi);
      if (ctx > p.c.cap && tid == W::kConsumers) report(p.err, QSA_DERR_CONTEXT);
      const int32_t seg_end = min(w_end, w + (at.count - at.tile));
      TileAt next = at;
      int next_col = 0;
      int32_t next_id = -1;
      if (kv == 0) {                                       // the segment's queries
        const int qs = segments & 1;
        if (segments >= 2 && !wait_empty(bar_qempty + 8 * qs, (uint32_t)((segments / 2 - 1) & 1)))
          break;
        const uint32_t full = bar_qfull + 8 * qs;
        if (lane == 0) mbar_expect_tx(full, (uint32_t)(n_rows * D * 2));
        __syncwarp();
        for (int i = lane; i < n_rows; i += 32)
          bulk_load(queries + qs * W::kQBytes + i * W::kQPitch * 2,
                    row_ptr(p.q, p.q_row, p.q_head, at.b, i), D * 2, full);
        ++segments;
      }
      for (int t = at.tile; w < seg_end; ++w, ++t) {
        const int32_t e0 = (first + t) * TT;
        const int col = e0 >> lg;
        if (col + tile_cols > chunk_col + 32) {
          chunk_col = col;
          chunk_id = page_ids(at.b, col);
        }
        const int32_t id = __shfl_sync(0xffffffffu, chunk_id,
                                       col - chunk_col + (lane < n_boxes ? (lane * box_rows) >> lg : 0));
        const int32_t be = e0 + lane * box_rows;
        const bool want = lane < n_boxes && be < hi && be + box_rows > lo;
        const bool good = want && id >= 0 && id < p.c.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, good);
        const uint32_t unseen = ~__ballot_sync(0xffffffffu, want);   // and not asked about
        if (__any_sync(0xffffffffu, want && !good) && tid == W::kConsumers)
          report(p.err, QSA_DERR_KV_PAGE);
        if (round > 0 && !wait_empty(bar_empty + 8 * s, (uint32_t)((round - 1) & 1))) break;
        const uint32_t full = bar_full + 8 * s, dst = ring + s * W::kSlot;
#ifdef QSA_WAIT_TEST
        // test build: leave this fill without a copy, so the consumers'
        // wait on it runs out (the failure-detection test)
        const bool withhold = blockIdx.x == 0 && 2 * issued + kv == p.test_withhold;
        if (withhold) withheld = issued;
        if (!withhold)
#endif
        {
          if (lane == 0) {
            tb.boxes[s] = mask | unseen;
            mbar_expect_tx(full, (uint32_t)(__popc(mask) * box_rows * W::kRowBytes));
          }
          __syncwarp();
          if (good) {
#pragma unroll
            for (int i = 0; i < W::kChunks; ++i)
              tma_load_4d(dst + i * (TT * W::kChunkBytes) + lane * box_rows * W::kChunkBytes,
                          kv ? &vmap : &kmap, i * (W::kChunkBytes / (kFp8 ? 1 : 2)), head,
                          be & ((1 << lg) - 1), id, full, policy);
          }
        }
        ++issued;
        s += 2;
        if (s >= S) {
          s -= S;
          ++round;
        }
        if (t == at.tile && seg_end < w_end) {             // on their way during the others
          next = tile_behind(pre, p.batch, at);
          next_col = first_col(next);
          next_id = page_ids(next.b, next_col);
        }
      }
      at = next;
      chunk_col = next_col;
      chunk_id = next_id;
    }
  } else {
    // ---------------- consumers ----------------
    const int wm = warp % WM, wk = warp / WM;
    const int g = lane >> 2, q4 = lane & 3;
    const int lg = p.c.page_log2;
    const int box_log2 = min(lg, TT == 256 ? 8 : TT == 128 ? 7 : 6);
    // ldmatrix source rows and the swizzle's exclusive-or, constant a lane
    const int k_row = wk * W::kSlice + ((lane >> 4) << 3) + (lane & 7);       // K: tokens by 8
    const int v_row = wk * W::kSlice + (((lane >> 3) & 1) << 3) + (lane & 7); // V: transposed
    const int k_c = (lane >> 3) & 1, v_c = lane >> 4;
    const int sw = W::kChunkBytes == 128 ? lane & 7 : (lane >> 1) & 3;
    constexpr int kPer = W::kChunkBytes / 16;              // 16-byte pieces of a TMA row
    const auto piece = [&](int row, int c) -> uint32_t {   // 16-byte piece c of a row of a slot
      return (uint32_t)(row * W::kChunkBytes + ((c ^ sw) << 4));
    };
    const uint32_t q_lane = queries + (uint32_t)(((wm * 16 + (lane & 15)) * W::kQPitch +
                                                  (lane >> 4) * 8) * 2);
    // a slot's wait: after a time-out every warp runs its loops to their end
    // without waiting, so that the barriers between them stay matched
    int slot = 0;                                          // ring position, and its phase
    uint32_t phase = 0;
    const auto wait_for = [&](uint32_t bar, uint32_t ph) {
      if (!mbar_try_wait(bar, ph) && *s_abort == 0 && !mbar_wait(bar, ph)) {
        *s_abort = 1;
        if (lane == 0) report(p.err, QSA_DERR_TIMEOUT);
      }
    };
    const auto wait_full = [&]() { wait_for(bar_full + 8 * slot, phase); };
    const auto release = [&]() {                           // and on to the next slot
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_empty + 8 * slot);
      if (++slot == S) {
        slot = 0;
        phase ^= 1;
      }
    };

    // requests without a visible entry: zeros, here because no tile is theirs
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
      if (pre[b + 1] != pre[b]) continue;
      const int64_t r0 = (int64_t)(p.b0 + b) * p.next_n;
      if (tb.ctx[b] > p.c.cap && tid == 0) report(p.err, QSA_DERR_CONTEXT);
      const int n = p.next_n * p.heads;
      for (int i = tid; i < n * (D / 8); i += W::kConsumers) {
        const int rh = i / (D / 8), o = i % (D / 8);
        *reinterpret_cast<uint4*>(p.out + (r0 + rh / p.heads) * p.out_row +
                                  (rh % p.heads) * p.out_head + o * 16) = make_uint4(0, 0, 0, 0);
      }
      for (int i = tid; i < n; i += W::kConsumers) {
        if (p.lse) p.lse[r0 * p.heads + i] = -INFINITY;
        if (p.stats) p.stats[r0 * p.heads + i] = make_float2(-INFINITY, 0.f);
      }
    }

    // merging: the real rows of every slice side by side, as many columns at a time
    // as the buffer holds (all of them for up to 16 rows and slices)
    const int cols = min(D, (W::kMergeBytes / 4 / (WK * n_rows) - 8) & ~31);
    const int pitch = cols + 8;
    int32_t w = w_begin;
    TileAt at = {0, 0, 0};
    for (int seg = 0; w < w_end; ++seg) {
      at = seg == 0 ? tile_at(pre, p.batch, w) : tile_behind(pre, p.batch, at);
      const int32_t seg_begin = w, seg_end = min(w_end, w + (at.count - at.tile));
      const bool whole = at.tile == 0 && seg_end - seg_begin == at.count;
      const int32_t ctx = tb.ctx[at.b];
      int32_t first, lo_all, hi_all, x;
      tiles_of<TT>(p, ctx, &first);
      visible(p, ctx, 0, &lo_all, &x);
      visible(p, ctx, p.next_n - 1, &x, &hi_all);
      // the entries that every row sees: a tile inside them needs no mask
      int32_t lo_in, hi_in;
      visible(p, ctx, p.next_n - 1, &lo_in, &x);
      visible(p, ctx, 0, &x, &hi_in);
      const int64_t q_row = (int64_t)(p.b0 + at.b) * p.next_n;

      // the queries: as they came, or for E4M3 as FP16 in the third slot
      const int qs = seg & 1;
      wait_for(bar_qfull + 8 * qs, (uint32_t)((seg >> 1) & 1));
      const uint32_t q_addr = q_lane + (kFp8 ? 2 : qs) * W::kQBytes;
      if constexpr (kFp8) {
        const unsigned char* src = base + S * W::kSlot + qs * W::kQBytes;
        uint32_t* fp16 = reinterpret_cast<uint32_t*>(base + S * W::kSlot + 2 * W::kQBytes);
        consumers_sync<W::kConsumers>();                   // all are done with the last ones
        for (int i = tid; i < W::kRows * (D / 8); i += W::kConsumers) {
          // D/8 lanes (8, 16 or 32, aligned) hold one row: its largest
          // magnitude, then FP16 with each 16 dims in the order in which the
          // E4M3 fragments hold them (dims 4q, 4q+1 at 2q and 4q+2, 4q+3 at 8 + 2q)
          const int r = i / (D / 8), o = i % (D / 8);
          const uint4 v = *reinterpret_cast<const uint4*>(src + r * W::kQPitch * 2 + o * 16);
          float f[8];
          const T* h = reinterpret_cast<const T*>(&v);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = (float)h[k];
          float mul = 1.f;
          if constexpr (__is_same(T, __nv_bfloat16)) {
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(f[k]));
#pragma unroll
            for (int k = 1; k < D / 8; k <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, k));
            // largest magnitude to [2^14, 2^15); as it is where that has no exponent
            const int e = (int)(__float_as_uint(a) >> 23);
            if (e > 0 && e < 255) {
              const int up = min(14 + 127 - e, 120);
              mul = __uint_as_float((uint32_t)(127 - up) << 23);      // 2^-up
              const float by = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
              for (int k = 0; k < 8; ++k) f[k] *= by;
            }
          }
          uint32_t* dst = fp16 + (r * W::kQPitch + (o >> 1) * 16) / 2;
          const int q2 = (o & 1) * 2;
          dst[q2] = pack2<false>(f[0], f[1]);
          dst[q2 + 4] = pack2<false>(f[2], f[3]);
          dst[q2 + 1] = pack2<false>(f[4], f[5]);
          dst[q2 + 5] = pack2<false>(f[6], f[7]);
          if (o == 0) tb.qs[r] = mul;
        }
        consumers_sync<W::kConsumers>();
      }

      // this thread's rows, k = 0 and 1
      const auto row_of = [&](int k) { return wm * 16 + g + 8 * k; };
      const auto token_of = [&](int i) { return (int)tb.token[i]; };
      float mult[2];
      float* z_at[2];                                     // its logits' row, or null
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mult[k] = p.scale_log2;
        if constexpr (kFp8) {
          if (p.c.k_scale) mult[k] *= p.c.k_scale[head];
          mult[k] *= tb.qs[row_of(k)];
        }
        const int r = min(row0 + row_of(k), p.rows - 1), j = token_of(row_of(k));
        const int64_t rh = ((int64_t)(p.b0 + at.b) * p.next_n + j) * p.heads + head * p.group + r -
                           j * p.group;
        z_at[k] = p.z && row_of(k) < n_rows ? p.z + rh * p.z_pitch : nullptr;
      }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

      for (int t = at.tile; w < seg_end; ++w, ++t) {
        const int32_t e0 = (first + t) * TT;
        const int32_t we = e0 + wk * W::kSlice;            // the warp's first entry
        wait_full();
        const uint32_t mask = tb.boxes[slot];
        const bool edge = e0 < lo_in || e0 + TT > hi_in || mask != 0xffffffffu;
        float sc[NS][2][4];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            sc[s][n][0] = sc[s][n][1] = sc[s][n][2] = sc[s][n][3] = 0.f;
#pragma unroll
        for (int ch = 0; ch < W::kChunks; ++ch) {
          const uint32_t kb = ring + slot * W::kSlot + ch * (TT * W::kChunkBytes);
#pragma unroll
          for (int kk = 0; kk < kPer / 2; ++kk) {          // two 16-byte pieces at a time
            const int k = ch * (kPer / 2) + kk;
            if constexpr (!kFp8) {
              uint32_t a[4];
              ldsm4(q_addr + k * 32, a);
#pragma unroll
              for (int st = 0; st < NS; ++st) {
                uint32_t b[4];
                ldsm4(kb + piece(k_row + st * 16, 2 * kk + k_c), b);
                mma16816<kBf16>(sc[st][0], a, b[0], b[1]);
                mma16816<kBf16>(sc[st][1], a, b[2], b[3]);
              }
            } else {
              uint32_t a0[4], a1[4];
              ldsm4(q_addr + k * 64, a0);
              ldsm4(q_addr + k * 64 + 32, a1);
#pragma unroll
              for (int st = 0; st < NS; ++st) {
                uint32_t b[4];
                ldsm4(kb + piece(k_row + st * 16, 2 * kk + k_c), b);
                mma16816<false>(sc[st][0], a0, e4m3_lo(b[0]), e4m3_hi(b[0]));
                mma16816<false>(sc[st][1], a0, e4m3_lo(b[2]), e4m3_hi(b[2]));
                mma16816<false>(sc[st][0], a1, e4m3_lo(b[1]), e4m3_hi(b[1]));
                mma16816<false>(sc[st][1], a1, e4m3_lo(b[3]), e4m3_hi(b[3]));
              }
            }
          }
        }
        release();
        // logits; masked ones -inf
        float ref[2], al[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              sc[s][n][2 * k] *= mult[k];
              sc[s][n][2 * k + 1] *= mult[k];
            }
          if (edge) {
            int32_t lo, hi;
            visible(p, ctx, token_of(row_of(k)), &lo, &hi);
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int32_t e = we + s * 16 + n * 8 + 2 * q4 + x;
                  const bool in = (mask >> ((e - e0) >> box_log2)) & 1u;
                  if (!in || e < lo || e >= hi) sc[s][n][2 * k + x] = -INFINITY;
                }
          }
          if (z_at[k]) {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const int32_t e = we + s * 16 + n * 8 + 2 * q4;
                if (e < hi_all)
                  *reinterpret_cast<float2*>(z_at[k] + e) =
                      make_float2(sc[s][n][2 * k], sc[s][n][2 * k + 1]);
              }
          }
          float mx = -INFINITY;
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int n = 0; n < 2; ++n) mx = fmaxf(mx, fmaxf(sc[s][n][2 * k], sc[s][n][2 * k + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[k], __fadd_ru(mx, -paged_shift(kBf16)));
          ref[k] = mn == -INFINITY ? 0.f : mn;             // nothing seen yet: all weights 0
          al[k] = mn == m[k] ? 1.f : ex2(m[k] - mn);
          m[k] = mn;
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
          l[0] *= al[0];
          l[1] *= al[1];
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= al[0];
            o[i][1] *= al[0];
            o[i][2] *= al[1];
            o[i][3] *= al[1];
          }
        }
        uint32_t ph[NS][4], pl[NS][4];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float p0 = ex2(sc[s][n][2 * k] - ref[k]), p1 = ex2(sc[s][n][2 * k + 1] - ref[k]);
              l[k] += p0 + p1;
              const uint32_t h = pack2<kBf16>(p0, p1);
              ph[s][2 * n + k] = h;
              if constexpr (W::kPair) {
                const float2 f = unpack2<kBf16>(h);
                pl[s][2 * n + k] = pack2<kBf16>(p0 - f.x, p1 - f.y);
              }
            }
        // P V.  Where an entry is hidden, 0 times what it holds may be NaN: in an
        // edge tile V enters with the entries zeroed that not all of the warp's
        // rows see; those that some see, a few at each end, are added one by one
        // to the rows that see them.
        int32_t lo_a = 0, hi_a = 0, lo_b = 0, hi_b = 0;    // of the first and the last row's token
        if (edge) {
          visible(p, ctx, token_of(wm * 16), &lo_a, &hi_a);
          visible(p, ctx, token_of(wm * 16 + 15), &lo_b, &hi_b);
        }
        wait_full();
#pragma unroll
        for (int ch = 0; ch < W::kChunks; ++ch) {
          const uint32_t vb = ring + slot * W::kSlot + ch * (TT * W::kChunkBytes);
          constexpr int kTiles = kFp8 ? kPer * 2 : kPer;   // of 8 dims
          if (!edge) {
#pragma unroll
            for (int st = 0; st < NS; ++st)
#pragma unroll
              for (int i = 0; i < kPer / 2; ++i) {
                uint32_t b[4];
                ldsm4t(vb + piece(v_row + st * 16, 2 * i + v_c), b);
                if constexpr (!kFp8) {
                  float(&o0)[4] = o[ch * kTiles + 2 * i], (&o1)[4] = o[ch * kTiles + 2 * i + 1];
                  mma16816<kBf16>(o0, ph[st], b[0], b[1]);
                  mma16816<kBf16>(o1, ph[st], b[2], b[3]);
                  if constexpr (W::kPair) {
                    mma16816<kBf16>(o0, pl[st], b[0], b[1]);
                    mma16816<kBf16>(o1, pl[st], b[2], b[3]);
                  }
                } else {
                  // a pair of tokens' E4M3 bytes (t0: d0 d1, t1: d0 d1) regrouped
                  // by dim, so that even and odd dims are two products
#pragma unroll
                  for (int k = 0; k < 4; ++k) b[k] = __byte_perm(b[k], 0, 0x3120);
                  const int n = ch * kTiles + 4 * i;
                  mma16816<false>(o[n], ph[st], e4m3_lo(b[0]), e4m3_lo(b[1]));
                  mma16816<false>(o[n + 1], ph[st], e4m3_hi(b[0]), e4m3_hi(b[1]));
                  mma16816<false>(o[n + 2], ph[st], e4m3_lo(b[2]), e4m3_lo(b[3]));
                  mma16816<false>(o[n + 3], ph[st], e4m3_hi(b[2]), e4m3_hi(b[3]));
                }
              }
          } else {
#pragma unroll
            for (int st = 0; st < NS; ++st) {
              uint32_t keep[2];
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const int32_t e = we + st * 16 + n * 8 + 2 * q4;
                const bool in = (mask >> ((e - e0) >> box_log2)) & 1u;
                keep[n] = (in && e >= lo_b && e < hi_a ? 0xffffu : 0u) |
                          (in && e + 1 >= lo_b && e + 1 < hi_a ? 0xffff0000u : 0u);
              }
              const auto add = [&](int n, uint32_t b0, uint32_t b1) {
                mma16816<kBf16>(o[n], ph[st], b0 & keep[0], b1 & keep[1]);
                if constexpr (W::kPair) mma16816<kBf16>(o[n], pl[st], b0 & keep[0], b1 & keep[1]);
              };
#pragma unroll
              for (int i = 0; i < kPer / 2; ++i) {
                uint32_t b[4];
                ldsm4t(vb + piece(v_row + st * 16, 2 * i + v_c), b);
                if constexpr (!kFp8) {
                  add(ch * kTiles + 2 * i, b[0], b[1]);
                  add(ch * kTiles + 2 * i + 1, b[2], b[3]);
                } else {
#pragma unroll
                  for (int k = 0; k < 4; ++k) b[k] = __byte_perm(b[k], 0, 0x3120);
                  const int n = ch * kTiles + 4 * i;
                  add(n, e4m3_lo(b[0]), e4m3_lo(b[1]));
                  add(n + 1, e4m3_hi(b[0]), e4m3_hi(b[1]));
                  add(n + 2, e4m3_lo(b[2]), e4m3_lo(b[3]));
                  add(n + 3, e4m3_hi(b[2]), e4m3_hi(b[3]));
                }
              }
            }
          }
        }
        if (edge && (lo_a != lo_b || hi_a != hi_b)) {
          int32_t lo[2], hi[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) visible(p, ctx, token_of(row_of(k)), &lo[k], &hi[k]);
          // [lo_a, mid) and [from, hi_b): what some rows see and not all
          const int32_t mid = min(lo_b, hi_b), from = max(hi_a, mid);
#pragma unroll
          for (int st = 0; st < NS; ++st) {
            const int32_t t0 = we + st * 16, t1 = t0 + 16;
            for (int32_t e = max(lo_a, t0); e < min(hi_b, t1); ++e) {
              if (e >= mid && e < from) {                  // all rows see it
                e = from - 1;
                continue;
              }
              if (!((mask >> ((e - e0) >> box_log2)) & 1u)) continue;
              const int at = e - t0, owner = (lane & 28) | (at & 7) >> 1, upper = at >> 3;
              float w[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t h = __shfl_sync(0xffffffffu, upper ? ph[st][2 + k] : ph[st][k], owner);
                const float2 f = unpack2<kBf16>(h);
                w[k] = at & 1 ? f.y : f.x;
                if constexpr (W::kPair) {
                  const uint32_t r = __shfl_sync(0xffffffffu, upper ? pl[st][2 + k] : pl[st][k], owner);
                  const float2 d = unpack2<kBf16>(r);
                  w[k] += at & 1 ? d.y : d.x;
                }
              }
              const int row = e - e0, rsw = W::kChunkBytes == 128 ? row & 7 : (row >> 1) & 3;
              const bool sees[2] = {e >= lo[0] && e < hi[0], e >= lo[1] && e < hi[1]};
              const unsigned char* v = base + slot * W::kSlot + row * W::kChunkBytes + q4 * 4;
#pragma unroll
              for (int c = 0; c < W::kRowBytes / 16; ++c) {  // four bytes of each 16-byte piece
                const uint32_t x = *reinterpret_cast<const uint32_t*>(
                    v + (c / kPer) * (TT * W::kChunkBytes) + (((c % kPer) ^ rsw) << 4));
                const auto add = [&](float (&acc)[4], float2 f) {
#pragma unroll
                  for (int k = 0; k < 2; ++k)
                    if (sees[k]) {
                      acc[2 * k] = fmaf(w[k], f.x, acc[2 * k]);
                      acc[2 * k + 1] = fmaf(w[k], f.y, acc[2 * k + 1]);
                    }
                };
                if constexpr (!kFp8) {
                  add(o[c], unpack2<kBf16>(x));
                } else {                                   // even and odd dims
                  const uint32_t y = __byte_perm(x, 0, 0x3120);
                  add(o[2 * c], h2f2(e4m3_lo(y)));
                  add(o[2 * c + 1], h2f2(e4m3_hi(y)));
                }
              }
            }
          }
        }
        release();
      }

      // ---- the segment's end: merge the WK slices, write the result or a piece
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_qempty + 8 * qs);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
      }
      const int which = seg_begin == w_begin ? 0 : 1;      // first segment, or the last
      const int64_t id = 2 * (int64_t)blockIdx.x + which;
      if (kCluster && !whole && at.tile == 0) {
        own_b = at.b;
        own_piece = which;
        own_runs = run_of(runs, seg_begin + at.count - 1) - run + 1;
      }
      const float vscale = kFp8 && p.c.v_scale ? p.c.v_scale[head] : 1.f;
      for (int c0 = 0; c0 < D; c0 += cols) {
        const int c1 = min(D, c0 + cols);
        consumers_sync<W::kConsumers>();                   // the buffer is free
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = row_of(k);
          if (i < n_rows) {
            float* b = merge + (wk * n_rows + i) * pitch - c0;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              if (n * 8 >= c0 && n * 8 < c1) {
                if constexpr (!kFp8) {
                  *reinterpret_cast<float2*>(b + n * 8 + 2 * q4) =
                      make_float2(o[n][2 * k], o[n][2 * k + 1]);
                } else {
                  // tile n holds the even (odd) dims of the 16 from 16 (n / 2)
                  b[(n >> 1) * 16 + 4 * q4 + (n & 1)] = o[n][2 * k];
                  b[(n >> 1) * 16 + 4 * q4 + 2 + (n & 1)] = o[n][2 * k + 1];
                }
              }
            }
            if (q4 == 0) {
              tb.ml[warp][g + 8 * k][0] = m[k];
              tb.ml[warp][g + 8 * k][1] = l[k];
            }
          }
        }
        consumers_sync<W::kConsumers>();
        const int groups = (c1 - c0) / 8;
        for (int it = tid; it < n_rows * groups; it += W::kConsumers) {
          const int i = it / groups, c = (it - i * groups) * 8;
          const float* ml[WK];
          float M = -INFINITY, L = 0.f, f[WK];
#pragma unroll
          for (int k = 0; k < WK; ++k) {
            ml[k] = tb.ml[(i >> 4) + k * WM][i & 15];
            M = fmaxf(M, ml[k][0]);
          }
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < WK; ++k) {
            f[k] = M == -INFINITY ? 0.f : ex2(ml[k][0] - M);
            L += ml[k][1] * f[k];
            const float4* b = reinterpret_cast<const float4*>(merge + (k * n_rows + i) * pitch + c);
            const float4 a0 = b[0], a1 = b[1];
            v[0] += a0.x * f[k]; v[1] += a0.y * f[k]; v[2] += a0.z * f[k]; v[3] += a0.w * f[k];
            v[4] += a1.x * f[k]; v[5] += a1.y * f[k]; v[6] += a1.z * f[k]; v[7] += a1.w * f[k];
          }
          if (whole) {
            const float inv = L == 0.f ? 0.f : vscale / L;   // 0: a row that saw nothing
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = pack2<__is_same(T, __nv_bfloat16)>(v[2 * k] * inv, v[2 * k + 1] * inv);
            *reinterpret_cast<uint4*>(
                const_cast<unsigned char*>(row_ptr(p.out, p.out_row, p.out_head, at.b, i)) +
                (c0 + c) * 2) = make_uint4(h[0], h[1], h[2], h[3]);
            if (c0 + c == 0) {
              const int r = row0 + i, j = token_of(i);
              const int64_t rh = ((int64_t)(p.b0 + at.b) * p.next_n + j) * p.heads +
                                 head * p.group + r - j * p.group;
              store_stats(p, rh, M, L);
            }
          } else if constexpr (kCluster) {
            float* d = pieces + (which * 16 + i) * (D + 4);
            reinterpret_cast<float4*>(d + c0 + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(d + c0 + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
            if (c0 + c == 0) *reinterpret_cast<float2*>(d + D) = make_float2(M, L);
          } else {
            float4* d = reinterpret_cast<float4*>(p.part_o + (id * p.chunk_rows + i) * D + c0 + c);
            d[0] = make_float4(v[0], v[1], v[2], v[3]);
            d[1] = make_float4(v[4], v[5], v[6], v[7]);
            if (c0 + c == 0)
              *reinterpret_cast<float2*>(p.part_ml + (id * p.chunk_rows + i) * 2) = make_float2(M, L);
          }
        }
      }
    }
  }
  if constexpr (kCluster) {
    // every thread of the cluster comes here, also after a time-out
    auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    if (own_b >= 0) {                                      // consumers of the owner
      const float vscale = kFp8 && p.c.v_scale ? p.c.v_scale[head] : 1.f;
      for (int it = tid; it < n_rows * (D / 4); it += W::kConsumers) {
        const int i = it / (D / 4), ln = it % (D / 4);
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < own_runs; ++k) {
          // the later runs hold theirs as a first segment
          const float* d = cluster.map_shared_rank(pieces, run + k) +
                           ((k == 0 ? own_piece : 0) * 16 + i) * (D + 4);
          const float2 ml = *reinterpret_cast<const float2*>(d + D);
          const float4 v = *reinterpret_cast<const float4*>(d + ln * 4);
          const float mn = fmaxf(M, ml.x);
          const float a = mn == M ? 1.f : ex2(M - mn), f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mn);
          L = L * a + ml.y * f;
          acc.x = acc.x * a + v.x * f;
          acc.y = acc.y * a + v.y * f;
          acc.z = acc.z * a + v.z * f;
          acc.w = acc.w * a + v.w * f;
          M = mn;
        }
        const float inv = L == 0.f ? 0.f : vscale / L;
        constexpr bool kOut = __is_same(T, __nv_bfloat16);
        *reinterpret_cast<uint2*>(
            const_cast<unsigned char*>(row_ptr(p.out, p.out_row, p.out_head, own_b, i)) + ln * 8) =
            make_uint2(pack2<kOut>(acc.x * inv, acc.y * inv), pack2<kOut>(acc.z * inv, acc.w * inv));
        if (ln == 0) {
          const int r = row0 + i, j = tb.token[i];
          const int64_t rh = ((int64_t)(p.b0 + own_b) * p.next_n + j) * p.heads + head * p.group +
                             r - j * p.group;
          store_stats(p, rh, M, L);
        }
      }
    }
    cluster.sync();                                        // its pieces have been read
  }
  __syncthreads();
  // after a time-out, let the copies this CTA issued land before it exits
  if (*s_abort != 0 && warp >= W::NW && lane == 0) {
    for (int i = max(0, issued - (S + 1) / 2); i < issued; ++i) {
      const int n = 2 * i + warp - W::NW;
      if (i != withheld) mbar_wait(bar_full + 8 * (n % S), (uint32_t)((n / S) & 1), kDrainLimitNs);
    }
    for (int n = segments > 2 ? segments - 2 : 0; n < segments; ++n)
      mbar_wait(bar_qfull + 8 * (n & 1), (uint32_t)((n >> 1) & 1), kDrainLimitNs);
  }
}

// CTA (c - 1, i, unit): row i of the unit in the request that the start of run
// c cuts, if it is the first such cut.  D/4 threads hold a row; the others take
// further pieces of it, or, where there are few, further rows (then the CTAs of
// those rows have nothing to do).
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedParams p, int n_runs) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  constexpr int kFew = 8;                                  // pieces that one group walks
  __shared__ __align__(16) float s_o[kGroups][D];
  __shared__ float s_m[kGroups], s_l[kGroups];
  const int tid = threadIdx.x, c = blockIdx.x + 1, unit = blockIdx.z;
  const int grp = tid / kLanes, ln = tid % kLanes;
  pdl_wait();
  const int units = p.c.heads * p.chunks;
  // run 0 has said how many tiles there are; a run without tiles says nothing
  const Runs runs = cut_runs(p.starts[0].w, n_runs);
  const int32_t cut = run_start(runs, c);
  if (runs.total == 0 || cut >= runs.total) return;
  const int4 at = p.starts[c];                             // request, tile, its tiles, all
  const int32_t x0 = cut - at.y;
  // between requests, or an earlier run's start cuts this one too
  if (at.y == 0 || run_start(runs, c - 1) > x0) return;
  const int c0 = c - 1, n = run_of(runs, x0 + at.z - 1) - c0 + 1;
  const bool few = n <= kFew;
  if (few && blockIdx.y % kGroups != 0) return;
  const int i = blockIdx.y + (few ? grp : 0);              // the row, and its pieces:
  const int k0 = few ? 0 : grp, dk = few ? 1 : kGroups;
  const int head = unit / p.chunks, chunk = unit - head * p.chunks;
  const int row0 = chunk * kPagedMaxRows, r = row0 + i;
  const bool there = i < min(kPagedMaxRows, p.rows - row0);
  // piece k's place in the workspace: a run's first segment, or its other one
  const int second = run_start(runs, c0) != x0;
  const auto piece_row = [&](int k) {
    return (int64_t)(2 * ((c0 + k) * units + unit) + (k == 0 ? second : 0)) * p.chunk_rows + i;
  };
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (there) {
#pragma unroll 4
    for (int k = k0; k < n; k += dk) {
      const int64_t at_k = piece_row(k);
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at_k * 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at_k * D + ln * 4);
      const float mn = fmaxf(m, ml.x);
      const float a = mn == m ? 1.f : ex2(m - mn), f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mn);
      l = l * a + ml.y * f;
      acc.x = acc.x * a + v.x * f;
      acc.y = acc.y * a + v.y * f;
      acc.z = acc.z * a + v.z * f;
      acc.w = acc.w * a + v.w * f;
      m = mn;
    }
  }
  if (!few) {                                              // the groups' parts of the row
    if (ln == 0) {
      s_m[grp] = m;
      s_l[grp] = l;
    }
    *reinterpret_cast<float4*>(&s_o[grp][ln * 4]) = acc;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int k = 1; k < kGroups; ++k) {
      const float mk = s_m[k], mn = fmaxf(m, mk);
      const float a = mn == m ? 1.f : ex2(m - mn), f = mk == -INFINITY ? 0.f : ex2(mk - mn);
      const float4 v = *reinterpret_cast<const float4*>(&s_o[k][ln * 4]);
      l = l * a + s_l[k] * f;
      acc.x = acc.x * a + v.x * f;
      acc.y = acc.y * a + v.y * f;
      acc.z = acc.z * a + v.z * f;
      acc.w = acc.w * a + v.w * f;
      m = mn;
    }
  }
  if (!there) return;
  const int j = r / p.group, h = head * p.group + r - j * p.group;
  const int64_t row = (int64_t)(p.b0 + at.x) * p.next_n + j;
  const float inv = l == 0.f ? 0.f : (p.c.v_scale ? p.c.v_scale[head] : 1.f) / l;
  constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
  *reinterpret_cast<uint2*>(p.out + row * p.out_row + h * p.out_head + ln * 8) =
      make_uint2(pack2<kBf16>(acc.x * inv, acc.y * inv), pack2<kBf16>(acc.z * inv, acc.w * inv));
  if (ln == 0) store_stats(p, row * p.heads + h, m, l);
}

// The SMs of the current device; the kernel's set-up once per device.
template <typename T, bool kFp8, int D, int WM, bool kCluster>
cudaError_t walk_device(int* n_sms) {
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
    e = cudaFuncSetAttribute(paged_walk_kernel<T, kFp8, D, WM, kCluster>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)WalkShape<kFp8, D, WM, kCluster>::kSmem);
    if (e != cudaSuccess) return e;
    sms[dev] = n;
  }
  *n_sms = sms[dev];
  return cudaSuccess;
}

template <typename T, bool kFp8, int D, int WM>
cudaError_t launch_walk(const PagedParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        cudaStream_t st) {
  using W = WalkShape<kFp8, D, WM, false>;
  int n_sms = 0;
  cudaError_t e = walk_device<T, kFp8, D, WM, false>(&n_sms);
  if (e != cudaSuccess) return e;
  // runs: as many as fill one wave, no more than there can be tiles
  const int units = p.c.heads * p.chunks;
  const int64_t tiles =
      (int64_t)p.batch * (p.mode == kPagedWhole ? 1 : ((int64_t)p.c.cap + W::TT - 1) / W::TT);
  int64_t n_runs = std::min(n_sms * W::kCtas, kPagedMaxCtas) / units;
  n_runs = std::max<int64_t>(1, std::min(n_runs, tiles));
  e = launch_after(paged_walk_kernel<T, kFp8, D, WM, false>, dim3((unsigned)(n_runs * units)),
                   dim3(W::kThreads), W::kSmem, st, p, kmap, vmap);
  if (e != cudaSuccess || n_runs == 1 || p.mode == kPagedWhole) return e;   // nothing has been cut
  return launch_after(paged_join_kernel<T, D>,
                      dim3((unsigned)n_runs - 1, (unsigned)p.chunk_rows, (unsigned)units),
                      dim3(kJoinThreads), 0, st, p, (int)n_runs);
}

// As launch_walk for up to 16 rows, in one kernel: a cluster of up to 8 runs a unit.
template <typename T, bool kFp8, int D>
cudaError_t launch_cluster(const PagedParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                           cudaStream_t st) {
  using W = WalkShape<kFp8, D, 1, true>;
  int n_sms = 0;
  const cudaError_t e = walk_device<T, kFp8, D, 1, true>(&n_sms);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.batch * (((int64_t)p.c.cap + W::TT - 1) / W::TT);
  const unsigned n_runs = (unsigned)std::min<int64_t>(kPagedCluster8, tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_runs * (unsigned)(p.c.heads * p.chunks));
  cfg.blockDim = dim3(W::kThreads);
  cfg.dynamicSmemBytes = W::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n_runs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, paged_walk_kernel<T, kFp8, D, 1, true>, p, kmap, vmap);
}

template <typename T, bool kFp8, int D>
cudaError_t launch_rows(const PagedParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        cudaStream_t st) {
  if (p.mode == kPagedCluster) return launch_cluster<T, kFp8, D>(p, kmap, vmap, st);
  switch (paged_sets(p.chunk_rows)) {
    case 1: return launch_walk<T, kFp8, D, 1>(p, kmap, vmap, st);
    case 2: return launch_walk<T, kFp8, D, 2>(p, kmap, vmap, st);
    default: return launch_walk<T, kFp8, D, 4>(p, kmap, vmap, st);
  }
}

template <int D>
cudaError_t launch_paged(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, cudaStream_t st) {
  if (bf16) return fp8 ? launch_rows<__nv_bfloat16, true, D>(p, kmap, vmap, st)
                       : launch_rows<__nv_bfloat16, false, D>(p, kmap, vmap, st);
  return fp8 ? launch_rows<__half, true, D>(p, kmap, vmap, st)
             : launch_rows<__half, false, D>(p, kmap, vmap, st);
}

}  // namespace
}  // namespace qsa
