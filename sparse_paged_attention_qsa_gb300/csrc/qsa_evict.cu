// qsa_evict.cu -- evicting the entries of a paged K/V cache that received
// the least attention weight, declared in include/qsa_cache.h
// (qsa_evict_entries, qsa_evict_entries_strided).
//
// rank_kernel  a cluster of 1 to 8 CTAs per request, each over a slice of its
//              entries: the budget-th largest key (protected entries, then the
//              weight sums' order-preserving bits) by radix select, histograms
//              summed through distributed shared memory; then, in entry order,
//              which entries of equal key stay, which places below the budget
//              fall free (holes) and which kept entries lie above it (movers).
//              As many of one as of the other, so the i-th mover goes to the
//              i-th hole: no entry is written that is read, so the moves need
//              no order, and only what has to move moves.  kept[] is the list
//              of moves, so there is no workspace.
// move_kernel  a warp looks 32 places of kept[] over and copies the K and V of
//              those that move, every lane's pieces in flight at once.  Where a
//              request can move but little (a decode step's eviction), the rank
//              kernel's own warps do it, in one launch.
#include "qsa_cache.h"
#include "qsa_cache_host.h"
#include "qsa_device.cuh"
#include "qsa_host.h"
#include "qsa_internal.h"

#include <algorithm>
#include <climits>
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>
#include <mutex>

namespace qsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kRankThreads = 1024;
constexpr int kRankWarps = kRankThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSpare = 8;
constexpr int kMaxSlice = 24576;          // entries of a CTA whose keys fit in shared memory
constexpr int kLoads = 4;
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
  int32_t head_log2;          // log2 of the 16-byte pieces of an entry's head
  int32_t move_here;          // the rank kernel moves K and V itself
  int32_t* kept;              // [reqs, budget]
  int32_t* new_lens;
  float* sums_out;            // rows of budget
  int64_t sums_out_s0;
  int32_t* pos_out;
  int64_t pos_out_s0;
  uint32_t* err;
};

// Order-preserving bits of a weight sum: NaN 0, -inf next, +0 and -0 equal;
// +inf stays below kProtected.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kMovePieces = 8;            // 16-byte pieces of a lane in flight

// A warp copies the K and V of up to 32 entries, one a lane (`from` to `to`; the
// same number twice: nothing to do), the lanes sharing the 16-byte pieces of
// each; up to kMovePieces blocks of 32 pieces, of one entry or of several, are in
// flight at once.
__device__ __forceinline__ void move_entries(const CacheView& c, const int32_t* bt, int head_log2,
                                             int from, int to, uint32_t* err) {
  const int lane = threadIdx.x & 31;
  const int row = c.heads << head_log2;                    // pieces of an entry's K
  const int slot_mask = (1 << c.page_log2) - 1;
  const bool moves = from != to;
  int32_t page_from = -1, page_to = -1;
  if (moves) {
    page_from = bt[from >> c.page_log2];
    page_to = bt[to >> c.page_log2];
  }
  const bool fine = moves && page_from >= 0 && page_from < c.num_pages && page_to >= 0 &&
                    page_to < c.num_pages;
  if (moves && !fine) report(err, QSA_DERR_KV_PAGE);
  uint32_t todo = __ballot_sync(0xffffffffu, fine);
  int f = 0, t = 0;                                        // the entry at hand
  int64_t pf = 0, pt = 0;
  int i0 = 2 * row;                                        // its next block
  while (todo != 0 || i0 < 2 * row) {
    uint4 x[kMovePieces];
    unsigned char* dst[kMovePieces];
#pragma unroll
    for (int j = 0; j < kMovePieces; ++j) {
      dst[j] = nullptr;
      if (i0 >= 2 * row && todo != 0) {
        const int who = __ffs(todo) - 1;
        todo &= todo - 1;
        f = __shfl_sync(0xffffffffu, from, who);
        t = __shfl_sync(0xffffffffu, to, who);
        pf = __shfl_sync(0xffffffffu, page_from, who);
        pt = __shfl_sync(0xffffffffu, page_to, who);
        i0 = 0;
      }
      const int i = i0 + lane;
      if (i < 2 * row) {
        const bool is_v = i >= row;
        const int u = is_v ? i - row : i, h = u >> head_log2, o = u & ((1 << head_log2) - 1);
        unsigned char* at = (is_v ? c.v + h * c.v_head : c.k + h * c.k_head) + o * 16;
        const int64_t ps = is_v ? c.v_page : c.k_page, ts = is_v ? c.v_token : c.k_token;
        x[j] = *reinterpret_cast<const uint4*>(at + pf * ps + (f & slot_mask) * ts);
        dst[j] = at + pt * ps + (t & slot_mask) * ts;
      }
      if (i0 < 2 * row) i0 += 32;
    }
#pragma unroll
    for (int j = 0; j < kMovePieces; ++j)
      if (dst[j]) *reinterpret_cast<uint4*>(dst[j]) = x[j];
  }
}

struct RankShared {
  // one a pass: each is read by the other CTAs while the next fills
  int hist[3][kBins];
  int coarse[3][kBins / 32];  // sums of 32 bins
  int warp[kRankWarps];
  // of the slice
  uint32_t lo, hi;            // keys (of unprotected and protected entries alike)
  int newest;                 // positions
  int holes, movers;
  // of the request, as warp 0 put it together
  uint32_t all_lo, all_hi;
  int all_newest;
  int digit, need, ties;      // of the pass: its bin, what is still to take, what it holds
  int ties_before;            // of the slice
  int first_hole[kMaxCluster + 1], first_mover[kMaxCluster + 1];   // then all of them
};

// Sum of v over the warps before this one (one value a warp, from lane 0);
// *total over all of them.
__device__ __forceinline__ int warps_before(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();                       // s_warp free again
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  const int c = s_warp[lane];
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
  *total = __reduce_add_sync(0xffffffffu, c);
  return before;
}

// ranks: CTAs of a request's cluster.
// kCached: the slice's keys are kept in shared memory (and, later, the lists of
// its holes and movers in place of the positions); else every sweep forms the
// keys from the inputs again, and the movers pass through pos_out.
template <bool kCached, int ranks>
__global__ void __launch_bounds__(kRankThreads) rank_kernel(const EvictParams p, int max_slice) {
  extern __shared__ __align__(16) unsigned char rank_smem[];
  RankShared& sh = *reinterpret_cast<RankShared*>(rank_smem);
  // [max_slice + kSpare] and [max_slice]
  uint32_t* s_key = reinterpret_cast<uint32_t*>(rank_smem + sizeof(RankShared));
  int32_t* s_pos = reinterpret_cast<int32_t*>(s_key + (kCached ? max_slice + kSpare : 0));
  // which entries stay, 32 a word
  uint32_t* s_keep = reinterpret_cast<uint32_t*>(s_pos + (kCached ? max_slice : 0));
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = ranks > 1 ? (int)cluster.block_rank() : 0;
  // a lone CTA needs no cluster barrier
  const auto sync_all = [&] {
    if (ranks > 1) cluster.sync(); else __syncthreads();
  };
  const auto of_rank = [&](int r) -> const RankShared& {
    return ranks > 1 ? *cluster.map_shared_rank(&sh, r) : sh;
  };
  pdl_wait();          // on every path: the grid's end must mean its predecessor's
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* w = p.sums + b * p.sums_s0;
  const int32_t* pos = p.pos + b * p.pos_s0;
  const int32_t ctx = p.ctx[b];
  const int n = max(0, min(ctx, p.cap));
  const int len = min(n, p.budget);
  int32_t* kept = p.kept + (int64_t)b * p.budget;
  float* sums_out = p.sums_out + b * p.sums_out_s0;
  int32_t* pos_out = p.pos_out + b * p.pos_out_s0;
  pdl_trigger();
  if (rank == 0 && tid == 0) {
    if (ctx > p.cap) report(p.err, QSA_DERR_CONTEXT);
    p.new_lens[b] = len;
  }
  if (n <= p.budget) {                   // the same for the whole cluster
    for (int i = rank * kRankThreads + tid; i < p.budget; i += ranks * kRankThreads) {
      kept[i] = i < len ? i : -1;
      sums_out[i] = i < len ? w[i] : 0.f;
      pos_out[i] = i < len ? pos[i] : -1;
    }
    return;
  }
  const int slice = (n + ranks - 1) / ranks;
  const int e0 = min(n, rank * slice), ne = min(n, e0 + slice) - e0;

  // keys and the newest position; every place below the budget starts as if
  // its entry stayed
  for (int i = tid; i < 3 * kBins; i += kRankThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) {
    sh.lo = 0xFFFFFFFFu;
    sh.hi = 0u;
    sh.newest = INT32_MIN;
  }
  __syncthreads();
  {
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    int newest = INT32_MIN;
    // a thread's loads in flight before the stores that could alias them: with
    // four of each, 26 requests of 47685 entries take 61.9 us, 40 of 5261 15.1
    // (one after another 65.5 and 15.9, eight 62.0 and 16.2)
    for (int i0 = tid; i0 < ne; i0 += kLoads * kRankThreads) {
      float f[kLoads];
      int32_t q[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int i = min(i0 + j * kRankThreads, ne - 1);
        f[j] = w[e0 + i];
        q[j] = pos[e0 + i];
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int i = i0 + j * kRankThreads;
        if (i >= ne) break;
        const uint32_t k = weight_key(f[j]);
        if constexpr (kCached) {
          s_key[i] = k;
          s_pos[i] = q[j];
        }
        if (e0 + i < p.budget) {
          kept[e0 + i] = e0 + i;
          if constexpr (kCached) {
            sums_out[e0 + i] = f[j];
            pos_out[e0 + i] = q[j];
          }
        }
        lo = min(lo, k);
        hi = max(hi, k);
        newest = max(newest, q[j]);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) {
      atomicMin(&sh.lo, lo);
      atomicMax(&sh.hi, hi);
      atomicMax(&sh.newest, newest);
    }
  }
  sync_all();
  if (warp == 0) {                       // a lane a rank
    const RankShared& o = of_rank(lane < ranks ? lane : 0);
    const uint32_t l = __reduce_min_sync(0xffffffffu, o.lo);
    const uint32_t h = __reduce_max_sync(0xffffffffu, o.hi);
    const int q = __reduce_max_sync(0xffffffffu, o.newest);
    if (lane == 0) {
      sh.all_lo = l;
      sh.all_hi = h;
      sh.all_newest = q;
    }
  }
  __syncthreads();
  const uint32_t lo = sh.all_lo, hi = sh.all_hi;
  const int newest = sh.all_newest;
  // position > newest - recent, in 64 bits: neither may wrap
  const int64_t after = (int64_t)newest - p.recent;
  // Keys relative to the smallest, so that the digits spread over the range
  // that occurs: span + 1 stands for the protected entries (hi is at most that
  // of +inf, so it does not wrap).
  const uint32_t span = hi - lo;
  const auto final_key = [&](uint32_t k, int32_t q) {
    return q < p.sink || q > after ? span + 1 : k - lo;
  };
  const auto key_of = [&](int i) {
    if constexpr (kCached) return s_key[i];
    return final_key(weight_key(w[e0 + i]), pos[e0 + i]);
  };
  const int bits = 32 - __clz(span + 1);

  // the budget-th largest key, up to 11 bits at a time from the top
  uint32_t prefix = 0, mask = 0;
  int need = p.budget, left = bits, pass = 0;
  while (left > 0) {
    const int width = min(left, 11), shift = left - width;
    const int bins = 1 << width;
    for (int i = tid; i < ne; i += kRankThreads) {
      uint32_t k;
      if (kCached && pass == 0) {
        k = final_key(s_key[i], s_pos[i]);
        s_key[i] = k;
      } else {
        k = key_of(i);
      }
      if ((k & mask) == prefix) atomicAdd(&sh.hist[pass][(k >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    for (int c = warp; c < kBins / 32; c += kRankWarps) {
      const int x = __reduce_add_sync(0xffffffffu, sh.hist[pass][c * 32 + lane]);
      if (lane == 0) sh.coarse[pass][c] = x;
    }
    sync_all();
    // From the top, the bin in which the count reaches `need`: first among the
    // sums of 32 bins, two a lane, then among the 32 (a few loads from each
    // rank, where the whole histograms would be 8 KB from each).
    if (warp == 0) {
      int c0 = 0, c1 = 0;                // sums 63 - 2 lane and 62 - 2 lane
#pragma unroll
      for (int r = 0; r < ranks; ++r) {
        const int2 h = *reinterpret_cast<const int2*>(&of_rank(r).coarse[pass][62 - 2 * lane]);
        c0 += h.y;
        c1 += h.x;
      }
      int x = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const int before = x - c0 - c1;
      const uint32_t here = __ballot_sync(0xffffffffu, before < need && x >= need);
      const int who = __ffs(here) - 1;
      const bool second = before + c0 < need;
      const int group = __shfl_sync(0xffffffffu, 63 - 2 * lane - (second ? 1 : 0), who);
      const int above = __shfl_sync(0xffffffffu, before + (second ? c0 : 0), who);
      int c = 0, earlier = 0;            // bin 31 - lane of the group; the lower ranks' part
#pragma unroll
      for (int r = 0; r < ranks; ++r) {
        const int h = of_rank(r).hist[pass][group * 32 + 31 - lane];
        c += h;
        if (r < rank) earlier += h;
      }
      x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (above + x - c < need && above + x >= need) {
        sh.digit = group * 32 + 31 - lane;
        sh.need = need - (above + x - c);
        sh.ties = c;
        sh.ties_before = earlier;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh.digit << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    need = sh.need;
    left = shift;
    ++pass;
    if (sh.ties == need) break;            // the whole bin stays: no need to look into it
  }
  // the first `need` of the bin's entries stay (of equal key, where the bin
  // holds more)
  int ties_before = sh.ties_before;
  const bool some = sh.ties != need;
  // Each warp takes a contiguous part of the slice, 32 entries at a time.
  const int part = ((ne + kRankThreads - 1) / kRankThreads) * 32;
  const int i0 = min(ne, warp * part), i1 = min(ne, i0 + part);
  const uint32_t below = (1u << lane) - 1u;
  if (some) {
    int mine = 0, total;
    for (int i = i0; i < i1; i += 32)
      mine += __popc(__ballot_sync(0xffffffffu,
                                   i + lane < i1 && (key_of(i + lane) & mask) == prefix));
    ties_before += warps_before(mine, sh.warp, &total);
  }
  // which of the 32 entries from i on stay; `ties` counts the bin's on the way
  const auto kept_of = [&](int i, int* ties) {
    const bool there = i + lane < i1;
    const uint32_t k = (there ? key_of(i + lane) : 0u) & mask;
    if (!some) return __ballot_sync(0xffffffffu, there && k >= prefix);
    const uint32_t tied = __ballot_sync(0xffffffffu, there && k == prefix);
    const uint32_t keep = __ballot_sync(
        0xffffffffu, there && (k > prefix || (k == prefix && *ties + __popc(tied & below) < need)));
    *ties += __popc(tied);
    return keep;
  };
  // the first n of 32 places
  const auto first = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; };
  // of the places from i on that `keep` says stay: holes and movers
  const auto holes_of = [&](int i, uint32_t keep) {
    return first(min(i1 - i, p.budget - e0 - i)) & ~keep;
  };
  const auto movers_of = [&](int i, uint32_t keep) { return keep & ~first(p.budget - e0 - i); };
  int holes = 0, movers = 0;
  if (!some) {                           // each lane counts its own
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
      const bool there = i + lane < i1, low = e0 + i + lane < p.budget;
      const bool stays = there && (key_of(there ? i + lane : i) & mask) >= prefix;
      holes += there && low && !stays;
      movers += stays && !low;
      if constexpr (kCached) {
        const uint32_t keep = __ballot_sync(0xffffffffu, stays);
        if (lane == 0) s_keep[i >> 5] = keep;
      }
    }
    holes = __reduce_add_sync(0xffffffffu, holes);
    movers = __reduce_add_sync(0xffffffffu, movers);
  } else {
    for (int i = i0, t = ties_before; i < i1; i += 32) {
      const uint32_t keep = kept_of(i, &t);
      if (kCached && lane == 0) s_keep[i >> 5] = keep;
      holes += __popc(holes_of(i, keep));
      movers += __popc(movers_of(i, keep));
    }
  }
  int hole_at = holes, mover_at = movers;
  hole_at = warps_before(hole_at, sh.warp, &holes);
  mover_at = warps_before(mover_at, sh.warp, &movers);
  if (tid == 0) {
    sh.holes = holes;
    sh.movers = movers;
  }
  // holes and movers of the ranks before each one
  const auto ranks_before = [&] {
    if (warp == 0) {
      const RankShared& o = of_rank(lane < ranks ? lane : 0);
      const int h = o.holes, m = o.movers;
      int x = lane < ranks ? h : 0, y = lane < ranks ? m : 0;
#pragma unroll
      for (int d = 1; d < kMaxCluster; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) {
          x += u;
          y += v;
        }
      }
      if (lane < ranks) {
        sh.first_hole[lane + 1] = x;
        sh.first_mover[lane + 1] = y;
      }
      if (lane == 0) sh.first_hole[0] = sh.first_mover[0] = 0;
    }
    __syncthreads();
  };
  if constexpr (kCached) {
    // holes from the front of the list, movers from its back (an entry is at
    // most one of the two)
#pragma unroll 2
    for (int i = i0; i < i1; i += 32) {
      const uint32_t keep = s_keep[i >> 5];
      if (e0 + i < p.budget) {
        const uint32_t h = holes_of(i, keep);
        if (h >> lane & 1u) s_pos[hole_at + __popc(h & below)] = e0 + i + lane;
        hole_at += __popc(h);
      }
      if (e0 + i + 32 > p.budget) {
        const uint32_t m = movers_of(i, keep);
        if (m >> lane & 1u) s_pos[max_slice - 1 - (mover_at + __popc(m & below))] = e0 + i + lane;
        mover_at += __popc(m);
      }
    }
    sync_all();
    ranks_before();
    // hole i of the request takes mover i, whichever CTAs' lists they are in;
    // the CTAs share the request's holes evenly
    const int all = sh.first_hole[ranks], share = (all + ranks - 1) / ranks;
    const int begin = min(all, rank * share), end = min(all, begin + share);
    const auto list_of = [&](const int* firsts, int i, int* in) {
      int r = 0;
#pragma unroll
      for (int q = 1; q < ranks; ++q)
        if (i >= firsts[q]) r = q;
      *in = i - firsts[r];
      return ranks > 1 ? cluster.map_shared_rank(s_pos, r) : s_pos;
    };
    for (int i = begin + tid; i < end; i += kRankThreads) {
      int ih, im;
      const int32_t* lh = list_of(sh.first_hole, i, &ih);
      const int32_t* lm = list_of(sh.first_mover, i, &im);
      const int to = lh[ih], from = lm[max_slice - 1 - im];
      kept[to] = from;
      sums_out[to] = w[from];
      pos_out[to] = pos[from];
      if (p.move_here) {
        // in place of the keys: at most half of the request's entries are
        // holes, so a CTA's share of pairs is a slice and a rounding
        s_key[2 * (i - begin)] = from;
        s_key[2 * (i - begin) + 1] = to;
      }
    }
    if (p.move_here) {
      __syncthreads();
      const int32_t* bt = p.c.bt + (int64_t)b * p.c.bt_s0;
      // neighbouring pairs to different warps
      for (int i0 = warp; i0 < end - begin; i0 += 32 * kRankWarps) {
        const int i = i0 + lane * kRankWarps;
        const bool there = i < end - begin;
        move_entries(p.c, bt, p.head_log2, there ? (int)s_key[2 * i] : 0,
                     there ? (int)s_key[2 * i + 1] : 0, p.err);
      }
    }
    sync_all();                          // no CTA leaves while another reads its shared memory
  } else {
    sync_all();
    ranks_before();
    const int hole_base = sh.first_hole[rank] + hole_at;
    const int mover_base = sh.first_mover[rank] + mover_at;
    int m_at = mover_base, h_at = hole_base;
    for (int i = i0, t = ties_before; i < i1; i += 32) {
      const uint32_t m = movers_of(i, kept_of(i, &t));
      if (m >> lane & 1u) pos_out[m_at + __popc(m & below)] = e0 + i + lane;
      m_at += __popc(m);
    }
    sync_all();
    for (int i = i0, t = ties_before; i < i1; i += 32) {
      const uint32_t h = holes_of(i, kept_of(i, &t));
      if (h >> lane & 1u) kept[e0 + i + lane] = __ldcg(pos_out + h_at + __popc(h & below));
      h_at += __popc(h);
    }
    sync_all();
    for (int i = rank * kRankThreads + tid; i < p.budget; i += ranks * kRankThreads) {
      const int e = __ldcg(kept + i);
      sums_out[i] = w[e];
      pos_out[i] = pos[e];
    }
  }
}

// A warp of request b looks over 32 places of kept[] at a time; its lanes share
// the 16-byte pieces of a moving entry's K and V.
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int32_t* kept = p.kept + (int64_t)b * p.budget;
  const int32_t* bt = p.c.bt + (int64_t)b * p.c.bt_s0;
  pdl_wait();
  const int warp = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const int stride = gridDim.x * (kMoveThreads / 32);
  // one place a lane, the places of a warp `stride` apart so that a run of
  // moves is spread over the warps
  for (int i0 = warp; i0 < p.budget; i0 += 32 * stride) {
    const int mine = i0 + lane * stride;
    const int src = mine < p.budget ? kept[mine] : -1;     // -1: behind the end
    move_entries(p.c, bt, p.head_log2, src < 0 ? 0 : src, src < 0 ? 0 : mine, p.err);
  }
}

// Shared memory for a slice whose keys it holds: keys, positions, a bit each.
size_t rank_smem_bytes(int64_t slice) {
  return sizeof(RankShared) + (size_t)(2 * slice + kSpare + (slice + 31) / 32) * 4;
}

// The SMs of the current device; the rank kernels' set-up once per device.
cudaError_t evict_device(int* n_sms) {
  static std::mutex mu;
  static int sms[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (sms[dev] == 0) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    for (auto k : {rank_kernel<true, 1>, rank_kernel<true, 2>, rank_kernel<true, 4>,
                   rank_kernel<true, 8>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)rank_smem_bytes(kMaxSlice));
      if (e != cudaSuccess) return e;
    }
    sms[dev] = n;
  }
  *n_sms = sms[dev];
  return cudaSuccess;
}

// CTAs of a request's cluster: as many as leave every request a cluster of its
// own, with at least kMinSlice entries each (16 requests of up to 65536 entries
// took 132, 76, 31 and 31 us with 1, 2, 4 and 8 CTAs, where slices of 65536 and
// 32768 do not fit in shared memory; with a slice of 4096 at least 8 requests of
// 16384 take 62.7 us, with 2048 or less 59.8, but 64 of 2064 9.6 and 10.9).
constexpr int64_t kMinSlice = 2048;

// Bytes that the rank kernel's CTAs move themselves for a request: more are
// sooner moved by a kernel over the whole GPU (16 entries of 4 KB in each of 64
// requests: 9.6 us against 13.0; 515 of 512 bytes in 3: 16.9 against 8.7).
constexpr int64_t kMoveHereBytes = 64 << 10;

// `most` entries can move in a request; *moved says whether they have been.
cudaError_t launch_rank(EvictParams& p, int reqs, int64_t most, int sms, cudaStream_t st,
                        bool* moved) {
  int ranks = 1;
  while (ranks < kMaxCluster && (int64_t)reqs * ranks * 2 <= sms &&
         (int64_t)p.cap >= kMinSlice * ranks * 2)
    ranks *= 2;
  const int64_t slice = ((int64_t)p.cap + ranks - 1) / ranks;
  const bool cached = slice <= kMaxSlice;
  const int64_t entry_bytes = (int64_t)2 * p.c.heads * (16 << p.head_log2);
  p.move_here = cached && most * entry_bytes <= kMoveHereBytes;
  *moved = p.move_here;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(reqs * ranks));
  cfg.blockDim = dim3(kRankThreads);
  cfg.dynamicSmemBytes = cached ? rank_smem_bytes(slice) : sizeof(RankShared);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const auto kernel = cached ? (ranks == 1   ? rank_kernel<true, 1>
                                : ranks == 2 ? rank_kernel<true, 2>
                                : ranks == 4 ? rank_kernel<true, 4>
                                             : rank_kernel<true, 8>)
                             : (ranks == 1   ? rank_kernel<false, 1>
                                : ranks == 2 ? rank_kernel<false, 2>
                                : ranks == 4 ? rank_kernel<false, 4>
                                             : rank_kernel<false, 8>);
  return cudaLaunchKernelEx(&cfg, kernel, p, (int)slice);
}

}  // namespace
}  // namespace qsa

extern "C" qsa_status qsa_evict_entries_strided(
    const qsa_paged_cache* cache, const float* weight_sums, int64_t weight_sums_stride0,
    const int32_t* entry_positions, int64_t entry_positions_stride0, int64_t entry_cols,
    const int32_t* context_lens, int64_t budget, int64_t num_sink, int64_t num_recent,
    int32_t* kept, int32_t* new_lens, float* weight_sums_out, int64_t weight_sums_out_stride0,
    int32_t* entry_positions_out, int64_t entry_positions_out_stride0, uint32_t* error_word,
    qsa_stream_t stream) {
  using namespace qsa;
  using namespace qsa::cache_host;
  EvictParams p{};
  CacheSpans cs{};
  const qsa_status st = check_cache(cache, &p.c, &cs);
  if (st != QSA_OK) return st;
  if (budget < 1 || budget > kMaxEntries || num_sink < 0 || num_recent < 0 || num_sink > budget ||
      num_recent > budget - num_sink)
    return QSA_ERR_CONTRACT;
  if (entry_cols < 0 || entry_cols > INT32_MAX) return QSA_ERR_SHAPE;
  if (!row_stride_ok(weight_sums_stride0, entry_cols) ||
      !row_stride_ok(entry_positions_stride0, entry_cols) ||
      !row_stride_ok(weight_sums_out_stride0, budget) ||
      !row_stride_ok(entry_positions_out_stride0, budget))
    return QSA_ERR_STRIDE;
  const int64_t R = cache->num_reqs;
  if (R == 0) return QSA_OK;
  if (!context_lens || !kept || !new_lens || !weight_sums_out || !entry_positions_out)
    return QSA_ERR_NULL;
  if (entry_cols > 0 && (!weight_sums || !entry_positions)) return QSA_ERR_NULL;
  if (!aligned(weight_sums, 4) || !aligned(entry_positions, 4) || !aligned(context_lens, 4) ||
      !aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(weight_sums_out, 4) ||
      !aligned(entry_positions_out, 4) || !aligned(error_word, 4))
    return QSA_ERR_ALIGN;
  const Span outs[5] = {rows_span(kept, R, budget, budget), span(new_lens, R * 4),
                        rows_span(weight_sums_out, R, budget, weight_sums_out_stride0),
                        rows_span(entry_positions_out, R, budget, entry_positions_out_stride0),
                        span(error_word, 4)};
  const Span ins[6] = {rows_span(weight_sums, R, entry_cols, weight_sums_stride0),
                       rows_span(entry_positions, R, entry_cols, entry_positions_stride0),
                       span(context_lens, R * 4), cs.tables, cs.k_scale, cs.v_scale};
  if (any_overlap(outs, 5, ins, 6)) return QSA_ERR_ALIAS;
  for (const Span& o : {cs.k, cs.v}) {
    if (any_overlap(&o, 1, ins, 6) || any_overlap(&o, 1, outs, 5)) return QSA_ERR_ALIAS;
  }
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
  p.sums_out_s0 = weight_sums_out_stride0;
  p.pos_out = entry_positions_out;
  p.pos_out_s0 = entry_positions_out_stride0;
  p.err = error_word;
  bind_calling_thread();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if (evict_device(&sms) != cudaSuccess) return QSA_ERR_CUDA;
  while (((int64_t)16 << p.head_log2) < cache->head_dim * dtype_size(cache->dtype)) ++p.head_log2;
  const int64_t most = std::min<int64_t>(budget, std::max<int64_t>(0, p.cap - budget));
  bool moved = false;
  if (launch_rank(p, (int)R, most, sms, s, &moved) != cudaSuccess) return QSA_ERR_CUDA;
  if (moved || most == 0) return QSA_OK;   // 0: no request can have an entry too many
  const int64_t warps = kMoveThreads / 32;
  const int64_t wave = std::max<int64_t>(1, (int64_t)sms * (2048 / kMoveThreads) / R);
  // every place is looked at; a warp's share is at least one, at most 32
  const int64_t ctas = std::max((most + warps - 1) / warps, (budget + 32 * warps - 1) / (32 * warps));
  const dim3 grid((unsigned)std::min(ctas, wave), (unsigned)R);
  return launch_after(move_kernel, grid, dim3(kMoveThreads), 0, s, p) == cudaSuccess ? QSA_OK
                                                                                     : QSA_ERR_CUDA;
}

extern "C" qsa_status qsa_evict_entries(
    const qsa_paged_cache* cache, const float* weight_sums, int64_t weight_sums_stride0,
    const int32_t* entry_positions, int64_t entry_positions_stride0, int64_t entry_cols,
    const int32_t* context_lens, int64_t budget, int64_t num_sink, int64_t num_recent,
    int32_t* kept, int32_t* new_lens, float* weight_sums_out, int32_t* entry_positions_out,
    uint32_t* error_word, qsa_stream_t stream) {
  return qsa_evict_entries_strided(cache, weight_sums, weight_sums_stride0, entry_positions,
                                   entry_positions_stride0, entry_cols, context_lens, budget,
                                   num_sink, num_recent, kept, new_lens, weight_sums_out, budget,
                                   entry_positions_out, budget, error_word, stream);
}
