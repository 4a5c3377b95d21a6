// qsa_chunk_attn.h -- launch interface between the entry points of the chunk
// attention (include/qsa_chunk.h, qsa_chunk.cu) and its kernels, compiled per
// head width (qsa_chunk_attn_{64,128,256}.cu).
#pragma once

#include "qsa_cache_host.h"

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace qsa {

constexpr int kChunkMaxCtas = 152;     // CTAs of the tile walk, one an SM (what the workspace is sized for)

// Tokens of a K/V tile, and the accumulators of 128 query rows that share a walk
// over the tiles: two in tensor memory, one for heads of 256.
constexpr int chunk_tile(int dim) { return dim == 256 ? 64 : 128; }
constexpr int chunk_accs(int dim) { return dim == 256 ? 1 : 2; }
// Query heads whose rows one accumulator holds side by side: the K/V head's group, or
// the largest part of it that divides it and fits.
inline int chunk_heads(int group) {
  int n = group < 128 ? group : 128;
  while (group % n != 0) --n;
  return n;
}
// What a K/V tile costs a row tile, and what the row tile costs beside, where two
// accumulators share it (heads of 256: where one holds more than 32 rows) and where
// not.  Measured, a row tile of 1, 2, 4, 8, 16 K/V tiles, in us an SM:
//   heads of 128, 256 rows  6.3  8.3 11.9 18.8 31.7;  4 rows  3.0  4.0  6.6 12.5 23.7
//   (over E4M3              8.4 10.2 13.7 20.8 32.8;          4.0  5.0  6.4 10.2 20.4)
//   heads of 64,  256 rows  5.5  6.8  9.5 14.1 24.6;  4 rows  3.3  4.0  5.1  8.1 14.8
//   heads of 256, 128 rows  5.7  7.3 10.1 16.0 27.2;  4 rows  2.8  3.5  6.4 11.7 22.9
// A heavy extra of 11 takes 12 prompts 561 us, of 14 552, of 17 571 (24 E4M3 chunks with
// 14 557, 17 553, 20 548); a light one of 6 and 8 differ
// in nothing that was timed; few rows' tiles at 3 for 4 took 256 requests behind
// 32768 entries 290 us in place of 253.
constexpr int kTileCostLog2 = 2, kTileCost = 4, kHeavyExtra = 14, kHeavyExtraE4M3 = 20,
              kLightExtra = 8;
// A CTA's share of a batch behind a prefix, below which it gets a run of the prefix's
// or of the requests' own alone: both cost it the start of a second row tile (8 requests
// behind 2000 entries 24.5 us, with both 25.9; 64 drafts behind 100000, far above it,
// 109 either way).
constexpr int kChunkShare = 60;
// K/V tiles from which on two warpgroups share a row tile of one accumulator (from 6
// on: 256 requests behind 32768 entries 241 us in place of 234, when all widths did).
constexpr int kChunkSplit = 12;
// Pieces of a row tile, from which on runs are longer, and how long at least (one
// request of 9215 entries 21.9 us, with runs of one K/V tile 28).
constexpr int kChunkPieces = 36, kChunkMinRun = 14;

// Query rows of one set of heads that walk K/V tiles together: the tokens [tok0, tok0
// + toks) of a request, 128 / sub of them in each accumulator.
struct ChunkTile {
  int32_t req;                  // its request; -1: the prefix, whose rows are all requests'
  int32_t tok0, toks, tiles;    // its tokens, and the K/V tiles they see
};
struct ChunkList {
  int64_t total;                // cost of its row tiles, for one set of heads
  int32_t k0, k1;               // they are [k0, k1)
  int32_t longest;              // the largest cost
  int32_t cta0, ctas;           // the CTAs that walk them
};
struct ChunkPlan {
  ChunkList list[2];            // the prefix's row tiles, the requests' own
  int32_t token0, tokens;       // rows of q that belong to requests
};

// A row tile of a request that runs cut: its pieces lie with the runs [c0, c1], in c0
// as its second segment or its first.
struct ChunkCut {
  int32_t set, c0, c1, second, by_head;
  int32_t token, toks;          // its rows of q
};

// With a prefix, for the join: the runs [c0, c1] of a row tile (c0 -1: other ones for
// each set of heads), in c0 as its second segment or its first; its rows of q.
struct ChunkOwner {
  int32_t c0, c1, second, token, toks;
};
constexpr int32_t kBySet = 1 << 30;

struct ChunkParams {
  CacheView c;
  const int32_t* prefix_table;  // nullable: no prefix, or no entries of it
  int32_t prefix_cap;           // entries that its columns can hold
  const int32_t* prefix_len;    // nullable: no prefix
  const unsigned char* q;
  int64_t q_row, q_head;        // bytes
  unsigned char* out;
  int64_t out_row, out_head;    // bytes
  const int32_t* starts;        // [num_reqs + 1]
  const int32_t* ctx;
  int32_t tokens, heads;
  int32_t sub;                  // query heads of a set, whose rows walk together
  int32_t sets, per_kv;         // sets in all, and of one K/V head
  int32_t acc_toks;             // tokens of an accumulator: 128 / sub
  int32_t heavy_rows;           // more rows than that cost heavy_extra
  int32_t heavy_extra;
  float scale_log2;             // scale * log2(e)
  int32_t window;               // 0: none
  int32_t sink;                 // 0 without a window
  float* lse;                   // nullable
  uint32_t* err;
  // workspace
  int32_t max_tiles;
  ChunkPlan* plan;
  ChunkTile* tiles;             // [max_tiles]
  int64_t* pos;                 // [max_tiles + 1] cost of the row tiles before each
  int32_t* first;               // [num_reqs] each request's first row tile
  ChunkCut* cuts;               // [kChunkMaxCtas] the one that a run's start cuts first (set -1: none)
  ChunkOwner* owners;           // with a prefix: [max_tiles]
  int32_t max_own;              // row tiles of requests, at most
  int32_t part_rows;            // rows of a row tile, at most; accumulators 128 apart
  float* part_ml;               // [2 * kChunkMaxCtas, twice that with a prefix][part_rows][2]
  float* part_o;                // [the same][part_rows][dim]
  float* res_ml[2];             // with a prefix: whole results [tokens][heads][2], of the
  float* res_o[2];              //   prefix and of the requests' own entries [..][dim]
#ifdef QSA_WAIT_TEST
  int32_t test_withhold;        // test build: CTA 0 issues no copy for this slot fill (-1: none)
#endif
};

cudaError_t launch_chunk_64(const ChunkParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, const CUtensorMap& qmap, cudaStream_t st);
cudaError_t launch_chunk_128(const ChunkParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, const CUtensorMap& qmap, cudaStream_t st);
cudaError_t launch_chunk_256(const ChunkParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, const CUtensorMap& qmap, cudaStream_t st);

}  // namespace qsa
