// qsa_paged_attn.h -- launch interface between the entry point of the dense
// paged attention (qsa_paged_attention.cu) and its kernels, compiled per head
// width (qsa_paged_attn_{64,128,256}.cu).
#pragma once

#include "qsa_cache_host.h"

#include <cuda.h>
#include <cstdint>
#include <cuda_runtime.h>

namespace qsa {

constexpr int kPagedBatch = 1024;   // requests per launch (their tile counts in shared memory)
constexpr int kPagedMaxCtas = 512;  // CTAs of the tile walk (what the workspace is sized for)
constexpr int kPagedMaxRows = 64;   // query rows of one K/V head that share a walk

struct PagedParams {
  CacheView c;
  const unsigned char* q;
  int64_t q_row, q_head;      // bytes
  unsigned char* out;
  int64_t out_row, out_head;  // bytes
  const int32_t* ctx;
  int32_t b0, batch;          // this launch's requests [b0, b0 + batch)
  int32_t next_n, heads, group;
  int32_t rows;               // query rows of a K/V head: next_n * group
  int32_t chunks;             // of at most kPagedMaxRows of them
  int32_t chunk_rows;         // rows of a full chunk
  float scale_log2;           // scale * log2(e)
  int64_t window;
  float* lse;                 // nullable
  float* lse2;                // workspace: [rows][heads] log2 sums, or null
  float* z;                   // workspace: [rows][heads][z_pitch] logits (base 2), or null
  int64_t z_pitch;
  int4* starts;               // workspace: [kPagedMaxCtas] request, tile, its tiles, all tiles
  float* part_ml;             // workspace: [2 * kPagedMaxCtas][chunk_rows][2]
  float* part_o;              // workspace: [2 * kPagedMaxCtas][chunk_rows][dim]
  uint32_t* err;
};

// The kernels' part of a call: the walk over the tiles and the join of what
// it left in pieces, for the requests [b0, b0 + batch).
cudaError_t launch_paged_64(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, cudaStream_t st);
cudaError_t launch_paged_128(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, cudaStream_t st);
cudaError_t launch_paged_256(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, cudaStream_t st);

// Tokens of a tile, for an element of `dim * esize` bytes and `wm` groups of
// 16 query rows: 128 where they take at most 128 bytes each and no more than
// two row groups share the walk, else 64.
constexpr int paged_tile(int row_bytes, int wm) { return row_bytes <= 128 && wm <= 2 ? 128 : 64; }

}  // namespace qsa
