// qsa_paged_attn.h -- launch interface between the entry point of the dense
// paged attention (qsa_paged_attention.cu) and its kernels, compiled per head
// width (qsa_paged_attn_{64,128,256}.cu).
#pragma once

#include "qsa_cache_host.h"

#include <cuda.h>
#include <cstdint>
#include <cuda_runtime.h>

namespace qsa {

constexpr int kPagedBatch = 512;    // requests per launch (their tables in shared memory)
constexpr int kPagedMaxCtas = 512;  // CTAs of the tile walk (what the workspace is sized for)
constexpr int kPagedMaxRows = 64;   // query rows of one K/V head that share a walk

// How the requests' tiles are dealt out.
enum PagedMode : int32_t {
  kPagedCut,       // equal runs over the GPU; a second kernel joins the requests they cut
  kPagedWhole,     // runs that end where a request does: nothing to join
  kPagedCluster,   // up to 8 equal runs a K/V head, one cluster, joined through its shared memory
};
// A request whose K and V of one head take no more than this is not cut: a CTA
// streams it in about the time that a second launch takes (a cluster, which needs
// none, was not tried below this size).  And where a K/V
// head's requests take no more than that for each CTA of a cluster, up to 16
// query rows are walked by one.
constexpr int64_t kPagedWholeBytes = 256 << 10;
constexpr int kPagedCluster8 = 8;

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
  int32_t mode;               // a PagedMode
  float scale_log2;           // scale * log2(e)
  int32_t window;             // 0: none; at most INT32_MAX - 16
  float* lse;                 // nullable
  float2* stats;              // workspace: [rows][heads] reference and log2 of the sum, or null
  float* z;                   // workspace: [rows][heads][z_pitch] logits (base 2), or null
  int64_t z_pitch;
  int4* starts;               // workspace: [kPagedMaxCtas] request, tile, its tiles, all tiles
  float* part_ml;             // workspace: [2 * kPagedMaxCtas][chunk_rows][2]
  float* part_o;              // workspace: [2 * kPagedMaxCtas][chunk_rows][dim]
  uint32_t* err;
#ifdef QSA_WAIT_TEST
  int32_t test_withhold;      // test build: CTA 0 issues no copy for this slot fill (-1: none)
#endif
};

// The kernels' part of a call: the walk over the tiles and the join of what
// it left in pieces, for the requests [b0, b0 + batch).
cudaError_t launch_paged_64(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, cudaStream_t st);
cudaError_t launch_paged_128(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, cudaStream_t st);
cudaError_t launch_paged_256(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, cudaStream_t st);

// The shape of a CTA that walks up to `rows` query rows of heads of `dim`, with
// row_bytes of K (or V) a token; what was measured, in us:
//   wm sets of warps, each with 16 rows.  Up to 16 rows of heads below 256 two
//   CTAs an SM with four consumer warps each; for more rows one CTA with eight
//   (16-bit heads of 128, 32 rows: 92 with eight warps, 111 with four; 64 rows:
//   260 and 305).  Two sets of rows in one warp, which share what it reads and
//   converts of K and V, leave too few warps: 16-bit 32 rows 103 against 88,
//   E4M3 117 against 108.  Heads of 256 hold twice the output a row, so four
//   warps with all registers (32 rows: 181 against 331).
//   Ring slots of 16 KB, but of 32 KB for heads of 256 (E4M3: 138 against 167)
//   and, where a warp's part of 16 KB is 32 tokens or fewer, for 17 rows and more
//   of 256-byte rows of K (32 rows: 92 against 108; 64: 198 against 230, 256 short
//   requests 137 against 129) and for 17 to 32 of 128-byte rows (FP16 heads of 64:
//   128 against 166; E4M3 heads of 128: 102 against 112, 32 requests of about 1000
//   tokens 37.2 against 35.5).  At most 64 tokens a warp, whose logits are in its
//   registers (64 rows with 128 tokens: E4M3 heads of 64 206 against 242, but short
//   requests of heads of 128 211 against 179).  Narrower heads with up to 16 rows
//   in one CTA an SM and 32 KB slots instead: 84 against 83 (131072 tokens), but 65
//   against 48 where requests are short, and 344 against 285 for E4M3 heads of 128.
constexpr int paged_sets(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
constexpr int paged_warps(int dim, int wm) { return wm == 1 || dim == 256 ? 4 : 8; }
constexpr int paged_ctas(int dim, int wm) { return wm == 1 && dim < 256 ? 2 : 1; }
// tokens of a tile
constexpr int paged_tile(int dim, int row_bytes, int wm) {
  const bool large = dim == 256 || (wm >= 2 && row_bytes == 256) || (wm == 2 && row_bytes == 128);
  const int most = 64 * (paged_warps(dim, wm) / wm), t = (large ? 32768 : 16384) / row_bytes;
  return t < most ? t : most;
}

}  // namespace qsa
