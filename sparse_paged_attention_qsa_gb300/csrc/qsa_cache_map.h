// qsa_cache_map.h -- TMA descriptors of a paged cache's views, for the kernels
// that load its tiles.
#pragma once

#include "qsa_cache_host.h"

#include <algorithm>
#include <cstring>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <mutex>

namespace qsa {

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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
inline bool encode_view(CUtensorMap* map, const unsigned char* p, const CacheView& c, int esize,
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

}  // namespace qsa
