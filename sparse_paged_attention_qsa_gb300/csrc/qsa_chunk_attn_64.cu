// qsa_chunk_attn_64.cu -- the chunk attention's kernels for heads of 64
// (qsa_chunk_attn_impl.cuh).
#include "qsa_chunk_attn_impl.cuh"

namespace qsa {

cudaError_t launch_chunk_64(const ChunkParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, const CUtensorMap& qmap, cudaStream_t st) {
  return launch_chunk<64>(p, bf16, fp8, kmap, vmap, qmap, st);
}

}  // namespace qsa
