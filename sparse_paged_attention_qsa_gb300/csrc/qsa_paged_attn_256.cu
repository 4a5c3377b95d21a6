// qsa_paged_attn_256.cu -- the dense paged attention's kernels for heads of 256
// (qsa_paged_attn_impl.cuh).
#include "qsa_paged_attn_impl.cuh"

namespace qsa {

cudaError_t launch_paged_256(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, cudaStream_t st) {
  return launch_paged<256>(p, bf16, fp8, kmap, vmap, st);
}

}  // namespace qsa
