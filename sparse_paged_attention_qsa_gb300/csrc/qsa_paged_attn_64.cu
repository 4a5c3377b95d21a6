// qsa_paged_attn_64.cu -- the dense paged attention's kernels for heads of 64
// (qsa_paged_attn_impl.cuh).
#include "qsa_paged_attn_impl.cuh"

namespace qsa {

cudaError_t launch_paged_64(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, cudaStream_t st) {
  return launch_paged<64>(p, bf16, fp8, kmap, vmap, st);
}

}  // namespace qsa
