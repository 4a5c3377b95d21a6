// qsa_paged_attn_128.cu -- the dense paged attention's kernels for heads of 128
// (qsa_paged_attn_impl.cuh).
#include "qsa_paged_attn_impl.cuh"

namespace qsa {

cudaError_t launch_paged_128(const PagedParams& p, bool bf16, bool fp8, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, cudaStream_t st) {
  return launch_paged<128>(p, bf16, fp8, kmap, vmap, st);
}

}  // namespace qsa
