// Prefill kernels with a scale for each 16-token block and head for head_dim 128 (the kernel is in
// prefill.cuh).
#include "prefill.cuh"

namespace pafp8 {

cudaError_t launch_prefill_blocks_d128(const PrefillParams& p, const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                  const CUtensorMap& tmap_v, const CUtensorMap& tmap_o, int num_ctas,
                                  cudaStream_t stream) {
    return launch_prefill_head<128, kVarBlocks>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
}

}  // namespace pafp8
