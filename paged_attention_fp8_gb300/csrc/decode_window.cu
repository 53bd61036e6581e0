// The decode kernel with a sliding window and sinks (the kernel is in decode.cuh).
#include "decode.cuh"

namespace pafp8 {

cudaError_t launch_decode_window(const DecodeParams& p, const CUtensorMap& tmap_k, const CUtensorMap& tmap_v, int num_ctas,
                             int hpc, int group, int heads_per_box, cudaStream_t stream) {
    return launch_decode_var<kVarWindow>(p, tmap_k, tmap_v, num_ctas, hpc, group, heads_per_box, stream);
}

}  // namespace pafp8
