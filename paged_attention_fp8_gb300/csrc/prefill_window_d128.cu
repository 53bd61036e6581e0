// Prefill kernels with a sliding window and sinks for head_dim 128: a 2-byte
// cache under a long window on CTA pairs (prefill_pair.cuh), the rest on single
// CTAs (prefill.cuh).
#include "prefill_pair.cuh"

namespace pafp8 {

cudaError_t launch_prefill_window_d128(const PrefillParams& p, const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                       const CUtensorMap& tmap_v, const CUtensorMap& tmap_o, int num_ctas,
                                       cudaStream_t stream) {
    if (prefill_pairs(128, p.kv_dtype, p.window))
        return launch_prefill_pair<kVarWindow>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
    return launch_prefill_head<128, kVarWindow>(p, tmap_q, tmap_k, tmap_v, tmap_o, num_ctas, stream);
}

}  // namespace pafp8
