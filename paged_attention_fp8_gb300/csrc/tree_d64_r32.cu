// Tree attention kernels for head_dim 64 and row tiles of up to 32 rows (the
// kernel is in tree.cuh).
#include "tree.cuh"

namespace pafp8 {

cudaError_t launch_tree_d64_r32(const TreeParams& p, const CUtensorMap& tmap_k, const CUtensorMap& tmap_v, int num_ctas,
                              int num_merge, cudaStream_t stream) {
    return launch_tree_rows<64, 32>(p, tmap_k, tmap_v, num_ctas, num_merge, stream);
}

}  // namespace pafp8
