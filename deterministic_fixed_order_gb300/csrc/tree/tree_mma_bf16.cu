// Attention of trees on the matrix units: bfloat16.
#include "tree_mma.cuh"

namespace detfold_tree {

cudaError_t launch_mma_bf16(const TreeWork &w, int slabs, cudaStream_t stream)
{
    switch (slabs) {
    case 1: return launch_mma<MmaShape<__nv_bfloat16, 1>>(w, stream);
    case 2: return launch_mma<MmaShape<__nv_bfloat16, 2>>(w, stream);
    case 3: return launch_mma<MmaShape<__nv_bfloat16, 3>>(w, stream);
    default: return launch_mma<MmaShape<__nv_bfloat16, 4>>(w, stream);
    }
}

}  // namespace detfold_tree
