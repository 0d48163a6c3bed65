// Attention of trees on the matrix units: float16.
#include "tree_mma.cuh"

namespace detfold_tree {

cudaError_t launch_mma_f16(const TreeWork &w, int slabs, cudaStream_t stream)
{
    switch (slabs) {
    case 1: return launch_mma<MmaShape<__half, 1>>(w, stream);
    case 2: return launch_mma<MmaShape<__half, 2>>(w, stream);
    case 3: return launch_mma<MmaShape<__half, 3>>(w, stream);
    default: return launch_mma<MmaShape<__half, 4>>(w, stream);
    }
}

}  // namespace detfold_tree
