// Attention of trees: how a call is cut and which kernel takes it, by element type.
#include "tree_mma.cuh"

namespace detfold_tree {

cudaError_t launch_simt(const TreeWork &w, cudaStream_t stream);
cudaError_t launch_mma_bf16(const TreeWork &w, int slabs, cudaStream_t stream);
cudaError_t launch_mma_f16(const TreeWork &w, int slabs, cudaStream_t stream);

namespace {

int slabs_of(int head_dim) { return (head_dim + 63) / 64; }

TreeRule rule_of(int dtype, int rows, int head_dim)
{
    if (dtype == DETFOLD_F32) return simt_rule(rows);
    switch (slabs_of(head_dim)) {  // the same for both 16-bit types
    case 1: return MmaShape<__half, 1>::rule();
    case 2: return MmaShape<__half, 2>::rule();
    case 3: return MmaShape<__half, 3>::rule();
    default: return MmaShape<__half, 4>::rule();
    }
}

}  // namespace

int64_t tree_workspace(int dtype, int batch, int nodes, int kv_heads, int group, int head_dim, int64_t max_len)
{
    return tree_need(rule_of(dtype, nodes * group, head_dim), batch, kv_heads, group, nodes, head_dim, max_len);
}

cudaError_t launch_tree(const TreeParams &p, int dtype, void *workspace, cudaStream_t stream)
{
    const int slabs = slabs_of(p.head_dim);
    const TreeWork w = tree_work(p, rule_of(dtype, p.nodes * p.group, p.head_dim), dtype == DETFOLD_F32 ? 4 : 2, workspace);
    switch (dtype) {
    case DETFOLD_F32: return launch_simt(w, stream);
    case DETFOLD_BF16: return launch_mma_bf16(w, slabs, stream);
    default: return launch_mma_f16(w, slabs, stream);
    }
}

}  // namespace detfold_tree
