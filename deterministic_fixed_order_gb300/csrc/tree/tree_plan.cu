// Lays out trees of drafted tokens: ancestor bits by doubling. Node i holds the bits of the
// nodes on its way up so far and the node that comes after them; each round adds that node's
// bits and jumps to where it points, so a path of depth D takes log2 D rounds.
//
// Bound by latency: a sequence's bits pass through shared memory a few times; one CTA a sequence, a node a thread. 128 sequences of
// 256 nodes take 3.3 us, one of 26 nodes 3.1.
#include "tree_common.cuh"

namespace detfold_tree {
namespace {

template <int WORDS>
__global__ void __launch_bounds__(DETFOLD_TREE_MAX_NODES) plan_kernel(const __grid_constant__ PlanParams p)
{
    __shared__ uint64_t s_bits[WORDS][DETFOLD_TREE_MAX_NODES];
    __shared__ short s_next[DETFOLD_TREE_MAX_NODES];
    enter_grid();
    const int b = blockIdx.x, i = threadIdx.x;
    const int64_t at = (int64_t)b * p.nodes + i;
    const bool here = i < p.nodes;
    int n = p.lens[b], c = p.counts ? p.counts[b] : p.nodes;
    const int parent = here ? p.parents[at] : -1;
    bool bad = n < 0 || n > DETFOLD_ATTN_MAX_LEN - p.nodes || c < 0 || c > p.nodes;
    bad = __syncthreads_or(bad || (i < c && (parent < -1 || parent >= i)));
    if (bad) n = 0, c = 0;
    uint64_t bits[WORDS];
#pragma unroll
    for (int w = 0; w < WORDS; ++w) bits[w] = i < c && i / 64 == w ? 1ull << (i % 64) : 0;
    int next = i < c ? parent : -1;
    while (__syncthreads_or(next >= 0)) {
#pragma unroll
        for (int w = 0; w < WORDS; ++w) s_bits[w][i] = bits[w];
        s_next[i] = (short)next;
        __syncthreads();
        if (next >= 0) {
#pragma unroll
            for (int w = 0; w < WORDS; ++w) bits[w] |= s_bits[w][next];
            next = s_next[next];
        }
    }
    if (bad && i == 0) flag_bad_index(p.status);
    if (!here) return;
    int depth = -1;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
        p.mask[at * WORDS + w] = (int64_t)bits[w];
        depth += __popcll(bits[w]);
    }
    if (p.positions) p.positions[at] = i < c ? (int64_t)n + depth : 0;
    if (p.slots) {
        int64_t slot = -1;
        if (i < c) {
            const unsigned t = (unsigned)n + i, col = t / (unsigned)p.page_size;
            const int page = col < p.table_cols ? p.table[b * p.table_stride + col] : -1;
            if (page >= 0 && page < p.num_pages)
                slot = (int64_t)page * p.page_size + (t - col * (unsigned)p.page_size);
            else
                flag_bad_index(p.status);
        }
        p.slots[at] = slot;
    }
}

}  // namespace

cudaError_t launch_plan(const PlanParams &p, cudaStream_t stream)
{
    const int threads = (p.nodes + 31) / 32 * 32;
    const auto kernel = p.nodes <= 64 ? plan_kernel<1> : p.nodes <= 128 ? plan_kernel<2> : p.nodes <= 192 ? plan_kernel<3> : plan_kernel<4>;
    return launch_early(kernel, dim3(p.batch), threads, 0, stream, p);
}

}  // namespace detfold_tree
