// Shared pieces of the operators of a step with drafted tokens: launch parameters and
// the refusals of indexes from device memory.
#pragma once

#include "attn/attn_common.cuh"
#include "detfold_tree.h"

namespace detfold_tree {

using namespace detfold_attn;

constexpr int kSms = 152;
constexpr int kMaxWords = DETFOLD_TREE_WORDS(DETFOLD_TREE_MAX_NODES);

struct PlanParams {
    int64_t *mask, *positions, *slots;
    const int32_t *parents, *lens, *counts, *table;
    int64_t table_stride, table_cols, num_pages;
    int page_size, batch, nodes;
    int *status;
};

struct TreeParams {
    void *out;
    float *lse;
    const void *q;
    int64_t out_bs, out_ns, out_hs, q_bs, q_ns, q_hs;
    const void *k, *v;
    int64_t num_pages, page_stride, token_stride, head_stride;
    const int32_t *table, *lens, *counts;
    const int64_t *mask;
    int64_t table_stride;
    int page_size, kv_heads, head_dim, group;
    int batch, nodes, words, q_heads, max_len, window;  // window 0: none
    float scale;
    int *status;
};

struct CompactParams {
    detfold_kv_cache cache;
    const int32_t *table, *lens, *path, *path_lens;
    int64_t table_stride, table_cols, path_stride;
    int batch, max_path;
    int *status;
};

struct CopyParams {
    detfold_kv_cache cache;
    const int32_t *src, *dst, *rows;
    int64_t count;
    int *status;
};

struct PagesParams {
    int32_t *refs_out, *table_out, *lens_out, *copy_src, *copy_dst, *copy_rows;
    const int32_t *refs, *table, *lens, *origin, *keep, *want;
    int64_t table_out_stride, table_stride;
    int num_pages, cols, page_size, rows_in, rows_out;
    int *status;
    Divide page;  // by the page size
};

cudaError_t launch_plan(const PlanParams &p, cudaStream_t stream);
// `max_len` of the call, for the sizes alone.
int64_t tree_workspace(int dtype, int batch, int nodes, int kv_heads, int group, int head_dim, int64_t max_len);
cudaError_t launch_tree(const TreeParams &p, int dtype, void *workspace, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream);
cudaError_t launch_copy(const CopyParams &p, cudaStream_t stream);
cudaError_t launch_pages(const PagesParams &p, cudaStream_t stream);

}  // namespace detfold_tree
