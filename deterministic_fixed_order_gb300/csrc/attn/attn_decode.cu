// One-token attention: the grid and workspace of a call, by element type.
#include "attn_decode.cuh"

namespace detfold_attn {

cudaError_t launch_decode_f32(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream);
cudaError_t launch_decode_bf16(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream);
cudaError_t launch_decode_f16(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream);

namespace {

// The call's grid: query heads a pair as the tiles take them, tokens a round.
DecodeGrid grid_of(int dtype, int batch, int kv_heads, int group, int head_dim, int64_t max_seen)
{
    const bool f32 = dtype == DETFOLD_F32;
    const int heads = f32 ? (group == 1 ? 1 : group <= 4 ? 4 : 8) : group > 8 && head_dim <= 128 ? 16 : 8;
    return decode_grid(batch, kv_heads, group, head_dim, max_seen, heads, tile_of(f32 ? 4 : 2, head_dim, heads));
}

}  // namespace

int64_t decode_workspace(int dtype, int batch, int kv_heads, int group, int head_dim, int64_t max_seen)
{
    return batch == 0 ? 0 : workspace_need(grid_of(dtype, batch, kv_heads, group, head_dim, max_seen));
}

cudaError_t launch_decode(const DecodeParams &p, int dtype, void *workspace, cudaStream_t stream)
{
    const DecodeGrid g = grid_of(dtype, p.batch, p.kv_heads, p.group, p.head_dim, p.window);
    DecodeWork w = {};
    w.p = p;
    w.pairs = g.pairs, w.blocks = g.pairs / p.kv_heads, w.heads = g.heads;
    w.slots = g.direct == 1 ? 0 : g.slots, w.by_pair = g.by_pair, w.most_chunks = g.most, w.slot_chunks = g.chunks;
    w.most = divide_by(w.most_chunks), w.grid = divide_by(g.ctas);
    w.direct = g.direct;
    if (g.direct) w.by_chunks = divide_by(g.direct);
    w.by_pairs = divide_by(g.pairs);
    w.short_line = (double)p.batch * g.pairs * (p.window / 32 + 2) < (1 << 30);
    w.pair_floats = g.pair_floats, w.slot_floats = g.slot_floats;
    w.page = divide_by(p.page_size);
    const int four = dtype == DETFOLD_F32 ? 16 : 8;
    w.q_vec = (uintptr_t)p.q % (four / 2) == 0 && p.q_bs % 2 == 0 && p.q_hs % 2 == 0;
    w.out_vec = (uintptr_t)p.out % four == 0 && p.out_bs % 4 == 0 && p.out_hs % 4 == 0;
    w.headers = (int4 *)workspace;
    w.slot = (float *)((char *)workspace + (int64_t)g.slots * 16);
    switch (dtype) {
    case DETFOLD_F32: return launch_decode_f32(w, g, stream);
    case DETFOLD_BF16: return launch_decode_bf16(w, g, stream);
    default: return launch_decode_f16(w, g, stream);
    }
}

}  // namespace detfold_attn
