// Joins the partial results of rows whose tokens lie in several units of work: half a warp a row, or a warp. The units'
// triples are folded in ascending order. Bound by instructions (57% of the issue slots, 18% of the memory's rate) and by latency:
// each accumulator is read once, several in flight. In a batch of 32 sequences of 128 rows a key-value head it takes 10 of 54 us.
#include "tree_attn.cuh"

namespace detfold_tree {
namespace {

constexpr int kWarps = 8;

// A CTA has rows of one sequence, so that what follows from the sequence is worked out once.
// LANES: of a row, each with PER groups of four places of the head. AHEAD: units whose accumulators a warp has in flight.
template <typename T, int LANES, int PER, int AHEAD, bool LOG2>
__global__ void __launch_bounds__(kWarps * 32) tree_join_kernel(const __grid_constant__ TreeWork w, int across)
{
    const TreeParams &p = w.p;
    const int lane = threadIdx.x % LANES;
    enter_grid();
    const int b = blockIdx.x / across, of = p.nodes * p.q_heads;
    const TreeSeq s = tree_seq_of(w, b);
    if (s.units <= 1) return;
    const int64_t step = (int64_t)s.pairs * w.slot_rows;
    // lengths that change under the call: no unit past the workspace
    const int units = min(s.units, over(w.slots, max(s.pairs, 1)));
    const int in = (blockIdx.x - b * across) * (kWarps * 32 / LANES) + threadIdx.x / LANES;
    if (in >= of) return;
    const int node = in / p.q_heads, head = in - node * p.q_heads;
    if (node >= s.c) return;
    const int kv = (int)quotient(head, w.by_heads), r = node * p.group + head - kv * p.group, block = r >> w.log_rows;
    const int pair = kv * s.blocks + block;
    const int64_t first = ((int64_t)b * w.slots + pair) * w.slot_rows + (r - block * w.rule.rows);
    float m = neg_inf(), l = 0.0f;
    float4 a[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) a[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int fours = p.head_dim / 4;
    for (int u0 = 0; u0 < units; u0 += AHEAD) {
        float2 ml[AHEAD];
        float4 x[AHEAD][PER];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (u0 + k >= units) continue;
            const int64_t at = first + (u0 + k) * step;
            ml[k] = w.ml[at];
            const float4 *acc = reinterpret_cast<const float4 *>(w.acc + at * p.head_dim);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + LANES * i < fours) x[k][i] = acc[lane + LANES * i];
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (u0 + k >= units) continue;
            float top, fa, fb;
            fold_factors<LOG2>(m, ml[k].x, top, fa, fb);
            m = top, l = fold_in(l, ml[k].y, fa, fb);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                a[i].x = fold_in(a[i].x, x[k][i].x, fa, fb), a[i].y = fold_in(a[i].y, x[k][i].y, fa, fb);
                a[i].z = fold_in(a[i].z, x[k][i].z, fa, fb), a[i].w = fold_in(a[i].w, x[k][i].w, fa, fb);
            }
        }
    }
    T *out = (T *)p.out + b * p.out_bs + node * p.out_ns + head * p.out_hs;
    const float inverse = inverse_of(l);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (lane + LANES * i >= fours) continue;
        Pack<T, 4> y;
        y.v[0] = quotient_of<T>(a[i].x, l, inverse), y.v[1] = quotient_of<T>(a[i].y, l, inverse);
        y.v[2] = quotient_of<T>(a[i].z, l, inverse), y.v[3] = quotient_of<T>(a[i].w, l, inverse);
        T *to = out + (lane + LANES * i) * 4;
        if (w.out_vec) {
            *reinterpret_cast<Pack<T, 4> *>(to) = y;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) to[k] = y.v[k];
        }
    }
    if (lane == 0 && p.lse) p.lse[(int64_t)b * of + in] = log_sum<LOG2>(m, l);
}

template <typename T, bool LOG2, int LANES, int PER, int AHEAD>
cudaError_t launch_lanes(const TreeWork &w, cudaStream_t stream)
{
    const int rows = kWarps * 32 / LANES, across = (w.p.nodes * w.p.q_heads + rows - 1) / rows;
    const dim3 grid((unsigned)((int64_t)w.p.batch * across));
    return launch_early(tree_join_kernel<T, LANES, PER, AHEAD, LOG2>, grid, kWarps * 32, 0, stream, w, across);
}

// What comes before the loads is as much as the rest: two rows a warp have it once. A batch of 32 sequences, 32 nodes of 32 heads of
// 128 each, takes 54.3 us with them, four units in flight, 55.5 with eight; 56.0 with a row a warp, 56.7 with four. Heads of 256 take
// a row a warp: 18.6 us for eight sequences in windows, 19.4 with two.
template <typename T, bool LOG2>
cudaError_t launch_type(const TreeWork &w, cudaStream_t stream)
{
    if (w.p.head_dim <= 64) return launch_lanes<T, LOG2, 16, 1, 8>(w, stream);
    if (w.p.head_dim <= 128) return launch_lanes<T, LOG2, 16, 2, 4>(w, stream);
    return launch_lanes<T, LOG2, 32, 2, 8>(w, stream);
}

}  // namespace

cudaError_t launch_tree_join(const TreeWork &w, int dtype, cudaStream_t stream)
{
    switch (dtype) {
    case DETFOLD_F32: return launch_type<float, false>(w, stream);
    case DETFOLD_BF16: return launch_type<__nv_bfloat16, true>(w, stream);
    default: return launch_type<__half, true>(w, stream);
    }
}

}  // namespace detfold_tree
