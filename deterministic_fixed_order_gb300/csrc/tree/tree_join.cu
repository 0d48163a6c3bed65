// Joins the partial results of rows whose tokens lie in several units of work: a warp a row. The units'
// triples are folded in ascending order. Bound by memory and latency: each accumulator is read once, several in flight. In a batch of
// 32 sequences of 128 rows a key-value head it takes 10 of 56 us; with two or four rows a warp, one after the other, the batch
// took 2 and 5 us more.
#include "tree_attn.cuh"

namespace detfold_tree {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 8;  // units whose accumulators a warp has in flight

// A CTA has rows of one sequence, so that what follows from the sequence is worked out once.
// PER: groups of four places of the head that a lane has.
template <typename T, int PER, bool LOG2>
__global__ void __launch_bounds__(kWarps * 32) tree_join_kernel(const __grid_constant__ TreeWork w, int across)
{
    const TreeParams &p = w.p;
    const int lane = threadIdx.x % 32;
    enter_grid();
    const int b = blockIdx.x / across, of = p.nodes * p.q_heads;
    const TreeSeq s = tree_seq_of(w, b);
    if (s.units <= 1) return;
    const int64_t step = (int64_t)s.pairs * w.slot_rows;
    // lengths that change under the call: no unit past the workspace
    const int units = min(s.units, over(w.slots, max(s.pairs, 1)));
    const int in = (blockIdx.x - b * across) * kWarps + threadIdx.x / 32;
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
    for (int u0 = 0; u0 < units; u0 += kAhead) {
        float2 ml[kAhead];
        float4 x[kAhead][PER];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (u0 + k >= units) continue;
            const int64_t at = first + (u0 + k) * step;
            ml[k] = w.ml[at];
            const float4 *acc = reinterpret_cast<const float4 *>(w.acc + at * p.head_dim);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < fours) x[k][i] = acc[lane + 32 * i];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
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
        if (lane + 32 * i >= fours) continue;
        Pack<T, 4> y;
        y.v[0] = quotient_of<T>(a[i].x, l, inverse), y.v[1] = quotient_of<T>(a[i].y, l, inverse);
        y.v[2] = quotient_of<T>(a[i].z, l, inverse), y.v[3] = quotient_of<T>(a[i].w, l, inverse);
        T *to = out + (lane + 32 * i) * 4;
        if (w.out_vec) {
            *reinterpret_cast<Pack<T, 4> *>(to) = y;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) to[k] = y.v[k];
        }
    }
    if (lane == 0 && p.lse) p.lse[(int64_t)b * of + in] = log_sum<LOG2>(m, l);
}

template <typename T, bool LOG2>
cudaError_t launch_type(const TreeWork &w, cudaStream_t stream)
{
    const int across = (w.p.nodes * w.p.q_heads + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)((int64_t)w.p.batch * across));
    const auto kernel = w.p.head_dim <= 128 ? tree_join_kernel<T, 1, LOG2> : tree_join_kernel<T, 2, LOG2>;
    return launch_early(kernel, grid, kWarps * 32, 0, stream, w, across);
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
