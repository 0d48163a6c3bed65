// Rank-order join of W partial attentions.
//
// Per row: M = max lse_r, w_r = exp(lse_r - M), then two serial ascending
// chains, sum w_r and sum w_r part_r, in binary32. Bound by memory: every part
// is read once.
#include "attn_common.cuh"

namespace detfold_attn {
namespace {

// One warp a row.
template <typename T>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ JoinParams p)
{
    const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (row >= p.rows) return;
    const int lane = threadIdx.x % 32;
    float top = neg_inf();
    for (int r = 0; r < p.W; ++r) top = fmaxf(top, p.lses[r][row]);
    const float base = top == neg_inf() ? 0.0f : top;
    float total = 0.0f;
    for (int r = 0; r < p.W; ++r) total = __fadd_rn(total, expf(p.lses[r][row] - base));
    for (int d = lane; d < p.head_dim; d += 32) {
        float acc = 0.0f;
        for (int r = 0; r < p.W; ++r) {
            const float w = expf(p.lses[r][row] - base);
            if (!(w == 0.0f)) acc = __fmaf_rn(w, to_f32(((const T *)p.parts[r])[row * p.head_dim + d]), acc);
        }
        ((T *)p.out)[row * p.head_dim + d] = from_f32<T>(total == 0.0f ? 0.0f : __fdiv_rn(acc, total));
    }
    if (p.lse && lane == 0) p.lse[row] = base + logf(total);
}

}  // namespace

cudaError_t launch_join(const JoinParams &p, int dtype, cudaStream_t stream)
{
    const dim3 grid((unsigned)((p.rows + 3) / 4)), block(128);
    switch (dtype) {
    case DETFOLD_F32: join_kernel<float><<<grid, block, 0, stream>>>(p); break;
    case DETFOLD_BF16: join_kernel<__nv_bfloat16><<<grid, block, 0, stream>>>(p); break;
    default: join_kernel<__half><<<grid, block, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace detfold_attn
