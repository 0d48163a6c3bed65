// Attention of one new token a sequence over a paged cache.
//
// Per query head: s_t = scale (q . k_t); with the running maximum m, p_t =
// exp(s_t - m), l = sum p_t, o = sum p_t v_t / l, in one pass over the cache.
#include "attn_common.cuh"

namespace detfold_attn {
namespace {

constexpr int kPerLane = DETFOLD_ATTN_MAX_HEAD_DIM / 32;

// One CTA a (sequence, query head): each warp takes every fourth token, lanes
// share the head's elements; the four warps' triples are joined in warp order.
template <typename T>
__global__ void __launch_bounds__(128) decode_kernel(const __grid_constant__ DecodeParams p)
{
    __shared__ float s_m[4], s_l[4], s_acc[4][DETFOLD_ATTN_MAX_HEAD_DIM];
    __shared__ int s_bad;
    const int b = blockIdx.x / p.q_heads, h = blockIdx.x % p.q_heads, hk = h / p.group;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, D = p.head_dim;
    const int n = p.lens[b];
    if (threadIdx.x == 0) s_bad = n < 0 || n > p.max_len;
    __syncthreads();
    float q[kPerLane], acc[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int d = lane + 32 * j;
        q[j] = d < D ? __fmul_rn(to_f32(((const T *)p.q)[b * p.q_bs + h * p.q_hs + d]), p.scale) : 0.0f;
        acc[j] = 0.0f;
    }
    float m = neg_inf(), l = 0.0f;
    const bool len_ok = n >= 0 && n <= p.max_len;
    const int64_t first = len_ok && n > p.window ? n - p.window : 0;
    for (int64_t t = first + warp; len_ok && t < n; t += 4) {
        const int64_t page = p.table[b * p.table_stride + t / p.page_size];
        if (page < 0 || page >= p.num_pages) {
            s_bad = 1;
            continue;
        }
        const int64_t at = page * p.page_stride + (t % p.page_size) * p.token_stride + hk * p.head_stride;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < kPerLane; ++j)
            if (lane + 32 * j < D) s = __fmaf_rn(q[j], to_f32(((const T *)p.k)[at + lane + 32 * j]), s);
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
        const float top = fmaxf(m, s), base = top == neg_inf() ? 0.0f : top;
        const float fade = expf(m - base), w = expf(s - base);
        l = __fmaf_rn(l, fade, w);
#pragma unroll
        for (int j = 0; j < kPerLane; ++j)
            if (lane + 32 * j < D)
                acc[j] = __fmaf_rn(acc[j], fade, w * to_f32(((const T *)p.v)[at + lane + 32 * j]));
        m = top;
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) s_acc[warp][lane + 32 * j] = acc[j];
    __syncthreads();
    float top = neg_inf();
    for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[w]);
    const float base = top == neg_inf() ? 0.0f : top;
    float total = 0.0f;
    for (int w = 0; w < 4; ++w) total = __fmaf_rn(s_l[w], expf(s_m[w] - base), total);
    if (s_bad) total = quiet_nan();
    for (int d = threadIdx.x; d < D; d += 128) {
        float o = 0.0f;
        for (int w = 0; w < 4; ++w) o = __fmaf_rn(s_acc[w][d], expf(s_m[w] - base), o);
        ((T *)p.out)[b * p.out_bs + h * p.out_hs + d] = from_f32<T>(total == 0.0f ? 0.0f : __fdiv_rn(o, total));
    }
    if (threadIdx.x == 0) {
        if (p.lse) p.lse[(int64_t)b * p.q_heads + h] = base + logf(total);
        if (s_bad) flag_bad_index(p.status);
    }
}

}  // namespace

cudaError_t launch_decode(const DecodeParams &p, int dtype, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.batch * p.q_heads)), block(128);
    switch (dtype) {
    case DETFOLD_F32: decode_kernel<float><<<grid, block, 0, stream>>>(p); break;
    case DETFOLD_BF16: decode_kernel<__nv_bfloat16><<<grid, block, 0, stream>>>(p); break;
    default: decode_kernel<__half><<<grid, block, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace detfold_attn
