// Append to a paged cache with the position rotation on the way.
//
// Per pair (a, b) of a head's rotated elements: (a cos - b sin, b cos + a sin),
// each as one rounded product and one fused multiply-add in binary32, then one
// rounding to the element type. Everything else is a copy. Bound by memory.
#include "attn_common.cuh"

namespace detfold_attn {
namespace {

// One CTA a token; a thread takes whole pairs (or single copied elements) of
// the token's query, key and value heads in turn.
template <typename T>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p)
{
    const int64_t t = blockIdx.x;
    const detfold_kv_cache &c = p.cache;
    const int D = c.head_dim, half = p.rot_dim / 2, units = D - half;  // pairs, then single elements
    const int64_t slot = p.slots[t];
    const int64_t page = slot / c.page_size;
    const bool keep = slot >= 0 && page < c.num_pages;
    if (slot >= 0 && !keep && threadIdx.x == 0) flag_bad_index(p.status);
    const int64_t dst = keep ? page * c.page_stride + (slot % c.page_size) * c.token_stride : 0;
    const float *cs = nullptr;
    bool rotate_ok = true;
    if (p.cos_sin) {
        const int64_t pos = p.positions[t];
        rotate_ok = pos >= 0 && pos < p.rope_rows;
        if (!rotate_ok && threadIdx.x == 0) flag_bad_index(p.status);
        cs = p.cos_sin + (rotate_ok ? pos : 0) * p.rot_dim;
    }
    const int64_t total = (int64_t)(p.q_heads + 2 * c.kv_heads) * units;
    for (int64_t i = threadIdx.x; i < total; i += blockDim.x) {
        int row = (int)(i / units);
        const int u = (int)(i % units);
        const T *from;
        T *to;
        bool turn = u < half;
        if (row < p.q_heads) {
            from = (const T *)p.q + t * p.q_ts + row * p.q_hs;
            to = (T *)p.q_out + t * p.qo_ts + row * p.qo_hs;
        } else if (!keep) {
            continue;
        } else if (row < p.q_heads + c.kv_heads) {
            row -= p.q_heads;
            from = (const T *)p.k + t * p.k_ts + row * p.k_hs;
            to = (T *)c.k + dst + row * c.head_stride;
        } else {
            row -= p.q_heads + c.kv_heads;
            from = (const T *)p.v + t * p.v_ts + row * p.v_hs;
            to = (T *)c.v + dst + row * c.head_stride;
            turn = false;
        }
        if (u < half) {
            const int ia = p.interleaved ? 2 * u : u, ib = p.interleaved ? 2 * u + 1 : u + half;
            const T ra = from[ia], rb = from[ib];
            if (turn) {
                const float a = to_f32(ra), b = to_f32(rb);
                const float co = rotate_ok ? cs[u] : quiet_nan(), si = rotate_ok ? cs[half + u] : quiet_nan();
                to[ia] = from_f32<T>(__fmaf_rn(a, co, -__fmul_rn(b, si)));
                to[ib] = from_f32<T>(__fmaf_rn(b, co, __fmul_rn(a, si)));
            } else {
                to[ia] = ra;
                to[ib] = rb;
            }
        } else {
            to[half + u] = from[half + u];
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)p.tokens), block(256);
    switch (p.cache.dtype) {
    case DETFOLD_F32: append_kernel<float><<<grid, block, 0, stream>>>(p); break;
    case DETFOLD_BF16: append_kernel<__nv_bfloat16><<<grid, block, 0, stream>>>(p); break;
    default: append_kernel<__half><<<grid, block, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace detfold_attn
