// Append to a paged cache with the position rotation on the way.
//
// Per pair (a, b) of a head's rotated elements: (a cos - b sin, b cos + a sin),
// each as one rounded product and one fused multiply-add in binary32, then one
// rounding to the element type. Everything else is a copy.
//
// Bound by memory: a token's queries, keys and values are read and written
// once. A token is one column of the grid; a thread keeps one place in the head
// -- N elements and the N that they turn with -- and takes head after head there,
// so it reads the cosines and sines of its place once for all heads. N is the
// widest access that every operand's address and stride allow.
#include "attn_common.cuh"

namespace detfold_attn {
namespace {

constexpr int kMost = 256;  // threads a CTA, at most
constexpr int kAhead = 4;   // heads whose elements a thread has in flight

// `units` places a head: first those of pairs, then those of single copies.
template <typename T, int N, bool PAIRS>
__global__ void __launch_bounds__(kMost) append_kernel(const __grid_constant__ AppendParams p, int units)
{
    using V = Pack<T, N>;
    const detfold_kv_cache &c = p.cache;
    const int half = p.rot_dim / 2, turning = half / N;
    const int abreast = min(units, kMost), rows = p.q_heads + 2 * c.kv_heads;
    const int step = blockDim.x / abreast * gridDim.y;
    const int64_t t = blockIdx.x;
    enter_grid();
    // one place a thread, several only in heads of more than kMost places
    for (int u = threadIdx.x % abreast; u < units; u += abreast) {
        // this place's elements: [ia, ia + N) and, where they turn, [ib, ib + N)
        const bool turns = u < turning;
        const int ia = !turns ? half + u * N : PAIRS ? 2 * u * N : u * N;
        const int ib = PAIRS ? ia + N : ia + half;
        const int64_t slot = p.slots[t];
        float co[N], si[N];
        bool known = true;
        if (turns) {
            const int64_t pos = p.positions[t];
            known = pos >= 0 && pos < p.rope_rows;
            const float *row = p.cos_sin + (known ? pos : 0) * p.rot_dim + u * N;
            constexpr int F = N < 4 ? N : 4;
#pragma unroll
            for (int j = 0; j < N; j += F) {
                const Pack<float, F> x = *reinterpret_cast<const Pack<float, F> *>(row + j);
                const Pack<float, F> y = *reinterpret_cast<const Pack<float, F> *>(row + half + j);
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    co[j + i] = known ? x.v[i] : quiet_nan();
                    si[j + i] = known ? y.v[i] : quiet_nan();
                }
            }
        }
        int64_t page, at;
        if (slot >= 0 && slot < ((int64_t)1 << 30)) {
            page = quotient((unsigned)slot, p.page);
            at = (unsigned)slot - (unsigned)page * (unsigned)c.page_size;
        } else {
            page = slot / c.page_size;
            at = slot % c.page_size;
        }
        const bool keep = slot >= 0 && page < c.num_pages;
        if (((slot >= 0 && !keep) || !known) && u == (int)threadIdx.x && blockIdx.y == 0) flag_bad_index(p.status);
        const int64_t dst = keep ? page * c.page_stride + at * c.token_stride : 0;

        const T *q = (const T *)p.q + t * p.q_ts, *k = (const T *)p.k + t * p.k_ts, *v = (const T *)p.v + t * p.v_ts;
        T *qo = (T *)p.q_out + t * p.qo_ts, *ck = (T *)c.k + dst, *cv = (T *)c.v + dst;
        const int last = keep ? rows : p.q_heads;
        for (int r0 = (blockIdx.y * blockDim.x + threadIdx.x) / abreast; r0 < last; r0 += kAhead * step) {
            V a[kAhead], b[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int r = r0 + j * step;
                if (r >= last) break;
                const T *from = r < p.q_heads               ? q + r * p.q_hs
                                : r < p.q_heads + c.kv_heads ? k + (r - p.q_heads) * p.k_hs
                                                             : v + (r - p.q_heads - c.kv_heads) * p.v_hs;
                a[j] = *reinterpret_cast<const V *>(from + ia);
                if (turns) b[j] = *reinterpret_cast<const V *>(from + ib);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int r = r0 + j * step;
                if (r >= last) break;
                T *to = r < p.q_heads               ? qo + r * p.qo_hs
                        : r < p.q_heads + c.kv_heads ? ck + (r - p.q_heads) * c.head_stride
                                                     : cv + (r - p.q_heads - c.kv_heads) * c.head_stride;
                if (turns && r < p.q_heads + c.kv_heads) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        // a pair: the same element of both packs, or two neighbours of one after the other
                        T &first = PAIRS ? (2 * i < N ? a[j].v[2 * i] : b[j].v[2 * i - N]) : a[j].v[i];
                        T &second = PAIRS ? (2 * i + 1 < N ? a[j].v[2 * i + 1] : b[j].v[2 * i + 1 - N]) : b[j].v[i];
                        const float x = to_f32(first), y = to_f32(second);
                        first = from_f32<T>(__fmaf_rn(x, co[i], -__fmul_rn(y, si[i])));
                        second = from_f32<T>(__fmaf_rn(y, co[i], __fmul_rn(x, si[i])));
                    }
                }
                *reinterpret_cast<V *>(to + ia) = a[j];
                if (turns) *reinterpret_cast<V *>(to + ib) = b[j];
            }
        }
    }
}

// Whether every operand can be accessed N elements at a time.
bool fits(const AppendParams &p, int es, int n)
{
    const detfold_kv_cache &c = p.cache;
    const int half = p.rot_dim / 2;
    if (half % n || c.head_dim % n) return false;
    for (const void *x : {(const void *)c.k, (const void *)c.v, p.k, p.v, p.q, (const void *)p.q_out})
        if ((uintptr_t)x % (uintptr_t)(es * n)) return false;
    for (int64_t s : {c.page_stride, c.token_stride, c.head_stride, p.k_ts, p.k_hs, p.v_ts, p.v_hs, p.q_ts, p.q_hs,
                      p.qo_ts, p.qo_hs})
        if (s % n) return false;
    return (uintptr_t)p.cos_sin % (4 * (n < 4 ? n : 4)) == 0;
}

template <typename T, int N>
cudaError_t launch_packs(const AppendParams &p, cudaStream_t stream)
{
    const detfold_kv_cache &c = p.cache;
    const int units = p.rot_dim / 2 / N + (c.head_dim - p.rot_dim) / N;
    const int rows = p.q_heads + 2 * c.kv_heads;
    const int abreast = units < kMost ? units : kMost;
    // whole heads a CTA: a thread stays at its place
    int heads = kMost / abreast;
    heads = heads > rows ? rows : heads;
    // a few tokens: their heads spread over more CTAs, one head a thread
    int across = (double)p.tokens * rows * units < 152 * 1024 ? (rows + heads - 1) / heads : 1;
    across = across > 1024 ? 1024 : across;
    const dim3 grid((unsigned)p.tokens, (unsigned)across);
    return p.interleaved ? launch_early(append_kernel<T, N, true>, grid, heads * abreast, 0, stream, p, units)
                         : launch_early(append_kernel<T, N, false>, grid, heads * abreast, 0, stream, p, units);
}

template <typename T>
cudaError_t launch_type(const AppendParams &p, cudaStream_t stream)
{
    constexpr int es = sizeof(T);
    if constexpr (es == 2)
        if (fits(p, es, 8)) return launch_packs<T, 8>(p, stream);
    if (fits(p, es, 4)) return launch_packs<T, 4>(p, stream);
    if (fits(p, es, 2)) return launch_packs<T, 2>(p, stream);
    return launch_packs<T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream)
{
    switch (p.cache.dtype) {
    case DETFOLD_F32: return launch_type<float>(p, stream);
    case DETFOLD_BF16: return launch_type<__nv_bfloat16>(p, stream);
    default: return launch_type<__half>(p, stream);
    }
}

}  // namespace detfold_attn
