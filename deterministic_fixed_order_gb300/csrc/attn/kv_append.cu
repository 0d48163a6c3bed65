// Append to a paged cache with the position rotation on the way.
//
// Per pair (a, b) of a head's rotated elements: (a cos - b sin, b cos + a sin),
// each as one rounded product and one fused multiply-add in binary32, then one
// rounding to the element type. Everything else is a copy.
//
// Bound by memory: a token's queries, keys and values are read and written
// once. A team of threads takes token after token; a thread keeps one place in the head --
// N elements and the N that they turn with -- and takes head after head there, so
// it reads the cosines and sines of its place once for all heads. N is the widest
// access that every operand's address and stride allow. The next token's slot and
// position are read one token ahead, so that its elements and its cosines are
// asked for together: one load's latency a token, not three in a row. 16381 tokens of
// 32 query and 8 key-value heads of 128 bfloat16: 65 us, 93% of the measured copy rate. (Six CTAs an SM leave its kernel 80
// registers a thread and 28 bytes of spills; with five, and none, 64.4 us for 64.5.)
#include "attn_common.cuh"

namespace detfold_attn {
namespace {

constexpr int kMost = 128;  // threads a CTA, at most
constexpr int kAhead = 3;   // heads whose elements a thread has in flight: 65 us below, 71 with two, 90 with four

// Where a token's heads are read and written: queries, then keys, then values.
template <typename T>
struct Heads {
    const T *q, *k, *v;
    T *qo, *ck, *cv;

    __device__ __forceinline__ const T *from(const AppendParams &p, int r) const
    {
        const int hk = p.cache.kv_heads;
        return r < p.q_heads ? q + r * p.q_hs : r < p.q_heads + hk ? k + (r - p.q_heads) * p.k_hs
                                                                   : v + (r - p.q_heads - hk) * p.v_hs;
    }
    __device__ __forceinline__ T *to(const AppendParams &p, int r) const
    {
        const int hk = p.cache.kv_heads;
        return r < p.q_heads ? qo + r * p.qo_hs : r < p.q_heads + hk ? ck + (r - p.q_heads) * p.cache.head_stride
                                                                     : cv + (r - p.q_heads - hk) * p.cache.head_stride;
    }
};

// Turns the pairs of a place: element i of `a` with element i of `b`, or
// neighbours with each other, `a` followed by `b`.
template <typename T, int N, bool PAIRS>
__device__ __forceinline__ void rotate(T *a, T *b, const float *co, const float *si)
{
    if constexpr (N == 1) {
        const float x = to_f32(a[0]), y = to_f32(b[0]);
        a[0] = from_f32<T>(__fmaf_rn(x, co[0], -__fmul_rn(y, si[0])));
        b[0] = from_f32<T>(__fmaf_rn(y, co[0], __fmul_rn(x, si[0])));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            // pairs i and i + 1
            T *p0 = PAIRS ? (2 * i < N ? a + 2 * i : b + 2 * i - N) : a + i;
            T *p1 = PAIRS ? (2 * i + 2 < N ? a + 2 * i + 2 : b + 2 * i + 2 - N) : b + i;
            const float2 u = to_f32x2(p0), v = to_f32x2(p1);
            const float2 x = PAIRS ? make_float2(u.x, v.x) : u, y = PAIRS ? make_float2(u.y, v.y) : v;
            const float2 c = make_float2(co[i], co[i + 1]), s = make_float2(si[i], si[i + 1]);
            const float2 ys = mul2(y, s), xs = mul2(x, s);
            const float2 d = fma2(x, c, make_float2(-ys.x, -ys.y)), e = fma2(y, c, xs);
            from_f32x2(p0, PAIRS ? make_float2(d.x, e.x) : d);
            from_f32x2(p1, PAIRS ? make_float2(d.y, e.y) : e);
        }
    }
}

// `units` places a head: first those of pairs, then those of copies, which take `twos` of N
// elements or one. `team` threads take a token together.
template <typename T, int N, bool PAIRS>
__global__ void __launch_bounds__(kMost, 6) append_kernel(const __grid_constant__ AppendParams p, int units,
                                                           int team, bool twos)
{
    using V = Pack<T, N>;
    const detfold_kv_cache &c = p.cache;
    const int half = p.rot_dim / 2, turning = half / N;
    const int abreast = min(units, kMost), rows = p.q_heads + 2 * c.kv_heads;
    const int member = threadIdx.x % team, teams = blockDim.x / team;
    const int step = team / abreast * gridDim.y;
    const int first = (blockIdx.y * team + member) / abreast;
    enter_grid();
    const int64_t t0 = (int64_t)blockIdx.x * teams + threadIdx.x / team, apart = (int64_t)gridDim.x * teams;
    int64_t slot = t0 < p.tokens ? p.slots[t0] : -1, pos = t0 < p.tokens && p.cos_sin ? p.positions[t0] : 0;
    for (int64_t t = t0; t < p.tokens; t += apart) {
        const int64_t next = t + apart;
        const int64_t next_slot = next < p.tokens ? p.slots[next] : -1;
        const int64_t next_pos = next < p.tokens && p.cos_sin ? p.positions[next] : 0;
        Heads<T> heads;
        heads.q = (const T *)p.q + t * p.q_ts;
        heads.k = (const T *)p.k + t * p.k_ts;
        heads.v = (const T *)p.v + t * p.v_ts;
        heads.qo = (T *)p.q_out + t * p.qo_ts;
        // one place a thread, several only in heads of more than kMost places
        for (int u = member % abreast; u < units; u += abreast) {
            // this place's elements: [ia, ia + N) and, where they turn or are copied by twos, [ib, ib + N)
            const bool turns = u < turning, two = turns || twos;
            const int ia = !turns ? p.rot_dim + (u - turning) * (twos ? 2 * N : N) : PAIRS ? 2 * u * N : u * N;
            const int ib = PAIRS || !turns ? ia + N : ia + half;
            V a[kAhead], b[kAhead];
            auto load = [&](int r0) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (r0 + j * step < rows) {
                        const T *from = heads.from(p, r0 + j * step);
                        a[j] = *reinterpret_cast<const V *>(from + ia);
                        if (two) b[j] = *reinterpret_cast<const V *>(from + ib);
                    }
            };
            load(first);
            float co[N], si[N];
            bool known = true;
            if (turns) {
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
            if (((slot >= 0 && !keep) || !known) && u == member && blockIdx.y == 0) flag_bad_index(p.status);
            const int64_t dst = keep ? page * c.page_stride + at * c.token_stride : 0;
            heads.ck = (T *)c.k + dst;
            heads.cv = (T *)c.v + dst;
            const int last = keep ? rows : p.q_heads;  // a token without a place: its queries only
            for (int r0 = first; r0 < last; r0 += kAhead * step) {
                if (r0 != first) load(r0);
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int r = r0 + j * step;
                    if (r >= last) break;
                    if (turns && r < p.q_heads + c.kv_heads) rotate<T, N, PAIRS>(a[j].v, b[j].v, co, si);
                    T *to = heads.to(p, r);
                    *reinterpret_cast<V *>(to + ia) = a[j];
                    if (two) *reinterpret_cast<V *>(to + ib) = b[j];
                }
            }
        }
        slot = next_slot;
        pos = next_pos;
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
    const int copied = c.head_dim - p.rot_dim;
    const bool twos = copied % (2 * N) == 0;
    const int units = p.rot_dim / 2 / N + copied / (twos ? 2 * N : N);
    const int rows = p.q_heads + 2 * c.kv_heads;
    const int abreast = units < kMost ? units : kMost;
    // whole heads a CTA: a thread stays at its place. A few tokens spread a head a
    // thread over as many CTAs as that takes; many give each thread several heads,
    // which share what a token costs anyway. (One token of 48 heads of 128: 2.0 us, 3.5 as if of many;
    // 16381 of them 110 us as if of few.)
    const int widest = kMost / abreast;
    const bool few = (double)p.tokens * rows * units < 152 * 1024;
    // Of many tokens a thread takes as many heads as it has in flight, 65 us for those 16381 (67.4 with
    // twice as many, 73.8 with four times); twice as many where an eighth of the places would stay
    // empty: 80078 tokens of 10 heads 74.7 us for 77.8, 400390 of 4 heads of 64 83.0 for 90.6.
    const auto by = [&](int heads_a_thread) { return (rows + heads_a_thread - 1) / heads_a_thread; };
    int heads = few ? rows : by(kAhead);
    if (!few && 8 * rows < 7 * kAhead * heads) heads = by(2 * kAhead);
    heads = heads > widest ? widest : heads;
    int across = few ? (rows + heads - 1) / heads : 1;
    across = across > 1024 ? 1024 : across;
    const int team = heads * abreast, teams = few ? 1 : kMost / team, threads = team * teams;
    // as many CTAs as are resident at 80 registers a thread
    const int64_t ctas = (p.tokens + teams - 1) / teams, resident = 152 * (65536 / 80 / ((threads + 31) / 32 * 32));
    const dim3 grid((unsigned)(ctas < resident ? ctas : resident), (unsigned)across);
    return p.interleaved ? launch_early(append_kernel<T, N, true>, grid, threads, 0, stream, p, units, team, twos)
                         : launch_early(append_kernel<T, N, false>, grid, threads, 0, stream, p, units, team, twos);
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
