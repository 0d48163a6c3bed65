// Rank-order join of W partial attentions.
//
// Per row: M = max lse_r, w_r = exp(lse_r - M), then two serial ascending
// chains, sum w_r and sum w_r part_r, in binary32.
//
// Bound by memory: each part is read once. A thread takes N neighbouring
// elements of a row -- the widest access that every operand's address and the row
// allow -- and has up to eight ranks' elements in flight; the row's weights are
// worked out by each of its threads again (one exponential a rank and access).
#include <type_traits>

#include "attn_common.cuh"

namespace detfold_attn {
namespace {

constexpr int kMost = 128;  // threads a CTA, at most
constexpr int kRanks = 8;   // ranks whose elements a thread has in flight
// CTAs an SM, which go from row to row: as many as have registers for the ranks' elements (but
// for 4 bytes of spills at two ranks of bfloat16 and 12 at one of float32). 131168 rows of 128
// bfloat16 from 8 ranks: 47.2 us (96% of the measured copy rate); 50.6 us with a CTA a row's
// worth, 54 with a division an element, 86 with seven CTAs an SM, which spill more.
constexpr int resident(int ranks) { return ranks == 0 ? 5 : ranks <= 2 ? 12 : ranks <= 4 ? 8 : 5; }

// Keeps the widening of 16-bit elements here: done as they arrive it takes twice their registers, which
// then spill. 32768 rows of 128 bfloat16 from 16 ranks: 27 us; 52 without, and 42 with eight ranks
// loaded, folded, and then the next eight.
template <typename V>
__device__ __forceinline__ void as_read(V &x)
{
    if constexpr (sizeof(V) == 16) {
        uint4 &u = reinterpret_cast<uint4 &>(x);
        asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w));
    }
}

// What the kernel is given: with up to kRanks ranks a small table, a quarter of a microsecond less of a
// launch's time than the largest.
template <int MOST>
struct Ranks {
    void *out;
    float *lse;
    const void *parts[MOST];
    const float *lses[MOST];
    int64_t rows;
    int W, head_dim;
};
constexpr int most_ranks(int W) { return W ? kRanks : DETFOLD_MAX_W; }

// W == 0: any number of ranks, kRanks at a time; else exactly W <= kRanks.
// `places` accesses a row, `abreast` of them at a time.
template <typename T, int N, int W>
__global__ void __launch_bounds__(kMost, resident(W)) join_kernel(const __grid_constant__ Ranks<most_ranks(W)> p,
                                                                       int places, int abreast)
{
    using V = Pack<T, N>;
    constexpr int R = W ? W : kRanks;
    const int world = W ? W : p.W;
    const int first = threadIdx.x % abreast, rows = blockDim.x / abreast;
    enter_grid();
    for (int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / abreast; row < p.rows;
         row += (int64_t)gridDim.x * rows) {
        const auto place = [&](int u) { return row * p.head_dim + (int64_t)u * N; };
        V x[R];
        const auto load = [&](int r, int rank, int64_t at) {
            if (rank < world) x[r] = *reinterpret_cast<const V *>((const T *)p.parts[rank] + at);
        };
        float lse[R];
        const auto weigh = [&](int r, int rank) { lse[r] = rank < world ? p.lses[rank][row] : neg_inf(); };
        // the elements do not need the weights: asked for first
#pragma unroll
        for (int r = 0; r < R; ++r) load(r, r, place(first));
        float top = neg_inf();
        for (int r0 = (world - 1) / R * R; r0 >= 0; r0 -= R) {  // ends with the first ranks' in hand
#pragma unroll
            for (int r = 0; r < R; ++r) weigh(r, r0 + r);
#pragma unroll
            for (int r = 0; r < R; ++r) top = fmaxf(top, lse[r]);
        }
        const float base = base_of(top);
        for (int u = first; u < places; u += abreast) {
            const int64_t at = place(u);
            float total = 0.0f, acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.0f;
            if (u != first) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    load(r, r, at);
                    if (W == 0) weigh(r, r);
                }
            }
            for (int r0 = 0; r0 < world; r0 += R) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float w = exp_neg(__fsub_rn(lse[r], base));
                    total = __fadd_rn(total, w);
                    // no weight: whatever the part holds stays out
                    if (!(w == 0.0f)) {
                        if (W == 0) as_read(x[r]);
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[i] = __fmaf_rn(w, to_f32(x[r].v[i]), acc[i]);
                    }
                    if (W == 0) {  // its place goes to the rank kRanks further on
                        load(r, r0 + R + r, at);
                        weigh(r, r0 + R + r);
                    }
                }
            }
            V y;
            // 16-bit results: one reciprocal a row, its half unit in the last place of binary32 far below theirs
            const float inv = total == 0.0f ? 0.0f : __frcp_rn(total);
#pragma unroll
            for (int i = 0; i < N; ++i)
                y.v[i] = from_f32<T>(sizeof(T) == 2     ? __fmul_rn(acc[i], inv)
                                     : total == 0.0f ? 0.0f
                                                     : __fdiv_rn(acc[i], total));
            *reinterpret_cast<V *>((T *)p.out + at) = y;
            if (u == 0 && p.lse) p.lse[row] = __fadd_rn(base, logf(total));
        }
    }
}

// Whether every operand can be accessed N elements at a time.
bool fits(const JoinParams &p, int es, int n)
{
    if (p.head_dim % n || (uintptr_t)p.out % (uintptr_t)(es * n)) return false;
    for (int r = 0; r < p.W; ++r)
        if ((uintptr_t)p.parts[r] % (uintptr_t)(es * n)) return false;
    return true;
}

template <typename T, int N>
cudaError_t launch_packs(const JoinParams &p, cudaStream_t stream)
{
    const int places = p.head_dim / N, abreast = places < kMost ? places : kMost, rows = kMost / abreast;
    const int64_t need = (p.rows + rows - 1) / rows, most = 152 * resident(p.W <= kRanks ? p.W : 0);
    const dim3 grid((unsigned)(need < most ? need : most));
    const auto launch = [&](auto world) {
        constexpr int W = decltype(world)::value;
        Ranks<most_ranks(W)> ranks;
        ranks.out = p.out, ranks.lse = p.lse, ranks.rows = p.rows, ranks.W = p.W, ranks.head_dim = p.head_dim;
        for (int r = 0; r < p.W; ++r) ranks.parts[r] = p.parts[r], ranks.lses[r] = p.lses[r];
        return launch_early(join_kernel<T, N, W>, grid, rows * abreast, 0, stream, ranks, places, abreast);
    };
    switch (p.W) {
    case 1: return launch(std::integral_constant<int, 1>());
    case 2: return launch(std::integral_constant<int, 2>());
    case 3: return launch(std::integral_constant<int, 3>());
    case 4: return launch(std::integral_constant<int, 4>());
    case 5: return launch(std::integral_constant<int, 5>());
    case 6: return launch(std::integral_constant<int, 6>());
    case 7: return launch(std::integral_constant<int, 7>());
    case 8: return launch(std::integral_constant<int, 8>());
    default: return launch(std::integral_constant<int, 0>());
    }
}

template <typename T>
cudaError_t launch_type(const JoinParams &p, cudaStream_t stream)
{
    constexpr int wide = 16 / sizeof(T);
    return fits(p, sizeof(T), wide) ? launch_packs<T, wide>(p, stream) : launch_packs<T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_join(const JoinParams &p, int dtype, cudaStream_t stream)
{
    switch (dtype) {
    case DETFOLD_F32: return launch_type<float>(p, stream);
    case DETFOLD_BF16: return launch_type<__nv_bfloat16>(p, stream);
    default: return launch_type<__half>(p, stream);
    }
}

}  // namespace detfold_attn
