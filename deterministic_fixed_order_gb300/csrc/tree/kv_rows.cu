// Rows and pages of a paged cache moved in place: an accepted path's rows to the end of the
// committed tokens, and whole pages. Copies of bytes, bound by memory: what moves is read and
// written once, by the widest accesses that pointers and strides allow.
#include "tree_common.cuh"

namespace detfold_tree {
namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 8;  // rows that a thread has in flight

// Elements of B bytes that are moved at once.
template <int B>
struct Bytes;
template <>
struct Bytes<2> { using type = uint16_t; };
template <>
struct Bytes<4> { using type = uint32_t; };
template <>
struct Bytes<8> { using type = uint2; };
template <>
struct Bytes<16> { using type = uint4; };

// A cache in units of B bytes.
struct Units {
    char *k, *v;
    int64_t page, token, head;  // strides in bytes
    int64_t a_head, a_row;      // units a head, units a row of all heads
};
Units units_of(const detfold_kv_cache &c, int es, int bytes)
{
    const int64_t a = (int64_t)c.head_dim * es / bytes;
    return {(char *)c.k, (char *)c.v, c.page_stride * es, c.token_stride * es, c.head_stride * es, a, a * c.kv_heads};
}

// The widest unit that divides a head and every address: a stride whose count is 1 is not used.
int widest(const detfold_kv_cache &c, int es)
{
    uint64_t all = (uint64_t)(uintptr_t)c.k | (uint64_t)(uintptr_t)c.v | (uint64_t)c.head_dim * es | 16;
    if (c.num_pages > 1) all |= (uint64_t)c.page_stride * es;
    if (c.page_size > 1) all |= (uint64_t)c.token_stride * es;
    if (c.kv_heads > 1) all |= (uint64_t)c.head_stride * es;
    return (int)(all & (0 - all));
}

// Row n + path[i] goes to row n + i, i ascending. A thread takes one place of the rows and all
// of the path there. Within a group of kFlight all are read before one is written; an earlier group wrote
// rows under n + i, and path[j] >= j >= i for the later ones, so every row is read as it was. Bound by latency: lengths, path, table
// and rows, the path with the lengths; 192 paths of 8 rows, 8 heads of 128 in 16 bits, take 3.1 us, one of 4 rows 2.2.
template <int B>
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactParams p, const Units u, const Divide by_page)
{
    using T = typename Bytes<B>::type;
    __shared__ int64_t s_from[DETFOLD_TREE_MAX_NODES], s_to[DETFOLD_TREE_MAX_NODES];
    enter_grid();
    const int b = blockIdx.x, tid = threadIdx.x;
    // asked for together; a path's numbers behind its length are not looked at
    const int32_t *path = p.path + b * p.path_stride;
    const int n = p.lens[b], count = p.path_lens[b], j = tid < p.max_path ? path[tid] : 0, before = tid && tid < p.max_path ? path[tid - 1] : -1;
    bool bad = n < 0 || n > DETFOLD_ATTN_MAX_LEN - DETFOLD_TREE_MAX_NODES || count < 0 || count > p.max_path;
    if (!bad && tid < count) {
        bad = j <= before || j >= DETFOLD_TREE_MAX_NODES;
        int64_t at[2] = {0, 0};
        if (!bad && j != tid) {
            const unsigned t[2] = {(unsigned)(n + j), (unsigned)(n + tid)};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const unsigned col = quotient(t[k], by_page);
                const int page = col < p.table_cols ? p.table[b * p.table_stride + col] : -1;
                if (page < 0 || page >= p.cache.num_pages) bad = true;
                at[k] = page * u.page + (int64_t)(t[k] - col * (unsigned)p.cache.page_size) * u.token;
            }
        }
        s_from[tid] = at[0], s_to[tid] = at[1];
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0 && blockIdx.y == 0) flag_bad_index(p.status);
        return;
    }
    // ascending from 0 on: what stays comes first
    int first = 0;
    while (first < count && s_from[first] == s_to[first]) ++first;
    for (int64_t place = (int64_t)blockIdx.y * kThreads + tid; place < 2 * u.a_row; place += (int64_t)gridDim.y * kThreads) {
        const bool value = place >= u.a_row;
        const int64_t in = place - (value ? u.a_row : 0), h = in / u.a_head;
        char *base = (value ? u.v : u.k) + h * u.head + (in - h * u.a_head) * B;
        for (int i0 = first; i0 < count; i0 += kFlight) {
            T x[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (i0 + i < count) x[i] = *reinterpret_cast<const T *>(base + s_from[i0 + i]);
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (i0 + i < count) *reinterpret_cast<T *>(base + s_to[i0 + i]) = x[i];
        }
    }
}

// How a page's rows lie: all one after the other, the rows of a head one after the other, or apart.
enum Lie { kPage, kHeads, kApart };

// Page src to page dst. A CTA takes a part of one pair's keys or values; threads go along the rows that lie side by
// side in memory. The next pair's numbers are read ahead of this one's rows.
template <int B, int LIE>
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ CopyParams p, const Units u, int parts)
{
    using T = typename Bytes<B>::type;
    enter_grid();
    const int64_t units = p.count * 2 * parts;
    struct Pair {
        int src, dst, rows;
    };
    const auto look = [&](int64_t w) {
        Pair x = {-1, -1, 0};
        if (w < units) {
            const int64_t i = w / (2 * parts);
            x = {p.src[i], p.dst[i], p.rows ? p.rows[i] : p.cache.page_size};
        }
        return x;
    };
    Pair next = look(blockIdx.x);
    for (int64_t w = blockIdx.x; w < units; w += gridDim.x) {
        const int64_t i = w / (2 * parts);
        const int rest = (int)(w - i * 2 * parts), part = rest >> 1;
        const Pair now = next;
        next = look(w + gridDim.x);
        if (now.src < 0 || now.dst < 0 || now.src == now.dst) continue;
        if (now.src >= p.cache.num_pages || now.dst >= p.cache.num_pages || now.rows < 0 || now.rows > p.cache.page_size) {
            if (threadIdx.x == 0 && rest == 0) flag_bad_index(p.status);
            continue;
        }
        const char *from = (rest & 1 ? u.v : u.k) + now.src * u.page;
        char *to = (rest & 1 ? u.v : u.k) + now.dst * u.page;
        const unsigned rows = (unsigned)now.rows, total = rows * (unsigned)u.a_row;  // units of this pair
        const auto place = [&](unsigned x) -> int64_t {
            if (LIE == kPage) return (int64_t)x * B;
            const unsigned a = (unsigned)u.a_head;
            if (LIE == kHeads) {
                const unsigned line = rows * a, h = x / line;
                return h * u.head + (int64_t)(x - h * line) * B;
            }
            const unsigned t = x / a, row = t / (unsigned)p.cache.kv_heads;
            return row * u.token + (t - row * (unsigned)p.cache.kv_heads) * u.head + (int64_t)(x - t * a) * B;
        };
        const unsigned step = parts * kThreads;
        for (unsigned x0 = part * kThreads + threadIdx.x; x0 < total; x0 += step * kFlight) {
            T x[kFlight];
#pragma unroll
            for (int j = 0; j < kFlight; ++j)
                if (x0 + j * step < total) x[j] = *reinterpret_cast<const T *>(from + place(x0 + j * step));
#pragma unroll
            for (int j = 0; j < kFlight; ++j)
                if (x0 + j * step < total) *reinterpret_cast<T *>(to + place(x0 + j * step)) = x[j];
        }
    }
}

template <int B>
cudaError_t compact(const CompactParams &p, int es, cudaStream_t stream)
{
    const Units u = units_of(p.cache, es, B);
    const int64_t across = (2 * u.a_row + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)p.batch, (unsigned)(across < 65535 ? across : 65535));
    return launch_early(compact_kernel<B>, grid, kThreads, 0, stream, p, u, divide_by(p.cache.page_size));
}

template <int B>
cudaError_t copy(const CopyParams &p, int es, cudaStream_t stream)
{
    const Units u = units_of(p.cache, es, B);
    const detfold_kv_cache &c = p.cache;
    const bool heads = c.kv_heads == 1 || c.head_stride == c.head_dim;  // a row's heads side by side
    const bool tokens = c.page_size == 1 || c.token_stride == c.head_dim;  // a head's rows side by side
    const bool page = heads && (c.page_size == 1 || c.token_stride == (int64_t)c.kv_heads * c.head_dim);
    const int64_t units = (int64_t)c.page_size * u.a_row;
    const int parts = (int)((units + kThreads * kFlight - 1) / (kThreads * kFlight));
    // 2047 pages of 32 KB and 32 KB: 41.6 us (95% of the measured copy rate); 42.7 with half the CTAs, 46.3 with a quarter
    const int64_t need = p.count * 2 * parts, most = kSms * 16;
    const dim3 grid((unsigned)(need < most ? need : most));
    const auto kernel = page ? copy_kernel<B, kPage> : tokens ? copy_kernel<B, kHeads> : copy_kernel<B, kApart>;
    return launch_early(kernel, grid, kThreads, 0, stream, p, u, parts);
}

}  // namespace

cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream)
{
    const int es = p.cache.dtype == DETFOLD_F32 ? 4 : 2;
    switch (widest(p.cache, es)) {
    case 16: return compact<16>(p, es, stream);
    case 8: return compact<8>(p, es, stream);
    case 4: return compact<4>(p, es, stream);
    default: return compact<2>(p, es, stream);
    }
}

cudaError_t launch_copy(const CopyParams &p, cudaStream_t stream)
{
    const int es = p.cache.dtype == DETFOLD_F32 ? 4 : 2;
    switch (widest(p.cache, es)) {
    case 16: return copy<16>(p, es, stream);
    case 8: return copy<8>(p, es, stream);
    case 4: return copy<4>(p, es, stream);
    default: return copy<2>(p, es, stream);
    }
}

}  // namespace detfold_tree
