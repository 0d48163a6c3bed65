// The bookkeeping of a pool of pages between two steps, in one launch of one cluster.
//
// Counts are whole numbers, so the atomics' order does not show. What is given out does not
// depend on it either: the free pages' numbers in ascending order go to the rows in ascending
// order, found by counting the free pages of each part of the pool and the needs of each row.
//
// Phases, with the whole cluster meeting between them:
//   1. the counts are copied (unless they are changed in place);
//   2. old rows' pages are released, kept pages counted, and kept pages written to the new table. A
//      row that goes on in its own place only releases what it does not keep;
//   3. each CTA works out every row's need and its sum over the rows before (the same in each), and counts
//      the free pages of its part of the pool;
//   4. each CTA hands out its part's free pages, and rows leave the pages that they copy.
// Bound by latency: a few loads and atomics a phase, each phase a barrier of the cluster. The
// counts are read past the L1, since other SMs change them.
#include "tree_common.cuh"

namespace detfold_tree {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kRows = DETFOLD_PAGES_MAX_ROWS;
constexpr int kEach = kRows / kThreads;

__device__ __forceinline__ void meet()
{
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// A new row: where it comes from and what it keeps. A row that does not make sense is empty.
struct Row {
    int origin, keep, want, kept, pages;  // `kept` columns kept, `pages` in the end
    bool bad;
};

__device__ __forceinline__ int up(int tokens, int page) { return (int)(((int64_t)tokens + page - 1) / page); }

// Tokens of an old row, or -1.
__device__ __forceinline__ int old_len(const PagesParams &p, int f)
{
    const int n = p.lens[f];
    return n >= 0 && n <= (int64_t)p.cols * p.page_size ? n : -1;
}

__device__ __forceinline__ Row row_of(const PagesParams &p, int b)
{
    Row r = {p.origin[b], p.keep[b], p.want[b], 0, 0, false};
    int most = 0;
    if (r.origin >= 0 && r.origin < p.rows_in) most = max(old_len(p, r.origin), 0);
    r.bad = r.origin < -1 || r.origin >= p.rows_in || r.keep < 0 || r.keep > most || r.want < r.keep ||
            r.want > (int64_t)p.cols * p.page_size;
    if (r.bad) r.origin = -1, r.keep = 0, r.want = 0;
    r.kept = up(r.keep, p.page_size);
    r.pages = up(r.want, p.page_size);
    return r;
}

// A held page, or -1 where the table's entry is none.
__device__ __forceinline__ int page_at(const PagesParams &p, int f, int col)
{
    const int page = p.table[f * p.table_stride + col];
    return page >= 0 && page < p.num_pages ? page : -1;
}

__device__ __forceinline__ int block_sum(int x, int *s_warp, int &before)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int sum = x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int y = __shfl_up_sync(~0u, sum, k);
        if (lane >= k) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        int t = s_warp[lane];
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int y = __shfl_up_sync(~0u, t, k);
            if (lane >= k) t += y;
        }
        s_warp[lane] = t;
    }
    __syncthreads();
    before = sum - x + (warp ? s_warp[warp - 1] : 0);
    const int total = s_warp[kThreads / 32 - 1];
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    pages_kernel(const __grid_constant__ PagesParams p)
{
    __shared__ int s_end[kRows];    // pages that rows up to this one need, this one's among them
    __shared__ int s_first[kRows];  // first column that a fresh page goes to
    __shared__ int s_warp[32];
    __shared__ int s_free;
    const int tid = threadIdx.x, rank = blockIdx.x;
    enter_grid();
    const int at = rank * kThreads + tid, all = kCluster * kThreads;
    int *refs = p.refs_out;
    if (p.refs != p.refs_out) {
        for (int i = at; i < p.num_pages; i += all) __stcg(refs + i, p.refs[i]);
        meet();
    }
    // Old rows. A row that the new row of the same number goes on from: that one's kept pages stay counted.
    const int warp = at / 32, warps = all / 32, lane = tid % 32;
    for (int f = warp; f < p.rows_in; f += warps) {
        const int n = old_len(p, f);
        if (n < 0) {
            if (lane == 0) flag_bad_index(p.status);
            continue;
        }
        int from = 0;
        if (f < p.rows_out) {
            const Row r = row_of(p, f);
            if (r.origin == f) from = r.kept;
        }
        for (int j = from + lane; j < up(n, p.page_size); j += 32) {
            const int page = page_at(p, f, j);
            if (page >= 0)
                atomicSub(refs + page, 1);
            else
                flag_bad_index(p.status);
        }
    }
    for (int b = warp; b < p.rows_out; b += warps) {
        const Row r = row_of(p, b);
        int32_t *to = p.table_out + b * p.table_out_stride;
        for (int j = lane; j < p.cols; j += 32) {
            int page = -1;
            if (j < r.kept) {
                page = page_at(p, r.origin, j);
                if (page < 0)
                    flag_bad_index(p.status);
                else if (r.origin != b)
                    atomicAdd(refs + page, 1);
            }
            to[j] = page;
        }
        if (lane == 0) {
            if (r.bad) flag_bad_index(p.status);
            p.lens_out[b] = r.want;
            p.copy_src[b] = -1, p.copy_dst[b] = -1, p.copy_rows[b] = 0;
        }
    }
    meet();
    // Needs: thread t has rows kEach t and on.
    int need[kEach], sum = 0;
    int leaves[kEach];  // the page that a row copies, or -1
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int b = tid * kEach + k;
        need[k] = 0, leaves[k] = -1;
        if (b < p.rows_out) {
            const Row r = row_of(p, b);
            if (r.keep % p.page_size != 0 && r.want > r.keep) {
                const int page = page_at(p, r.origin, r.kept - 1);
                if (page >= 0 && __ldcg(refs + page) > 1) leaves[k] = page;
            }
            need[k] = r.pages - r.kept + (leaves[k] >= 0);
            s_first[b] = r.kept - (leaves[k] >= 0);
        }
        sum += need[k];
    }
    int before;
    const int wanted = block_sum(sum, s_warp, before);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        before += need[k];
        if (tid * kEach + k < p.rows_out) s_end[tid * kEach + k] = before;
    }
    // Free pages of this CTA's part.
    const int part = (p.num_pages + kCluster - 1) / kCluster, lo = min(rank * part, p.num_pages);
    const int hi = min(lo + part, p.num_pages);
    int mine = 0;
    for (int i = lo + tid; i < hi; i += kThreads) mine += __ldcg(refs + i) == 0;
    int dummy;
    mine = block_sum(mine, s_warp, dummy);
    if (tid == 0) s_free = mine;
    meet();
    int nth = 0, have = 0;
    for (int r = 0; r < kCluster; ++r) {
        uint32_t there;
        int x;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"((uint32_t)__cvta_generic_to_shared(&s_free)), "r"(r));
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(there) : "memory");
        if (r < rank) nth += x;
        have += x;
    }
    // The rows that are served, and what they leave.
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int b = tid * kEach + k;
            if (need[k] == 0) continue;
            if (s_end[b] > have) {
                p.lens_out[b] = p.keep[b];
                flag(p.status, DETFOLD_ERR_SCRATCH_LIMIT);
            } else if (leaves[k] >= 0) {
                p.copy_src[b] = leaves[k];
                p.copy_rows[b] = p.keep[b] % p.page_size;
            }
        }
    }
    // Free pages in ascending order to what is needed in ascending order.
    for (int i0 = lo; i0 < hi && nth < min(wanted, have); i0 += kThreads) {
        const int i = i0 + tid;
        const bool free = i < hi && __ldcg(refs + i) == 0;
        int k;
        const int found = block_sum(free, s_warp, k);
        k += nth;
        nth += found;
        if (free && k < wanted) {
            // the first row whose end is past k
            int a = 0, z = p.rows_out - 1;
            while (a < z) {
                const int m = (a + z) / 2;
                if (s_end[m] > k)
                    z = m;
                else
                    a = m + 1;
            }
            if (s_end[a] <= have) {
                const int start = a ? s_end[a - 1] : 0, col = s_first[a] + (k - start);
                p.table_out[a * p.table_out_stride + col] = i;
                __stcg(refs + i, 1);
                const Row r = row_of(p, a);
                if (col < r.kept) p.copy_dst[a] = i;
            }
        }
    }
    // Others' counts of free pages have been read by now, and a page that is left had a count above 1:
    // it is none of them.
    meet();
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (leaves[k] >= 0 && s_end[tid * kEach + k] <= have) atomicSub(refs + leaves[k], 1);
    }
}

}  // namespace

cudaError_t launch_pages(const PagesParams &p, cudaStream_t stream)
{
    return launch_early(pages_kernel, dim3(kCluster), kThreads, 0, stream, p);
}

}  // namespace detfold_tree
