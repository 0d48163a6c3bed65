// Kernels and launches of the one-token attention, for one element type a unit.
#pragma once

#include <atomic>

#include "attn_decode.cuh"

namespace detfold_attn {

template <typename Tile>
inline constexpr TileShape kShape = tile_of(sizeof(typename Tile::T), Tile::kDP, Tile::kHeads);

template <typename Tile, int SLOTS>
__global__ void __launch_bounds__(kThreads, kShape<Tile>.ctas) decode_kernel(const __grid_constant__ DecodeWork w)
{
    DecodeKernel<Tile, SLOTS>::run(w);
}

template <typename T, int DP, int TOK>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const __grid_constant__ DecodeWork w)
{
    join_chunks<T, DP, TOK>(w);
}

// Shared memory above 48 KB is allowed once a device.
inline cudaError_t allow_shared(const void *kernel, size_t bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)) return e;
    done.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}

template <typename Tile, int SLOTS>
cudaError_t launch_tile(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    using K = DecodeKernel<Tile, SLOTS>;
    // of an SM's 228 KB the system keeps 1 KB a CTA
    static_assert((sizeof(typename K::Shared) + 1024) * kShape<Tile>.ctas <= 228 * 1024, "CTAs an SM");
    static_assert(K::R::kRound == kShape<Tile>.round, "as the grid is sized");
    static std::atomic<uint64_t> done{0};
    const size_t bytes = sizeof(typename K::Shared);
    if (cudaError_t e = allow_shared((const void *)decode_kernel<Tile, SLOTS>, bytes, done)) return e;
    if (cudaError_t e = launch_early(decode_kernel<Tile, SLOTS>, dim3(g.ctas), kThreads, bytes, stream, w)) return e;
    if (w.slots)
        return launch_early(decode_join_kernel<typename Tile::T, K::DP, K::TOK>, dim3(g.slots, g.heads), kThreads, 0, stream, w);
    return cudaSuccess;
}

}  // namespace detfold_attn
