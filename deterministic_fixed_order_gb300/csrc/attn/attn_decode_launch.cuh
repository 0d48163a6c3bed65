// Kernels and launches of the one-token attention, for one element type a unit.
#pragma once

#include <atomic>

#include "attn_decode.cuh"

namespace detfold_attn {

template <typename Tile, int SLOTS>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const __grid_constant__ DecodeWork w)
{
    DecodeKernel<Tile, SLOTS>::run(w);
}

template <typename Tile, int SLOTS>
__global__ void __launch_bounds__(kThreads, 2) decode_few_kernel(const __grid_constant__ DecodeWork w)
{
    DecodeKernel<Tile, SLOTS>::run_few(w);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(const __grid_constant__ DecodeWork w)
{
    join_chunks<T>(w);
}

// A kernel's attribute is set once a device.
inline cudaError_t allow(const void *kernel, cudaFuncAttribute attribute, int value, std::atomic<uint64_t> &done)
{
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, attribute, value)) return e;
    done.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}
inline cudaError_t allow_shared(const void *kernel, size_t bytes, std::atomic<uint64_t> &done)
{
    return allow(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes, done);
}

// The cluster launch of a few sequences.
template <typename Tile, int SLOTS>
cudaError_t launch_few(const DecodeWork &w, const DecodeGrid &g, size_t bytes, cudaStream_t stream)
{
    const auto kernel = decode_few_kernel<Tile, SLOTS>;
    static std::atomic<uint64_t> done{0}, wide{0};
    if (cudaError_t e = allow_shared((const void *)kernel, 227 * 1024, done)) return e;
    if (g.ranks > 8)
        if (cudaError_t e = allow((const void *)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, wide)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(g.ranks, w.pairs, w.p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = g.ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, w);
}

template <typename Tile, int SLOTS>
cudaError_t launch_tile(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    using K = DecodeKernel<Tile, SLOTS>;
    using Few = DecodeKernel<Tile, SLOTS>;
    static_assert(sizeof(typename K::Shared) <= 113 * 1024, "two CTAs an SM");
    static_assert(K::R::kRound == tile_of(sizeof(typename K::T), K::DP).round, "as the grid is sized");
    const size_t few = sizeof(typename Few::Shared) + (size_t)w.chunks * (w.own * 16 + g.heads * 8);
    if (g.ranks && few <= 227 * 1024) return launch_few<Tile, SLOTS>(w, g, few, stream);
    static std::atomic<uint64_t> done{0};
    const size_t bytes = sizeof(typename K::Shared);
    if (cudaError_t e = allow_shared((const void *)decode_kernel<Tile, SLOTS>, bytes, done)) return e;
    if (cudaError_t e = launch_early(decode_kernel<Tile, SLOTS>, dim3(g.ctas), kThreads, bytes, stream, w)) return e;
    if (g.slots)
        return launch_early(decode_join_kernel<typename Tile::T>, dim3(g.slots, g.heads), kThreads, 0, stream, w);
    return cudaSuccess;
}

}  // namespace detfold_attn
