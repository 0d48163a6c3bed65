// The 16-bit launches: which tile a call takes.
#pragma once

#include "attn_decode_launch.cuh"
#include "attn_decode_mma.cuh"

namespace detfold_attn {

template <typename T>
cudaError_t launch_16bit(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    const bool wide = g.heads > 8;
    if (w.p.head_dim <= 64)
        return wide ? launch_tile<MmaTile<T, 64, 32, 2>, 4>(w, g, stream)
                    : launch_tile<MmaTile<T, 64, 32, 1>, 3>(w, g, stream);
    if (w.p.head_dim <= 128)
        return wide ? launch_tile<MmaTile<T, 128, 32, 2>, 3>(w, g, stream)
                    : launch_tile<MmaTile<T, 128, 32, 1>, 3>(w, g, stream);
    return launch_tile<MmaTile<T, 256, 16, 1>, 3>(w, g, stream);
}

}  // namespace detfold_attn
