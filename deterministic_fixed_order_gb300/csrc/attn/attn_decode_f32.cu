// One-token attention over float32 caches.
#include "attn_decode_f32.cuh"
#include "attn_decode_launch.cuh"

namespace detfold_attn {
cudaError_t launch_decode_f32(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    if (w.p.head_dim <= 64) return launch_tile<F32Tile<64, 16>, 3>(w, g, stream);
    if (w.p.head_dim <= 128) return launch_tile<F32Tile<128, 16>, 3>(w, g, stream);
    return launch_tile<F32Tile<256, 8>, 3>(w, g, stream);
}
}  // namespace detfold_attn
