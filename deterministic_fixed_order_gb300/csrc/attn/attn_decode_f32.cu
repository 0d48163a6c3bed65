// One-token attention over float32 caches.
#include "attn_decode_f32.cuh"
#include "attn_decode_launch.cuh"

namespace detfold_attn {
namespace {

template <int HB>
cudaError_t launch_heads(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    if (w.p.head_dim <= 64) return launch_tile<F32Tile<64, 32, HB>, 3>(w, g, stream);
    if (w.p.head_dim <= 128) return launch_tile<F32Tile<128, 16, HB>, 3>(w, g, stream);
    return launch_tile<F32Tile<256, 8, HB>, 3>(w, g, stream);
}

}  // namespace

cudaError_t launch_decode_f32(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    return g.heads == 1 ? launch_heads<1>(w, g, stream)
           : g.heads <= 4 ? launch_heads<4>(w, g, stream)
                          : launch_heads<8>(w, g, stream);
}

}  // namespace detfold_attn
