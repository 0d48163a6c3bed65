// One-token attention over float16 caches.
#include "attn_decode_16bit.cuh"

namespace detfold_attn {
cudaError_t launch_decode_f16(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    return launch_16bit<__half>(w, g, stream);
}
}  // namespace detfold_attn
