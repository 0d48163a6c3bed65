// One-token attention over bfloat16 caches.
#include "attn_decode_16bit.cuh"

namespace detfold_attn {
cudaError_t launch_decode_bf16(const DecodeWork &w, const DecodeGrid &g, cudaStream_t stream)
{
    return launch_16bit<__nv_bfloat16>(w, g, stream);
}
}  // namespace detfold_attn
