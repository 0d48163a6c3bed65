// Shared pieces of the decode-step attention operators: launch parameters,
// element conversions, the chunk rule and the fold of softmax triples.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "detfold_attn.h"

namespace detfold_attn {

// Both 16-bit conversions from binary32 round to nearest-even.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// The device status word: written only where an index is out of range.
__device__ __forceinline__ void flag_bad_index(int *status)
{
    if (status) *(volatile int *)status = DETFOLD_ERR_ARG;
}

struct AppendParams {
    detfold_kv_cache cache;
    const void *k, *v, *q;
    void *q_out;
    const int64_t *slots, *positions;
    const float *cos_sin;
    int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs;
    int64_t tokens, rope_rows;
    int rot_dim, interleaved, q_heads;
    int *status;
};

struct DecodeParams {
    void *out;
    float *lse;
    const void *q;
    int64_t out_bs, out_hs, q_bs, q_hs;
    const void *k, *v;
    int64_t num_pages, page_stride, token_stride, head_stride;
    const int32_t *table, *lens;
    int64_t table_stride, window;
    int page_size, kv_heads, head_dim, group;
    int batch, q_heads, max_len;
    float scale;
    int *status;
};

struct JoinParams {
    void *out;
    float *lse;
    const void *parts[DETFOLD_MAX_W];
    const float *lses[DETFOLD_MAX_W];
    int64_t rows;
    int W, head_dim;
};

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);
// `max_seen`: the most tokens that a sequence attends to (p.window of a call).
int64_t decode_workspace(int dtype, int batch, int kv_heads, int group, int head_dim, int64_t max_seen);
cudaError_t launch_decode(const DecodeParams &p, int dtype, void *workspace, cudaStream_t stream);
cudaError_t launch_join(const JoinParams &p, int dtype, cudaStream_t stream);

}  // namespace detfold_attn
