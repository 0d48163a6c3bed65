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

// Two neighbours at once.
__device__ __forceinline__ float2 to_f32x2(const float *x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ float2 to_f32x2(const __nv_bfloat16 *x)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(x));
}
__device__ __forceinline__ float2 to_f32x2(const __half *x)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(x));
}
__device__ __forceinline__ void from_f32x2(float *x, float2 y) { x[0] = y.x, x[1] = y.y; }
__device__ __forceinline__ void from_f32x2(__nv_bfloat16 *x, float2 y)
{
    *reinterpret_cast<__nv_bfloat162 *>(x) = __float22bfloat162_rn(y);
}
__device__ __forceinline__ void from_f32x2(__half *x, float2 y)
{
    *reinterpret_cast<__half2 *>(x) = __float22half2_rn(y);
}

// Two binary32 products, or fused multiply-adds, an instruction; each rounded as alone.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{ .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n"
        " mov.b64 {%0, %1}, z; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{ .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// The device status word: written only where something is wrong.
__device__ __forceinline__ void flag(int *status, int code)
{
    if (status) *(volatile int *)status = code;
}
__device__ __forceinline__ void flag_bad_index(int *status) { flag(status, DETFOLD_ERR_ARG); }

// e^x for x <= 0: one product and the hardware's 2^x (2 units in the last place). The roundings
// of the product and of log2 e become relative errors that grow with |x|: 3.6 units more for |x| up
// to 4, 15 up to 16, 62 up to 80. The scores whose difference x is bring as much by their own
// rounding. Results below 2^-126 become 0.
__device__ __forceinline__ float exp_neg(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__fmul_rn(x, kLog2e)));
    return y;
}
// The same times 2^SHIFT by one fused multiply-add. A SHIFT of 14 rounds the exponent at 2^-21, the
// weight by 3e-7; the weights' sum is taken of the same weights.
template <int SHIFT>
__device__ __forceinline__ float exp_neg_scaled(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(SHIFT ? __fmaf_rn(x, kLog2e, (float)SHIFT) : __fmul_rn(x, kLog2e)));
    return y;
}
// The point that exponents are taken from: the maximum, or 0 where no score is above -inf.
__device__ __forceinline__ float base_of(float m) { return m == neg_inf() ? 0.0f : m; }

// Waits for the work before this launch, then lets the next launch start its prologue.
__device__ __forceinline__ void enter_grid()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// N elements that are read or written at once.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

// t / size = t * mul >> shift for t < 2^30: with s = ceil(log2 size) and mul =
// ceil(2^(30 + s) / size), mul * size - 2^(30 + s) < 2^s, so the quotient is exact.
struct Divide {
    unsigned mul, shift;
};
inline Divide divide_by(int size)
{
    int s = 0;
    while ((1 << s) < size) ++s;
    return {(unsigned)((((uint64_t)1 << (30 + s)) + size - 1) / size), (unsigned)(30 + s)};
}
__device__ __forceinline__ unsigned quotient(unsigned t, Divide d)
{
    return (unsigned)((uint64_t)t * d.mul >> d.shift);
}

// A launch whose prologue may overlap the end of the launch before it.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t shared, cudaStream_t stream,
                         const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
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
    Divide page;  // by the page size
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
    int64_t table_stride, table_cols, window;
    int page_size, kv_heads, head_dim, group;
    int batch, q_heads, max_len;
    float scale;
    int *status;
};

struct JoinParams {
    void *out;
    float *lse;
    const void *const *parts;  // host arrays of the call
    const float *const *lses;
    int64_t rows;
    int W, head_dim;
};

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);
// `max_seen`: the most tokens that a sequence attends to (p.window of a call).
int64_t decode_workspace(int dtype, int batch, int kv_heads, int group, int head_dim, int64_t max_seen);
cudaError_t launch_decode(const DecodeParams &p, int dtype, void *workspace, cudaStream_t stream);
cudaError_t launch_join(const JoinParams &p, int dtype, cudaStream_t stream);

}  // namespace detfold_attn
