// Softmax weights as pairs of 16-bit parts for the matrix units.
#pragma once

#include <cstring>

#include "attn_common.cuh"

namespace detfold_attn {

template <typename T>
__device__ __forceinline__ uint32_t pack2(T x, T y)
{
    uint16_t a, b;
    memcpy(&a, &x, 2);
    memcpy(&b, &y, 2);
    return (uint32_t)b << 16 | a;
}

// Two weights as 16-bit pairs, hi + lo: hi truncated, so that lo, what hi leaves, is not negative, and neither part 0
// where the weight is not. So both products with an infinite value are that infinity, as the weight's own
// is. (Rounded to nearest, a weight of 1 leaves lo = 0, others a negative lo: NaN.) A weight of bfloat16 is off by 2^-16 of
// itself at most, one of float16 by 2^-22 of itself or, far below the largest, by 2^-23 of the units that it is held in.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo, __nv_bfloat16)
{
    // weights are normal numbers or 0: their upper halves are the truncated ones
    const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
    hi = __byte_perm(u, v, 0x7632);
    const __nv_bfloat162 rest = __floats2bfloat162_rn(__fsub_rn(x, __uint_as_float(u & 0xffff0000u)),
                                                      __fsub_rn(y, __uint_as_float(v & 0xffff0000u)));
    memcpy(&lo, &rest, 4);
    lo = __vmaxu2(lo, __vminu2(hi, 0x00010001u));
}
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo, __half)
{
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
    __half2 part;
    memcpy(&part, &hi, 4);
    const float2 held = __half22float2(part);
    part = __floats2half2_rn(__fsub_rn(x, held.x), __fsub_rn(y, held.y));
    memcpy(&lo, &part, 4);
    // the least number where the weight is not 0 (its upper half is not)
    const uint32_t least = __vminu2(__byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632), 0x00010001u);
    hi = __vmaxu2(hi, least);
    lo = __vmaxu2(lo, least);
}

}  // namespace detfold_attn
