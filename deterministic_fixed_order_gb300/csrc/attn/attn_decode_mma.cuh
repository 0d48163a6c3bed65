// One warp's share of the attention in 16-bit types, on the matrix units.
//
// Scores: S^T = K Q^T, 16 tokens by 8 query heads a product, so that a group of up to eight
// heads costs what one does; a tile of 32 tokens is two of them side by side, whose chains of
// dependent instructions overlap. P stays in registers: S^T's layout,
// packed to 16 bits and transposed 8x8 by movmatrix, is the second product's
// right operand, O^T = V^T P^T (V^T by transposing loads). P is split in two
// 16-bit parts, p = hi + lo, both multiplied (split2): one part alone would round each
// weight to the type's 8 or 11 bits and add as much error as rounding the output
// does. float16 has few exponents: its weights are held times 2^14, so that the weights of
// many tokens far below the largest keep their bits too. Scores, maxima, sums and O^T are
// binary32.
#pragma once

#include <type_traits>

#include "attn_decode.cuh"

namespace detfold_attn {

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// c += a b, 16x8x16.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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

template <typename T_, int DP, int TOK, int NT>
struct MmaTile {
    using T = T_;
    static constexpr int kDP = DP, kTok = TOK, kHeads = 8 * NT;
    static constexpr bool kSharedQueries = false;
    static constexpr int kSub = TOK / 16;
    static constexpr int kShift = std::is_same_v<T, __half> ? 14 : 0;  // weights, sums and O^T are times 2^kShift
    struct Shared {
        int unused;
    };

    uint32_t q[DP / 16][NT][2];  // Q^T: dims 16 ks + 2t (+1) and + 8, head 8 nt + g
    float o[DP / 16][NT][4];     // O^T: dims 16 mt + g, + 8; heads 8 nt + 2t, + 1
    float m[NT][2], l[NT][2];    // of heads 2t, 2t + 1; l of this lane's tokens only
    uint32_t hi[kSub][NT][2], lo[kSub][NT][2];  // the tile's weights, tokens 8 half + 2t (+1), head g

    __device__ __forceinline__ void load_q(const DecodeWork &w, Shared &, int b, int head0, int heads, int, int lane)
    {
        const int g = lane / 4, t = lane % 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // lanes past the last head repeat it: their columns are never written out
            const int h = min(nt * 8 + g, heads - 1);
            const T *from = (const T *)w.p.q + b * w.p.q_bs + (int64_t)(head0 + h) * w.p.q_hs;
            // head_dim is a multiple of 8: a pair is inside or outside
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                for (int half = 0; half < 2; ++half) q[ks][nt][half] = 0;
            if (w.q_vec) {
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int d = ks * 16 + half * 8 + 2 * t;
                        if (d < w.p.head_dim) q[ks][nt][half] = *reinterpret_cast<const uint32_t *>(from + d);
                    }
            } else {
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int d = ks * 16 + half * 8 + 2 * t;
                        if (d < w.p.head_dim) q[ks][nt][half] = pack2<T>(from[d], from[d + 1]);
                    }
            }
        }
    }

    __device__ __forceinline__ void reset()
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) m[nt][j] = neg_inf(), l[nt][j] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[mt][nt][j] = 0.0f;
        }
    }

    // The weights of a tile of `count` tokens (TOK or fewer), and what they do to the triple.
    __device__ __forceinline__ void scores(const DecodeWork &w, Shared &, const unsigned char *keys, int count, int,
                                           int lane)
    {
        const float scale = w.p.scale;
        const int g = lane / 4;
        const uint32_t at = smem_addr(keys);
        // two sums a score, joined at the end: half the length of the chain of products
        float s[kSub][NT][4], s2[kSub][NT][4];
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[u][nt][j] = s2[u][nt][j] = 0.0f;
        // a batch of loads goes ahead of its products, since the loads keep their order among themselves
        constexpr int kBatch = 4;
#pragma unroll
        for (int k0 = 0; k0 < DP / 16; k0 += kBatch) {
            uint32_t a[kSub][kBatch][4];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int u = 0; u < kSub; ++u)
                    ldmatrix4(a[u][i], at + piece_at<TOK>(u * 16 + lane % 16, (k0 + i) * 2 + lane / 16));
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma(i % 2 ? s2[u][nt] : s[u][nt], a[u][i], q[k0 + i][nt][0], q[k0 + i][nt][1], T());
        }
        bool moved = false;
        float fade[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float top[2] = {neg_inf(), neg_inf()};
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float &x = s[u][nt][j];
                    x = __fmul_rn(__fadd_rn(x, s2[u][nt][j]), scale);
                    if (u * 16 + g + (j / 2) * 8 >= count) x = neg_inf();
                    top[j % 2] = fmaxf(top[j % 2], x);
                }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                const float y0 = __shfl_xor_sync(~0u, top[0], x), y1 = __shfl_xor_sync(~0u, top[1], x);
                top[0] = fmaxf(top[0], y0);
                top[1] = fmaxf(top[1], y1);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                top[j] = fmaxf(top[j], m[nt][j]);
                const float base = base_of(top[j]);
                fade[nt][j] = exp_neg(m[nt][j] - base);
                moved |= top[j] != m[nt][j];
                m[nt][j] = top[j];
                float sum = 0.0f;
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    s[u][nt][j] = exp_neg_scaled<kShift>(s[u][nt][j] - base);
                    s[u][nt][j + 2] = exp_neg_scaled<kShift>(s[u][nt][j + 2] - base);
                    const float two = __fadd_rn(s[u][nt][j], s[u][nt][j + 2]);
                    sum = u ? __fadd_rn(sum, two) : two;
                }
                l[nt][j] = __fmaf_rn(l[nt][j], fade[nt][j], sum);
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    split2(s[u][nt][half * 2], s[u][nt][half * 2 + 1], hi[u][nt][half], lo[u][nt][half], T());
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    hi[u][nt][half] = transpose8(hi[u][nt][half]);
                    lo[u][nt][half] = transpose8(lo[u][nt][half]);
                }
        }
        // where no maximum moved every factor is 1
        if (__any_sync(~0u, moved)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[mt][nt][j] = __fmul_rn(o[mt][nt][j], fade[nt][j % 2]);
        }
    }

    // Adds the tile's weighted values.
    __device__ __forceinline__ void values(Shared &, const unsigned char *from, int count, int, int lane)
    {
        const uint32_t at = smem_addr(from);
        constexpr int kBatch = 4;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            if (u * 16 >= count) break;  // not copied
#pragma unroll
            for (int m0 = 0; m0 < DP / 16; m0 += kBatch) {
                uint32_t a[kBatch][4];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    ldmatrix4_trans(a[i], at + piece_at<TOK>(u * 16 + (lane / 16) * 8 + lane % 8,
                                                            (m0 + i) * 2 + lane / 8 % 2));
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(o[m0 + i][nt], a[i], hi[u][nt][0], hi[u][nt][1], T());
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(o[m0 + i][nt], a[i], lo[u][nt][0], lo[u][nt][1], T());
            }
        }
    }

    // Leaves the triple in shared memory, its scale taken out again; a `bad` chunk's sums are NaN.
    __device__ __forceinline__ void leave(float *acc, int pitch, float *sm, float *sl, bool bad, int lane)
    {
        constexpr float kUnscale = 1.0f / (1 << kShift);
        const int g = lane / 4, t = lane % 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                const float y0 = __shfl_xor_sync(~0u, l[nt][0], x), y1 = __shfl_xor_sync(~0u, l[nt][1], x);
                l[nt][0] = __fadd_rn(l[nt][0], y0);
                l[nt][1] = __fadd_rn(l[nt][1], y1);
            }
            if (g == 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    sm[nt * 8 + 2 * t + j] = m[nt][j];
                    sl[nt * 8 + 2 * t + j] = bad ? quiet_nan() : __fmul_rn(l[nt][j], kUnscale);
                }
            }
#pragma unroll
            for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[(nt * 8 + 2 * t + j % 2) * pitch + mt * 16 + g + (j / 2) * 8] =
                        __fmul_rn(o[mt][nt][j], kUnscale);
        }
    }
};

}  // namespace detfold_attn
