// One warp's share of the attention in binary32, on the FMA units.
//
// Scores: a lane takes one token and one part of the dimensions for all eight
// heads, so a score needs few exchanges. Values: a lane takes DP / 32 dimensions for
// all eight heads, the weights come from shared memory. 2 x 8 fused multiply-adds a
// cached element pair whatever the group: at 32 bits an element they keep up
// with memory.
#pragma once

#include "attn_decode.cuh"

namespace detfold_attn {

__device__ __forceinline__ float4 lds4(uint32_t at)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

template <int DP, int TOK>
struct F32Tile {
    using T = float;
    static constexpr int kDP = DP, kTok = TOK, kHeads = 8, kRow = DP * 4 + 16;
    static constexpr int kParts = 32 / TOK, kPart = DP / kParts;  // dimensions a lane sums in a score
    static constexpr int kOwn = DP / 32;                          // dimensions a lane holds of the output
    static constexpr int kVec = kOwn >= 4 ? 4 : kOwn;
    struct Shared {
        float q[8][DP];
        float p[kWarps][TOK][8];
        float fade[kWarps][8];
    };
    // Softmax statistics: the lanes of part i hold heads i * kMine ..., for their token.
    static constexpr int kMine = 8 / kParts;
    float m[kMine], l[kMine];
    float o[8][kOwn];

    __device__ __forceinline__ void load_q(const DecodeWork &w, Shared &sh, int b, int head0, int heads, int, int)
    {
        for (int i = threadIdx.x; i < 8 * DP; i += kThreads) {
            const int h = i / DP, d = i % DP;
            sh.q[h][d] = h < heads && d < w.p.head_dim
                             ? ((const float *)w.p.q)[b * w.p.q_bs + (int64_t)(head0 + h) * w.p.q_hs + d]
                             : 0.0f;
        }
        __syncthreads();
    }

    __device__ __forceinline__ void reset()
    {
#pragma unroll
        for (int i = 0; i < kMine; ++i) m[i] = neg_inf(), l[i] = 0.0f;
#pragma unroll
        for (int h = 0; h < 8; ++h)
#pragma unroll
            for (int i = 0; i < kOwn; ++i) o[h][i] = 0.0f;
    }

    // The dimension of a lane's i-th output element.
    static __device__ __forceinline__ int dim(int lane, int i) { return (i / kVec) * 32 * kVec + lane * kVec + i % kVec; }

    __device__ __forceinline__ void step(Shared &sh, const unsigned char *kt, const unsigned char *vt, int count,
                                         float scale, int warp, int lane)
    {
        const int token = lane % TOK, part = lane / TOK;
        float s[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) s[h] = 0.0f;
        const uint32_t ka = smem_addr(kt) + token * kRow + part * kPart * 4;
        const uint32_t qa = smem_addr(&sh.q[0][0]) + part * kPart * 4;
#pragma unroll 4
        for (int i = 0; i < kPart / 4; ++i) {
            const float4 k = lds4(ka + i * 16);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float4 q = lds4(qa + h * DP * 4 + i * 16);
                s[h] = __fmaf_rn(q.x, k.x, s[h]);
                s[h] = __fmaf_rn(q.y, k.y, s[h]);
                s[h] = __fmaf_rn(q.z, k.z, s[h]);
                s[h] = __fmaf_rn(q.w, k.w, s[h]);
            }
        }
#pragma unroll
        for (int h = 0; h < 8; ++h)
#pragma unroll
            for (int x = TOK; x < 32; x <<= 1) s[h] = __fadd_rn(s[h], __shfl_xor_sync(~0u, s[h], x));
        bool moved = false;
        __syncwarp();  // the previous tile's weights have been read
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            float x = s[i];  // head part * kMine + i
#pragma unroll
            for (int k = 1; k < kParts; ++k) x = part == k ? s[k * kMine + i] : x;
            x = token < count ? __fmul_rn(x, scale) : neg_inf();
            float top = x;
#pragma unroll
            for (int y = 1; y < TOK; y <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, y));
            top = fmaxf(top, m[i]);
            const float base = base_of(top), fade = exp_neg(m[i] - base), p = exp_neg(x - base);
            moved |= top != m[i];
            m[i] = top;
            l[i] = __fmaf_rn(l[i], fade, p);
            sh.p[warp][token][part * kMine + i] = p;
            if (token == 0) sh.fade[warp][part * kMine + i] = fade;
        }
        __syncwarp();
        if (__any_sync(~0u, moved)) {
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float f = sh.fade[warp][h];
#pragma unroll
                for (int i = 0; i < kOwn; ++i) o[h][i] = __fmul_rn(o[h][i], f);
            }
        }
        const uint32_t pa = smem_addr(&sh.p[warp][0][0]);
        const float *v0 = reinterpret_cast<const float *>(vt);
#pragma unroll 4
        for (int t = 0; t < TOK; ++t) {
            const float4 p0 = lds4(pa + t * 32), p1 = lds4(pa + t * 32 + 16);
            const float p[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
            float v[kOwn];
#pragma unroll
            for (int i = 0; i < kOwn; i += kVec) {
                const float *at = v0 + t * (kRow / 4) + dim(lane, i);
                if constexpr (kVec == 4)
                    *reinterpret_cast<float4 *>(v + i) = *reinterpret_cast<const float4 *>(at);
                else
                    *reinterpret_cast<float2 *>(v + i) = *reinterpret_cast<const float2 *>(at);
            }
#pragma unroll
            for (int h = 0; h < 8; ++h)
#pragma unroll
                for (int i = 0; i < kOwn; ++i) o[h][i] = __fmaf_rn(p[h], v[i], o[h][i]);
        }
    }

    __device__ __forceinline__ void leave(float *acc, int pitch, float *sm, float *sl, bool bad, int lane)
    {
        const int token = lane % TOK, part = lane / TOK;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            float sum = l[i];
#pragma unroll
            for (int x = 1; x < TOK; x <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(~0u, sum, x));
            if (token == 0) {
                sm[part * kMine + i] = m[i];
                sl[part * kMine + i] = bad ? quiet_nan() : sum;
            }
        }
#pragma unroll
        for (int h = 0; h < 8; ++h)
#pragma unroll
            for (int i = 0; i < kOwn; ++i) acc[h * pitch + dim(lane, i)] = o[h][i];
    }
};

}  // namespace detfold_attn
