// One warp's share of the attention in binary32, on the FMA units.
//
// Scores: a lane takes one token and every kParts-th group of four dimensions, for
// all HB heads, so a score needs few exchanges. Values: a lane takes DP / 32 dimensions
// for all heads, the weights come from shared memory. HB is the group rounded up to
// 1, 4 or 8: 2 x HB multiply-adds a cached element pair, two an instruction, keep up
// with memory at 32 bits an element.
#pragma once

#include "attn_decode.cuh"

namespace detfold_attn {

template <int DP, int TOK, int HB>
struct F32Tile {
    using T = float;
    static constexpr int kDP = DP, kTok = TOK, kHeads = HB;
    static constexpr bool kSharedQueries = true;
    static constexpr int kParts = 32 / TOK;  // lanes that share a token's score
    static constexpr int kOwn = DP / 32;     // dimensions a lane holds of the output
    static constexpr int kVec = kOwn >= 4 ? 4 : kOwn;
    // Softmax statistics: the lanes of part i hold kMine heads for their token, several parts
    // the same ones where there are fewer heads than parts.
    static constexpr int kMine = HB > kParts ? HB / kParts : 1;
    struct Shared {
        alignas(16) float q[HB][DP];
        alignas(16) float p[kWarps][TOK][HB];
        float fade[kWarps][HB];
    };
    float m[kMine], l[kMine];
    float2 o[HB][kOwn / 2];

    static __device__ __forceinline__ int head(int part, int i) { return part * kMine % HB + i; }

    __device__ __forceinline__ void load_q(const DecodeWork &w, Shared &sh, int b, int head0, int heads, int, int)
    {
        for (int i = threadIdx.x; i < HB * DP; i += kThreads) {
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
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int i = 0; i < kOwn / 2; ++i) o[h][i] = make_float2(0.0f, 0.0f);
    }

    // The dimension of a lane's i-th output element.
    static __device__ __forceinline__ int dim(int lane, int i) { return (i / kVec) * 32 * kVec + lane * kVec + i % kVec; }

    // The weights of a tile of `count` tokens (TOK or fewer), and what they do to the triple.
    __device__ __forceinline__ void scores(const DecodeWork &w, Shared &sh, const unsigned char *keys, int count,
                                           int warp, int lane)
    {
        const int token = lane % TOK, part = lane / TOK;
        float2 sum[HB];
#pragma unroll
        for (int h = 0; h < HB; ++h) sum[h] = make_float2(0.0f, 0.0f);
        const int fours = w.p.head_dim / 4;
#pragma unroll 8
        for (int i = part; i < fours; i += kParts) {
            const float4 k = *reinterpret_cast<const float4 *>(keys + piece_at<TOK>(token, i));
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                const float4 q = reinterpret_cast<const float4 *>(sh.q[h])[i];
                sum[h] = fma2(make_float2(q.x, q.y), make_float2(k.x, k.y), sum[h]);
                sum[h] = fma2(make_float2(q.z, q.w), make_float2(k.z, k.w), sum[h]);
            }
        }
        __syncwarp();
        float s[HB];
#pragma unroll
        for (int h = 0; h < HB; ++h) {
            s[h] = __fadd_rn(sum[h].x, sum[h].y);
#pragma unroll
            for (int x = TOK; x < 32; x <<= 1) s[h] = __fadd_rn(s[h], __shfl_xor_sync(~0u, s[h], x));
        }
        bool moved = false;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            float x = s[i];  // of head(part, i)
#pragma unroll
            for (int k = 1; k < kParts; ++k) x = part == k ? s[head(k, i)] : x;
            x = token < count ? __fmul_rn(x, w.p.scale) : neg_inf();
            float top = x;
#pragma unroll
            for (int y = 1; y < TOK; y <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, y));
            top = fmaxf(top, m[i]);
            const float base = base_of(top), fade = exp_neg(m[i] - base), p = exp_neg(x - base);
            moved |= top != m[i];
            m[i] = top;
            l[i] = __fmaf_rn(l[i], fade, p);
            if (part * kMine < HB) {
                sh.p[warp][token][head(part, i)] = p;
                if (token == 0) sh.fade[warp][head(part, i)] = fade;
            }
        }
        __syncwarp();
        // where no maximum moved every factor is 1
        if (__any_sync(~0u, moved)) {
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                const float f = sh.fade[warp][h];
#pragma unroll
                for (int i = 0; i < kOwn / 2; ++i) o[h][i] = mul2(o[h][i], make_float2(f, f));
            }
        }
    }

    // Adds the tile's weighted values.
    __device__ __forceinline__ void values(Shared &sh, const unsigned char *from, int count, int warp, int lane)
    {
        const int last = min(TOK, (count + 7) & ~7);  // zeros up to there
#pragma unroll 8
        for (int t = 0; t < last; ++t) {
            float p[HB];
            const float *pt = sh.p[warp][t];
            if constexpr (HB % 4 == 0) {
#pragma unroll
                for (int h = 0; h < HB; h += 4) *reinterpret_cast<float4 *>(p + h) = *reinterpret_cast<const float4 *>(pt + h);
            } else {
#pragma unroll
                for (int h = 0; h < HB; ++h) p[h] = pt[h];
            }
            float2 v[kOwn / 2];
#pragma unroll
            for (int i = 0; i < kOwn; i += kVec) {
                const unsigned char *at = from + piece_at<TOK>(t, dim(lane, i) / 4) + dim(lane, i) % 4 * 4;
                if constexpr (kVec == 4)
                    *reinterpret_cast<float4 *>(v + i / 2) = *reinterpret_cast<const float4 *>(at);
                else
                    v[i / 2] = *reinterpret_cast<const float2 *>(at);
            }
#pragma unroll
            for (int h = 0; h < HB; ++h)
#pragma unroll
                for (int i = 0; i < kOwn / 2; ++i) o[h][i] = fma2(make_float2(p[h], p[h]), v[i], o[h][i]);
        }
        __syncwarp();  // the weights have been read
    }

    __device__ __forceinline__ void leave(float *acc, int pitch, float *sm, float *sl, bool bad, int lane)
    {
        const int token = lane % TOK, part = lane / TOK;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            float sum = l[i];
#pragma unroll
            for (int x = 1; x < TOK; x <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(~0u, sum, x));
            if (token == 0 && part * kMine < HB) {
                sm[head(part, i)] = m[i];
                sl[head(part, i)] = bad ? quiet_nan() : sum;
            }
        }
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                acc[h * pitch + dim(lane, i)] = i % 2 ? o[h][i / 2].y : o[h][i / 2].x;
    }
};

}  // namespace detfold_attn
