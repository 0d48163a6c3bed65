// Attention of one new token a sequence over a paged cache: the pieces that
// every element type shares -- the chunk rule, the spread of the work over
// CTAs, the copy pipeline, the fold of chunk triples and the join.
//
// Mathematics. Per query head: s_t = scale (q . k_t), m = max s_t, p_t =
// exp(s_t - m), l = sum p_t, o = sum p_t v_t / l. A set of tokens is summed up by
// its triple (m, l, a = sum p_t v_t); two triples join to
//     m' = max(m, m_i), l' = l e^(m - m') + l_i e^(m_i - m'), a' likewise.
//
// Fixed order. A sequence's tokens are cut into chunks; the cut follows from
// its length and the head counts alone (sequence). Within a chunk warp w
// takes tiles w, w + 4, ... and the four warps' triples join in warp order; the
// chunks' triples are folded in ascending order. Which CTA takes which chunks is
// free: a CTA that begins a sequence folds in registers, any other leaves its
// chunks' triples in the workspace for the join kernel, which goes on with the
// same operations on the same values. So the bits do not depend on the batch.
//
// Bound. Each cached key and value is read once for all the query heads of a tile (8,
// or 16 in 16-bit types up to 128 dimensions): 4 x group flops an element pair, so memory bound while the
// arithmetic keeps up. One pass; nothing but the triples of split sequences
// goes back to memory. A wider group is several blocks of heads, and each reads the cache again: 16 sequences
// of 8192 tokens, 2 key-value heads, groups of 8, 16 and 32: 33.7, 40.9 and 73.1 us for bfloat16 of 128, 58.8, 100
// and 176 for 256, 63.3, 115 and 209 for float32 of 128.
#pragma once

#include "attn_common.cuh"

namespace detfold_attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSms = 152;
// Tokens a chunk, at least, us with 128 and with 256: one sequence of 4093 tokens 7.7 and 8.6, 32 mixed
// sequences of one key-value head 9.4 and 10.3, float32 14.6 and 15.9; 24 windows of 1024 tokens of 256-wide heads 17.6 and
// 15.9, 64 mixed sequences 51.4 and 51.1. 64 brings float32 to 13.1 and the windows to 19.7. One length for every
// tile: a length by type and width would take both gains.
constexpr int kMinChunk = 128;
// Chunks a sequence: enough for one sequence to fill every CTA, within limits that keep
// the join short.
constexpr int kMinChunks = 16, kMaxChunks = 128;

// A (key-value head, block of at most `heads` query heads) of a sequence is a
// "pair": the unit that has a triple a query head. `resident`: CTAs that the GPU holds.
inline int max_chunks(int pairs, int resident)
{
    const int c = resident / pairs;
    return c < kMinChunks ? kMinChunks : c > kMaxChunks ? kMaxChunks : c;
}

// The tile that a head dimension takes: tokens a warp has at once, so that their keys are 8 KB
// (4 KB at 64 16-bit dimensions), and tokens a round; and the CTAs that an SM holds.
//
// Two, so that one's arithmetic goes on while the other folds a chunk: four warps with three slots of
// 8 KB take under half an SM's shared memory, and its registers go round at 255 a thread. (One CTA of eight
// warps: the same for one long sequence, 71 us where this took 54 on 64 mixed ones. Three CTAs with slots of
// 4 KB at 128 16-bit dimensions: 82.5 us for 84.1 on one sequence of 131071 tokens, 63.0 for 51.9 on 64 mixed ones.)
// At 64 16-bit dimensions a tile has half the bytes and takes nearly as long, and half the registers: four, with
// three slots of 4 KB. 64 mixed sequences of 16 heads 60.4 us for 65.5, one of 131071 tokens 48.6 for
// 51.6, 100 of 64 tokens 8.4 for 11.5; 32 mixed ones of one head 9.5 for 8.9. Of more than eight query heads
// three, with four slots: 64 mixed sequences of 4 key-value heads 32.9 us, 36.3 with two CTAs and 40.1 with four,
// which spill.
struct TileShape {
    int dims, tokens, round, ctas;
};
constexpr TileShape tile_of(int element_bytes, int head_dim, int heads)
{
    const int dims = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    const int by_size = 8192 / (dims * element_bytes), tokens = by_size < 32 ? by_size : 32;
    return {dims, tokens, kWarps * tokens, dims > 64 || element_bytes > 2 ? 2 : heads > 8 ? 3 : 4};
}

struct DecodeGrid {
    int ctas;    // CTAs of the main kernel
    int most;    // max_chunks
    int slots;   // workspace slots, 0: no sequence can be split
    bool by_pair;  // a slot a pair, else a slot a CTA for the pair that its share breaks off in
    int chunks;  // most chunks of a sequence
    int pairs;   // pairs a sequence
    int heads;   // query heads a pair, at most
    int64_t pair_floats, slot_floats;  // floats of a slot's (m, l) pairs; of a slot
    int direct;  // CTAs a pair: a CTA a chunk, or 1: a CTA has it all; else 0
};

// Few chunks in all, as the longest sequence allows: a CTA a chunk, without working shares out, for up to
// kDirect times as many CTAs as are resident. One sequence of 4093 tokens (0.8 times) 7.7 us for 8.4 with
// shares, 96 windows of 1024 tokens (2.5 times) 17.6 for 19.1; 32 sequences that are mostly shorter than the
// longest (3.4 times) 10.6 for 9.4.
constexpr int kDirect = 3;
// More chunks than resident CTAs, none of a pair of over kWhole rounds, at most kDirect pairs a resident CTA: a CTA a
// pair, and no join. 300 sequences of 288 tokens, one key-value head: 13.3 us for 26.0 in chunks; 600 of them
// 24.6 for 31.4 in shares; 300 mixed ones of up to 480 tokens 12.1 for 16.0, 16 of 8 heads 10.6 for 7.9.
constexpr int kWhole = 4;

// Workspace: a header of four ints a slot, then the slots: for each chunk and head (m, l),
// then for each chunk and head the accumulator.
inline DecodeGrid decode_grid(int batch, int kv_heads, int group, int head_dim, int64_t max_seen, int heads,
                              const TileShape &tile)
{
    const int round = tile.round, resident = kSms * tile.ctas;
    DecodeGrid g;
    g.heads = heads < group ? heads : group;
    const int blocks = (group + heads - 1) / heads;
    g.pairs = kv_heads * blocks;
    const int rounds = (int)((max_seen + round - 1) / round);
    // shorter sequences may have more chunks than the longest: as many as there can be at all, so
    // that a larger max_seen never needs less
    g.most = max_chunks(g.pairs, resident);
    const int least = kMinChunk / round, up_to = (rounds + least - 1) / least;
    g.chunks = up_to < g.most ? up_to : g.most;
    const int each = g.chunks > 0 ? g.chunks : 1;
    const int64_t pairs = (int64_t)batch * g.pairs, units = pairs * each;
    // A slot a pair; where there are more pairs than CTAs, a slot a CTA, since at most one pair
    // begins in a CTA's share and ends beyond it. So slots and their size only grow with max_seen.
    g.by_pair = pairs <= resident;
    g.slots = g.chunks <= 1 ? 0 : g.by_pair ? (int)pairs : resident;
    const bool whole = units > resident && pairs <= kDirect * resident && rounds <= kWhole;
    g.direct = whole ? 1 : units <= kDirect * resident && (g.by_pair || !g.slots) ? each : 0;
    g.ctas = g.direct ? (int)(pairs * g.direct) : units < resident ? (int)units : resident;
    g.pair_floats = ((int64_t)g.chunks * g.heads * 2 + 3) / 4 * 4;
    g.slot_floats = g.pair_floats + ((int64_t)g.chunks * g.heads * head_dim + 3) / 4 * 4;
    return g;
}

inline int64_t workspace_need(const DecodeGrid &g)
{
    return g.slots == 0 ? 0 : (int64_t)g.slots * (16 + g.slot_floats * 4);
}

struct DecodeWork {
    DecodeParams p;
    int pairs, blocks, heads, slots, by_pair;
    int slot_chunks;                // a slot has room for
    int most_chunks;                // max_chunks
    Divide most, grid;              // by most_chunks, by the number of CTAs
    int short_line;                 // the shares' line is shorter than 2^30
    Divide page;                    // by the page size
    int direct;                     // CTAs a pair, else 0
    Divide by_chunks, by_pairs;     // by `direct` and by `pairs`
    int out_vec;                    // four elements of out start at a multiple of their size
    int q_vec;                      // two elements of q do
    int64_t pair_floats, slot_floats;
    int4 *headers;
    float *slot;
};

#ifdef __CUDACC__

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes from global to shared memory; `bytes` == 0 fills with zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A sequence as the kernel sees it.
struct Seq {
    int n, first;     // attended tokens, the first one's index
    int rounds, per;  // rounds, and rounds a chunk: kMinChunk tokens, or more where that made too many chunks
    bool bad;      // its length is out of range
};

template <int TOK>
__device__ __forceinline__ Seq sequence_of(const DecodeWork &w, int len)
{
    Seq s;
    s.bad = len < 0 || len > w.p.max_len;
    constexpr int kRound = kWarps * TOK;
    const int n = s.bad ? 0 : len;
    s.n = n < w.p.window ? n : (int)w.p.window;
    s.first = n - s.n;
    s.rounds = (s.n + kRound - 1) / kRound;
    s.per = max(kMinChunk / kRound, (int)quotient(s.rounds + w.most_chunks - 1, w.most));
    return s;
}

template <int TOK>
__device__ __forceinline__ Seq sequence(const DecodeWork &w, int b)
{
    return sequence_of<TOK>(w, w.p.lens[b]);
}

// A pair's share of the work: its rounds, and one for what each pair costs anyway (53.3 us for 51.8 on 64 mixed
// sequences without the one).
__device__ __forceinline__ int64_t cost(const Seq &s) { return s.rounds + 1; }

// Walks the pairs of a CTA's share [lo, hi) of the line on which all pairs of
// all sequences lie, each as long as it costs. A chunk belongs to the share
// that its first round lies in, a pair's output to the share that its start lies in.
template <int TOK>
struct Walk {
    int64_t at, lo, hi;  // start of the current pair on the line; the share
    Seq s;
    int b, pair;
    int round, end;  // the share's rounds of this pair: [round, end)

    __device__ __forceinline__ bool done(const DecodeWork &w) const { return at >= hi || b >= w.p.batch; }
    __device__ __forceinline__ int chunks() const { return (s.rounds + s.per - 1) / s.per; }
    __device__ __forceinline__ void enter()
    {
        // chunks whose start at + c * per lies in [lo, hi); both bounds as far as the pair reaches
        const int64_t far = cost(s);
        round = 0;
        end = s.rounds;
        if (at < lo) {
            const unsigned from = (unsigned)(lo - at < far ? lo - at : far);
            round = min((int)((from + s.per - 1) / (unsigned)s.per * s.per), s.rounds);
        }
        if (hi - at < far) {
            const unsigned to = (unsigned)(hi - at);
            end = min((int)((to + s.per - 1) / (unsigned)s.per * s.per), s.rounds);
        }
    }
    __device__ __forceinline__ void next_pair(const DecodeWork &w)
    {
        at += cost(s);
        if (++pair == w.pairs) {
            pair = 0;
            if (++b < w.p.batch) s = sequence<TOK>(w, b);
        }
        if (!done(w)) enter();
    }
};

// The line cut into one share a CTA: share j begins at floor(j line / CTAs), so that
// equal chunks meet equal shares.
struct Shares {
    int64_t line, each;
    int over;

    __device__ __forceinline__ void cut(const DecodeWork &w, int64_t length)
    {
        line = length;
        each = w.short_line ? quotient((unsigned)line, w.grid) : line / gridDim.x;
        over = (int)(line - each * gridDim.x);
    }
    __device__ __forceinline__ int64_t begin(const DecodeWork &w, unsigned j) const
    {
        return j * each + quotient(j * over, w.grid);
    }
    // The share that a point of the line lies in.
    __device__ __forceinline__ int of(const DecodeWork &w, int64_t x) const
    {
        const int64_t up = (x + 1) * gridDim.x + line - 1;
        return (int)(up >> 32 ? up / line : (unsigned)up / (unsigned)line) - 1;
    }
};

// The sequence that this CTA's share begins in and its start, and the cut of the line into shares: each lane
// adds up the costs of a block of sequences, and the block that the share begins in is looked through. I
// holds the line's length. (608 mixed sequences of up to 900 tokens, 64 wide, one key-value head: 20.2 us,
// 23.7 where all sequences were looked through 32 at a time.)
template <int TOK, typename I>
__device__ __forceinline__ void find_sequence(const DecodeWork &w, Shares &shares, int64_t &lo, int &b, int64_t &at)
{
    const int lane = threadIdx.x & 31, block = (w.p.batch + 31) / 32;
    const auto scan = [&](I up) {
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const I y = __shfl_up_sync(~0u, up, x);
            if (lane >= x) up += y;
        }
        return up;
    };
    I mine = 0;
    constexpr int kAhead = 4;  // lengths asked for at once
    const int end = min(lane * block + block, w.p.batch);
    for (int i = lane * block; i < end; i += kAhead) {
        int len[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) len[k] = i + k < end ? w.p.lens[i + k] : 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k < end) mine += (I)cost(sequence_of<TOK>(w, len[k])) * w.pairs;
    }
    __syncwarp();
    I up = scan(mine);
    shares.cut(w, __shfl_sync(~0u, up, 31));
    lo = shares.begin(w, blockIdx.x);
    int i = __ffs(__ballot_sync(~0u, up > (I)lo)) - 1;
    I before = __shfl_sync(~0u, up - mine, i);
    if (block == 1) {
        b = i;
        at = before;
        return;
    }
    for (int b0 = i * block; b0 < w.p.batch; b0 += 32) {
        const I c = b0 + lane < w.p.batch ? (I)cost(sequence<TOK>(w, b0 + lane)) * w.pairs : (I)0;
        up = scan(c);
        const unsigned past = __ballot_sync(~0u, before + up > (I)lo);
        if (past) {
            i = __ffs(past) - 1;
            b = b0 + i;
            at = before + __shfl_sync(~0u, up - c, i);
            return;
        }
        before += __shfl_sync(~0u, up, 31);
    }
    // lengths that changed meanwhile: any place that is one
    b = w.p.batch - 1;
    at = lo;
}

// This CTA's share, or its chunk of the pair that is its own. Every warp does the same: no barrier.
template <int TOK>
__device__ __forceinline__ Walk<TOK> begin_walk(const DecodeWork &w, Shares &shares)
{
    Walk<TOK> k;
    if (w.direct) {
        const unsigned pair = quotient(blockIdx.x, w.by_chunks), c = blockIdx.x - pair * w.direct;
        k.b = (int)quotient(pair, w.by_pairs);
        k.pair = (int)(pair - (unsigned)k.b * (unsigned)w.pairs);
        k.s = sequence<TOK>(w, k.b);
        k.at = 0;
        k.lo = c > 0;
        k.hi = 1;
        k.round = min((int)c * k.s.per, k.s.rounds);
        k.end = w.direct == 1 ? k.s.rounds : min(k.round + k.s.per, k.s.rounds);
        return k;
    }
    if (w.p.batch == 1) {
        k.b = 0;
        k.at = 0;
        k.s = sequence<TOK>(w, 0);
        shares.cut(w, cost(k.s) * w.pairs);
        k.lo = shares.begin(w, blockIdx.x);
    } else {
        if (w.short_line)
            find_sequence<TOK, int>(w, shares, k.lo, k.b, k.at);
        else
            find_sequence<TOK, int64_t>(w, shares, k.lo, k.b, k.at);
        k.s = sequence<TOK>(w, k.b);
    }
    k.hi = shares.begin(w, blockIdx.x + 1);
    const int64_t in = k.lo - k.at;
    k.pair = w.pairs == 1 ? 0 : (int)(in >> 32 ? in / cost(k.s) : (unsigned)in / (unsigned)cost(k.s));
    k.pair = min(k.pair, w.pairs - 1);
    k.at += k.pair * cost(k.s);
    k.enter();
    return k;
}

// A running triple of one element and its fold with the next chunk's.
__device__ __forceinline__ void fold_weights(float m, float mi, float &top, float &fa, float &fb)
{
    top = fmaxf(m, mi);
    const float base = base_of(top);
    fa = exp_neg(m - base);
    fb = exp_neg(mi - base);
}
__device__ __forceinline__ float fold_value(float a, float ai, float fa, float fb)
{
    return __fmaf_rn(a, fa, __fmul_rn(ai, fb));
}

__device__ __forceinline__ float4 fold_four(float4 a, float4 ai, float fa, float fb)
{
    return make_float4(fold_value(a.x, ai.x, fa, fb), fold_value(a.y, ai.y, fa, fb), fold_value(a.z, ai.z, fa, fb),
                       fold_value(a.w, ai.w, fa, fb));
}

// Four elements of a head's output, from d on (head_dim is a multiple of 4).
template <typename T>
__device__ __forceinline__ void write_out(const DecodeWork &w, int b, int head, int d, float m, float l, float4 a)
{
    T *to = (T *)w.p.out + b * w.p.out_bs + head * w.p.out_hs + d;
    T v[4];
    // 16-bit results: one reciprocal, its half unit in the last place of binary32 far below theirs
    const float inv = sizeof(T) == 2 && l != 0.0f ? __frcp_rn(l) : 0.0f;
    const auto quotient_of = [&](float x) {
        return from_f32<T>(sizeof(T) == 2 ? __fmul_rn(x, inv) : l == 0.0f ? 0.0f : __fdiv_rn(x, l));
    };
    v[0] = quotient_of(a.x);
    v[1] = quotient_of(a.y);
    v[2] = quotient_of(a.z);
    v[3] = quotient_of(a.w);
    if (w.out_vec) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<uint4 *>(v);
        else
            *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<uint2 *>(v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = v[j];
    }
    if (d == 0 && w.p.lse) w.p.lse[(int64_t)b * w.p.q_heads + head] = __fadd_rn(base_of(m), logf(l));
}

// One warp's ring: slots that hold TOK tokens of keys or of values in turn. A slot is cut into
// columns of 128 bytes; in a column a token's eight 16-byte pieces are exchanged by the low
// bits of the token's number, so that eight tokens' same pieces lie in different banks.
template <typename T, int DP, int TOK, int SLOTS>
struct Ring {
    static constexpr int kRowBytes = DP * (int)sizeof(T);
    static constexpr int kSlot = TOK * kRowBytes;
    static constexpr int kBytes = SLOTS * kSlot;
    static constexpr int kVecs = kRowBytes / 16;  // 16-byte pieces a row
    static constexpr int kRound = kWarps * TOK;
};
// The offset of piece `vec` of token `row` in a slot.
template <int TOK>
__device__ __forceinline__ int piece_at(int row, int vec)
{
    return vec / 8 * (TOK * 128) + row * 128 + (((vec & 7) ^ (row & 7)) << 4);
}

// Copies keys and values ahead of their use, across chunks and pairs of the CTA's share, by
// 16-byte pieces (cp.async): one call a slot, keys and values in turn, and one commit group a
// call. Each lane looks a token's page up and the lanes exchange the rows' places. Pieces that
// are not copied are filled with zeros, so nothing that lies in unwritten cache rows reaches
// the arithmetic.
//
// Measured against it, times of 64 mixed sequences and of one of 131071 tokens: bulk copies, a lane a
// row, 72 and 113 us (a warp starts its copies one after the other); tensor copies of 16 tokens
// by 128 bytes 57 and 86 us; pieces 53 and 86 us, the shortest path at few tokens, and any page size.
template <typename T, int DP, int TOK, int SLOTS>
struct Loader {
    using R = Ring<T, DP, TOK, SLOTS>;
    static constexpr int kTimes = TOK * R::kVecs / 32;  // pieces a lane copies a slot
    static_assert(TOK * R::kVecs % 32 == 0, "every lane copies the same number of pieces");

    Walk<TOK> walk;
    uint32_t ring;  // shared address of this warp's ring
    int slot;
    bool values;    // the next slot takes the values of the tile whose keys went before
    int rows;       // its tokens of this warp, rounded up to what the arithmetic reads; 0: none
    unsigned bad;   // bit i: the tile looked up i tiles before the last one needs a page outside the cache
    unsigned mask;  // bit t: token t is copied
    int64_t off;    // where in the cache this lane's token lies, in bytes; 0 where it is not copied

    __device__ __forceinline__ void start(const Walk<TOK> &k, unsigned char *at)
    {
        walk = k;
        ring = smem_addr(at);
        slot = 0;
        values = false;
        bad = 0;
    }
    __device__ __forceinline__ void look(const DecodeWork &w, int warp, int lane)
    {
        rows = 0;
        bad <<= 1;
        while (!walk.done(w) && walk.round >= walk.end) walk.next_pair(w);  // pairs without rounds in this share
        if (walk.done(w)) return;
        const int i0 = walk.round * R::kRound + warp * TOK, token = lane % TOK;
        ++walk.round;
        const int count = walk.s.n - i0;
        if (count <= 0) return;
        rows = min(TOK, (count + 15) & ~15);
        const bool live = token < count;
        const unsigned t = (unsigned)(walk.s.first + i0 + token), page = quotient(t, w.page);
        const int e = live ? w.p.table[walk.b * w.p.table_stride + page] : 0;
        const bool ok = e >= 0 && e < w.p.num_pages;
        if (live && !ok) flag_bad_index(w.p.status);
        bad |= __any_sync(~0u, live && !ok) ? 1u : 0u;
        const int hk = w.blocks == 1 ? walk.pair : walk.pair / w.blocks;
        mask = __ballot_sync(~0u, live && ok);
        off = live && ok ? (e * w.p.page_stride + hk * w.p.head_stride +
                            (int)(t - page * (unsigned)w.p.page_size) * w.p.token_stride) * (int64_t)sizeof(T)
                         : 0;
    }
    __device__ __forceinline__ void issue(const DecodeWork &w, int warp, int lane)
    {
        if (!values) look(w, warp, lane);
        if (rows) {
            // Turn i copies rows row_of(i) + lr, pieces from vec_of(i) + lv on: what depends on the lane alone is
            // worked out once.
            constexpr int kAbreast = R::kVecs < 32 ? 32 / R::kVecs : 1;
            const int lr = lane / R::kVecs, lv = lane % R::kVecs;
            const auto row_of = [](int i) { return R::kVecs < 32 ? i * kAbreast : i * 32 / R::kVecs; };
            const auto vec_of = [](int i) { return R::kVecs < 32 ? 0 : i * 32 % R::kVecs; };
            const char *from = (const char *)(values ? w.p.v : w.p.k) + lv * 16;
            const uint32_t to = ring + slot * R::kSlot + lv / 8 * (TOK * 128) + lr * 128;
            const uint32_t swizzle = ((lv & 7) ^ lr) << 4;
            const int valid = w.p.head_dim * (int)sizeof(T) / 16 - lv;
            const unsigned rows_here = mask >> lr;
            // all rows' places first: the exchanges keep their order, and copies between them would wait for
            // each. A short tile's second half goes uncopied.
            constexpr int kHalf = TOK > 16 ? kTimes / 2 : kTimes;
#pragma unroll
            for (int i0 = 0; i0 < kTimes; i0 += kHalf) {
                if (i0 && rows <= 16) break;
                int64_t o[kHalf];
#pragma unroll
                for (int i = 0; i < kHalf; ++i) o[i] = __shfl_sync(~0u, off, row_of(i0 + i) + lr);
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    const int row = row_of(i0 + i), vec = vec_of(i0 + i);
                    const int bytes = (rows_here >> row & 1) && vec < valid ? 16 : 0;
                    copy16(to + vec / 8 * (TOK * 128) + row * 128 + (swizzle ^ (row & 7) << 4), from + o[i] + vec * 16,
                           bytes);
                }
            }
        }
        copy_commit();
        values = !values;
        slot = slot + 1 == SLOTS ? 0 : slot + 1;
    }
    // Whether the tile whose keys have just been waited for needs a page outside the cache.
    __device__ __forceinline__ bool bad_tile() const { return bad >> ((SLOTS + 1) / 2 - 1) & 1; }
    // Waits for the oldest slot that has not been waited for, and starts the next copy.
    __device__ __forceinline__ void turn(const DecodeWork &w, int warp, int lane)
    {
        copy_wait<SLOTS - 2>();
        __syncwarp();
        issue(w, warp, lane);
    }
};

// The main kernel's skeleton. Tile computes one warp's triple:
//   Tile::kHeads, kTok, kDP, T; load_q / reset / scores / values / leave (see the users).
template <typename Tile, int SLOTS>
struct DecodeKernel {
    using T = typename Tile::T;
    static constexpr int DP = Tile::kDP, TOK = Tile::kTok, HB = Tile::kHeads;
    using R = Ring<T, DP, TOK, SLOTS>;
    using Loader = detfold_attn::Loader<T, DP, TOK, SLOTS>;
    // Floats a head of an accumulator that a warp leaves: lanes that store together hit different
    // banks, where a slot has room for that.
    static constexpr int kPitch = HB * (DP + 4) * 4 <= R::kSlot ? DP + 4 : DP;
    // The fold: kTeam threads a head, each kFours groups of four dimensions.
    static constexpr int kTeam = kThreads / HB < DP / 4 ? kThreads / HB : DP / 4, kFours = DP / 4 / kTeam;
    struct Shared {
        alignas(128) unsigned char ring[kWarps][R::kBytes];
        float m[kWarps][HB], l[kWarps][HB];
        typename Tile::Shared tile;
    };
    static_assert(HB * kTeam <= kThreads && DP % (4 * kTeam) == 0, "every thread folds the same number of elements");
    // A warp leaves its accumulator in the slot that it has just used up: the next
    // copy into it starts after the fold.
    static_assert(HB * kPitch * 4 <= R::kSlot, "the accumulator fits a slot");

    // A chunk's triple, of this thread's head and dimensions, from the warps' triples.
    static __device__ __forceinline__ void join_warps(const Shared &sh, int used, int h, int d0, float &top, float &l,
                                                      float4 (&a)[kFours])
    {
        top = sh.m[0][h];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) top = fmaxf(top, sh.m[k][h]);
        const float base = base_of(top);
        float f[kWarps];
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            f[k] = exp_neg(sh.m[k][h] - base);
            l = __fmaf_rn(sh.l[k][h], f[k], l);
        }
#pragma unroll
        for (int i = 0; i < kFours; ++i) {
            a[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 x = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(sh.ring[k] + used * R::kSlot) + h * kPitch + d0 + i * kTeam * 4);
                a[i].x = __fmaf_rn(x.x, f[k], a[i].x);
                a[i].y = __fmaf_rn(x.y, f[k], a[i].y);
                a[i].z = __fmaf_rn(x.z, f[k], a[i].z);
                a[i].w = __fmaf_rn(x.w, f[k], a[i].w);
            }
        }
    }
    // Folds a chunk's triple into the running one.
    static __device__ __forceinline__ void fold_chunk(float &rm, float &rl, float4 (&ra)[kFours], float top, float l,
                                                      const float4 (&a)[kFours])
    {
        float m, fa, fb;
        fold_weights(rm, top, m, fa, fb);
        rl = fold_value(rl, l, fa, fb);
#pragma unroll
        for (int i = 0; i < kFours; ++i) ra[i] = fold_four(ra[i], a[i], fa, fb);
        rm = m;
    }

    __device__ static void run(const DecodeWork &w)
    {
        extern __shared__ __align__(128) unsigned char raw[];
        Shared &sh = *reinterpret_cast<Shared *>(raw);
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        // this thread's head in the fold (the last one again where there are threads to spare) and first dimension
        const bool folds = threadIdx.x < HB * kTeam;
        const int h = folds ? threadIdx.x / kTeam : HB - 1, d0 = threadIdx.x % kTeam * 4;
        enter_grid();
        Shares shares;
        Walk<TOK> walk = begin_walk<TOK>(w, shares);
        Loader load;
        load.start(walk, sh.ring[warp]);
        int slot_now = 0;
        int4 header = make_int4(0, 0, 0, 0);
        bool started = false;
        Tile tile;
        for (; !walk.done(w); walk.next_pair(w)) {
            const bool begins = walk.at >= walk.lo;
            if (!begins && walk.round >= walk.end) continue;
            const int hk = w.blocks == 1 ? walk.pair : walk.pair / w.blocks, block = walk.pair - hk * w.blocks;
            const int head0 = hk * w.p.group + block * w.heads;
            const int heads = min(w.heads, w.p.group - block * w.heads);
            float *slot = nullptr;
            if (w.slots)
                slot = w.slot + (w.by_pair ? walk.b * w.pairs + walk.pair
                                 : begins  ? (int)blockIdx.x
                                           : shares.of(w, walk.at)) *
                                    w.slot_floats;
            // the first copies: after the first queries are asked for, where these go to registers, before them where
            // all warps wait for them
            if (!Tile::kSharedQueries) tile.load_q(w, sh.tile, walk.b, head0, heads, warp, lane);
            if (!started) {
                started = true;
#pragma unroll 1
                for (int i = 0; i < SLOTS - 1; ++i) load.issue(w, warp, lane);
            }
            if (Tile::kSharedQueries) tile.load_q(w, sh.tile, walk.b, head0, heads, warp, lane);
            tile.reset();
            float rm = neg_inf(), rl = 0.0f;
            float4 ra[kFours];
#pragma unroll
            for (int i = 0; i < kFours; ++i) ra[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            bool bad = false;
            int chunk = walk.round / walk.s.per, left = walk.s.per;
            for (int g = walk.round; g < walk.end; ++g) {
                const int count = min(walk.s.n - (g * R::kRound + warp * TOK), TOK);  // tokens of this tile
                const int used = slot_now + 1 == SLOTS ? 0 : slot_now + 1;
                load.turn(w, warp, lane);
                bad |= load.bad_tile();
                if (count > 0) tile.scores(w, sh.tile, sh.ring[warp] + slot_now * R::kSlot, count, warp, lane);
                load.turn(w, warp, lane);
                unsigned char *at = sh.ring[warp] + used * R::kSlot;
                if (count > 0) tile.values(sh.tile, at, count, warp, lane);
                slot_now = used + 1 == SLOTS ? 0 : used + 1;
                if (--left && g + 1 < walk.end) continue;
                // the chunk's end: the warps' triples, joined in warp order
                __syncwarp();
                tile.leave(reinterpret_cast<float *>(at), kPitch, sh.m[warp], sh.l[warp], bad, lane);
                tile.reset();
                bad = false;
                __syncthreads();
                float top, l;
                float4 a[kFours];
                join_warps(sh, used, h, d0, top, l, a);
                if (begins) {
                    fold_chunk(rm, rl, ra, top, l, a);
                } else if (folds && h < heads) {
#pragma unroll
                    for (int i = 0; i < kFours; ++i) {
                        const int d = d0 + i * kTeam * 4;
                        if (d < w.p.head_dim) put_four(w, slot, chunk, h, d, a[i]);
                    }
                    if (d0 == 0) put_pair(w, slot, chunk, h, top, l);
                }
                __syncthreads();
                ++chunk;
                left = walk.s.per;
            }
            if (!begins) continue;
            const bool whole = walk.end >= walk.s.rounds;
            if (walk.s.bad) {
                rl = quiet_nan();
                if (threadIdx.x == 0) flag_bad_index(w.p.status);
            }
            if (folds && h < heads) {
#pragma unroll
                for (int i = 0; i < kFours; ++i) {
                    const int d = d0 + i * kTeam * 4;
                    if (d >= w.p.head_dim) continue;
                    if (whole)
                        write_out<T>(w, walk.b, head0 + h, d, rm, rl, ra[i]);
                    else
                        put_four(w, slot, chunk - 1, h, d, ra[i]);
                }
                if (!whole && d0 == 0) put_pair(w, slot, chunk - 1, h, rm, rl);
            }
            if (w.slots && !w.direct && (w.by_pair || !whole)) {
                header = make_int4(walk.b, walk.pair, chunk - 1, whole ? 0 : walk.chunks());
                if (w.by_pair && threadIdx.x == 0) w.headers[walk.b * w.pairs + walk.pair] = header;
            }
        }
        copy_wait<0>();
        if (w.slots && !w.by_pair && threadIdx.x == 0) w.headers[blockIdx.x] = header;
    }

    // A chunk's triple in a slot: (m, l) of each head, then the accumulators.
    static __device__ __forceinline__ void put_pair(const DecodeWork &w, float *slot, int chunk, int h, float m, float l)
    {
        *reinterpret_cast<float2 *>(slot + ((int64_t)chunk * w.heads + h) * 2) = make_float2(m, l);
    }
    static __device__ __forceinline__ void put_four(const DecodeWork &w, float *slot, int chunk, int h, int d, float4 a)
    {
        *reinterpret_cast<float4 *>(slot + w.pair_floats + ((int64_t)chunk * w.heads + h) * w.p.head_dim + d) = a;
    }
};

// Joins the split pairs: a CTA a (slot, query head) of kThreads threads. The triples
// from the first stored one on are folded in ascending order, with the main
// kernel's operations. The folds' factors follow from the running maxima alone
// and are made first; the accumulators pass through shared memory so that a whole
// batch of them is in flight at once. Bound by latency: a few tens of KB a CTA.
template <typename T, int DP, int TOK>
__device__ __forceinline__ void join_chunks(const DecodeWork &w)
{
    constexpr int kPer = 12, kBatch = kPer * kThreads * 4 / DP;  // float4s in flight a thread, chunks a batch
    __shared__ float4 s_fold[kMaxChunks];  // fa, fb, top, l
    __shared__ float s_top[kWarps];
    __shared__ float4 s_acc[kPer * kThreads];
    const int slot_index = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int fours = w.p.head_dim / 4;
    // float4 i of a batch: chunk i / fours, group i % fours; divided once, stepped from there
    const int step_c = kThreads / fours, step_d = kThreads % fours;
    const int c_first = tid / fours, d_first = tid % fours;
    const float *slot = w.slot + slot_index * w.slot_floats;
    // Every kernel that may start early waits before it reads anything, the lengths too: what earlier launches wrote is
    // visible after this wait only.
    enter_grid();
    // (sequence, pair, first stored triple, chunks; 0: whole). A CTA a chunk stores every one: all of it follows from
    // the length.
    int4 header;
    if (w.direct) {
        const int b = (int)quotient(slot_index, w.by_pairs);
        const Seq s = sequence<TOK>(w, b);
        const int chunks = (s.rounds + s.per - 1) / s.per;
        header = make_int4(b, slot_index - b * w.pairs, 0, chunks > 1 ? chunks : 0);
    } else {
        header = w.headers[slot_index];
        // written by one CTA's share, unless lengths changed under the call
        if ((unsigned)header.x >= (unsigned)w.p.batch || (unsigned)header.y >= (unsigned)w.pairs || header.z < 0 ||
            header.z >= header.w || header.w > w.slot_chunks)
            return;
    }
    if (header.w == 0) return;
    const int hk = header.y / w.blocks, block = header.y % w.blocks;
    if (h >= min(w.heads, w.p.group - block * w.heads)) return;
    const int first = header.z, count = header.w - first;
    const float4 *acc = reinterpret_cast<const float4 *>(slot + w.pair_floats);
    float4 x[kPer];
    const auto fetch = [&](int c0) {
        int c = c_first, d = d_first;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (c < kBatch && c0 + c < count) x[k] = acc[((int64_t)(first + c0 + c) * w.heads + h) * fours + d];
            c += step_c;
            d += step_d;
            if (d >= fours) d -= fours, ++c;
        }
    };
    // factors: thread c takes chunk c
    static_assert(kMaxChunks <= kThreads, "a thread a chunk");
    float2 ml = make_float2(neg_inf(), 0.0f);
    if (tid < count) ml = *reinterpret_cast<const float2 *>(slot + ((int64_t)(first + tid) * w.heads + h) * 2);
    fetch(0);
    float top = ml.x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const float y = __shfl_up_sync(~0u, top, k);
        if (lane >= k) top = fmaxf(top, y);
    }
    float before = __shfl_up_sync(~0u, top, 1);
    if (lane == 0) before = neg_inf();
    if (count > 32) {
        if (lane == 31) s_top[warp] = top;
        __syncthreads();
        for (int k = 0; k < warp; ++k) before = fmaxf(before, s_top[k]);
    }
    float m, fa, fb;
    fold_weights(before, ml.x, m, fa, fb);
    if (tid < count) s_fold[tid] = make_float4(fa, fb, m, ml.y);
    float l = 0.0f;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c0 = 0; c0 < count; c0 += kBatch) {
        const int have = min(kBatch, count - c0);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (tid + k * kThreads < have * fours) s_acc[tid + k * kThreads] = x[k];
        __syncthreads();
        if (c0 + kBatch < count) fetch(c0 + kBatch);
        if (tid < fours) {
#pragma unroll 8
            for (int k = 0; k < have; ++k) {
                const float4 f = s_fold[c0 + k];
                l = fold_value(l, f.w, f.x, f.y);
                a = fold_four(a, s_acc[k * fours + tid], f.x, f.y);
            }
        }
        __syncthreads();
    }
    if (tid < fours)
        write_out<T>(w, header.x, hk * w.p.group + block * w.heads + h, tid * 4, s_fold[count - 1].z, l, a);
}

#endif  // __CUDACC__

}  // namespace detfold_attn
