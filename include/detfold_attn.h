/*
 * libdetfold_attn -- the decode step's attention over a paged key-value cache,
 * for GB300 (sm_103a), in the fixed-order manner of libdetfold (detfold.h).
 *
 * Three operators that a rank runs before the fold that joins a decode step:
 *   detfold_kv_append    append new tokens' keys and values to a paged cache,
 *                        with the position rotation applied on the way;
 *   detfold_attn_decode  attention of one new token per sequence over that
 *                        cache, split over the cache's length and joined;
 *   detfold_attn_join    join W ranks' partial attentions (each rank holds a
 *                        part of the cache) in ascending rank order.
 *
 * Fixed order: a sequence's attention is computed over chunks of its tokens
 * whose bounds follow from its own length and the head counts alone; each chunk
 * gives a triple (maximum, sum, accumulator) and the triples are folded in
 * ascending order. How chunks are spread over the GPU never changes the bits:
 * a sequence gives the same output alone or in any batch, in any pages.
 *
 * Conventions are those of detfold.h: status codes, no allocation, no
 * synchronisation, stream-ordered work on `stream`, host structures read only
 * during the call, nothing enqueued on an error. In addition:
 *   - Element types are DETFOLD_F32, DETFOLD_BF16 and DETFOLD_F16; every
 *     operand of a call that is not otherwise typed has the cache's type (the
 *     parts' type in detfold_attn_join). Sums, maxima and accumulators are
 *     binary32; each output is rounded once.
 *   - Strides are in elements. The head dimension is always contiguous. Where
 *     an operand is written, neighbours (two heads, rows, tokens or pages) are at
 *     least head_dim elements apart (DETFOLD_ERR_ARG).
 *   - A call whose count (tokens, batch, rows) is 0 is a no-op, and operands that
 *     have no elements then may be NULL.
 *   - `d_status` is an optional DEVICE int (NULL = none) that the caller sets
 *     to DETFOLD_OK. It is written only when a kernel meets an index out of
 *     range in device memory (a slot, a position, a page, a length), and then
 *     becomes DETFOLD_ERR_ARG. Such an index is never used as an address; what
 *     depends on it is stated at each call.
 */
#ifndef DETFOLD_ATTN_H
#define DETFOLD_ATTN_H

#include "detfold.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define DETFOLD_F32 0
#define DETFOLD_BF16 1
#define DETFOLD_F16 2

/* Largest head dimension that detfold_attn_decode takes. */
#define DETFOLD_ATTN_MAX_HEAD_DIM 256
/* Largest sequence length (and max_len). */
#define DETFOLD_ATTN_MAX_LEN ((int64_t)1 << 30)
/* Largest batch, head count and page size. */
#define DETFOLD_ATTN_MAX_COUNT ((int64_t)1 << 20)

/*
 * A paged cache: num_pages pages of page_size tokens of kv_heads heads of
 * head_dim elements, for keys and for values. Element (page, row, head, d) of
 * either lies at page * page_stride + row * token_stride + head * head_stride + d,
 * so pages may be stored token by token, head by head, or inside one buffer
 * that holds both. Pages of keys and of values have the same strides. No two
 * elements that are written may share an address. A stride whose count is 1 is not used.
 */
typedef struct detfold_kv_cache {
    void *k;             /* device */
    void *v;             /* device */
    int64_t num_pages;   /* >= 1 */
    int64_t page_stride;
    int64_t token_stride;
    int64_t head_stride;
    int dtype;     /* DETFOLD_F32, DETFOLD_BF16 or DETFOLD_F16 */
    int page_size; /* tokens a page, >= 1 */
    int kv_heads;  /* >= 1 */
    int head_dim;  /* >= 1 */
} detfold_kv_cache;

/*
 * A position rotation: row p of the table holds cos(angle_i) for i < rot_dim / 2,
 * then sin(angle_i). Pair i of a head is elements (i, i + rot_dim / 2), or
 * (2i, 2i + 1) when interleaved; it becomes (a cos - b sin, b cos + a sin).
 * Elements from rot_dim on are copied.
 */
typedef struct detfold_rope {
    const float *cos_sin; /* device, [positions][rot_dim] f32, 4-byte aligned */
    int64_t positions;    /* rows of the table, >= 1 */
    int rot_dim;          /* even, 2 .. head_dim */
    int interleaved;      /* 0 or 1 */
} detfold_rope;

/*
 * Append: for each token t with slots[t] >= 0, the rotated key and the value of
 * every head go to page slots[t] / page_size, row slots[t] % page_size of the
 * cache. For every token, the rotated queries go to q_out.
 *   k, v      device, element (t, head, d) at t * token_stride + head * head_stride + d.
 *   slots     device, int64, one a token. A negative slot is padding: that
 *             token leaves the cache as it is. Two tokens must not have the
 *             same slot. A slot past the cache is not written (d_status).
 *   rope      host, or NULL: keys and queries are copied unrotated.
 *   positions device, int64, one a token; needed with rope. The rotated
 *             elements of a token whose position is outside the table become
 *             NaN (d_status).
 *   q, q_out  device, or q_heads == 0 and both NULL. q_out may be q itself with
 *             the same strides (rotation in place).
 * tokens == 0 is a no-op. k, v, q and q_out need only their element's
 * alignment; wide accesses are used where every operand is 16-byte aligned.
 */
DETFOLD_API int detfold_kv_append(const detfold_kv_cache *cache, const void *k, int64_t k_token_stride,
                                  int64_t k_head_stride, const void *v, int64_t v_token_stride,
                                  int64_t v_head_stride, const int64_t *slots, int64_t tokens,
                                  const detfold_rope *rope, const int64_t *positions, void *q_out,
                                  int64_t q_out_token_stride, int64_t q_out_head_stride, const void *q,
                                  int64_t q_token_stride, int64_t q_head_stride, int q_heads,
                                  int *d_status, void *stream);

/*
 * Bytes of device workspace that detfold_attn_decode needs for these sizes
 * (cache: host, its pointers are not looked at). Returns a negative status for
 * invalid sizes.
 */
DETFOLD_API int64_t detfold_attn_decode_workspace_bytes(const detfold_kv_cache *cache, int batch,
                                                        int q_heads, int64_t max_len);

/*
 * Attention of one new token a sequence over the cache: for sequence b of
 * n = seq_lens[b] tokens and query head h (which reads key-value head
 * h / (q_heads / kv_heads)), over the tokens t of the last `window` (all when
 * window == 0):
 *     s_t = scale * (q . k_t),  m = max s_t,  l = sum exp(s_t - m)
 *     out = (sum exp(s_t - m) v_t) / l,  lse = m + ln l
 * A sequence of length 0 gives out = 0 and lse = -inf. Token t of sequence b is
 * row t % page_size of page block_table[b][t / page_size]. Cache rows outside
 * the attended tokens, and table entries of pages that hold none, are not read.
 *   out         device, element (b, h, d) at b * out_batch_stride + h * out_head_stride + d.
 *   lse         device f32 [batch][q_heads], or NULL.
 *   q           device, strides as out's.
 *   cache       head_dim <= DETFOLD_ATTN_MAX_HEAD_DIM; its pointers and, in
 *               bytes, its strides and head_dim must be multiples of 16
 *               (DETFOLD_ERR_ALIGN).
 *   block_table device int32, row b at b * table_stride, table_cols entries each
 *               (NULL when table_cols == 0).
 *   seq_lens    device int32 [batch].
 *   max_len     no length is larger; max_len <= table_cols * page_size.
 *   workspace   device, >= detfold_attn_decode_workspace_bytes bytes, 16-byte
 *               aligned; contents on entry are ignored, on return undefined.
 *               Calls that may run at the same time need workspaces of their own.
 * A sequence whose length is negative or over max_len, or that needs a page
 * outside the cache, gives NaN in out and lse (d_status). q_heads must be a
 * multiple of kv_heads. batch == 0 is a no-op.
 */
DETFOLD_API int detfold_attn_decode(void *out, int64_t out_batch_stride, int64_t out_head_stride, float *lse,
                                    const void *q, int64_t q_batch_stride, int64_t q_head_stride,
                                    const detfold_kv_cache *cache, const int32_t *block_table,
                                    int64_t table_stride, int64_t table_cols, const int32_t *seq_lens,
                                    int batch, int q_heads, int64_t max_len, float scale, int64_t window,
                                    void *workspace, int64_t workspace_bytes, int *d_status, void *stream);

/*
 * Join W ranks' partial attentions of the same queries over disjoint parts of
 * the cache, per row: M = max_r lse_r, w_r = exp(lse_r - M),
 *     out = (sum_r w_r part_r) / (sum_r w_r),  lse = M + ln(sum_r w_r)
 * with both sums as serial chains in ascending rank order from rank 0. A rank
 * with lse_r = -inf contributes nothing, whatever its part holds; a row that
 * is -inf on every rank gives out = 0 and lse = -inf.
 *   out    device, [rows][head_dim]; may be exactly one of the parts, no other
 *          overlap with a part or an lses entry (DETFOLD_ERR_OVERLAP).
 *   lse    device f32 [rows], or NULL; disjoint from everything read.
 *   parts  host array of W device pointers, each [rows][head_dim].
 *   lses   host array of W device pointers, each f32 [rows].
 * Pointers need their element's alignment. rows == 0 is a no-op.
 */
DETFOLD_API int detfold_attn_join(void *out, float *lse, const void *const *parts,
                                  const float *const *lses, int W, int64_t rows, int head_dim, int dtype,
                                  void *stream);

/* The cudaError_t value of the last DETFOLD_ERR_CUDA that this library
 * returned on the calling thread (0 if none). */
DETFOLD_API int detfold_attn_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DETFOLD_ATTN_H */
