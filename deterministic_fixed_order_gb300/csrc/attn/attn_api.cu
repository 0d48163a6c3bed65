// The C ABI of libdetfold_attn (declared in include/detfold_attn.h): argument
// checks and dispatch. Nothing here allocates, synchronizes or touches device
// memory other than through stream-ordered launches.
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_common.cuh"

namespace {

using namespace detfold_attn;

thread_local int g_last_cuda_error = 0;

int cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return DETFOLD_OK;
    g_last_cuda_error = (int)e;
    (void)cudaGetLastError();  // clear a non-sticky launch error
    return DETFOLD_ERR_CUDA;
}

int esize(int dtype) { return dtype == DETFOLD_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == DETFOLD_F32 || dtype == DETFOLD_BF16 || dtype == DETFOLD_F16; }
bool aligned(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// Half-open byte ranges [a, a+na) and [b, b+nb) intersect.
bool intersects(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t ua = (uintptr_t)a, ub = (uintptr_t)b;
    return ua < ub + (uintptr_t)nb && ub < ua + (uintptr_t)na;
}

constexpr int64_t kMaxElems = (int64_t)1 << 48;

// Elements from the first to the last of a strided block, or -1 when a count
// or stride is negative or the block is too large to address.
int64_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t inner)
{
    if (s0 < 0 || s1 < 0 || s2 < 0 || n0 < 1 || n1 < 1 || n2 < 1 || inner < 1) return -1;
    const __int128 e = (__int128)(n0 - 1) * s0 + (__int128)(n1 - 1) * s1 + (__int128)(n2 - 1) * s2 + inner;
    return e > kMaxElems ? -1 : (int64_t)e;
}

// Whether neighbours of `n` blocks of `inner` elements share some: they may not where they are written.
bool shares(int64_t n, int64_t stride, int64_t inner) { return n > 1 && stride < inner; }

// A cache's shape; its pointers are checked by the calls that use them.
int check_cache_shape(const detfold_kv_cache *c)
{
    if (!c) return DETFOLD_ERR_NULL;
    if (!known(c->dtype)) return DETFOLD_ERR_ARG;
    if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1) return DETFOLD_ERR_ARG;
    if (c->page_size > DETFOLD_ATTN_MAX_COUNT || c->kv_heads > DETFOLD_ATTN_MAX_COUNT ||
        c->head_dim > DETFOLD_ATTN_MAX_COUNT || c->num_pages > kMaxElems)
        return DETFOLD_ERR_ARG;
    if (extent(c->num_pages, c->page_stride, c->page_size, c->token_stride, c->kv_heads, c->head_stride,
               c->head_dim) < 0)
        return DETFOLD_ERR_ARG;
    return DETFOLD_OK;
}

int64_t cache_bytes(const detfold_kv_cache *c)
{
    return extent(c->num_pages, c->page_stride, c->page_size, c->token_stride, c->kv_heads, c->head_stride,
                  c->head_dim) * esize(c->dtype);
}

// The decode call's sizes, as far as they do not concern pointers.
int check_decode_sizes(const detfold_kv_cache *c, int batch, int q_heads, int64_t max_len)
{
    if (int rc = check_cache_shape(c)) return rc;
    if (c->head_dim > DETFOLD_ATTN_MAX_HEAD_DIM) return DETFOLD_ERR_ARG;
    if (batch < 0 || batch > DETFOLD_ATTN_MAX_COUNT || q_heads < 1 || q_heads > DETFOLD_ATTN_MAX_COUNT ||
        q_heads % c->kv_heads != 0)
        return DETFOLD_ERR_ARG;
    if ((int64_t)batch * q_heads > ((int64_t)1 << 30)) return DETFOLD_ERR_ARG;
    if (max_len < 0 || max_len > DETFOLD_ATTN_MAX_LEN) return DETFOLD_ERR_LEN;
    return DETFOLD_OK;
}

}  // namespace

extern "C" {

int detfold_kv_append(const detfold_kv_cache *cache, const void *k, int64_t k_token_stride,
                      int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                      const int64_t *slots, int64_t tokens, const detfold_rope *rope,
                      const int64_t *positions, void *q_out, int64_t q_out_token_stride,
                      int64_t q_out_head_stride, const void *q, int64_t q_token_stride,
                      int64_t q_head_stride, int q_heads, int *d_status, void *stream)
{
    if (int rc = check_cache_shape(cache)) return rc;
    // operands without elements may have no address
    if (!cache->k || !cache->v || (tokens != 0 && (!k || !v || !slots))) return DETFOLD_ERR_NULL;
    if (q_heads < 0 || q_heads > DETFOLD_ATTN_MAX_COUNT) return DETFOLD_ERR_ARG;
    if (q_heads > 0 && tokens != 0 && (!q || !q_out)) return DETFOLD_ERR_NULL;
    if (q_heads == 0 && (q || q_out)) return DETFOLD_ERR_ARG;
    if (rope) {
        if (!rope->cos_sin || (tokens != 0 && !positions)) return DETFOLD_ERR_NULL;
        if (rope->rot_dim < 2 || rope->rot_dim > cache->head_dim || rope->rot_dim % 2 || rope->positions < 1 ||
            (rope->interleaved != 0 && rope->interleaved != 1))
            return DETFOLD_ERR_ARG;
        if (!aligned(rope->cos_sin, 4) || !aligned(positions, 8)) return DETFOLD_ERR_ALIGN;
    }
    if (tokens < 0 || tokens > DETFOLD_ATTN_MAX_LEN) return DETFOLD_ERR_LEN;
    const int es = esize(cache->dtype);
    if (!aligned(cache->k, es) || !aligned(cache->v, es) || !aligned(k, es) || !aligned(v, es) ||
        !aligned(q, es) || !aligned(q_out, es) || !aligned(slots, 8) || !aligned(d_status, 4))
        return DETFOLD_ERR_ALIGN;
    if (tokens == 0) return DETFOLD_OK;
    const int64_t kb = extent(tokens, k_token_stride, cache->kv_heads, k_head_stride, 1, 0, cache->head_dim) * es;
    const int64_t vb = extent(tokens, v_token_stride, cache->kv_heads, v_head_stride, 1, 0, cache->head_dim) * es;
    if (kb < 0 || vb < 0 || shares(cache->num_pages, cache->page_stride, cache->head_dim) ||
        shares(cache->page_size, cache->token_stride, cache->head_dim) ||
        shares(cache->kv_heads, cache->head_stride, cache->head_dim))
        return DETFOLD_ERR_ARG;
    const int64_t cb = cache_bytes(cache);
    for (const void *c : {cache->k, cache->v})
        if (intersects(c, cb, k, kb) || intersects(c, cb, v, vb)) return DETFOLD_ERR_OVERLAP;
    if (q_heads > 0) {
        const int64_t qb = extent(tokens, q_token_stride, q_heads, q_head_stride, 1, 0, cache->head_dim) * es;
        const int64_t ob =
            extent(tokens, q_out_token_stride, q_heads, q_out_head_stride, 1, 0, cache->head_dim) * es;
        if (qb < 0 || ob < 0 || shares(tokens, q_out_token_stride, cache->head_dim) ||
            shares(q_heads, q_out_head_stride, cache->head_dim))
            return DETFOLD_ERR_ARG;
        for (const void *c : {cache->k, cache->v})
            if (intersects(c, cb, q, qb) || intersects(c, cb, q_out, ob)) return DETFOLD_ERR_OVERLAP;
        // In place the layouts are one; elsewhere q_out meets nothing that is read.
        const bool in_place =
            q_out == q && q_out_token_stride == q_token_stride && q_out_head_stride == q_head_stride;
        if (!in_place && (intersects(q_out, ob, q, qb) || intersects(q_out, ob, k, kb) ||
                          intersects(q_out, ob, v, vb)))
            return DETFOLD_ERR_OVERLAP;
    }
    AppendParams p = {};
    p.cache = *cache;
    p.k = k, p.v = v, p.q = q, p.q_out = q_out;
    p.slots = slots, p.positions = positions;
    p.k_ts = k_token_stride, p.k_hs = k_head_stride, p.v_ts = v_token_stride, p.v_hs = v_head_stride;
    p.q_ts = q_token_stride, p.q_hs = q_head_stride, p.qo_ts = q_out_token_stride, p.qo_hs = q_out_head_stride;
    p.tokens = tokens, p.q_heads = q_heads, p.status = d_status;
    p.page = divide_by(cache->page_size);
    if (rope) {
        p.cos_sin = rope->cos_sin, p.rope_rows = rope->positions;
        p.rot_dim = rope->rot_dim, p.interleaved = rope->interleaved;
    }
    return cuda_status(launch_append(p, (cudaStream_t)stream));
}

int64_t detfold_attn_decode_workspace_bytes(const detfold_kv_cache *cache, int batch, int q_heads,
                                            int64_t max_len)
{
    if (int rc = check_decode_sizes(cache, batch, q_heads, max_len)) return rc;
    return decode_workspace(cache->dtype, batch, cache->kv_heads, q_heads / cache->kv_heads, cache->head_dim,
                            max_len);
}

int detfold_attn_decode(void *out, int64_t out_batch_stride, int64_t out_head_stride, float *lse,
                        const void *q, int64_t q_batch_stride, int64_t q_head_stride,
                        const detfold_kv_cache *cache, const int32_t *block_table, int64_t table_stride,
                        int64_t table_cols, const int32_t *seq_lens, int batch, int q_heads, int64_t max_len,
                        float scale, int64_t window, void *workspace, int64_t workspace_bytes, int *d_status,
                        void *stream)
{
    if (int rc = check_decode_sizes(cache, batch, q_heads, max_len)) return rc;
    if (!cache->k || !cache->v) return DETFOLD_ERR_NULL;
    if (batch > 0 && (!out || !q || !seq_lens || (table_cols > 0 && !block_table))) return DETFOLD_ERR_NULL;
    if (window < 0 || table_cols < 0 || table_stride < 0) return DETFOLD_ERR_ARG;
    if (max_len > 0 && (max_len - 1) / cache->page_size >= table_cols) return DETFOLD_ERR_LEN;
    const int es = esize(cache->dtype), per16 = 16 / es;
    if (!aligned(out, es) || !aligned(q, es) || !aligned(lse, 4) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(d_status, 4) || !aligned(cache->k, 16) || !aligned(cache->v, 16) ||
        cache->page_stride % per16 || cache->token_stride % per16 || cache->head_stride % per16 ||
        cache->head_dim % per16)
        return DETFOLD_ERR_ALIGN;
    if (batch == 0) return DETFOLD_OK;
    const int64_t ob = extent(batch, out_batch_stride, q_heads, out_head_stride, 1, 0, cache->head_dim) * es;
    const int64_t qb = extent(batch, q_batch_stride, q_heads, q_head_stride, 1, 0, cache->head_dim) * es;
    const int64_t tb = extent(batch, table_stride, 1, 0, 1, 0, table_cols > 0 ? table_cols : 1) * 4;
    if (ob < 0 || qb < 0 || tb < 0 || shares(batch, out_batch_stride, cache->head_dim) ||
        shares(q_heads, out_head_stride, cache->head_dim))
        return DETFOLD_ERR_ARG;
    const int64_t need = detfold_attn_decode_workspace_bytes(cache, batch, q_heads, max_len);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return DETFOLD_ERR_WORKSPACE;
    const int64_t cb = cache_bytes(cache), lb = (int64_t)batch * q_heads * 4;
    const void *written[3] = {out, lse, need > 0 ? workspace : nullptr};
    const int64_t wrote[3] = {ob, lb, need};
    const void *read[5] = {q, cache->k, cache->v, block_table, seq_lens};
    const int64_t reads[5] = {qb, cb, cb, tb, (int64_t)batch * 4};
    for (int a = 0; a < 3; ++a) {
        if (!written[a]) continue;
        for (int b = 0; b < 5; ++b)
            if (intersects(written[a], wrote[a], read[b], reads[b])) return DETFOLD_ERR_OVERLAP;
        for (int b = a + 1; b < 3; ++b)
            if (written[b] && intersects(written[a], wrote[a], written[b], wrote[b])) return DETFOLD_ERR_OVERLAP;
    }
    DecodeParams p = {};
    p.out = out, p.lse = lse, p.q = q;
    p.out_bs = out_batch_stride, p.out_hs = out_head_stride, p.q_bs = q_batch_stride, p.q_hs = q_head_stride;
    p.k = cache->k, p.v = cache->v, p.num_pages = cache->num_pages;
    p.page_stride = cache->page_stride, p.token_stride = cache->token_stride, p.head_stride = cache->head_stride;
    p.table = block_table, p.lens = seq_lens, p.table_stride = table_stride, p.table_cols = table_cols;
    p.window = window == 0 || window > max_len ? max_len : window;
    p.page_size = cache->page_size, p.kv_heads = cache->kv_heads, p.head_dim = cache->head_dim;
    p.group = q_heads / cache->kv_heads;
    p.batch = batch, p.q_heads = q_heads, p.max_len = (int)max_len;
    p.scale = scale, p.status = d_status;
    return cuda_status(launch_decode(p, cache->dtype, workspace, (cudaStream_t)stream));
}

int detfold_attn_join(void *out, float *lse, const void *const *parts, const float *const *lses, int W,
                      int64_t rows, int head_dim, int dtype, void *stream)
{
    if (!parts || !lses || (rows != 0 && !out)) return DETFOLD_ERR_NULL;
    if (W < 1 || W > DETFOLD_MAX_W) return DETFOLD_ERR_WORLD;
    for (int r = 0; rows != 0 && r < W; ++r)
        if (!parts[r] || !lses[r]) return DETFOLD_ERR_NULL;
    if (!known(dtype) || head_dim < 1 || head_dim > DETFOLD_ATTN_MAX_COUNT) return DETFOLD_ERR_ARG;
    if (rows < 0 || rows > DETFOLD_MAX_LEN / head_dim) return DETFOLD_ERR_LEN;
    const int es = esize(dtype);
    if (!aligned(out, es) || !aligned(lse, 4)) return DETFOLD_ERR_ALIGN;
    for (int r = 0; r < W; ++r)
        if (!aligned(parts[r], es) || !aligned(lses[r], 4)) return DETFOLD_ERR_ALIGN;
    if (rows == 0) return DETFOLD_OK;
    const int64_t pb = rows * head_dim * es, lb = rows * 4;
    if (lse && intersects(lse, lb, out, pb)) return DETFOLD_ERR_OVERLAP;
    for (int r = 0; r < W; ++r) {
        if (out != parts[r] && intersects(out, pb, parts[r], pb)) return DETFOLD_ERR_OVERLAP;
        if (intersects(out, pb, lses[r], lb)) return DETFOLD_ERR_OVERLAP;
        if (lse && (intersects(lse, lb, parts[r], pb) || intersects(lse, lb, lses[r], lb)))
            return DETFOLD_ERR_OVERLAP;
    }
    const JoinParams p = {out, lse, parts, lses, rows, W, head_dim};
    return cuda_status(launch_join(p, dtype, (cudaStream_t)stream));
}

int detfold_attn_last_cuda_error(void) { return g_last_cuda_error; }

}  // extern "C"
