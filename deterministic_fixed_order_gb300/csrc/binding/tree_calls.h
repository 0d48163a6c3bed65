// Python marshalling of libdetfold_tree for tensors, as attn_binding.cpp does it for libdetfold_attn.
#pragma once

#include "detfold_tree.h"
#include "marshal.h"

namespace {

// The device of a CUDA tensor.
int device_of(PyObject *x, const char *what)
{
    const at::Tensor &t = tensor(x, what);
    if (!t.is_cuda()) raise(PyExc_TypeError, std::string(what) + ": expected a CUDA tensor, got " + t.device().str());
    return (int)t.get_device();
}

// Address of a contiguous int32 tensor of this shape, or NULL where it is None.
const int32_t *optional_ints(PyObject *x, int device, at::IntArrayRef shape, const char *what)
{
    return x == Py_None ? nullptr : (const int32_t *)packed(x, at::kInt, device, shape, what);
}

// tree_plan(mask, parents, seq_lens, node_counts, block_table, page_size, num_pages, positions, slots, status, stream)
PyObject *tree_plan(PyObject *const *a)
{
    const int device = device_of(a[0], "mask");
    const int64_t any[2] = {-1, -1};
    const at::Tensor &parents = rows(a[1], at::kInt, device, any, "parents");
    const int64_t batch = parents.size(0), nodes = parents.size(1);
    if (batch > DETFOLD_ATTN_MAX_COUNT || nodes > DETFOLD_TREE_MAX_NODES)
        raise(PyExc_ValueError, "parents: shape " + shape_text(parents.sizes()) + " is too large");
    const int64_t per[2] = {batch, nodes}, words[3] = {batch, nodes, DETFOLD_TREE_WORDS(nodes)}, one[1] = {batch};
    packed(a[1], at::kInt, device, per, "parents");
    int64_t *mask = (int64_t *)packed(a[0], at::kLong, device, words, "mask");
    const int32_t *lens = (const int32_t *)packed(a[2], at::kInt, device, one, "seq_lens");
    const int32_t *counts = optional_ints(a[3], device, one, "node_counts");
    int64_t *positions = a[7] == Py_None ? nullptr : (int64_t *)packed(a[7], at::kLong, device, per, "positions");
    int64_t *slots = a[8] == Py_None ? nullptr : (int64_t *)packed(a[8], at::kLong, device, per, "slots");
    const int32_t *table = nullptr;
    int64_t stride = 0, cols = 0;
    if (a[4] != Py_None) {
        const int64_t shape[2] = {batch, -1};
        const at::Tensor &t = rows(a[4], at::kInt, device, shape, "block_table");
        table = t.data_ptr<int>(), stride = t.stride(0), cols = t.size(1);
    } else if (slots) {
        raise(PyExc_ValueError, "block_table: needed with slots");
    }
    const int page = small_integer(a[5], "page_size");
    const int64_t pages = integer(a[6]);
    int *status = status_word(a[9], device);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    return PyLong_FromLong(detfold_tree_plan(mask, positions, slots, parents.data_ptr<int>(), lens, counts, table, stride, cols,
                                             page, pages, (int)batch, (int)nodes, status, stream_of(a[10], device)));
}

// tree_workspace_bytes(cache, batch, nodes, q_heads, max_len) -> bytes or status
PyObject *tree_workspace_bytes(PyObject *const *a)
{
    const Cache &c = *unpack<Cache>(a[0], kCacheName);
    return PyLong_FromLongLong(detfold_attn_tree_workspace_bytes(&c.desc, small_integer(a[1], "batch"), small_integer(a[2], "nodes"),
                                                                 small_integer(a[3], "q_heads"), integer(a[4])));
}

// attn_tree(out, q, cache, block_table, seq_lens, mask, max_len, scale, node_counts, window, lse, workspace, status, stream)
PyObject *attn_tree(PyObject *const *a)
{
    const Cache &c = *unpack<Cache>(a[2], kCacheName);
    const int64_t d = c.desc.head_dim, any[4] = {-1, -1, -1, d};
    const at::Tensor &q = rows(a[1], c.type, c.device, any, "q");
    const int64_t batch = q.size(0), nodes = q.size(1), heads = q.size(2);
    if (batch > DETFOLD_ATTN_MAX_COUNT || nodes > DETFOLD_TREE_MAX_NODES || heads > DETFOLD_ATTN_MAX_COUNT)
        raise(PyExc_ValueError, "q: shape " + shape_text(q.sizes()) + " is too large");
    const int64_t shape[4] = {batch, nodes, heads, d}, of_table[2] = {batch, -1}, one[1] = {batch};
    const int64_t words[3] = {batch, nodes, DETFOLD_TREE_WORDS(nodes)}, of_lse[3] = {batch, nodes, heads};
    const at::Tensor &out = rows(a[0], c.type, c.device, shape, "out");
    const at::Tensor &table = rows(a[3], at::kInt, c.device, of_table, "block_table");
    const int32_t *lens = (const int32_t *)packed(a[4], at::kInt, c.device, one, "seq_lens");
    const int64_t *mask = (const int64_t *)packed(a[5], at::kLong, c.device, words, "mask");
    const int64_t max_len = integer(a[6]), window = integer(a[9]);
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const int32_t *counts = optional_ints(a[8], c.device, one, "node_counts");
    float *lse = a[10] == Py_None ? nullptr : (float *)packed(a[10], at::kFloat, c.device, of_lse, "lse");
    void *ws = nullptr;
    int64_t bytes = 0;
    if (a[11] != Py_None) {
        const at::Tensor &w = tensor(a[11], "workspace");
        if (!w.is_cuda() || w.get_device() != c.device || !w.is_contiguous())
            raise(PyExc_ValueError, "workspace: expected a contiguous tensor on cuda:" + std::to_string(c.device));
        ws = w.data_ptr();
        bytes = (int64_t)w.nbytes();
    }
    int *status = status_word(a[12], c.device);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    return PyLong_FromLong(detfold_attn_tree(out.data_ptr(), out.stride(0), out.stride(1), out.stride(2), lse, q.data_ptr(),
                                             q.stride(0), q.stride(1), q.stride(2), &c.desc, table.data_ptr<int>(),
                                             table.stride(0), table.size(1), lens, counts, mask, (int)batch, (int)nodes,
                                             (int)heads, max_len, (float)scale, window, ws, bytes, status,
                                             stream_of(a[13], c.device)));
}

// kv_compact(cache, block_table, seq_lens, path, path_lens, status, stream)
PyObject *kv_compact(PyObject *const *a)
{
    const Cache &c = *unpack<Cache>(a[0], kCacheName);
    const int64_t any[2] = {-1, -1};
    const at::Tensor &path = rows(a[3], at::kInt, c.device, any, "path");
    const int64_t batch = path.size(0), of_table[2] = {batch, -1}, one[1] = {batch};
    if (batch > DETFOLD_ATTN_MAX_COUNT || path.size(1) > DETFOLD_TREE_MAX_NODES)
        raise(PyExc_ValueError, "path: shape " + shape_text(path.sizes()) + " is too large");
    const at::Tensor &table = rows(a[1], at::kInt, c.device, of_table, "block_table");
    const int32_t *lens = (const int32_t *)packed(a[2], at::kInt, c.device, one, "seq_lens");
    const int32_t *path_lens = (const int32_t *)packed(a[4], at::kInt, c.device, one, "path_lens");
    int *status = status_word(a[5], c.device);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    return PyLong_FromLong(detfold_kv_compact(&c.desc, table.data_ptr<int>(), table.stride(0), table.size(1), lens,
                                              path.data_ptr<int>(), path.stride(0), path_lens, (int)batch, (int)path.size(1),
                                              status, stream_of(a[6], c.device)));
}

// kv_copy_pages(cache, src, dst, rows, status, stream)
PyObject *kv_copy_pages(PyObject *const *a)
{
    const Cache &c = *unpack<Cache>(a[0], kCacheName);
    const at::Tensor &src = tensor(a[1], "src");
    if (src.dim() != 1) raise(PyExc_ValueError, "src: expected one dimension, got shape " + shape_text(src.sizes()));
    const int64_t one[1] = {src.size(0)};
    const int32_t *from = (const int32_t *)packed(a[1], at::kInt, c.device, one, "src");
    const int32_t *to = (const int32_t *)packed(a[2], at::kInt, c.device, one, "dst");
    const int32_t *some = optional_ints(a[3], c.device, one, "rows");
    int *status = status_word(a[4], c.device);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    return PyLong_FromLong(detfold_kv_copy_pages(&c.desc, from, to, some, one[0], status, stream_of(a[5], c.device)));
}

// pages_step(refs_out, table_out, lens_out, copy_src, copy_dst, copy_rows, refs, table, lens, origin, keep, want, page_size,
//            status, stream)
PyObject *pages_step(PyObject *const *a)
{
    const int device = device_of(a[6], "refs");
    const at::Tensor &refs = tensor(a[6], "refs");
    if (refs.dim() != 1) raise(PyExc_ValueError, "refs: expected one dimension, got shape " + shape_text(refs.sizes()));
    const int64_t pages[1] = {refs.size(0)}, any[2] = {-1, -1};
    packed(a[6], at::kInt, device, pages, "refs");
    int32_t *refs_out = (int32_t *)packed(a[0], at::kInt, device, pages, "refs_out");
    const at::Tensor &table = rows(a[7], at::kInt, device, any, "table");
    const int64_t cols = table.size(1), in[1] = {table.size(0)}, after[2] = {-1, cols};
    const at::Tensor &table_out = rows(a[1], at::kInt, device, after, "table_out");
    const int64_t out[1] = {table_out.size(0)};
    if (in[0] > DETFOLD_PAGES_MAX_ROWS || out[0] > DETFOLD_PAGES_MAX_ROWS || cols > DETFOLD_ATTN_MAX_COUNT)
        raise(PyExc_ValueError, "table: shape " + shape_text(table.sizes()) + " or " + shape_text(table_out.sizes()) + " is too large");
    int32_t *to[4];
    const char *names[4] = {"lens_out", "copy_src", "copy_dst", "copy_rows"};
    for (int i = 0; i < 4; ++i) to[i] = (int32_t *)packed(a[2 + i], at::kInt, device, out, names[i]);
    const int32_t *lens = (const int32_t *)packed(a[8], at::kInt, device, in, "lens");
    const int32_t *origin = (const int32_t *)packed(a[9], at::kInt, device, out, "origin");
    const int32_t *keep = (const int32_t *)packed(a[10], at::kInt, device, out, "keep");
    const int32_t *want = (const int32_t *)packed(a[11], at::kInt, device, out, "want");
    const int page = small_integer(a[12], "page_size");
    int *status = status_word(a[13], device);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    return PyLong_FromLong(detfold_pages_step(refs_out, table_out.data_ptr<int>(), table_out.stride(0), to[0], to[1], to[2], to[3],
                                              refs.data_ptr<int>(), table.data_ptr<int>(), table.stride(0), lens, origin, keep,
                                              want, pages[0], cols, page, (int)in[0], (int)out[0], status,
                                              stream_of(a[14], device)));
}

}  // namespace
