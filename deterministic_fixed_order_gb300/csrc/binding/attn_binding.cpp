// Python marshalling of libdetfold_attn (and, in tree_calls.h, of libdetfold_tree) for tensors: checks the tensors that a call is
// given and passes their addresses and strides to the C entry points. No arithmetic.
//
// Small calls are bound by what happens on the host: the same checks written in
// Python with ctypes took 5 us of a call's 8 on a GB300's Grace cores, here 1.
#include "marshal.h"
#include "tree_calls.h"

namespace {

// cache(k, v) -> handle
PyObject *new_cache(PyObject *const *a)
{
    const at::Tensor &k = tensor(a[0], "k");
    const int code = type_code(k.scalar_type(), "k");
    if (!k.is_cuda()) raise(PyExc_TypeError, "k: expected a CUDA tensor, got " + k.device().str());
    const int64_t any[4] = {-1, -1, -1, -1};
    const int device = k.get_device();
    rows(a[0], k.scalar_type(), device, any, "k");
    const at::Tensor &v = rows(a[1], k.scalar_type(), device, any, "v");
    if (k.sizes() != v.sizes() || k.strides() != v.strides())
        raise(PyExc_ValueError, "k and v differ: shapes " + shape_text(k.sizes()) + " and " + shape_text(v.sizes()) +
                                    ", strides " + shape_text(k.strides()) + " and " + shape_text(v.strides()));
    for (int i = 1; i < 4; ++i)
        if (k.size(i) > DETFOLD_ATTN_MAX_COUNT) raise(PyExc_ValueError, "k: shape " + shape_text(k.sizes()) + " is too large");
    const detfold_kv_cache d = {k.data_ptr(), v.data_ptr(), k.size(0), k.stride(0), k.stride(1), k.stride(2),
                                code, (int)k.size(1), (int)k.size(2), (int)k.size(3)};
    Cache *c = new Cache{d, k.scalar_type(), device};
    return PyCapsule_New(c, kCacheName, [](PyObject *o) { delete (Cache *)PyCapsule_GetPointer(o, kCacheName); });
}

// rope(cos_sin, interleaved) -> handle
PyObject *new_rope(PyObject *const *a)
{
    const at::Tensor &t = tensor(a[0], "cos_sin");
    if (!t.is_cuda() || t.scalar_type() != at::kFloat)
        raise(PyExc_TypeError, "cos_sin: expected a CUDA float32 tensor, got " + std::string(c10::toString(t.scalar_type())) +
                                   " on " + t.device().str());
    if (t.dim() != 2 || !t.is_contiguous() || t.size(1) > DETFOLD_ATTN_MAX_COUNT)
        raise(PyExc_ValueError, "cos_sin: expected a contiguous [positions, rot_dim] tensor, got shape " + shape_text(t.sizes()));
    const int inter = PyObject_IsTrue(a[1]);
    if (inter < 0) throw Raised{};
    Rope *r = new Rope{{t.data_ptr<float>(), t.size(0), (int)t.size(1), inter}, (int)t.get_device()};
    return PyCapsule_New(r, kRopeName, [](PyObject *o) { delete (Rope *)PyCapsule_GetPointer(o, kRopeName); });
}

// kv_append(cache, k, v, slots, rope, positions, q, q_out, status, stream) -> status
PyObject *kv_append(PyObject *const *a)
{
    const Cache &c = *unpack<Cache>(a[0], kCacheName);
    const int64_t h = c.desc.kv_heads, d = c.desc.head_dim;
    const at::Tensor &k = rows(a[1], c.type, c.device, {-1, h, d}, "k");
    const int64_t tokens = k.size(0);
    const at::Tensor &v = rows(a[2], c.type, c.device, {tokens, h, d}, "v");
    const int64_t *slots = (const int64_t *)flat(a[3], at::kLong, c.device, tokens, "slots");
    const detfold_rope *rope = nullptr;
    const int64_t *positions = nullptr;
    if (a[4] != Py_None) {
        const Rope &r = *unpack<Rope>(a[4], kRopeName);
        if (r.device != c.device) raise(PyExc_TypeError, "rope: on another device than the cache");
        if (a[5] == Py_None) raise(PyExc_ValueError, "positions: needed with rope");
        rope = &r.desc;
        positions = (const int64_t *)flat(a[5], at::kLong, c.device, tokens, "positions");
    }
    const void *q = nullptr;
    void *qo = nullptr;
    int64_t qt = 0, qh = 0, ot = 0, oh = 0, heads = 0;
    if (a[6] != Py_None) {
        if (a[7] == Py_None) raise(PyExc_ValueError, "q_out: needed with q");
        const at::Tensor &x = rows(a[6], c.type, c.device, {tokens, -1, d}, "q");
        heads = x.size(1);
        const at::Tensor &y = rows(a[7], c.type, c.device, {tokens, heads, d}, "q_out");
        q = x.data_ptr(), qt = x.stride(0), qh = x.stride(1);
        qo = y.data_ptr(), ot = y.stride(0), oh = y.stride(1);
    } else if (a[7] != Py_None) {
        raise(PyExc_ValueError, "q_out without q");
    }
    int *status = status_word(a[8], c.device);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    return PyLong_FromLong(detfold_kv_append(&c.desc, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                                             v.stride(1), slots, tokens, rope, positions, qo, ot, oh, q, qt, qh, (int)heads,
                                             status, stream_of(a[9], c.device)));
}

// workspace_bytes(cache, batch, q_heads, max_len) -> bytes or status
PyObject *workspace_bytes(PyObject *const *a)
{
    const Cache &c = *unpack<Cache>(a[0], kCacheName);
    return PyLong_FromLongLong(detfold_attn_decode_workspace_bytes(&c.desc, small_integer(a[1], "batch"),
                                                                   small_integer(a[2], "q_heads"), integer(a[3])));
}

// attn_decode(out, q, cache, block_table, seq_lens, max_len, scale, window, lse, workspace, status, stream) -> status
PyObject *attn_decode(PyObject *const *a)
{
    const Cache &c = *unpack<Cache>(a[2], kCacheName);
    const int64_t d = c.desc.head_dim;
    const at::Tensor &q = rows(a[1], c.type, c.device, {-1, -1, d}, "q");
    const int64_t batch = q.size(0), heads = q.size(1);
    if (batch > DETFOLD_ATTN_MAX_COUNT || heads > DETFOLD_ATTN_MAX_COUNT)
        raise(PyExc_ValueError, "q: shape " + shape_text(q.sizes()) + " is too large");
    const at::Tensor &out = rows(a[0], c.type, c.device, {batch, heads, d}, "out");
    const at::Tensor &table = rows(a[3], at::kInt, c.device, {batch, -1}, "block_table");
    const int32_t *lens = (const int32_t *)flat(a[4], at::kInt, c.device, batch, "seq_lens");
    const int64_t max_len = integer(a[5]), window = integer(a[7]);
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const int64_t rows_heads[2] = {batch, heads};
    float *lse = a[8] == Py_None ? nullptr : (float *)packed(a[8], at::kFloat, c.device, rows_heads, "lse");
    void *ws = nullptr;
    int64_t bytes = 0;
    if (a[9] != Py_None) {
        const at::Tensor &w = tensor(a[9], "workspace");
        if (!w.is_cuda() || w.get_device() != c.device || !w.is_contiguous())
            raise(PyExc_ValueError, "workspace: expected a contiguous tensor on cuda:" + std::to_string(c.device));
        ws = w.data_ptr();
        bytes = (int64_t)w.nbytes();
    }
    int *status = status_word(a[10], c.device);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.device);
    return PyLong_FromLong(detfold_attn_decode(out.data_ptr(), out.stride(0), out.stride(1), lse, q.data_ptr(), q.stride(0),
                                               q.stride(1), &c.desc, table.data_ptr<int>(), table.stride(0), table.size(1),
                                               lens, (int)batch, (int)heads, max_len, (float)scale, window, ws, bytes, status,
                                               stream_of(a[11], c.device)));
}

// attn_join(out, parts, lses, lse, stream) -> status; parts and lses are sequences
PyObject *attn_join(PyObject *const *a)
{
    const at::Tensor &out = tensor(a[0], "out");
    const at::ScalarType type = out.scalar_type();
    const int code = type_code(type, "out");
    PyObject *parts = PySequence_Fast(a[1], "parts: expected a sequence of tensors");
    if (!parts) throw Raised{};
    struct Drop {
        PyObject *o;
        ~Drop() { Py_XDECREF(o); }
    } drop_parts{parts}, drop_lses{PySequence_Fast(a[2], "lses: expected a sequence of tensors")};
    PyObject *lses = drop_lses.o;
    if (!lses) throw Raised{};
    const Py_ssize_t world = PySequence_Fast_GET_SIZE(parts);
    if (PySequence_Fast_GET_SIZE(lses) != world)
        raise(PyExc_ValueError, std::to_string(world) + " parts, " + std::to_string(PySequence_Fast_GET_SIZE(lses)) + " lses");
    if (!out.is_cuda()) raise(PyExc_TypeError, "out: expected a CUDA tensor, got " + out.device().str());
    const int device = out.get_device();
    if (!out.dim()) raise(PyExc_ValueError, "out: expected rows of a head, got shape []");
    // every operand has out's shape, log-sums without the head's dimension
    const at::IntArrayRef shape = out.sizes(), shape_rows = shape.slice(0, shape.size() - 1);
    const int64_t width = shape.back(), n = c10::multiply_integers(shape_rows);
    if (width > DETFOLD_ATTN_MAX_COUNT) raise(PyExc_ValueError, "out: shape " + shape_text(out.sizes()) + " is too large");
    const void *p[DETFOLD_MAX_W];
    const float *l[DETFOLD_MAX_W];
    for (Py_ssize_t r = 0; r < world && r < DETFOLD_MAX_W; ++r) {
        p[r] = packed(PySequence_Fast_GET_ITEM(parts, r), type, device, shape, "parts");
        l[r] = (const float *)packed(PySequence_Fast_GET_ITEM(lses, r), at::kFloat, device, shape_rows, "lses");
    }
    void *to = packed(a[0], type, device, shape, "out");
    float *lse = a[3] == Py_None ? nullptr : (float *)packed(a[3], at::kFloat, device, shape_rows, "lse");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    return PyLong_FromLong(detfold_attn_join(to, lse, p, l, world > DETFOLD_MAX_W ? DETFOLD_MAX_W + 1 : (int)world, n,
                                             (int)width, code, stream_of(a[4], device)));
}

PyMethodDef g_methods[] = {
    method<new_cache, 2>("cache"),
    method<new_rope, 2>("rope"),
    method<kv_append, 10>("kv_append"),
    method<workspace_bytes, 4>("workspace_bytes"),
    method<attn_decode, 12>("attn_decode"),
    method<attn_join, 5>("attn_join"),
    method<tree_plan, 11>("tree_plan"),
    method<tree_workspace_bytes, 5>("tree_workspace_bytes"),
    method<attn_tree, 14>("attn_tree"),
    method<kv_compact, 7>("kv_compact"),
    method<kv_copy_pages, 6>("kv_copy_pages"),
    method<pages_step, 15>("pages_step"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&g_module); }
