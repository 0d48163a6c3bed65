// What the Python marshalling of tensors is made of: checks of the tensors that a call is given,
// the handles of caches and tables, and the wrapper that makes Python errors of what goes wrong.
#pragma once

#include <Python.h>

#include <string>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "detfold_attn.h"

namespace {

// What a PagedCache and a Rope keep: the library's structure and where it lives.
struct Cache {
    detfold_kv_cache desc;
    at::ScalarType type;
    int device;
};
struct Rope {
    detfold_rope desc;
    int device;
};

// Thrown with a Python error set.
struct Raised {};

[[noreturn]] void raise(PyObject *kind, const std::string &text)
{
    PyErr_SetString(kind, text.c_str());
    throw Raised{};
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i)
        t += (i ? ", " : "") + (s[i] < 0 ? std::string("any") : std::to_string(s[i]));
    return t + "]";
}

const at::Tensor &tensor(PyObject *x, const char *what)
{
    if (!THPVariable_Check(x)) raise(PyExc_TypeError, std::string(what) + ": expected a tensor, got " + Py_TYPE(x)->tp_name);
    return THPVariable_Unpack(x);
}

void check_kind(const at::Tensor &t, at::ScalarType type, int device, const char *what)
{
    if (!t.is_cuda() || t.scalar_type() != type || t.get_device() != device)
        raise(PyExc_TypeError, std::string(what) + ": expected a " + c10::toString(type) + " tensor on cuda:" +
                                   std::to_string(device) + ", got " + c10::toString(t.scalar_type()) + " on " +
                                   t.device().str());
}

// A tensor of this type, device and shape (-1: any length) with a contiguous last dimension.
template <size_t N>
const at::Tensor &rows(PyObject *x, at::ScalarType type, int device, const int64_t (&shape)[N], const char *what)
{
    const at::Tensor &t = tensor(x, what);
    check_kind(t, type, device, what);
    bool fits = t.dim() == (int64_t)N;
    for (size_t i = 0; fits && i < N; ++i) fits = shape[i] < 0 || t.size(i) == shape[i];
    if (!fits)
        raise(PyExc_ValueError, std::string(what) + ": expected shape " + shape_text(at::IntArrayRef(shape, N)) +
                                    ", got " + shape_text(t.sizes()));
    if (t.stride(N - 1) != 1 && t.size(N - 1) > 1)
        raise(PyExc_ValueError, std::string(what) + ": the last dimension must be contiguous, strides are " +
                                    shape_text(t.strides()));
    return t;
}

// Address of a contiguous tensor of this type with `count` elements.
void *flat(PyObject *x, at::ScalarType type, int device, int64_t count, const char *what)
{
    const at::Tensor &t = tensor(x, what);
    check_kind(t, type, device, what);
    if (!t.is_contiguous() || t.numel() != count)
        raise(PyExc_ValueError, std::string(what) + ": expected " + std::to_string(count) +
                                    " contiguous elements, got shape " + shape_text(t.sizes()) + ", strides " +
                                    shape_text(t.strides()));
    return t.data_ptr();
}

// Address of a contiguous tensor of this type and shape.
void *packed(PyObject *x, at::ScalarType type, int device, at::IntArrayRef shape, const char *what)
{
    const at::Tensor &t = tensor(x, what);
    check_kind(t, type, device, what);
    if (!t.is_contiguous() || t.sizes() != shape)
        raise(PyExc_ValueError, std::string(what) + ": expected a contiguous tensor of shape " + shape_text(shape) +
                                    ", got shape " + shape_text(t.sizes()) + ", strides " + shape_text(t.strides()));
    return t.data_ptr();
}

int *status_word(PyObject *x, int device)
{
    if (x == Py_None) return nullptr;
    const at::Tensor &t = tensor(x, "status");
    check_kind(t, at::kInt, device, "status");
    if (t.numel() < 1) raise(PyExc_ValueError, "status: expected one element");
    return t.data_ptr<int>();
}

int64_t integer(PyObject *x)
{
    const long long v = PyLong_AsLongLong(x);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
int small_integer(PyObject *x, const char *what)
{
    const int64_t v = integer(x);
    if (v != (int)v) raise(PyExc_OverflowError, std::string(what) + ": out of range");
    return (int)v;
}

// None: torch's current stream of the device.
void *stream_of(PyObject *x, int device)
{
    if (x == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    void *s = PyLong_AsVoidPtr(x);
    if (!s && PyErr_Occurred()) throw Raised{};
    return s;
}

template <typename C>
C *unpack(PyObject *x, const char *name)
{
    C *c = (C *)PyCapsule_GetPointer(x, name);
    if (!c) throw Raised{};
    return c;
}

int type_code(at::ScalarType t, const char *what)
{
    switch (t) {
    case at::kFloat: return DETFOLD_F32;
    case at::kBFloat16: return DETFOLD_BF16;
    case at::kHalf: return DETFOLD_F16;
    default:
        raise(PyExc_TypeError, std::string(what) + ": expected float32, bfloat16 or float16, got " + c10::toString(t));
    }
}

constexpr const char *kCacheName = "detfold.cache", *kRopeName = "detfold.rope";

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyMethodDef method(const char *name)
{
    return {name, (PyCFunction)(void *)(entry<F, N>), METH_FASTCALL, nullptr};
}

}  // namespace
