// Argument checks shared by the native bindings of the operators: each takes what
// Python gave and returns what the C ABI takes, or sets a ValueError and throws
// Refused.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>

#include "mq.h"

namespace {

// A failed check: the Python error is set; unwinds to the entry point.
struct Refused {};

template <class... A>
[[noreturn]] void refuse(const char *format, A... a) {
    PyErr_Format(PyExc_ValueError, format, a...);
    throw Refused{};
}

const char *type_name(const at::Tensor &t) { return c10::toString(t.scalar_type()); }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    return THPVariable_Unpack(o);
}
// an optional tensor: nullptr for None
const at::Tensor *optional(PyObject *o, const char *name) {
    return o == Py_None ? nullptr : &tensor(o, name);
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
// A size, format, activation or split as an int of the C ABI, whose ranges all end
// below INT32_MAX: what does not fit is refused there.  Not for strides, which
// may be any int (matrix_form).
int to_int(int64_t v) {
    if (v > INT32_MAX) return INT32_MAX;
    if (v < INT32_MIN) return INT32_MIN;
    return (int)v;
}

int device_of(const at::Tensor &x, const char *name) {
    if (!x.is_cuda()) refuse("%s must be a GPU tensor", name);
    return x.get_device();
}
void same_device(const at::Tensor &t, int dev, const char *name) {
    if (!t.is_cuda() || t.get_device() != dev)
        refuse("%s must be on the same GPU as the activations", name);
}

int element_type(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kFloat) return MQ_F32;
    if (t.scalar_type() == at::kHalf) return MQ_F16;
    refuse("%s must be float32 or float16, got %s", name, type_name(t));
}

void matrix_form(const at::Tensor &t, const char *name) {
    if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
        refuse("%s must be 2-D with unit column stride", name);
    // the C ABI takes row strides as int
    if (t.size(0) > 1 && t.stride(0) > INT32_MAX)
        refuse("the rows of %s must be at most %d elements apart, got %lld", name, INT32_MAX,
               (long long)t.stride(0));
}
// The row stride of a row-major matrix of at least rows × cols; for a single
// row, whose stride is never used (a slice may carry any), its width.
int matrix(const at::Tensor &t, int dev, int64_t rows, int64_t cols, const char *name) {
    matrix_form(t, name);
    if (t.size(0) < rows || t.size(1) < cols)
        refuse("%s must be at least %lld x %lld, got (%lld, %lld)", name, (long long)rows,
               (long long)cols, (long long)t.size(0), (long long)t.size(1));
    same_device(t, dev, name);
    return t.size(0) > 1 ? (int)t.stride(0) : to_int(cols);
}

// A bias or a norm's weights: of the layer's own size (a longer vector is another
// layer's; matrices may be wider, as parts of strided buffers are).
const float *vector(const at::Tensor &t, int dev, int64_t n, const char *name) {
    if (t.scalar_type() != at::kFloat)
        refuse("%s must be torch.float32, got %s", name, type_name(t));
    if (t.dim() != 1 || !t.is_contiguous() || t.size(0) != n)
        refuse("%s must be a contiguous vector of %lld elements", name, (long long)n);
    same_device(t, dev, name);
    return (const float *)t.const_data_ptr();
}

at::Tensor make(const at::Tensor &like, std::initializer_list<int64_t> shape, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

at::ScalarType scalar(int type) { return type == MQ_F32 ? at::kFloat : at::kHalf; }

PyObject *status_object(int rc) { return PyLong_FromLong(rc); }

void need_bound(bool bound, Py_ssize_t got, Py_ssize_t want, const char *name) {
    if (!bound) {
        PyErr_SetString(PyExc_RuntimeError, "the library's entry points are not bound");
        throw Refused{};
    }
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
        throw Refused{};
    }
}

// An entry point's body between Python's exceptions and ours.
template <class F>
PyObject *guarded(F body, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return body(a, n);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The address of one entry point out of bind()'s dict; false if it is missing.
template <class F>
bool get_entry(PyObject *dict, F &fn, const char *name) {
    PyObject *v = PyDict_Check(dict) ? PyDict_GetItemString(dict, name) : nullptr;   // borrowed
    void *p = v ? PyLong_AsVoidPtr(v) : nullptr;
    fn = reinterpret_cast<F>(p);
    return p != nullptr;
}

}  // namespace

// The attention operators (binding_attention.cpp).
PyObject *binding_rope(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *binding_kv_store(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *binding_kv_load(PyObject *, PyObject *const *a, Py_ssize_t n);
PyObject *binding_attend(PyObject *, PyObject *const *a, Py_ssize_t n);
bool bind_attention(PyObject *dict);
