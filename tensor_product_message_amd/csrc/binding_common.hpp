// What the bindings of the C ABI share: argument checks, outputs and workspaces
// from torch's allocator, the current stream, errors.  Included once by each
// binding module.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include "../../include/convtp.h"
#include "../../include/convtp_train.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

PyObject* status_check = nullptr;   // called with a non-zero status: raises

// A Python exception to raise at the boundary; type null: already set.
struct Raise {
    PyObject* type;
    std::string message;
};

template <class... A>
[[noreturn]] void refuse(PyObject* type, const A&... parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw Raise{type, s.str()};
}
template <class... A>
[[noreturn]] void bad_value(const A&... parts) {
    refuse(PyExc_ValueError, parts...);
}

void check(int32_t status) {
    if (status == CTP_OK) return;
    PyObject* r = PyObject_CallFunction(status_check, "i", (int)status);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "status %d", (int)status);
    throw Raise{nullptr, {}};
}

// ------------------------------------------------------------ arguments

const Tensor& tensor_of(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// Null for None.
const Tensor* maybe_tensor(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor_of(o, name); }

double number_of(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raise{nullptr, {}};
    return x;
}

int64_t integer_of(PyObject* o) {
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raise{nullptr, {}};
    return x;
}

// conv_tp_dtype of a type, or -1.
int code_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return CTP_F32;
        case at::kBFloat16: return CTP_BF16;
        case at::kHalf: return CTP_F16;
        default: return -1;
    }
}

int float_code(const Tensor& t, const char* name) {
    const int c = code_of(t.scalar_type());
    if (c < 0) bad_value(name, " must be float32, bfloat16 or float16, got ", t.scalar_type());
    return c;
}

int device_of(const Tensor& t, const char* name) {
    if (!t.is_cuda()) bad_value(name, " must be on a HIP device, got ", t.device());
    return t.get_device();
}

void on_device(const Tensor& t, const char* name, int index) {
    if (!t.is_cuda() || t.get_device() != index) bad_value(name, " is on ", t.device(), ", expected device ", index);
}

// Elements from row to row of a tensor of shape [..., tail] of rows of `width` dense values.
int64_t row_stride(const Tensor& t, const char* name, IntArrayRef shape, size_t tail, int64_t width, at::ScalarType type,
                   int index) {
    if (t.scalar_type() != type) bad_value(name, " must be ", type, ", got ", t.scalar_type());
    if (t.sizes() != shape) bad_value(name, " must have shape ", shape, ", got ", t.sizes());
    on_device(t, name, index);
    if (t.is_contiguous()) return width;
    const auto strides = t.strides();
    const size_t lead = shape.size() - tail;
    int64_t dense = 1;
    for (size_t d = shape.size(); d-- > lead;) {
        if (shape[d] > 1 && strides[d] != dense) bad_value(name, ": a row must be contiguous (strides ", strides, ")");
        dense *= shape[d];
    }
    int64_t stride = 0, next = 0;       // of the innermost leading dimension; what the next outer one has to be
    for (size_t d = lead; d-- > 0;) {
        if (shape[d] <= 1) continue;
        if (stride == 0) {
            stride = strides[d];
            if (stride < width) bad_value(name, ": its rows must not overlap (strides ", strides, ")");
        } else if (strides[d] != next) {
            bad_value(name, ": its rows must lie one stride apart (strides ", strides, ")");
        }
        next = strides[d] * shape[d];
    }
    return stride ? stride : width;
}

// A dense tensor of a shape, or the caller's (`given`).
Tensor dense(const Tensor* given, const char* name, IntArrayRef shape, const Tensor& like) {
    if (!given) return at::empty(shape, like.options().requires_grad(false));
    if (given->sizes() != shape || given->scalar_type() != like.scalar_type() || given->device() != like.device() ||
        !given->is_contiguous())
        bad_value(name, " must be a contiguous ", like.scalar_type(), " tensor of shape ", shape, " on ", like.device());
    return *given;
}

struct Workspace {
    Tensor t;
    int64_t bytes;
};

// Unless the caller gives one, from torch's allocator on the current stream, which orders its reuse.
Workspace workspace(const Tensor* given, int64_t bytes, const Tensor& like) {
    if (!given) {
        bytes = std::max<int64_t>(16, bytes);
        return {at::empty({bytes}, like.options().dtype(at::kByte).requires_grad(false)), bytes};
    }
    if (given->device() != like.device() || !given->is_contiguous())
        bad_value("workspace must be a contiguous tensor on the inputs' device");
    return {*given, (int64_t)given->nbytes()};
}

// After a call has written a tensor that the caller gave: a backward pass that saved it must see that it has
// changed.  Inference tensors cannot be saved and have no version.
void written(const Tensor* t) {
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

void* address(const Tensor& t) { return t.data_ptr(); }
void* address(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

void* stream_of(int index) { return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)index).stream(); }

PyObject* wrap_or_none(const std::optional<Tensor>& t) {
    if (t) return THPVariable_Wrap(*t);
    Py_RETURN_NONE;
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {     // takes the references
    PyObject* t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t k = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, k++, o);
    return t;
}

[[maybe_unused]] std::optional<Tensor> like(const Tensor* t) {
    if (!t) return std::nullopt;
    return at::empty(t->sizes(), t->options().requires_grad(false));
}

void* address(const std::optional<Tensor>& t) { return t ? t->data_ptr() : nullptr; }

// Nothing but Python exceptions leaves an entry point.
template <PyObject* (*F)(PyObject* const*), int Args>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != Args) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", Args, n);
    if (!status_check) return PyErr_Format(PyExc_RuntimeError, "bind() has not been called");
    try {
        return F(args);
    } catch (const Raise& e) {
        if (e.type) PyErr_SetString(e.type, e.message.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <class F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace
