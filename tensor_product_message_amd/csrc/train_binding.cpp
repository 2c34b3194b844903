// Python side of the training-step operators (include/convtp_train.h):
// argument checks, outputs and workspaces from torch's allocator, the current
// stream, and one call of the C ABI.  No computation.
//
// These operators are called on small tensors too, where the host decides: the
// same marshalling in Python took 7 us for a lookup and 21 us for the clipping
// of 21 tensors, of which a kernel launch is 3.
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

// The library's entry points, looked up in the copy that the package has loaded.
struct Library {
    decltype(&conv_tp_embed_fwd) embed_fwd;
    decltype(&conv_tp_embed_bwd) embed_bwd;
    decltype(&conv_tp_embed_bwd_workspace) embed_bwd_workspace;
    decltype(&conv_tp_norm_fwd) norm_fwd;
    decltype(&conv_tp_norm_bwd) norm_bwd;
    decltype(&conv_tp_norm_bwd_bwd) norm_bwd_bwd;
    decltype(&conv_tp_norm_bwd_workspace) norm_bwd_workspace;
    decltype(&conv_tp_clip) clip;
    decltype(&conv_tp_clip_workspace) clip_workspace;
    PyObject* check;    // called with a non-zero status: raises
} lib{};

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
    PyObject* r = PyObject_CallFunction(lib.check, "i", (int)status);
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

int index_bits(const Tensor& tokens, int index) {
    const auto type = tokens.scalar_type();
    if (type != at::kInt && type != at::kLong) bad_value("tokens must be int32 or int64, got ", type);
    on_device(tokens, "tokens", index);
    if (!tokens.is_contiguous()) bad_value("tokens must be contiguous");
    return type == at::kInt ? 32 : 64;
}

std::vector<int64_t> with_channels(const Tensor& tokens, int64_t c) {
    std::vector<int64_t> shape(tokens.sizes().begin(), tokens.sizes().end());
    shape.push_back(c);
    return shape;
}

// ------------------------------------------------------------ embedding

// (table, tokens, scale, out)
PyObject* embed_fwd(PyObject* const* a) {
    const Tensor& table = tensor_of(a[0], "table");
    const int code = float_code(table, "table"), index = device_of(table, "table");
    if (table.dim() != 2 || table.size(1) < 1) bad_value("table must be [rows, C], got ", table.sizes());
    const Tensor& tokens = tensor_of(a[1], "tokens");
    conv_tp_embed_problem p{};
    p.index_bits = index_bits(tokens, index);
    p.n_tokens = tokens.numel();
    p.n_rows = table.size(0);
    const int64_t c = table.size(1);
    p.channels = (int32_t)std::min<int64_t>(c, INT32_MAX);
    p.dtype = p.out_dtype = code;
    p.scale = (float)number_of(a[2]);
    p.src_stride = row_stride(table, "table", table.sizes(), 1, c, table.scalar_type(), index);
    p.dst_stride = c;
    const std::vector<int64_t> shape = with_channels(tokens, c);
    const Tensor* given = maybe_tensor(a[3], "out");
    const c10::DeviceGuard guard(table.device());
    if (given) p.dst_stride = row_stride(*given, "out", shape, 1, c, table.scalar_type(), index);
    const Tensor out = given ? *given : dense(nullptr, "out", shape, table);
    check(lib.embed_fwd(&p, address(table), address(tokens), address(out), stream_of(index)));
    written(given);
    return THPVariable_Wrap(out);
}

// (grad_out, tokens, n_rows, scale, out, dtype, workspace)
PyObject* embed_bwd(PyObject* const* a) {
    const Tensor& grad = tensor_of(a[0], "grad_out");
    conv_tp_embed_problem p{};
    p.dtype = float_code(grad, "grad_out");
    const int index = device_of(grad, "grad_out");
    const Tensor& tokens = tensor_of(a[1], "tokens");
    p.index_bits = index_bits(tokens, index);
    const int64_t c = grad.dim() ? grad.size(-1) : 0;
    if (c < 1 || grad.sizes().slice(0, grad.dim() - 1) != tokens.sizes())
        bad_value("grad_out must have tokens' shape ", tokens.sizes(), " and channels, got ", grad.sizes());
    p.n_tokens = tokens.numel();
    p.n_rows = integer_of(a[2]);
    if (p.n_rows < 0) bad_value("n_rows must be >= 0, got ", p.n_rows);
    p.channels = (int32_t)std::min<int64_t>(c, INT32_MAX);
    p.scale = (float)number_of(a[3]);
    p.src_stride = row_stride(grad, "grad_out", grad.sizes(), 1, c, grad.scalar_type(), index);
    p.dst_stride = c;
    const Tensor* given = maybe_tensor(a[4], "out");
    at::ScalarType type = given ? given->scalar_type() : grad.scalar_type();
    if (a[5] != Py_None) {
        if (!THPDtype_Check(a[5])) refuse(PyExc_TypeError, "dtype must be a torch.dtype");
        type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    }
    p.out_dtype = code_of(type);
    if (p.out_dtype < 0) bad_value("the gradient must be ", grad.scalar_type(), " or float32, got ", type);
    const int64_t shape[2] = {p.n_rows, c};
    if (given) p.dst_stride = row_stride(*given, "out", shape, 1, c, type, index);
    const Tensor* given_ws = maybe_tensor(a[6], "workspace");
    const c10::DeviceGuard guard(grad.device());
    int64_t bytes = 0;
    check(lib.embed_bwd_workspace(&p, &bytes));
    const Tensor out = given ? *given : at::empty(shape, grad.options().dtype(type).requires_grad(false));
    const Workspace ws = workspace(given_ws, bytes, grad);
    check(lib.embed_bwd(&p, address(grad), address(tokens), address(out), address(ws.t), ws.bytes, stream_of(index)));
    written(given);
    written(given_ws);
    return THPVariable_Wrap(out);
}

// ------------------------------------------------------------ norms

struct Norm {
    conv_tp_norm_problem p{};
    int index = 0;
    const Tensor *first = nullptr, *h = nullptr, *r = nullptr, *w_post = nullptr, *w_pre = nullptr, *gate = nullptr;
    const Tensor *grad_r = nullptr, *grad_u = nullptr;
};

// Checks what the two directions share; a: w_post, w_pre, gate, alpha, eps, lmax.
void read_norm(Norm& n, PyObject* const* a) {
    n.w_post = maybe_tensor(a[0], "w_post");
    n.w_pre = maybe_tensor(a[1], "w_pre");
    n.gate = maybe_tensor(a[2], "gate");
    conv_tp_norm_problem& p = n.p;
    p.alpha = (float)number_of(a[3]);
    p.eps = (float)number_of(a[4]);
    const int64_t lmax = integer_of(a[5]);
    if (lmax < 0 || lmax > 3) bad_value("lmax must be 0..3, got ", lmax);
    p.lmax = (int32_t)lmax;
    const char* name = n.h ? "h" : n.r ? "r" : "grad_r";
    n.first = n.h ? n.h : n.r ? n.r : n.grad_r;
    const Tensor& first = *n.first;
    p.dtype = p.param_dtype = float_code(first, name);
    n.index = device_of(first, name);
    const IntArrayRef shape = first.sizes();
    const size_t tail = lmax ? 2 : 1;
    const int64_t comps = (lmax + 1) * (lmax + 1);
    if (shape.size() < tail || shape.back() < 1 || (lmax && shape[shape.size() - 2] != comps))
        bad_value("features must be [..., C], for lmax > 0 [..., (lmax + 1)^2, C]; got ", shape, " for lmax = ", lmax);
    const size_t lead = shape.size() - tail;
    const int64_t c = shape.back(), width = c * comps;
    p.channels = (int32_t)std::min<int64_t>(c, INT32_MAX);
    p.n_rows = 1;
    for (size_t d = 0; d < lead; ++d) p.n_rows *= shape[d];
    const auto type = first.scalar_type();
    auto stride = [&](const Tensor* t, const char* which) {
        return t ? row_stride(*t, which, shape, tail, width, type, n.index) : 0;
    };
    p.h_stride = stride(n.h, "h");
    p.r_stride = stride(n.r, "r");
    p.grad_r_stride = stride(n.grad_r, "grad_r");
    p.grad_u_stride = stride(n.grad_u, "grad_u");
    std::vector<int64_t> per;
    if (lmax) per.push_back(lmax + 1);
    per.push_back(c);
    std::optional<at::ScalarType> param;
    auto parameter = [&](const Tensor* t, const char* which) {
        if (!t) return;
        if (!param) {
            param = t->scalar_type();
            if (*param != type && *param != at::kFloat) bad_value("parameters must be ", type, " or float32, got ", *param);
            p.param_dtype = code_of(*param);
        }
        if (t->scalar_type() != *param) bad_value(which, " must be ", *param, " like the other parameters, got ", t->scalar_type());
        if (t->sizes() != IntArrayRef(per)) bad_value(which, " must have shape ", IntArrayRef(per), ", got ", t->sizes());
        on_device(*t, which, n.index);
        if (!t->is_contiguous()) bad_value(which, " must be contiguous");
    };
    parameter(n.w_post, "w_post");
    parameter(n.w_pre, "w_pre");
    if (!n.gate) return;
    // a single row without a batch: its gate may have either type, and a batch's gate of every row has the features'
    if (n.gate->sizes() == IntArrayRef(per) && (lead > 0 || n.gate->scalar_type() != type)) {
        p.gate = 1;
        parameter(n.gate, "gate");
        return;
    }
    p.gate = 2;
    std::vector<int64_t> rows(shape.begin(), shape.begin() + lead);
    rows.insert(rows.end(), per.begin(), per.end());
    p.gate_stride = row_stride(*n.gate, "gate", rows, tail, c * (lmax + 1), type, n.index);
}

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

// (h, r, w_post, w_pre, gate, alpha, eps, lmax, r_out, u)
PyObject* norm_fwd(PyObject* const* a) {
    Norm n;
    n.h = maybe_tensor(a[0], "h");
    n.r = &tensor_of(a[1], "r");
    read_norm(n, a + 2);
    const Tensor *given_r = maybe_tensor(a[8], "r'"), *given_u = maybe_tensor(a[9], "u");
    const c10::DeviceGuard guard(n.first->device());
    std::optional<Tensor> r_out, u;
    if (n.h) r_out = dense(given_r, "r'", n.first->sizes(), *n.first);
    if (n.w_pre) u = dense(given_u, "u", n.first->sizes(), *n.first);
    check(lib.norm_fwd(&n.p, address(n.h), address(n.r), address(n.w_post), address(n.w_pre), address(n.gate),
                       r_out ? address(*r_out) : nullptr, u ? address(*u) : nullptr, stream_of(n.index)));
    if (r_out) written(given_r);
    if (u) written(given_u);
    PyObject* r;
    if (n.h) {
        r = THPVariable_Wrap(*r_out);
    } else {
        r = a[1];
        Py_INCREF(r);
    }
    return tuple_of({r, wrap_or_none(u)});
}

// a: grad_r, grad_u, h, r_out, w_post, w_pre, gate, alpha, eps, lmax.
void read_first_bwd(Norm& n, PyObject* const* a) {
    n.grad_r = maybe_tensor(a[0], "grad_r");
    n.grad_u = maybe_tensor(a[1], "grad_u");
    n.h = maybe_tensor(a[2], "h");
    n.r = maybe_tensor(a[3], "r_out");
    if (!n.grad_r && !n.grad_u) refuse(PyExc_TypeError, "grad_r and grad_u are both None");
    if (n.grad_u && a[5] == Py_None) bad_value("grad_u without w_pre");
    if (a[5] != Py_None && !n.r) refuse(PyExc_TypeError, "r_out must be a tensor where there is w_pre");
    read_norm(n, a + 4);
}

std::optional<Tensor> like(const Tensor* t) {
    if (!t) return std::nullopt;
    return at::empty(t->sizes(), t->options().requires_grad(false));
}

void* address(const std::optional<Tensor>& t) { return t ? t->data_ptr() : nullptr; }

Workspace norm_workspace(const Norm& n, const Tensor* given) {
    int64_t bytes = 0;
    check(lib.norm_bwd_workspace(&n.p, &bytes));
    return workspace(given, bytes, *n.first);
}

// (grad_r, grad_u, h, r_out, w_post, w_pre, gate, alpha, eps, lmax, workspace)
PyObject* norm_bwd(PyObject* const* a) {
    Norm n;
    read_first_bwd(n, a);
    const Tensor* given_ws = maybe_tensor(a[10], "workspace");
    const c10::DeviceGuard guard(n.first->device());
    const std::optional<Tensor> d_r = like(n.first), d_h = like(n.h), d_w_post = like(n.w_post), d_w_pre = like(n.w_pre),
                                d_gate = like(n.gate);
    const Workspace ws = norm_workspace(n, given_ws);
    check(lib.norm_bwd(&n.p, address(n.grad_r), address(n.grad_u), address(n.h), address(n.r), address(n.w_post),
                       address(n.w_pre), address(n.gate), address(d_h), address(d_r), address(d_w_post),
                       address(d_w_pre), address(d_gate), address(ws.t), ws.bytes, stream_of(n.index)));
    written(given_ws);
    return tuple_of({wrap_or_none(d_h), wrap_or_none(d_r), wrap_or_none(d_w_post), wrap_or_none(d_w_pre), wrap_or_none(d_gate)});
}

// (a_d_h, a_d_r, grad_r, grad_u, h, r_out, w_post, w_pre, gate, alpha, eps, lmax, workspace)
PyObject* norm_bwd_bwd(PyObject* const* a) {
    Norm n;
    read_first_bwd(n, a + 2);
    const Tensor *a_d_h = maybe_tensor(a[0], "a_d_h"), *a_d_r = maybe_tensor(a[1], "a_d_r");
    if (!a_d_h && !a_d_r) refuse(PyExc_TypeError, "a_d_h and a_d_r are both None");
    if (a_d_h && !n.h) bad_value("a_d_h without h");
    for (const Tensor* t : {a_d_h, a_d_r})
        if (t && (t->sizes() != n.first->sizes() || t->scalar_type() != n.first->scalar_type() ||
                  t->device() != n.first->device() || !t->is_contiguous()))
            bad_value("a_d_h and a_d_r must be contiguous and of the features' type, shape and device");
    const Tensor* given_ws = maybe_tensor(a[12], "workspace");
    const c10::DeviceGuard guard(n.first->device());
    const std::optional<Tensor> g_gr = like(n.grad_r), g_gu = like(n.grad_u), g_h = like(n.h),
                                g_r = like(n.w_pre ? n.r : nullptr), g_w_post = like(n.w_post), g_w_pre = like(n.w_pre),
                                g_gate = like(n.gate);
    const Workspace ws = norm_workspace(n, given_ws);
    check(lib.norm_bwd_bwd(&n.p, address(a_d_h), address(a_d_r), address(n.grad_r), address(n.grad_u), address(n.h),
                           address(n.r), address(n.w_post), address(n.w_pre), address(n.gate), address(g_gr),
                           address(g_gu), address(g_h), address(g_r), address(g_w_post), address(g_w_pre),
                           address(g_gate), address(ws.t), ws.bytes, stream_of(n.index)));
    written(given_ws);
    return tuple_of({wrap_or_none(g_gr), wrap_or_none(g_gu), wrap_or_none(g_h), wrap_or_none(g_r), wrap_or_none(g_w_post),
                     wrap_or_none(g_w_pre), wrap_or_none(g_gate)});
}

// ------------------------------------------------------------ clipping

struct TensorList {
    std::vector<void*> at;
    std::vector<int64_t> numel;
    std::vector<int32_t> dtype;

    // `o` is a list
    TensorList(PyObject* o, const char* name, int index) {
        const Py_ssize_t n = PyList_GET_SIZE(o);
        at.reserve(n), numel.reserve(n), dtype.reserve(n);
        for (Py_ssize_t k = 0; k < n; ++k) {
            const Tensor& t = tensor_of(PyList_GET_ITEM(o, k), name);
            dtype.push_back(float_code(t, name));
            on_device(t, name, index);
            if (!t.is_contiguous()) bad_value(name, " must be contiguous (strides ", t.strides(), ")");
            at.push_back(t.data_ptr());
            numel.push_back(t.numel());
        }
    }
};

// (tensors, out, max_norm, eps, norm): lists; out None: the norm alone.  The norm.
PyObject* clip(PyObject* const* a) {
    if (!PyList_Check(a[0]) || (a[1] != Py_None && !PyList_Check(a[1]))) refuse(PyExc_TypeError, "tensors and out must be lists");
    if (PyList_GET_SIZE(a[0]) == 0) bad_value("no tensors");
    const Tensor& first = tensor_of(PyList_GET_ITEM(a[0], 0), "tensors");
    const int index = device_of(first, "tensors");
    const TensorList in(a[0], "tensors", index);
    std::optional<TensorList> out;
    if (a[1] != Py_None) {
        out.emplace(a[1], "out", index);
        if (out->numel != in.numel || out->dtype != in.dtype) bad_value("out must have the tensors' number, sizes and types");
    }
    const Tensor* given = maybe_tensor(a[4], "norm");
    if (given && (given->scalar_type() != at::kFloat || given->numel() != 1 || given->device() != first.device()))
        bad_value("norm must be one float32 value on the tensors' device");
    const c10::DeviceGuard guard(first.device());
    const Tensor norm = given ? *given : at::empty({}, first.options().dtype(at::kFloat).requires_grad(false));
    const int32_t n = (int32_t)in.at.size();
    const Workspace ws = workspace(nullptr, lib.clip_workspace(n), first);
    check(lib.clip(n, in.at.data(), out ? out->at.data() : nullptr, in.numel.data(), in.dtype.data(), (float)number_of(a[2]),
                   (float)number_of(a[3]), norm.data_ptr<float>(), address(ws.t), ws.bytes, stream_of(index)));
    if (out)
        for (Py_ssize_t k = 0; k < PyList_GET_SIZE(a[1]); ++k) written(&tensor_of(PyList_GET_ITEM(a[1], k), "out"));
    written(given);
    return THPVariable_Wrap(norm);
}

// ------------------------------------------------------------ module

// Nothing but Python exceptions leaves an entry point.
template <PyObject* (*F)(PyObject* const*), int Args>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != Args) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", Args, n);
    if (!lib.check) return PyErr_Format(PyExc_RuntimeError, "bind() has not been called");
    try {
        return F(args);
    } catch (const Raise& e) {
        if (e.type) PyErr_SetString(e.type, e.message.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (handle of the loaded library, a callable that raises for a status)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "expected 2 arguments, got %zd", n);
    void* handle = PyLong_AsVoidPtr(args[0]);
    if (PyErr_Occurred()) return nullptr;
    Library l{};
    bool all = true;
    auto find = [&](auto& f, const char* name) { all &= (f = (std::decay_t<decltype(f)>)dlsym(handle, name)) != nullptr; };
    find(l.embed_fwd, "conv_tp_embed_fwd");
    find(l.embed_bwd, "conv_tp_embed_bwd");
    find(l.embed_bwd_workspace, "conv_tp_embed_bwd_workspace");
    find(l.norm_fwd, "conv_tp_norm_fwd");
    find(l.norm_bwd, "conv_tp_norm_bwd");
    find(l.norm_bwd_bwd, "conv_tp_norm_bwd_bwd");
    find(l.norm_bwd_workspace, "conv_tp_norm_bwd_workspace");
    find(l.clip, "conv_tp_clip");
    find(l.clip_workspace, "conv_tp_clip_workspace");
    if (!all) return PyErr_Format(PyExc_RuntimeError, "the library lacks an entry point of include/convtp_train.h");
    Py_INCREF(args[1]);
    l.check = args[1];
    lib = l;
    Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"embed_fwd", fast(entry<embed_fwd, 4>), METH_FASTCALL, nullptr},
    {"embed_bwd", fast(entry<embed_bwd, 7>), METH_FASTCALL, nullptr},
    {"norm_fwd", fast(entry<norm_fwd, 10>), METH_FASTCALL, nullptr},
    {"norm_bwd", fast(entry<norm_bwd, 11>), METH_FASTCALL, nullptr},
    {"norm_bwd_bwd", fast(entry<norm_bwd_bwd, 13>), METH_FASTCALL, nullptr},
    {"clip", fast(entry<clip, 5>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_train", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__train() { return PyModule_Create(&module); }
