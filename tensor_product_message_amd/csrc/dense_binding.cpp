// Python side of the dense operators (include/convtp_dense.h), as
// train_binding.cpp for the training step's.  No computation.
#include "binding_common.hpp"

#include "../../include/convtp_dense.h"

namespace {

// The library's entry points, looked up in the copy that the package has loaded.
struct Library {
    decltype(&conv_tp_linear_fwd) linear_fwd;
    decltype(&conv_tp_linear_fwd_workspace) linear_fwd_workspace;
    decltype(&conv_tp_linear_bwd) linear_bwd;
    decltype(&conv_tp_linear_bwd_workspace) linear_bwd_workspace;
    decltype(&conv_tp_linear_bwd_bwd) linear_bwd_bwd;
    decltype(&conv_tp_linear_bwd_bwd_workspace) linear_bwd_bwd_workspace;
    decltype(&conv_tp_orthogonalise) orthogonalise;
    decltype(&conv_tp_orthogonalise_workspace) orthogonalise_workspace;
} lib{};

// ------------------------------------------------------------ linear layers

struct Linear {
    conv_tp_linear_problem p{};
    int index = 0;
    const Tensor *x = nullptr, *w = nullptr;
    std::vector<int64_t> rows, in_shape, out_shape, z_shape, bias_shape;
    size_t tail = 1;
    int64_t comps = 1;
};

bool flag_of(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Raise{nullptr, {}};
    return x != 0;
}

// a: x, w; then act, lmax, gated.
void read_linear(Linear& n, PyObject* const* a, PyObject* const* how) {
    n.x = &tensor_of(a[0], "x");
    n.w = &tensor_of(a[1], "w");
    const Tensor &x = *n.x, &w = *n.w;
    conv_tp_linear_problem& p = n.p;
    p.act = (int32_t)integer_of(how[0]);
    const int64_t lmax = integer_of(how[1]);
    if (lmax < 0 || lmax > 3) bad_value("lmax must be 0..3, got ", lmax);
    p.lmax = (int32_t)lmax;
    p.gated = flag_of(how[2]);
    if (lmax && (p.gated || p.act != CTP_ACT_NONE)) bad_value("degrees above 0 have no activation (lmax = ", lmax, ")");
    p.dtype = float_code(x, "x");
    n.index = device_of(x, "x");
    n.tail = lmax ? 2 : 1;
    n.comps = (lmax + 1) * (lmax + 1);
    const IntArrayRef shape = x.sizes();
    if (shape.size() < n.tail || shape.back() < 1 || (lmax && shape[shape.size() - 2] != n.comps))
        bad_value("x must be [..., inner], for lmax > 0 [..., (lmax + 1)^2, inner]; got ", shape, " for lmax = ", lmax);
    const int64_t inner = shape.back();
    const bool stacked = lmax || p.gated;
    if (w.scalar_type() != x.scalar_type()) bad_value("w must be ", x.scalar_type(), ", got ", w.scalar_type());
    on_device(w, "w", n.index);
    if (w.dim() != (stacked ? 3 : 2) || w.size(-1) != inner || w.size(-2) < 1 ||
        (stacked && w.size(0) != (lmax ? lmax + 1 : 2)))
        bad_value("w must be ", p.gated ? "[2, outer, inner]" : lmax ? "[lmax + 1, outer, inner]" : "[outer, inner]",
                  " with x's inner = ", inner, ", got ", w.sizes());
    if (!w.is_contiguous()) bad_value("w must be contiguous (strides ", w.strides(), ")");
    const int64_t outer = w.size(-2);
    n.rows.assign(shape.begin(), shape.end() - (ptrdiff_t)n.tail);
    p.n_rows = 1;
    for (const int64_t s : n.rows) p.n_rows *= s;
    p.inner = (int32_t)std::min<int64_t>(inner, INT32_MAX);
    p.outer = (int32_t)std::min<int64_t>(outer, INT32_MAX);
    n.in_shape.assign(shape.begin(), shape.end());
    n.out_shape = n.in_shape;
    n.out_shape.back() = outer;
    n.z_shape = n.out_shape;
    if (p.gated) n.z_shape.insert(n.z_shape.end() - 1, 2);
    n.bias_shape = p.gated ? std::vector<int64_t>{2, outer} : std::vector<int64_t>{outer};
    p.x_stride = row_stride(x, "x", n.in_shape, n.tail, n.comps * inner, x.scalar_type(), n.index);
}

Workspace workspace_of(const Linear& n, decltype(&conv_tp_linear_bwd_workspace) size, const Tensor* given) {
    int64_t bytes = 0;
    check(size(&n.p, &bytes));
    return workspace(given, bytes, *n.x);
}

// (x, w, bias, residual, act, lmax, gated, keep_z, out)
PyObject* linear_fwd(PyObject* const* a) {
    Linear n;
    read_linear(n, a, a + 4);
    const Tensor *bias = maybe_tensor(a[2], "bias"), *residual = maybe_tensor(a[3], "residual");
    const auto type = n.x->scalar_type();
    if (bias && (bias->sizes() != IntArrayRef(n.bias_shape) || bias->scalar_type() != type || !bias->is_contiguous()))
        bad_value("bias must be a contiguous ", type, " tensor of shape ", IntArrayRef(n.bias_shape));
    if (bias) on_device(*bias, "bias", n.index);
    if (residual)
        n.p.residual_stride = row_stride(*residual, "residual", n.out_shape, n.tail, n.comps * n.p.outer, type, n.index);
    const bool keep_z = flag_of(a[7]);
    const Tensor* given = maybe_tensor(a[8], "out");
    const c10::DeviceGuard guard(n.x->device());
    const Tensor y = dense(given, "out", n.out_shape, *n.x);
    std::optional<Tensor> z;
    if (keep_z) z = dense(nullptr, "z", n.z_shape, *n.x);
    int64_t bytes = 0;
    check(lib.linear_fwd_workspace(&n.p, &bytes));
    std::optional<Workspace> ws;
    if (bytes > 0) ws = workspace(nullptr, bytes, *n.x);
    check(lib.linear_fwd(&n.p, address(n.x), address(n.w), address(bias), address(residual), address(y), address(z),
                         ws ? address(ws->t) : nullptr, ws ? ws->bytes : 0, stream_of(n.index)));
    written(given);
    return tuple_of({THPVariable_Wrap(y), wrap_or_none(z)});
}

struct Grad {
    const Tensor *grad, *z;
};

// grad, (x, w,) z
Grad read_grad(Linear& n, PyObject* grad, PyObject* z) {
    Grad g{&tensor_of(grad, "grad"), maybe_tensor(z, "z")};
    const auto type = n.x->scalar_type();
    n.p.grad_stride = row_stride(*g.grad, "grad", n.out_shape, n.tail, n.comps * n.p.outer, type, n.index);
    const bool need = n.p.gated || n.p.act != CTP_ACT_NONE;
    if (need && !g.z) refuse(PyExc_TypeError, "z must be a tensor where there is an activation");
    if (g.z && (g.z->sizes() != IntArrayRef(n.z_shape) || g.z->scalar_type() != type || !g.z->is_contiguous()))
        bad_value("z must be a contiguous ", type, " tensor of shape ", IntArrayRef(n.z_shape), ", got ", g.z->sizes());
    if (g.z) on_device(*g.z, "z", n.index);
    if (!need) g.z = nullptr;
    return g;
}

std::optional<Tensor> wanted(PyObject* need, IntArrayRef shape, const Tensor& like) {
    if (!flag_of(need)) return std::nullopt;
    return at::empty(shape, like.options().requires_grad(false));
}

// (grad, x, w, z, act, lmax, gated, need_x, need_w, need_bias, workspace)
PyObject* linear_bwd(PyObject* const* a) {
    Linear n;
    read_linear(n, a + 1, a + 4);
    const Grad g = read_grad(n, a[0], a[3]);
    const Tensor* given = maybe_tensor(a[10], "workspace");
    const c10::DeviceGuard guard(n.x->device());
    const std::optional<Tensor> d_x = wanted(a[7], n.in_shape, *n.x), d_w = wanted(a[8], n.w->sizes(), *n.x),
                                d_bias = wanted(a[9], n.bias_shape, *n.x);
    const Workspace ws = workspace_of(n, lib.linear_bwd_workspace, given);
    check(lib.linear_bwd(&n.p, address(g.grad), address(n.x), address(n.w), address(g.z), address(d_x), address(d_w),
                         address(d_bias), address(ws.t), ws.bytes, stream_of(n.index)));
    written(given);
    return tuple_of({wrap_or_none(d_x), wrap_or_none(d_w), wrap_or_none(d_bias)});
}

// (a_d_x, grad, x, w, z, act, lmax, gated, need_grad, need_x, need_w, need_bias, workspace)
PyObject* linear_bwd_bwd(PyObject* const* a) {
    Linear n;
    read_linear(n, a + 2, a + 5);
    const Grad g = read_grad(n, a[1], a[4]);
    const Tensor& u = tensor_of(a[0], "a_d_x");
    if (u.sizes() != IntArrayRef(n.in_shape) || u.scalar_type() != n.x->scalar_type() || !u.is_contiguous())
        bad_value("a_d_x must be a contiguous ", n.x->scalar_type(), " tensor of x's shape ", IntArrayRef(n.in_shape));
    on_device(u, "a_d_x", n.index);
    const Tensor* given = maybe_tensor(a[12], "workspace");
    const c10::DeviceGuard guard(n.x->device());
    const std::optional<Tensor> g_grad = wanted(a[8], n.out_shape, *n.x), g_x = wanted(a[9], n.in_shape, *n.x),
                                g_w = wanted(a[10], n.w->sizes(), *n.x), g_bias = wanted(a[11], n.bias_shape, *n.x);
    const Workspace ws = workspace_of(n, lib.linear_bwd_bwd_workspace, given);
    check(lib.linear_bwd_bwd(&n.p, address(u), address(g.grad), address(n.x), address(n.w), address(g.z), address(g_grad),
                             address(g_x), address(g_w), address(g_bias), address(ws.t), ws.bytes, stream_of(n.index)));
    written(given);
    return tuple_of({wrap_or_none(g_grad), wrap_or_none(g_x), wrap_or_none(g_w), wrap_or_none(g_bias)});
}

// ------------------------------------------------------------ orthogonalising

struct Matrices {
    std::vector<void*> at;
    std::vector<int64_t> batch;
    std::vector<int32_t> rows, cols, dtype;

    // `o` is a list
    Matrices(PyObject* o, const char* name, int index) {
        const Py_ssize_t n = PyList_GET_SIZE(o);
        at.reserve(n), batch.reserve(n), rows.reserve(n), cols.reserve(n), dtype.reserve(n);
        for (Py_ssize_t k = 0; k < n; ++k) {
            const Tensor& t = tensor_of(PyList_GET_ITEM(o, k), name);
            dtype.push_back(float_code(t, name));
            on_device(t, name, index);
            if (t.dim() < 2) bad_value(name, " must be matrices [..., rows, cols], got ", t.sizes());
            if (!t.is_contiguous()) bad_value(name, " must be contiguous (strides ", t.strides(), ")");
            int64_t b = 1;
            for (const int64_t s : t.sizes().slice(0, t.dim() - 2)) b *= s;
            at.push_back(t.data_ptr());
            batch.push_back(b);
            rows.push_back((int32_t)std::min<int64_t>(t.size(-2), INT32_MAX));
            cols.push_back((int32_t)std::min<int64_t>(t.size(-1), INT32_MAX));
        }
    }
};

// (tensors, out, steps, eps, scale, workspace): lists.
PyObject* orthogonalise(PyObject* const* a) {
    if (!PyList_Check(a[0]) || !PyList_Check(a[1])) refuse(PyExc_TypeError, "tensors and out must be lists");
    if (PyList_GET_SIZE(a[0]) == 0) bad_value("no tensors");
    const Tensor& first = tensor_of(PyList_GET_ITEM(a[0], 0), "tensors");
    const int index = device_of(first, "tensors");
    const Matrices in(a[0], "tensors", index), out(a[1], "out", index);
    if (out.batch != in.batch || out.rows != in.rows || out.cols != in.cols || out.dtype != in.dtype)
        bad_value("out must have the tensors' number, shapes and types");
    const Tensor* given = maybe_tensor(a[5], "workspace");
    const int64_t steps = integer_of(a[2]);
    if (steps < 1 || steps > 64) bad_value("steps must be 1..64, got ", steps);
    const c10::DeviceGuard guard(first.device());
    const int32_t n = (int32_t)in.at.size();
    int64_t bytes = 0;
    check(lib.orthogonalise_workspace(n, in.batch.data(), in.rows.data(), in.cols.data(), &bytes));
    const Workspace ws = workspace(given, bytes, first);
    check(lib.orthogonalise(n, in.at.data(), out.at.data(), in.batch.data(), in.rows.data(), in.cols.data(),
                            in.dtype.data(), (int32_t)steps, (float)number_of(a[3]), (float)number_of(a[4]),
                            address(ws.t), ws.bytes, stream_of(index)));
    for (Py_ssize_t k = 0; k < PyList_GET_SIZE(a[1]); ++k) written(&tensor_of(PyList_GET_ITEM(a[1], k), "out"));
    written(given);
    Py_RETURN_NONE;
}

// ------------------------------------------------------------ module

// (handle of the loaded library, a callable that raises for a status)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "expected 2 arguments, got %zd", n);
    void* handle = PyLong_AsVoidPtr(args[0]);
    if (PyErr_Occurred()) return nullptr;
    Library l{};
    bool all = true;
    auto find = [&](auto& f, const char* name) { all &= (f = (std::decay_t<decltype(f)>)dlsym(handle, name)) != nullptr; };
    find(l.linear_fwd, "conv_tp_linear_fwd");
    find(l.linear_fwd_workspace, "conv_tp_linear_fwd_workspace");
    find(l.linear_bwd, "conv_tp_linear_bwd");
    find(l.linear_bwd_workspace, "conv_tp_linear_bwd_workspace");
    find(l.linear_bwd_bwd, "conv_tp_linear_bwd_bwd");
    find(l.linear_bwd_bwd_workspace, "conv_tp_linear_bwd_bwd_workspace");
    find(l.orthogonalise, "conv_tp_orthogonalise");
    find(l.orthogonalise_workspace, "conv_tp_orthogonalise_workspace");
    if (!all) return PyErr_Format(PyExc_RuntimeError, "the library lacks an entry point of include/convtp_dense.h");
    Py_INCREF(args[1]);
    status_check = args[1];
    lib = l;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"linear_fwd", fast(entry<linear_fwd, 9>), METH_FASTCALL, nullptr},
    {"linear_bwd", fast(entry<linear_bwd, 11>), METH_FASTCALL, nullptr},
    {"linear_bwd_bwd", fast(entry<linear_bwd_bwd, 13>), METH_FASTCALL, nullptr},
    {"orthogonalise", fast(entry<orthogonalise, 6>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense() { return PyModule_Create(&module); }
