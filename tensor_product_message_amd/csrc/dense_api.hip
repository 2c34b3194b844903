// C ABI front of the dense operators (include/convtp_dense.h): argument
// validation (host only, before any HIP call), error reporting and dispatch.
// No exception leaves an entry point.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/convtp.h"
#include "../../include/convtp_dense.h"
#include "dense_kernels.hpp"
#include "train_common.hpp"

namespace {

thread_local char g_last_error[512] = "";

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return code;
}

int ok() {
    g_last_error[0] = 0;
    return CTP_OK;
}

int hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(CTP_EHIP, "%s: %s", what, hipGetErrorString(e));
}

// A pointer is required when its array has elements; alignment is checked whenever it is non-null.
int need(const void* p, int64_t count, uintptr_t align, const char* name) {
    if (count > 0 && p == nullptr) return fail(CTP_EINVAL, "%s is null but has %lld elements", name, (long long)count);
    if (reinterpret_cast<uintptr_t>(p) & (align - 1))
        return fail(CTP_EALIGN, "%s is not %u-byte aligned", name, (unsigned)align);
    return CTP_OK;
}

bool is_dtype(int d) { return d == CTP_F32 || d == CTP_BF16 || d == CTP_F16; }
uintptr_t size_of(int dtype) { return dtype == CTP_F32 ? 4 : 2; }

constexpr int64_t kMaxCount = 0x7fffffff;
constexpr int64_t kMaxStride = int64_t(1) << 40;    // row offsets stay far from 64 bits
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxSide = int64_t(1) << 17;

int check_stride(int64_t stride, int64_t row, int64_t n_rows, const char* name) {
    // one row has no next one, so its stride is not looked at
    if (n_rows > 1 && (stride < row || stride > kMaxStride))
        return fail(CTP_EINVAL, "%s = %lld, rows have %lld elements", name, (long long)stride, (long long)row);
    return CTP_OK;
}

bool has_act(const conv_tp_linear_problem* p) { return p->act != CTP_ACT_NONE || p->gated; }
int64_t comps_of(const conv_tp_linear_problem* p) { return (int64_t)(p->lmax + 1) * (p->lmax + 1); }

int check_linear(const conv_tp_linear_problem* p) {
    if (p == nullptr) return fail(CTP_EINVAL, "problem is null");
    if (p->n_rows < 0) return fail(CTP_EINVAL, "negative row count");
    if (p->n_rows > kMaxCount) return fail(CTP_EUNSUPPORTED, "%lld rows: above 2^31", (long long)p->n_rows);
    if (p->lmax < 0 || p->lmax > 3) return fail(CTP_EUNSUPPORTED, "lmax = %d outside 0..3", p->lmax);
    if (p->inner < 1 || p->outer < 1) return fail(CTP_EINVAL, "inner = %d and outer = %d must be >= 1", p->inner, p->outer);
    if (comps_of(p) * p->inner > kMaxWidth || comps_of(p) * p->outer > kMaxWidth)
        return fail(CTP_EUNSUPPORTED, "rows of %lld and %lld values: above 2^20", (long long)(comps_of(p) * p->inner),
                    (long long)(comps_of(p) * p->outer));
    if (!is_dtype(p->dtype)) return fail(CTP_EINVAL, "dtype = %d is no conv_tp_dtype", p->dtype);
    if (p->act < CTP_ACT_NONE || p->act > CTP_ACT_TANH) return fail(CTP_EINVAL, "act = %d is no conv_tp_act", p->act);
    if (p->gated != 0 && p->gated != 1) return fail(CTP_EINVAL, "gated = %d not 0 or 1", p->gated);
    if (p->lmax > 0 && has_act(p)) return fail(CTP_EINVAL, "an activation or a gate of components of degree > 0");
    return CTP_OK;
}

ctp::LinearArgs linear_args(const conv_tp_linear_problem* p) {
    ctp::LinearArgs a{};
    a.n_rows = p->n_rows;
    a.lmax = p->lmax;
    a.inner = p->inner;
    a.outer = p->outer;
    a.dtype = p->dtype;
    a.act = p->act;
    a.gated = p->gated != 0;
    // one row has no next one: a stride that nothing reads, but tiles count with it
    const bool one = p->n_rows <= 1;
    a.x_stride = one ? comps_of(p) * p->inner : p->x_stride;
    a.residual_stride = one ? comps_of(p) * p->outer : p->residual_stride;
    a.grad_stride = one ? comps_of(p) * p->outer : p->grad_stride;
    return a;
}

// What a workspace's size depends on, as the call itself checks it; it is the call's own strides that count.
int check_strides(const conv_tp_linear_problem* p, bool grad) {
    if (int r = check_stride(p->x_stride, comps_of(p) * p->inner, p->n_rows, "x_stride")) return r;
    return grad ? check_stride(p->grad_stride, comps_of(p) * p->outer, p->n_rows, "grad_stride") : CTP_OK;
}

int check_workspace(const void* ws, int64_t bytes, int64_t wants) {
    if (bytes < wants) return fail(CTP_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)bytes, (long long)wants);
    return need(ws, wants, 16, "workspace");
}

// x, w and what the backward passes read besides.
int check_inputs(const conv_tp_linear_problem* p, const void* x, const void* w, bool need_w) {
    const uintptr_t e = size_of(p->dtype);
    if (int r = need(x, p->n_rows, e, "x")) return r;
    if (int r = check_stride(p->x_stride, comps_of(p) * p->inner, p->n_rows, "x_stride")) return r;
    return need(w, need_w ? p->n_rows : 0, e, "w");
}
int check_grad(const conv_tp_linear_problem* p, const void* grad, const void* z) {
    const uintptr_t e = size_of(p->dtype);
    if (int r = need(grad, p->n_rows, e, "grad")) return r;
    if (int r = check_stride(p->grad_stride, comps_of(p) * p->outer, p->n_rows, "grad_stride")) return r;
    return need(z, has_act(p) ? p->n_rows : 0, e, "z");
}

int check_matrices(int32_t n_tensors, const int64_t* batch, const int32_t* rows, const int32_t* cols) {
    if (n_tensors < 0) return fail(CTP_EINVAL, "negative tensor count");
    if (n_tensors > 0 && (batch == nullptr || rows == nullptr || cols == nullptr))
        return fail(CTP_EINVAL, "batch, rows or cols is null");
    for (int k = 0; k < n_tensors; ++k) {
        if (batch[k] < 0 || rows[k] < 0 || cols[k] < 0) return fail(CTP_EINVAL, "tensor %d: a negative size", k);
        if (rows[k] > kMaxSide || cols[k] > kMaxSide)
            return fail(CTP_EUNSUPPORTED, "tensor %d: a side of %d above 2^17", k, rows[k] > cols[k] ? rows[k] : cols[k]);
        const int64_t size = (int64_t)rows[k] * cols[k];
        if (size > 0 && batch[k] > (int64_t(1) << 38) / size)
            return fail(CTP_EUNSUPPORTED, "tensor %d: above 2^38 elements", k);
        if (batch[k] > 1 << 16) return fail(CTP_EUNSUPPORTED, "tensor %d: %lld matrices, above 2^16", k, (long long)batch[k]);
    }
    return CTP_OK;
}

}  // namespace

extern "C" {

int32_t conv_tp_linear_fwd_workspace(const conv_tp_linear_problem* prob, int64_t* bytes) {
    if (int r = check_linear(prob)) return r;
    if (int r = check_strides(prob, false)) return r;
    if (bytes == nullptr) return fail(CTP_EINVAL, "bytes is null");
    *bytes = ctp::linear_fwd_workspace(linear_args(prob));
    return ok();
}

int32_t conv_tp_linear_fwd(const conv_tp_linear_problem* prob, const void* x, const void* w, const void* bias,
                           const void* residual, void* y, void* z, void* workspace, int64_t workspace_bytes,
                           void* stream) {
    if (int r = check_linear(prob)) return r;
    const uintptr_t e = size_of(prob->dtype);
    if (int r = check_inputs(prob, x, w, true)) return r;
    if (int r = need(bias, 0, e, "bias")) return r;
    if (int r = need(residual, 0, e, "residual")) return r;
    if (residual != nullptr) {
        if (prob->gated) return fail(CTP_EINVAL, "a residual of the gated form");
        if (int r = check_stride(prob->residual_stride, comps_of(prob) * prob->outer, prob->n_rows, "residual_stride")) return r;
    }
    if (int r = need(y, prob->n_rows, e, "y")) return r;
    if (int r = need(z, 0, e, "z")) return r;
    ctp::LinearArgs a = linear_args(prob);
    if (int r = check_workspace(workspace, workspace_bytes, ctp::linear_fwd_workspace(a))) return r;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.residual = residual;
    a.y = y;
    a.z_out = z;
    a.workspace = workspace;
    return hip_status(ctp::launch_linear_fwd(a, (hipStream_t)stream), "conv_tp_linear_fwd");
}

int32_t conv_tp_linear_bwd_workspace(const conv_tp_linear_problem* prob, int64_t* bytes) {
    if (int r = check_linear(prob)) return r;
    if (int r = check_strides(prob, true)) return r;
    if (bytes == nullptr) return fail(CTP_EINVAL, "bytes is null");
    *bytes = ctp::linear_bwd_workspace(linear_args(prob));
    return ok();
}

int32_t conv_tp_linear_bwd(const conv_tp_linear_problem* prob, const void* grad, const void* x, const void* w,
                           const void* z, void* d_x, void* d_w, void* d_bias, void* workspace,
                           int64_t workspace_bytes, void* stream) {
    if (int r = check_linear(prob)) return r;
    const uintptr_t e = size_of(prob->dtype);
    if (int r = check_inputs(prob, x, w, d_x != nullptr)) return r;
    if (int r = check_grad(prob, grad, z)) return r;
    if (int r = need(d_x, 0, e, "d_x")) return r;
    if (int r = need(d_w, 0, e, "d_w")) return r;
    if (int r = need(d_bias, 0, e, "d_bias")) return r;
    ctp::LinearArgs a = linear_args(prob);
    if (int r = check_workspace(workspace, workspace_bytes, ctp::linear_bwd_workspace(a))) return r;
    a.x = x;
    a.w = w;
    a.grad = grad;
    a.z = z;
    a.d_x = d_x;
    a.d_w = d_w;
    a.d_bias = d_bias;
    a.workspace = workspace;
    return hip_status(ctp::launch_linear_bwd(a, (hipStream_t)stream), "conv_tp_linear_bwd");
}

int32_t conv_tp_linear_bwd_bwd_workspace(const conv_tp_linear_problem* prob, int64_t* bytes) {
    if (int r = check_linear(prob)) return r;
    if (int r = check_strides(prob, true)) return r;
    if (bytes == nullptr) return fail(CTP_EINVAL, "bytes is null");
    *bytes = ctp::linear_bwd_bwd_workspace(linear_args(prob));
    return ok();
}

int32_t conv_tp_linear_bwd_bwd(const conv_tp_linear_problem* prob, const void* a_d_x, const void* grad, const void* x,
                               const void* w, const void* z, void* g_grad, void* g_x, void* g_w, void* g_bias,
                               void* workspace, int64_t workspace_bytes, void* stream) {
    if (int r = check_linear(prob)) return r;
    const uintptr_t e = size_of(prob->dtype);
    if (int r = need(a_d_x, prob->n_rows, e, "a_d_x")) return r;
    if (int r = check_inputs(prob, x, w, true)) return r;
    if (int r = check_grad(prob, grad, z)) return r;
    if (!has_act(prob) && (g_x != nullptr || g_bias != nullptr))
        return fail(CTP_EINVAL, "g_x or g_bias without an activation: they are zero");
    if (int r = need(g_grad, 0, e, "g_grad")) return r;
    if (int r = need(g_x, 0, e, "g_x")) return r;
    if (int r = need(g_w, 0, e, "g_w")) return r;
    if (int r = need(g_bias, 0, e, "g_bias")) return r;
    ctp::LinearArgs a = linear_args(prob);
    if (int r = check_workspace(workspace, workspace_bytes, ctp::linear_bwd_bwd_workspace(a))) return r;
    a.x = x;
    a.w = w;
    a.grad = grad;
    a.z = z;
    a.a_d_x = a_d_x;
    a.g_grad = g_grad;
    a.g_x = g_x;
    a.g_w = g_w;
    a.g_bias = g_bias;
    a.workspace = workspace;
    return hip_status(ctp::launch_linear_bwd_bwd(a, (hipStream_t)stream), "conv_tp_linear_bwd_bwd");
}

int32_t conv_tp_orthogonalise_workspace(int32_t n_tensors, const int64_t* batch, const int32_t* rows,
                                        const int32_t* cols, int64_t* bytes) {
    if (int r = check_matrices(n_tensors, batch, rows, cols)) return r;
    if (bytes == nullptr) return fail(CTP_EINVAL, "bytes is null");
    static_assert(sizeof(long) == sizeof(int64_t));
    *bytes = ctp::ortho_workspace(n_tensors, reinterpret_cast<const long*>(batch), rows, cols);
    return ok();
}

int32_t conv_tp_orthogonalise(int32_t n_tensors, const void* const* in, void* const* out, const int64_t* batch,
                              const int32_t* rows, const int32_t* cols, const int32_t* dtype, int32_t steps, float eps,
                              float scale, void* workspace, int64_t workspace_bytes, void* stream) {
    if (int r = check_matrices(n_tensors, batch, rows, cols)) return r;
    if (n_tensors > 0 && (in == nullptr || out == nullptr || dtype == nullptr))
        return fail(CTP_EINVAL, "in, out or dtype is null");
    for (int k = 0; k < n_tensors; ++k) {
        if (!is_dtype(dtype[k])) return fail(CTP_EINVAL, "tensor %d: dtype = %d is no conv_tp_dtype", k, dtype[k]);
        const int64_t size = batch[k] * rows[k] * cols[k];
        if (int r = need(in[k], size, size_of(dtype[k]), "a tensor of in")) return r;
        if (int r = need(out[k], size, size_of(dtype[k]), "a tensor of out")) return r;
    }
    if (steps < 1 || steps > 64) return fail(CTP_EINVAL, "steps = %d outside 1..64", steps);
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(CTP_EINVAL, "eps must be >= 0 and finite");
    if (!std::isfinite(scale)) return fail(CTP_EINVAL, "scale must be finite");
    ctp::OrthoArgs a{};
    a.n_tensors = n_tensors;
    a.in = in;
    a.out = out;
    a.batch = reinterpret_cast<const long*>(batch);
    a.rows = rows;
    a.cols = cols;
    a.dtype = dtype;
    a.steps = steps;
    a.eps = eps;
    a.scale = scale;
    a.workspace = workspace;
    if (int r = check_workspace(workspace, workspace_bytes, ctp::ortho_workspace(n_tensors, a.batch, rows, cols))) return r;
    return hip_status(ctp::launch_ortho(a, (hipStream_t)stream), "conv_tp_orthogonalise");
}

const char* conv_tp_dense_last_error(void) { return g_last_error; }

}  // extern "C"
