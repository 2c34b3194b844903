// C ABI front of the training-step operators (include/convtp_train.h):
// argument validation (host only, before any HIP call), error reporting and
// dispatch.  No exception leaves an entry point.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/convtp.h"
#include "../../include/convtp_train.h"
#include "train_common.hpp"
#include "train_kernels.hpp"

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
constexpr int64_t kMaxStride = int64_t(1) << 40;   // row offsets stay far from 64 bits

int check_stride(int64_t stride, int64_t row, int64_t n_rows, const char* name) {
    // one row has no next one, so its stride is not looked at
    if (n_rows > 1 && (stride < row || stride > kMaxStride))
        return fail(CTP_EINVAL, "%s = %lld, rows have %lld elements", name, (long long)stride, (long long)row);
    return CTP_OK;
}

int check_embed(const conv_tp_embed_problem* p, bool bwd) {
    if (p == nullptr) return fail(CTP_EINVAL, "problem is null");
    if (p->n_tokens < 0 || p->n_rows < 0) return fail(CTP_EINVAL, "negative token or row count");
    if (p->n_tokens > kMaxCount || p->n_rows > kMaxCount - 1)
        return fail(CTP_EUNSUPPORTED, "%lld tokens, %lld rows: above 2^31", (long long)p->n_tokens, (long long)p->n_rows);
    if (p->channels < 1) return fail(CTP_EINVAL, "channels = %d must be >= 1", p->channels);
    if (p->channels > 1 << 20) return fail(CTP_EUNSUPPORTED, "channels = %d above 2^20", p->channels);
    if (!is_dtype(p->dtype)) return fail(CTP_EINVAL, "dtype = %d is no conv_tp_dtype", p->dtype);
    if (p->out_dtype != p->dtype && !(bwd && p->out_dtype == CTP_F32))
        return fail(CTP_EINVAL, "out_dtype = %d must be dtype%s", p->out_dtype, bwd ? " or CTP_F32" : "");
    if (p->index_bits != 32 && p->index_bits != 64) return fail(CTP_EINVAL, "index_bits = %d not 32 or 64", p->index_bits);
    if (int r = check_stride(p->src_stride, p->channels, bwd ? p->n_tokens : p->n_rows, "src_stride")) return r;
    if (int r = check_stride(p->dst_stride, p->channels, bwd ? p->n_rows : p->n_tokens, "dst_stride")) return r;
    return CTP_OK;
}

ctp::EmbedArgs embed_args(const conv_tp_embed_problem* p, const void* tokens, const void* src, void* dst, void* ws) {
    ctp::EmbedArgs a{};
    a.n_tokens = p->n_tokens;
    a.n_rows = p->n_rows;
    a.channels = p->channels;
    a.dtype = p->dtype;
    a.out_dtype = p->out_dtype;
    a.wide_index = p->index_bits == 64;
    a.scale = p->scale;
    a.src_stride = p->src_stride;
    a.dst_stride = p->dst_stride;
    a.tokens = tokens;
    a.src = src;
    a.dst = dst;
    a.workspace = ws;
    return a;
}

int check_norm(const conv_tp_norm_problem* p) {
    if (p == nullptr) return fail(CTP_EINVAL, "problem is null");
    if (p->n_rows < 0) return fail(CTP_EINVAL, "negative row count");
    if (p->n_rows > kMaxCount) return fail(CTP_EUNSUPPORTED, "%lld rows: above 2^31", (long long)p->n_rows);
    if (p->lmax < 0 || p->lmax > 3) return fail(CTP_EUNSUPPORTED, "lmax = %d outside 0..3", p->lmax);
    if (p->channels < 1) return fail(CTP_EINVAL, "channels = %d must be >= 1", p->channels);
    const int64_t comps = (int64_t)(p->lmax + 1) * (p->lmax + 1);
    if (comps * p->channels > ctp::kMaxNormRow)
        return fail(CTP_EUNSUPPORTED, "a row of %lld values: above %d", (long long)(comps * p->channels), ctp::kMaxNormRow);
    if (!is_dtype(p->dtype)) return fail(CTP_EINVAL, "dtype = %d is no conv_tp_dtype", p->dtype);
    if (p->param_dtype != p->dtype && p->param_dtype != CTP_F32)
        return fail(CTP_EINVAL, "param_dtype = %d must be dtype or CTP_F32", p->param_dtype);
    if (p->gate < 0 || p->gate > 2) return fail(CTP_EINVAL, "gate = %d not 0, 1 or 2", p->gate);
    if (!(p->eps >= 0.0f)) return fail(CTP_EINVAL, "eps must be >= 0");
    return CTP_OK;
}

// What the forward and the backward pass check alike.
int check_norm_arrays(const conv_tp_norm_problem* p, const void* h, const void* w_post, const void* w_pre,
                      const void* gate) {
    const int64_t row = (int64_t)(p->lmax + 1) * (p->lmax + 1) * p->channels, par = (int64_t)(p->lmax + 1) * p->channels;
    const uintptr_t e = size_of(p->dtype), q = size_of(p->param_dtype);
    // without rows the features have no addresses, and no parameter's gradient depends on which are there
    if (p->n_rows > 0 && h == nullptr && w_pre == nullptr) return fail(CTP_EINVAL, "h and w_pre are both null: nothing to compute");
    if (p->n_rows > 0 && h == nullptr && (w_post != nullptr || p->gate != ctp::kGateNone))
        return fail(CTP_EINVAL, "w_post or a gate without h");
    if (int r = need(h, 0, e, "h")) return r;
    if (int r = need(w_post, 0, q, "w_post")) return r;
    if (int r = need(w_pre, 0, q, "w_pre")) return r;
    if (h != nullptr)
        if (int r = check_stride(p->h_stride, row, p->n_rows, "h_stride")) return r;
    if (p->gate == ctp::kGateChannel)
        if (int r = need(gate, par, q, "gate")) return r;
    if (p->gate == ctp::kGateRow) {
        if (int r = need(gate, p->n_rows, e, "gate")) return r;
        if (int r = check_stride(p->gate_stride, par, p->n_rows, "gate_stride")) return r;
    }
    return CTP_OK;
}

ctp::NormArgs norm_args(const conv_tp_norm_problem* p, const void* h, const void* r, const void* w_post,
                        const void* w_pre, const void* gate) {
    ctp::NormArgs a{};
    a.n_rows = p->n_rows;
    a.lmax = p->lmax;
    a.channels = p->channels;
    a.dtype = p->dtype;
    a.param_dtype = p->param_dtype;
    a.gate = p->gate;
    a.alpha = p->alpha;
    a.eps = p->eps;
    a.h_stride = p->h_stride;
    a.r_stride = p->r_stride;
    a.gate_stride = p->gate_stride;
    a.grad_r_stride = p->grad_r_stride;
    a.grad_u_stride = p->grad_u_stride;
    a.h = h;
    a.r = r;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.gate_p = gate;
    return a;
}

int check_workspace(const void* ws, int64_t bytes, int64_t wants) {
    if (bytes < wants) return fail(CTP_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)bytes, (long long)wants);
    return need(ws, wants, 16, "workspace");
}

// Checks the first backward pass's inputs and the workspace; fills them in.
int first_bwd_args(const conv_tp_norm_problem* prob, const void* grad_r, const void* grad_u, const void* h,
                   const void* r_out, const void* w_post, const void* w_pre, const void* gate, void* workspace,
                   int64_t workspace_bytes, ctp::NormArgs* out) {
    if (int r = check_norm(prob)) return r;
    const int64_t row = (int64_t)(prob->lmax + 1) * (prob->lmax + 1) * prob->channels, n = prob->n_rows;
    const uintptr_t e = size_of(prob->dtype);
    if (int r = check_norm_arrays(prob, h, w_post, w_pre, gate)) return r;
    if (int r = need(grad_r, 0, e, "grad_r")) return r;
    if (int r = need(grad_u, 0, e, "grad_u")) return r;
    if (grad_u != nullptr && w_pre == nullptr) return fail(CTP_EINVAL, "grad_u without w_pre");
    if (grad_r != nullptr)
        if (int r = check_stride(prob->grad_r_stride, row, n, "grad_r_stride")) return r;
    if (grad_u != nullptr)
        if (int r = check_stride(prob->grad_u_stride, row, n, "grad_u_stride")) return r;
    if (w_pre != nullptr) {
        if (int r = need(r_out, n, e, "r_out")) return r;
        if (int r = check_stride(prob->r_stride, row, n, "r_stride")) return r;
    }
    const int64_t wants = ctp::norm_bwd_workspace(n, prob->lmax, prob->channels);
    if (int r = check_workspace(workspace, workspace_bytes, wants)) return r;
    *out = norm_args(prob, h, r_out, w_post, w_pre, gate);
    out->grad_r = grad_r;
    out->grad_u = grad_u;
    out->workspace = workspace;
    return CTP_OK;
}

// Checks and fills in the gradients that both backward passes write for h and the parameters.
int gradient_args(const conv_tp_norm_problem* prob, ctp::NormArgs* a, void* d_h, void* d_w_post, void* d_w_pre, void* d_gate) {
    const uintptr_t e = size_of(prob->dtype), q = size_of(prob->param_dtype);
    const int64_t n = prob->n_rows, par = (int64_t)(prob->lmax + 1) * prob->channels;
    const bool of_row = prob->gate == ctp::kGateRow;
    if (int r = need(d_h, a->h ? n : 0, e, "the gradient of h")) return r;
    if (int r = need(d_w_post, a->w_post ? par : 0, q, "the gradient of w_post")) return r;
    if (int r = need(d_w_pre, a->w_pre ? par : 0, q, "the gradient of w_pre")) return r;
    if (prob->gate != ctp::kGateNone)
        if (int r = need(d_gate, of_row ? n : par, of_row ? e : q, "the gradient of gate")) return r;
    a->d_h = a->h ? d_h : nullptr;
    a->d_w_post = a->w_post ? d_w_post : nullptr;
    a->d_w_pre = a->w_pre ? d_w_pre : nullptr;
    a->d_gate = prob->gate != ctp::kGateNone ? d_gate : nullptr;
    return CTP_OK;
}

}  // namespace

extern "C" {

int32_t conv_tp_embed_fwd(const conv_tp_embed_problem* prob, const void* table, const void* tokens, void* out,
                          void* stream) {
    if (int r = check_embed(prob, false)) return r;
    const uintptr_t e = size_of(prob->dtype);
    if (int r = need(table, prob->n_tokens ? prob->n_rows : 0, e, "table")) return r;
    if (int r = need(tokens, prob->n_tokens, prob->index_bits / 8, "tokens")) return r;
    if (int r = need(out, prob->n_tokens, e, "out")) return r;
    return hip_status(ctp::launch_embed_fwd(embed_args(prob, tokens, table, out, nullptr), (hipStream_t)stream),
                      "conv_tp_embed_fwd");
}

int32_t conv_tp_embed_bwd_workspace(const conv_tp_embed_problem* prob, int64_t* bytes) {
    if (int r = check_embed(prob, true)) return r;
    if (bytes == nullptr) return fail(CTP_EINVAL, "bytes is null");
    *bytes = ctp::embed_bwd_workspace(prob->n_tokens, prob->n_rows, prob->channels);
    return ok();
}

int32_t conv_tp_embed_bwd(const conv_tp_embed_problem* prob, const void* grad_out, const void* tokens, void* d_table,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    if (int r = check_embed(prob, true)) return r;
    if (int r = need(grad_out, prob->n_tokens, size_of(prob->dtype), "grad_out")) return r;
    if (int r = need(tokens, prob->n_tokens, prob->index_bits / 8, "tokens")) return r;
    if (int r = need(d_table, prob->n_rows, size_of(prob->out_dtype), "d_table")) return r;
    const int64_t wants = ctp::embed_bwd_workspace(prob->n_tokens, prob->n_rows, prob->channels);
    if (int r = check_workspace(workspace, workspace_bytes, wants)) return r;
    return hip_status(ctp::launch_embed_bwd(embed_args(prob, tokens, grad_out, d_table, workspace), (hipStream_t)stream),
                      "conv_tp_embed_bwd");
}

int32_t conv_tp_norm_fwd(const conv_tp_norm_problem* prob, const void* h, const void* r, const void* w_post,
                         const void* w_pre, const void* gate, void* r_out, void* u, void* stream) {
    if (int e = check_norm(prob)) return e;
    const int64_t row = (int64_t)(prob->lmax + 1) * (prob->lmax + 1) * prob->channels;
    const uintptr_t e = size_of(prob->dtype);
    if (int x = check_norm_arrays(prob, h, w_post, w_pre, gate)) return x;
    if (int x = need(r, prob->n_rows, e, "r")) return x;
    if (int x = check_stride(prob->r_stride, row, prob->n_rows, "r_stride")) return x;
    if (int x = need(r_out, h ? prob->n_rows : 0, e, "r_out")) return x;
    if (int x = need(u, w_pre ? prob->n_rows : 0, e, "u")) return x;
    ctp::NormArgs a = norm_args(prob, h, r, w_post, w_pre, gate);
    a.r_out = r_out;
    a.u = u;
    return hip_status(ctp::launch_norm_fwd(a, (hipStream_t)stream), "conv_tp_norm_fwd");
}

int32_t conv_tp_norm_bwd_workspace(const conv_tp_norm_problem* prob, int64_t* bytes) {
    if (int r = check_norm(prob)) return r;
    if (bytes == nullptr) return fail(CTP_EINVAL, "bytes is null");
    *bytes = ctp::norm_bwd_workspace(prob->n_rows, prob->lmax, prob->channels);
    return ok();
}

int32_t conv_tp_norm_bwd(const conv_tp_norm_problem* prob, const void* grad_r, const void* grad_u, const void* h,
                         const void* r_out, const void* w_post, const void* w_pre, const void* gate, void* d_h,
                         void* d_r, void* d_w_post, void* d_w_pre, void* d_gate, void* workspace,
                         int64_t workspace_bytes, void* stream) {
    ctp::NormArgs a{};
    if (int r = first_bwd_args(prob, grad_r, grad_u, h, r_out, w_post, w_pre, gate, workspace, workspace_bytes, &a)) return r;
    if (int r = need(d_r, prob->n_rows, size_of(prob->dtype), "d_r")) return r;
    if (int r = gradient_args(prob, &a, d_h, d_w_post, d_w_pre, d_gate)) return r;
    a.d_r = d_r;
    return hip_status(ctp::launch_norm_bwd(a, (hipStream_t)stream), "conv_tp_norm_bwd");
}

int32_t conv_tp_norm_bwd_bwd(const conv_tp_norm_problem* prob, const void* a_d_h, const void* a_d_r, const void* grad_r,
                             const void* grad_u, const void* h, const void* r_out, const void* w_post,
                             const void* w_pre, const void* gate, void* g_grad_r, void* g_grad_u, void* g_h, void* g_r,
                             void* g_w_post, void* g_w_pre, void* g_gate, void* workspace, int64_t workspace_bytes,
                             void* stream) {
    ctp::NormArgs a{};
    if (int r = first_bwd_args(prob, grad_r, grad_u, h, r_out, w_post, w_pre, gate, workspace, workspace_bytes, &a)) return r;
    const uintptr_t e = size_of(prob->dtype);
    const int64_t n = prob->n_rows;
    if (int r = need(a_d_h, 0, e, "a_d_h")) return r;
    if (int r = need(a_d_r, 0, e, "a_d_r")) return r;
    if (n > 0 && a_d_h != nullptr && h == nullptr) return fail(CTP_EINVAL, "a_d_h without h");
    if (int r = need(g_grad_r, 0, e, "g_grad_r")) return r;
    if (int r = need(g_grad_u, 0, e, "g_grad_u")) return r;
    if (int r = need(g_r, w_pre ? n : 0, e, "g_r")) return r;
    if (int r = gradient_args(prob, &a, g_h, g_w_post, g_w_pre, g_gate)) return r;
    a.a_d_h = a_d_h;
    a.a_d_r = a_d_r;
    a.g_grad_r = g_grad_r;
    a.g_grad_u = w_pre ? g_grad_u : nullptr;
    a.d_r = w_pre ? g_r : nullptr;
    return hip_status(ctp::launch_norm_bwd_bwd(a, (hipStream_t)stream), "conv_tp_norm_bwd_bwd");
}

int64_t conv_tp_clip_workspace(int32_t n_tensors) { return ctp::clip_workspace(n_tensors < 0 ? 0 : n_tensors); }

int32_t conv_tp_clip(int32_t n_tensors, const void* const* in, void* const* out, const int64_t* numel,
                     const int32_t* dtype, float max_norm, float eps, float* norm, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    if (n_tensors < 0) return fail(CTP_EINVAL, "negative tensor count");
    if (n_tensors > 0 && (in == nullptr || numel == nullptr || dtype == nullptr))
        return fail(CTP_EINVAL, "in, numel or dtype is null");
    for (int k = 0; k < n_tensors; ++k) {
        if (!is_dtype(dtype[k])) return fail(CTP_EINVAL, "tensor %d: dtype = %d is no conv_tp_dtype", k, dtype[k]);
        if (numel[k] < 0 || numel[k] > kMaxStride) return fail(CTP_EINVAL, "tensor %d: %lld elements", k, (long long)numel[k]);
        if (int r = need(in[k], numel[k], size_of(dtype[k]), "a tensor of in")) return r;
        if (out != nullptr)
            if (int r = need(out[k], numel[k], size_of(dtype[k]), "a tensor of out")) return r;
    }
    if (out != nullptr && !(max_norm >= 0.0f)) return fail(CTP_EINVAL, "max_norm must be >= 0");
    if (out != nullptr && !(eps >= 0.0f)) return fail(CTP_EINVAL, "eps must be >= 0");
    if (int r = need(norm, 1, 4, "norm")) return r;
    if (int r = check_workspace(workspace, workspace_bytes, conv_tp_clip_workspace(n_tensors))) return r;
    ctp::ClipArgs a{};
    a.n_tensors = n_tensors;
    a.in = in;
    a.out = out;
    static_assert(sizeof(long) == sizeof(int64_t));
    a.numel = reinterpret_cast<const long*>(numel);
    a.dtype = dtype;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = norm;
    a.workspace = static_cast<double*>(workspace);
    return hip_status(ctp::launch_clip(a, (hipStream_t)stream), "conv_tp_clip");
}

const char* conv_tp_train_last_error(void) { return g_last_error; }

}  // extern "C"
