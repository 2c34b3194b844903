// Launch interface between the C ABI front of the training-step operators
// (train_api.hip) and their kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ctp {

struct EmbedArgs {
    long n_tokens, n_rows;  // tokens, rows of the table: each below 2^31
    int channels;
    int dtype;              // DType of table and out (forward), of grad_out (backward)
    int out_dtype;          // backward: DType of d_table (dtype or kF32)
    int wide_index;         // tokens are int64 (1) or int32 (0)
    float scale;
    long src_stride;        // elements from row to row of table (forward) or grad_out (backward)
    long dst_stride;        // of out or d_table
    const void* tokens;
    const void* src;
    void* dst;
    void* workspace;        // backward
};

long embed_bwd_workspace(long n_tokens, long n_rows, int channels);
hipError_t launch_embed_fwd(const EmbedArgs& a, hipStream_t st);
hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t st);

enum Gate : int { kGateNone = 0, kGateChannel = 1, kGateRow = 2 };

struct NormArgs {
    long n_rows;
    int lmax, channels;     // D = (lmax + 1)^2 components
    int dtype;              // DType of the features and of a gate for every row
    int param_dtype;        // DType of w_post, w_pre, a gate of one row and their gradients (dtype or kF32)
    int gate;               // Gate
    float alpha, eps;
    // element strides from row to row of the inputs; outputs are dense
    long h_stride, r_stride, gate_stride, grad_r_stride, grad_u_stride;
    const void *h, *r;      // h null: no block output, r' = r
    const void *w_post, *w_pre, *gate_p;        // w_post null: N(h) is h itself; w_pre null: no u
    void *r_out, *u;        // forward
    const void *grad_r, *grad_u;                // backward (null: zero)
    void *d_h, *d_r, *d_w_post, *d_w_pre, *d_gate;
    const void *a_d_h, *a_d_r;                  // second backward: cotangents of d_h and d_r, dense (null: zero);
    void *g_grad_r, *g_grad_u;                  // its gradients in h, r' and the parameters are d_*, these in grad_*
    void* workspace;
    bool stream, stream_out;    // set by the launch: reads, writes are non-temporal
};

// Largest row: D * channels values.
constexpr int kMaxNormRow = 16384;
long norm_bwd_workspace(long n_rows, int lmax, int channels);
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd_bwd(const NormArgs& a, hipStream_t st);

struct ClipArgs {
    int n_tensors;
    const void* const* in;      // host arrays of n_tensors entries
    void* const* out;           // null: the norm alone
    const long* numel;
    const int* dtype;
    float max_norm, eps;
    float* norm;
    double* workspace;
};

long clip_workspace(int n_tensors);
hipError_t launch_clip(const ClipArgs& a, hipStream_t st);

}  // namespace ctp
