// Launch interface between the C ABI front of the dense operators
// (dense_api.hip) and their kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ctp {

// Activations of the C ABI (conv_tp_act).
enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActSigmoid = 4, kActTanh = 5 };

struct LinearArgs {
    long n_rows;            // below 2^31
    int lmax;               // D = (lmax + 1)^2 components a row, one matrix a degree
    int inner, outer;       // values of a component of x, of y
    int dtype, act;
    bool gated;             // w is two matrices, y = act(z[0]) z[1], z [row][2][outer]; lmax = 0
    // element strides from row to row of the inputs; outputs and z are dense
    long x_stride, residual_stride, grad_stride;
    const void *x, *w, *bias, *residual;        // bias, residual null: none
    void *y, *z_out;        // forward; z_out null: not wanted
    const void *grad, *z;   // backward; z null without an activation
    void *d_x, *d_w, *d_bias;                   // null: not wanted
    const void* a_d_x;      // second backward: cotangent of d_x, dense; its gradients are g_*
    void *g_grad, *g_x, *g_w, *g_bias;
    void* workspace;
};

long linear_fwd_workspace(const LinearArgs& a);
long linear_bwd_workspace(const LinearArgs& a);
long linear_bwd_bwd_workspace(const LinearArgs& a);
hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_bwd_bwd(const LinearArgs& a, hipStream_t st);

struct OrthoArgs {
    int n_tensors;
    const void* const* in;  // host arrays of n_tensors entries
    void* const* out;
    const long* batch;      // matrices of each tensor, dense one after the other
    const int *rows, *cols;
    const int* dtype;
    int steps;
    float eps, scale;
    void* workspace;
};

long ortho_workspace(int n_tensors, const long* batch, const int* rows, const int* cols);
hipError_t launch_ortho(const OrthoArgs& a, hipStream_t st);

}  // namespace ctp
