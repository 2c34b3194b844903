// Launch functions of the dense operators, stubbed out for the sanitizer build
// of their C ABI front (as train_stubs.hip for the training step's): a stub
// succeeds where its call has nothing to launch and reports an error otherwise.
#include <hip/hip_runtime.h>

#include "../../tensor_product_message_amd/csrc/dense_kernels.hpp"

namespace ctp {

namespace {
long values(const LinearArgs& a) { return a.n_rows * a.outer * (a.gated ? 2 : 1); }
}  // namespace

long linear_fwd_workspace(const LinearArgs&) { return 0; }
long linear_bwd_workspace(const LinearArgs& a) { return 4 * values(a) + 256; }
long linear_bwd_bwd_workspace(const LinearArgs& a) { return 8 * values(a) + 256; }
hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t) { return a.n_rows == 0 ? hipSuccess : hipErrorNotSupported; }
hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t) { return a.n_rows == 0 ? hipSuccess : hipErrorNotSupported; }
hipError_t launch_linear_bwd_bwd(const LinearArgs&, hipStream_t) { return hipErrorNotSupported; }

long ortho_workspace(int n_tensors, const long* batch, const int* rows, const int* cols) {
    long bytes = 0;
    for (int k = 0; k < n_tensors; ++k) bytes += 12 * batch[k] * rows[k] * cols[k];
    return bytes;
}
hipError_t launch_ortho(const OrthoArgs& a, hipStream_t) {
    return ortho_workspace(a.n_tensors, a.batch, a.rows, a.cols) == 0 ? hipSuccess : hipErrorNotSupported;
}

}  // namespace ctp
