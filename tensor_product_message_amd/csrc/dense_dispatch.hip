// The linear layers' passes by element type.
#include "dense_linear.hpp"
#include "train_common.hpp"

namespace ctp {
namespace {

const LinearOps& ops_of(int dtype) {
    if (dtype == kBF16) return linear_ops<kBF16>();
    if (dtype == kF16) return linear_ops<kF16>();
    return linear_ops<kF32>();
}

}  // namespace

long linear_fwd_workspace(const LinearArgs& a) { return ops_of(a.dtype).fwd_workspace(a); }
long linear_bwd_workspace(const LinearArgs& a) { return ops_of(a.dtype).bwd_workspace(a, false); }
long linear_bwd_bwd_workspace(const LinearArgs& a) { return ops_of(a.dtype).bwd_workspace(a, true); }
hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t st) { return a.n_rows ? ops_of(a.dtype).fwd(a, st) : hipSuccess; }
hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t st) { return ops_of(a.dtype).bwd(a, st); }
hipError_t launch_linear_bwd_bwd(const LinearArgs& a, hipStream_t st) { return ops_of(a.dtype).bwd_bwd(a, st); }

}  // namespace ctp
