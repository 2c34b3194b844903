// Launch functions of the training-step operators, stubbed out for the
// sanitizer build of their C ABI front (as launch_stubs.hip for the
// convolution's): a stub succeeds where its call has nothing to launch and
// reports an error otherwise.
#include <hip/hip_runtime.h>

#include "../../tensor_product_message_amd/csrc/train_kernels.hpp"

namespace ctp {

long embed_bwd_workspace(long n_tokens, long, int) { return 64 * n_tokens + 256; }
hipError_t launch_embed_fwd(const EmbedArgs& a, hipStream_t) { return a.n_tokens == 0 ? hipSuccess : hipErrorNotSupported; }
hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t) { return a.n_rows == 0 ? hipSuccess : hipErrorNotSupported; }
long norm_bwd_workspace(long n_rows, int, int channels) { return 16 * n_rows * channels; }
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t) { return a.n_rows == 0 ? hipSuccess : hipErrorNotSupported; }
hipError_t launch_norm_bwd(const NormArgs&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_norm_bwd_bwd(const NormArgs&, hipStream_t) { return hipErrorNotSupported; }
long clip_workspace(int n_tensors) { return 256 + 8 * n_tensors; }
hipError_t launch_clip(const ClipArgs&, hipStream_t) { return hipErrorNotSupported; }

}  // namespace ctp
