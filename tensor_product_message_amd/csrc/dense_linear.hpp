// The linear layers' passes of one element type (dense_linear.hip), by DType.
#pragma once

#include "dense_kernels.hpp"

namespace ctp {

struct LinearOps {
    hipError_t (*fwd)(const LinearArgs&, hipStream_t);
    hipError_t (*bwd)(const LinearArgs&, hipStream_t);
    hipError_t (*bwd_bwd)(const LinearArgs&, hipStream_t);
    long (*fwd_workspace)(const LinearArgs&);
    long (*bwd_workspace)(const LinearArgs&, bool second);
};

template <int Code>
const LinearOps& linear_ops();
template <>
const LinearOps& linear_ops<0>();
template <>
const LinearOps& linear_ops<1>();
template <>
const LinearOps& linear_ops<2>();

}  // namespace ctp
