// The global norm of many gradients, and their clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + eps))
//
// The factor is known only when everything has been read, so clipping reads
// twice.  Squares are summed in 64 bits: neither large nor small gradients
// leave the range of the sum, and the vector units add 64-bit numbers faster
// than memory delivers 32-bit ones.  Every workgroup writes one partial sum
// and the second kernel adds them in a fixed order, so a repeated call gives
// the same bits.
//
// The tensors' addresses travel in the kernel arguments (no table to copy to
// the device, so a call can be captured in a graph); kPerLaunch of them fit
// into one launch.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "train_common.hpp"
#include "train_kernels.hpp"

namespace ctp {

namespace {

constexpr int kThreads = 256;
constexpr int kPerLaunch = 128;
constexpr long kChunk = 16384;      // elements a workgroup takes at a time
constexpr int kMaxGroups = 2048;    // workgroups, and partial sums, of a launch

struct Batch {
    const void* in[kPerLaunch];
    void* out[kPerLaunch];
    int64_t numel[kPerLaunch];
    int32_t first[kPerLaunch + 1];  // first chunk of each tensor
    uint8_t dtype[kPerLaunch];
    int n;
};

// Tensor of a chunk: the last one whose first chunk is not beyond it.
__device__ __forceinline__ int tensor_of(const Batch& b, int chunk) {
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (b.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <class T>
__device__ __forceinline__ double squares(const T* x, long n) {
    double s = 0.0;
    const long whole = n / kVec<T>;
#pragma unroll 4
    for (long v = threadIdx.x; v < whole; v += kThreads) {
        const vec_t<T> q = *reinterpret_cast<const typename Vec<T>::unaligned*>(x + v * kVec<T>);
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) {
            const double d = (double)(float)q[k];
            s = __builtin_fma(d, d, s);
        }
    }
    const long at = whole * kVec<T> + threadIdx.x;
    if (at < n) {
        const double d = (double)(float)x[at];
        s = __builtin_fma(d, d, s);
    }
    return s;
}

template <class T>
__device__ __forceinline__ void scaled(const T* x, T* y, long n, float factor) {
    const long whole = n / kVec<T>;
#pragma unroll 4
    for (long v = threadIdx.x; v < whole; v += kThreads) {
        Floats<T> f = widen<T>(*reinterpret_cast<const typename Vec<T>::unaligned*>(x + v * kVec<T>));
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) f.v[k] *= factor;
        *reinterpret_cast<typename Vec<T>::unaligned*>(y + v * kVec<T>) = narrow<T>(f);
    }
    const long at = whole * kVec<T> + threadIdx.x;
    if (at < n) y[at] = (T)((float)x[at] * factor);
}

// Sum over the workgroup in a fixed order, in every thread.
__device__ __forceinline__ double group_sum(double x, double* part) {
    x = wave_sum(x);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) s += part[w];
    return s;
}

__global__ void __launch_bounds__(kThreads) k_clip_squares(Batch b, int chunks, double* __restrict__ partial) {
    __shared__ double part[kThreads / 64];
    double s = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(b, c);
        const long at = (long)(c - b.first[t]) * kChunk, n = min(kChunk, (long)b.numel[t] - at);
        if (b.dtype[t] == kBF16) s += squares(static_cast<const __bf16*>(b.in[t]) + at, n);
        else if (b.dtype[t] == kF16) s += squares(static_cast<const _Float16*>(b.in[t]) + at, n);
        else s += squares(static_cast<const float*>(b.in[t]) + at, n);
    }
    s = group_sum(s, part);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// Every workgroup adds all partial sums for itself; the first one writes the norm.
__device__ __forceinline__ float total_norm(const double* partial, int n_partial, double* part) {
    double s = 0.0;
    for (int k = threadIdx.x; k < n_partial; k += kThreads) s += partial[k];
    return (float)sqrt(group_sum(s, part));
}

__global__ void __launch_bounds__(kThreads) k_clip_norm(const double* __restrict__ partial, int n_partial, float* norm) {
    __shared__ double part[kThreads / 64];
    const float x = total_norm(partial, n_partial, part);
    if (threadIdx.x == 0) *norm = x;
}

__global__ void __launch_bounds__(kThreads)
k_clip_scale(Batch b, int chunks, const double* __restrict__ partial, int n_partial, float max_norm, float eps, float* norm) {
    __shared__ double part[kThreads / 64];
    const float x = total_norm(partial, n_partial, part);
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = x;
    float factor = max_norm / (x + eps);
    if (factor > 1.0f) factor = 1.0f;       // a NaN norm stays NaN
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(b, c);
        // in place with nothing to clip: the values stay as they are
        if (factor == 1.0f && b.in[t] == b.out[t]) continue;
        const long at = (long)(c - b.first[t]) * kChunk, n = min(kChunk, (long)b.numel[t] - at);
        if (b.dtype[t] == kBF16) scaled(static_cast<const __bf16*>(b.in[t]) + at, static_cast<__bf16*>(b.out[t]) + at, n, factor);
        else if (b.dtype[t] == kF16) scaled(static_cast<const _Float16*>(b.in[t]) + at, static_cast<_Float16*>(b.out[t]) + at, n, factor);
        else scaled(static_cast<const float*>(b.in[t]) + at, static_cast<float*>(b.out[t]) + at, n, factor);
    }
}

long chunks_of(long numel) { return (numel + kChunk - 1) / kChunk; }

}  // namespace

long clip_workspace(int n_tensors) {
    const long launches = ((long)n_tensors + kPerLaunch - 1) / kPerLaunch;
    return std::max(1L, launches) * kMaxGroups * (long)sizeof(double);
}

hipError_t launch_clip(const ClipArgs& a, hipStream_t st) {
    Batch b;
    int n_partial = 0;
    auto batches = [&](auto&& go) {
        bool first = true;
        for (int t0 = 0; t0 < a.n_tensors; t0 += kPerLaunch) {
            b.n = std::min(kPerLaunch, a.n_tensors - t0);
            int32_t chunks = 0;
            for (int k = 0; k < b.n; ++k) {
                b.in[k] = a.in[t0 + k];
                b.out[k] = a.out ? a.out[t0 + k] : nullptr;
                b.numel[k] = a.numel[t0 + k];
                b.dtype[k] = (uint8_t)a.dtype[t0 + k];
                b.first[k] = chunks;
                chunks += (int32_t)chunks_of(b.numel[k]);
            }
            b.first[b.n] = chunks;
            if (chunks == 0) continue;
            go(chunks, std::min(chunks, (int32_t)kMaxGroups), first);
            first = false;
        }
        return first;
    };
    batches([&](int chunks, int grid, bool) {
        k_clip_squares<<<grid, kThreads, 0, st>>>(b, chunks, a.workspace + n_partial);
        n_partial += grid;
    });
    if (!a.out || n_partial == 0) {
        k_clip_norm<<<1, kThreads, 0, st>>>(a.workspace, n_partial, a.norm);
        return hipGetLastError();
    }
    batches([&](int chunks, int grid, bool first) {
        k_clip_scale<<<grid, kThreads, 0, st>>>(b, chunks, a.workspace, n_partial, a.max_norm, a.eps, first ? a.norm : nullptr);
    });
    return hipGetLastError();
}

}  // namespace ctp
