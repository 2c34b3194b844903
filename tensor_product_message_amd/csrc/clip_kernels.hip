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
//
// Memory bounds both kernels: 604 MB of bf16 are read in 105 us (5.8 TB/s), and
// read and written in 202 us (6.0 TB/s).  21 tensors of 850 KB take 4 and 5 us,
// little more than an empty kernel.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "train_common.hpp"
#include "train_kernels.hpp"

namespace ctp {

namespace {

constexpr int kThreads = 256;
constexpr int kPerLaunch = 128;
constexpr long kChunk = 2048;       // elements; a workgroup takes a run of chunks
constexpr int kMaxGroups = 1024;    // workgroups, and partial sums, of a launch: four a CU (eight are no faster)
constexpr int kAhead = 4;           // vectors that a lane has on their way

struct Batch {
    const void* in[kPerLaunch];
    void* out[kPerLaunch];
    int64_t numel[kPerLaunch];
    int32_t first[kPerLaunch + 1];  // first chunk of each tensor, and the number of chunks
    uint8_t dtype[kPerLaunch];
    int n;
};

// Calls f(tensor, begin, end) for the elements that a workgroup has of each
// tensor: the chunks of all tensors, in a row, are cut into equal runs.
template <class F>
__device__ __forceinline__ void each_span(const Batch& b, F&& f) {
    const long chunks = b.first[b.n];
    const int from = (int)(chunks * blockIdx.x / gridDim.x), to = (int)(chunks * (blockIdx.x + 1) / gridDim.x);
    // The last tensor whose first chunk is not beyond the run's.  All first
    // chunks are read at once, one a lane: the arguments lie in host memory, and
    // a search by halves would go there step by step.
    const int lane = threadIdx.x % 64;
    int t = -1;
#pragma unroll
    for (int k = 0; k < kPerLaunch; k += 64) t += __popcll(__ballot(k + lane < b.n && b.first[k + lane] <= from));
    for (; t < b.n && b.first[t] < to; ++t) {
        const long lo = max(from, b.first[t]) - b.first[t], hi = min(to, b.first[t + 1]) - b.first[t];
        if (hi > lo) f(t, lo * kChunk, min(hi * kChunk, (long)b.numel[t]));
    }
}

template <class T>
__device__ __forceinline__ double square(T x) {
    const double d = (double)(float)x;
    return d * d;
}

template <class T>
__device__ __forceinline__ double squares(const T* x, long n) {
    double s = 0.0;
    const long whole = n / kVec<T>;
    auto* xv = reinterpret_cast<const typename Vec<T>::unaligned*>(x);
    long v = threadIdx.x;
    for (; v + (kAhead - 1) * kThreads < whole; v += kAhead * kThreads) {
        vec_t<T> q[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) q[u] = xv[v + u * kThreads];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                const double d = (double)(float)q[u][k];
                s = __builtin_fma(d, d, s);
            }
    }
    for (; v < whole; v += kThreads) {
        const vec_t<T> q = xv[v];
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) s += square(q[k]);
    }
    const long at = whole * kVec<T> + threadIdx.x;
    if (at < n) s += square(x[at]);
    return s;
}

// What a value is multiplied by, in two steps.  The norm may be above fp32's
// largest number and the factor below its smallest normal one where the clipped
// values are neither: then `factor` is 2^64 times it, and `then` 2^-64.  Else
// `then` is 1, which leaves the first product as it is.
struct Factor {
    float factor, then;
};

__device__ __forceinline__ Factor factor_of(double norm, float max_norm, float eps) {
    float f = max_norm / ((float)norm + eps);
    if (f > 1.0f) f = 1.0f;       // a NaN norm stays NaN
    if (f < 0x1p-126f && norm < __builtin_inf())
        return {(float)(0x1p64 * ((double)max_norm / (norm + (double)eps))), 0x1p-64f};
    return {f, 1.0f};
}

// y = factor x.
template <class T, bool Stream>
__device__ __forceinline__ void scaled(const T* x, T* y, long n, Factor by) {
    const long whole = n / kVec<T>;
    auto* xv = reinterpret_cast<const typename Vec<T>::unaligned*>(x);
    auto* yv = reinterpret_cast<typename Vec<T>::unaligned*>(y);
    auto put = [&](long v, const vec_t<T>& q) {
        Floats<T> f = widen<T>(q);
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) f.v[k] = f.v[k] * by.factor * by.then;
        if (Stream) __builtin_nontemporal_store(narrow<T>(f), yv + v);
        else yv[v] = narrow<T>(f);
    };
    long v = threadIdx.x;
    for (; v + (kAhead - 1) * kThreads < whole; v += kAhead * kThreads) {
        vec_t<T> q[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) q[u] = Stream ? __builtin_nontemporal_load(xv + v + u * kThreads) : xv[v + u * kThreads];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) put(v + u * kThreads, q[u]);
    }
    for (; v < whole; v += kThreads) {
        const vec_t<T> q = xv[v];
        put(v, q);
    }
    const long at = whole * kVec<T> + threadIdx.x;
    if (at < n) y[at] = (T)((float)x[at] * by.factor * by.then);
}

// Calls f with a value of the type of a code.
template <class F>
__device__ __forceinline__ void typed(int dtype, F&& f) {
    if (dtype == kBF16) f(__bf16{});
    else if (dtype == kF16) f(_Float16{});
    else f(float{});
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

__global__ void __launch_bounds__(kThreads) k_clip_squares(Batch b, double* __restrict__ partial) {
    __shared__ double part[kThreads / 64];
    double s = 0.0;
    each_span(b, [&](int t, long begin, long end) {
        typed(b.dtype[t], [&](auto x) {
            using T = decltype(x);
            s += squares(static_cast<const T*>(b.in[t]) + begin, end - begin);
        });
    });
    s = group_sum(s, part);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// Every workgroup adds all partial sums for itself; the first one writes the norm.
__device__ __forceinline__ double total_norm(const double* partial, int n_partial, double* part) {
    double s = 0.0;
    for (int k = threadIdx.x; k < n_partial; k += kThreads) s += partial[k];
    return sqrt(group_sum(s, part));
}

__global__ void __launch_bounds__(kThreads) k_clip_norm(const double* __restrict__ partial, int n_partial, float* norm) {
    __shared__ double part[kThreads / 64];
    const double x = total_norm(partial, n_partial, part);
    if (threadIdx.x == 0) *norm = (float)x;
}

// Stream: where much is moved, neither what is read here nor what is written
// pushes out of the last-level cache what the first kernel left there (its
// reads are not marked; 604 MB of bf16: 309 us, 363 without the marks here, 332
// with the first kernel's reads marked too; 77 MB of float: 43 and 54 us).
template <bool Stream>
__global__ void __launch_bounds__(kThreads)
k_clip_scale(Batch b, const double* __restrict__ partial, int n_partial, float max_norm, float eps, float* norm) {
    __shared__ double part[kThreads / 64];
    const double x = total_norm(partial, n_partial, part);
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = (float)x;
    const Factor by = factor_of(x, max_norm, eps);
    each_span(b, [&](int t, long begin, long end) {
        // in place with nothing to clip: the values stay as they are
        if (by.factor == 1.0f && by.then == 1.0f && b.in[t] == b.out[t]) return;
        typed(b.dtype[t], [&](auto q) {
            using T = decltype(q);
            scaled<T, Stream>(static_cast<const T*>(b.in[t]) + begin, static_cast<T*>(b.out[t]) + begin, end - begin, by);
        });
    });
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
    long bytes = 0;
    auto batches = [&](auto&& go) {
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
            if (chunks > 0) go(std::min(chunks, (int32_t)kMaxGroups));
        }
    };
    for (int k = 0; k < a.n_tensors; ++k) bytes += a.numel[k] * (a.dtype[k] == kF32 ? 4 : 2);
    batches([&](int grid) {
        k_clip_squares<<<grid, kThreads, 0, st>>>(b, a.workspace + n_partial);
        n_partial += grid;
    });
    if (!a.out || n_partial == 0) {
        k_clip_norm<<<1, kThreads, 0, st>>>(a.workspace, n_partial, a.norm);
        return hipGetLastError();
    }
    float* norm = a.norm;       // the first launch writes it
    batches([&](int grid) {
        auto* kernel = streams(3 * bytes) ? k_clip_scale<true> : k_clip_scale<false>;
        kernel<<<grid, kThreads, 0, st>>>(b, a.workspace, n_partial, a.max_norm, a.eps, norm);
        norm = nullptr;
    });
    return hipGetLastError();
}

}  // namespace ctp
