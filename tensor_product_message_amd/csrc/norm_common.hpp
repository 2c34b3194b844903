// Norms after and before a block, fused with the block's gate and the scaled
// residual, and their gradient.  One row is [D][C] with D = (lmax + 1)^2
// components of the degrees 0..lmax (lmax = 0: a plain row of C values):
//
//   N(x; w)[d, c] = w[l(d), c] x[d, c] s(x)
//   s(x) = (eps + sum_{d, c} b_d x[d, c]^2)^(-1/2),  b_d = 1 / ((lmax + 1) (2 l(d) + 1) C)
//   r' = r + alpha g N(h; w_post)          u = N(r'; w_pre)
//
// and for gradients dr' and du
//
//   A = w_pre du        d  = dr' + s2 (A - b_d <A, s2 r'> s2 r')   (s2 = s(r'))
//   dy = alpha g d      B  = w_post dy
//   dh = s1 (B - b_d <B, s1 h> s1 h)                               (s1 = s(h))
//   dr = d,  dw_pre = sum du r' s2,  dw_post = sum dy h s1,  dg = sum alpha d N(h; w_post)
//
// with the sums over the rows, and the components of a degree, that share the
// parameter (s x and not s^3: the cube leaves fp32 for rows of 1e13).  A row
// is read once and stays in registers between the two reductions that it
// needs; memory bounds both directions.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "train_common.hpp"
#include "train_kernels.hpp"

namespace ctp {

__device__ __forceinline__ int degree_of(int d) { return d < 1 ? 0 : d < 4 ? 1 : d < 9 ? 2 : 3; }

// Where one of a lane's vectors sits in the row: its degree and its vector of
// the component's channels, and the elements of the row, and of a row of one
// component a degree, at which it is read and written.  All the offsets are 32
// bits from the start of a row that the whole wave shares, so that an access
// takes a scalar address and one offset register.
struct Place {
    int l, v, left;         // left: values from the vector's first to the component's end
    bool on;
    Span span;
    unsigned from, to, par_from, par_to;
};

template <class T>
__device__ __forceinline__ Place place_of(int i, int nvec, int comps, int channels) {
    Place p;
    const int d = comps == 1 ? 0 : i / nvec;
    p.v = i - d * nvec;
    p.on = i < nvec * comps;
    p.l = degree_of(d);
    p.left = channels - p.v * kVec<T>;
    p.span = span_of<T>(p.v, channels);
    p.from = d * channels + p.span.at;
    p.to = d * channels + p.v * kVec<T>;
    p.par_from = p.l * channels + p.span.at;
    p.par_to = p.l * channels + p.v * kVec<T>;
    return p;
}

// Row of the array of a lane's row (the whole wave's, but for rows of 16 lanes).
template <class T>
__device__ __forceinline__ T* row_of(const void* x, long row, long stride) {
    return static_cast<T*>(const_cast<void*>(x)) + row * stride;
}

// Row `sub` of those that a workgroup has at once, known to the compiler as the same in the wave where it is.
template <int Lanes>
__device__ __forceinline__ int row_in_group() {
    if (Lanes >= 256) return 0;
    const int sub = threadIdx.x / Lanes;
    return Lanes >= 64 ? __builtin_amdgcn_readfirstlane(sub) : sub;
}

// A row of parameters for every degree, in T or (`wide`) in fp32.
template <class T>
struct Params {
    const void* base;
    bool wide;
    int channels;
    __device__ __forceinline__ Floats<T> load(const Place& p) const {
        return load_param<T>(static_cast<const char*>(base) + (size_t)p.l * channels * (wide ? 4 : sizeof(T)), wide, p.v, channels);
    }
};

// Threads of a workgroup: one row of `Lanes` lanes each, several rows where they are short.
template <int Lanes>
constexpr int kNormThreads = Lanes < 256 ? 256 : Lanes;
constexpr int rows_at_once(int lanes) { return lanes < 256 ? 256 / lanes : 1; }

// Sums of a row's values over its lanes.  Rows of up to 64 lanes reduce in a
// wave; the waves of wider ones meet in LDS, `slot` alternating so that one
// barrier a reduction is enough.
template <int Lanes>
constexpr int kSumWaves = Lanes > 64 ? kNormThreads<Lanes> / 64 : 1;

template <int Lanes, int N>
struct RowSum {
    float (*part)[N][kSumWaves<Lanes>];
    int slot = 0;
    __device__ __forceinline__ void operator()(float (&x)[N]) {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = lane_sum<(Lanes < 64 ? Lanes : 64)>(x[k]);
        if constexpr (Lanes > 64) {
            constexpr int kOfRow = Lanes / 64;
            const int wave = threadIdx.x / 64, first = wave / kOfRow * kOfRow;
            if (threadIdx.x % 64 == 0)
#pragma unroll
                for (int k = 0; k < N; ++k) part[slot][k][wave] = x[k];
            lds_barrier();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if constexpr (kOfRow == 16) {
                    // a wave's part a lane: read by every lane, they take 16 registers a sum (second gradients
                    // of 4096 rows of 8192 bf16: 211 us, 439 with the spills; 8 waves a row: no difference)
                    x[k] = lane_sum<16>(part[slot][k][threadIdx.x % 16]);
                } else {
                    float s = 0.0f;
#pragma unroll
                    for (int w = 0; w < kOfRow; ++w) s += part[slot][k][first + w];
                    x[k] = s;
                }
            }
            slot ^= 1;
        }
    }
};

__device__ __forceinline__ float inv_root(float mean, float eps) { return rsqrtf(mean + eps); }

// Calls f(lanes, vectors a lane) for the smallest shape that holds a row of n
// vectors: one vector a lane as long as a workgroup has lanes, since a lane
// with two has twice the registers and half the waves to hide a row's latency
// (gradients of 16384 rows of 512 vectors: 137 us with one, 172 with two;
// forward, 8192 rows of 512: 59 and 69 us).
template <class F>
auto with_shape(int n, F&& f) {
    using std::integral_constant;
    constexpr integral_constant<int, 1> one;
    if (n <= 16) return f(integral_constant<int, 16>{}, one);
    if (n <= 64) return f(integral_constant<int, 64>{}, one);
    if (n <= 128) return f(integral_constant<int, 128>{}, one);
    if (n <= 256) return f(integral_constant<int, 256>{}, one);
    if (n <= 512) return f(integral_constant<int, 512>{}, one);
    if (n <= 1024) return f(integral_constant<int, 1024>{}, one);
    if (n <= 2048) return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

inline int row_vectors(int lmax, int channels, int kvec) {
    return (lmax + 1) * (lmax + 1) * ((channels + kvec - 1) / kvec);
}

}  // namespace ctp
