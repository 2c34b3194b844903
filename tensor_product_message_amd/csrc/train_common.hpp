// Shared pieces of the training-step kernels (embedding, gated residual norms,
// gradient clipping): element types, 16-byte row accesses, reductions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ctp {

// Element types of the C ABI (conv_tp_dtype).
enum DType : int { kF32 = 0, kBF16 = 1, kF16 = 2 };

template <class T>
struct TypeOf;
template <>
struct TypeOf<float> {
    static constexpr int code = kF32;
};
template <>
struct TypeOf<__bf16> {
    static constexpr int code = kBF16;
};
template <>
struct TypeOf<_Float16> {
    static constexpr int code = kF16;
};

// Calls f(T{}) for the element type of a code checked by the C ABI front.
template <class F>
auto with_type(int code, F&& f) {
    if (code == kBF16) return f(__bf16{});
    if (code == kF16) return f(_Float16{});
    return f(float{});
}

// One 16-byte access: kVec values of T.  The type asks for no more than the
// elements' own alignment, so that a row may begin anywhere (an odd channel
// count, a view into a wider array): global memory instructions of gfx950 take
// any address, and the same dwordx4 instruction serves aligned rows at full
// speed, so there is no second, aligned path.
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

template <class T>
struct Vec {
    typedef T type __attribute__((ext_vector_type(kVec<T>)));
    typedef T unaligned __attribute__((ext_vector_type(kVec<T>), aligned(alignof(T))));
};
template <class T>
using vec_t = typename Vec<T>::type;

// Vector v of a row of n values (n > v * kVec); what lies past the row's end reads as 0.
template <class T>
__device__ __forceinline__ vec_t<T> load_vec(const T* row, int v, int n) {
    const int at = v * kVec<T>;
    if (at + kVec<T> <= n) return *reinterpret_cast<const typename Vec<T>::unaligned*>(row + at);
    vec_t<T> x = {};
#pragma unroll
    for (int k = 0; k < kVec<T> - 1; ++k)
        if (at + k < n) x[k] = row[at + k];
    return x;
}

template <class T>
__device__ __forceinline__ void store_vec(T* row, int v, int n, vec_t<T> x) {
    const int at = v * kVec<T>;
    if (at + kVec<T> <= n) {
        *reinterpret_cast<typename Vec<T>::unaligned*>(row + at) = x;
        return;
    }
#pragma unroll
    for (int k = 0; k < kVec<T> - 1; ++k)
        if (at + k < n) row[at + k] = x[k];
}

// kVec<T> values in fp32, and back with one rounding to nearest even.
template <class T>
struct Floats {
    float v[kVec<T>];
};

template <class T>
__device__ __forceinline__ Floats<T> widen(vec_t<T> x) {
    Floats<T> f;
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) f.v[k] = (float)x[k];
    return f;
}

template <class T>
__device__ __forceinline__ vec_t<T> narrow(const Floats<T>& f) {
    vec_t<T> x;
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) x[k] = (T)f.v[k];
    return x;
}

// Vector v of a row of parameters, which are held in T or in fp32 (`wide`): kVec<T> values either way.
template <class T>
__device__ __forceinline__ Floats<T> load_param(const void* row, bool wide, int v, int n) {
    if (!wide) return widen<T>(load_vec<T>(static_cast<const T*>(row), v, n));
    Floats<T> f;
    constexpr int kParts = kVec<T> / 4;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
        const int at = v * kVec<T> + 4 * p;
        const Floats<float> q = at < n ? widen<float>(load_vec<float>(static_cast<const float*>(row), at / 4, n)) : Floats<float>{};
#pragma unroll
        for (int k = 0; k < 4; ++k) f.v[4 * p + k] = q.v[k];
    }
    return f;
}

// Sum over aligned groups of `Width` lanes (a power of two up to 64), the same in every lane, in a fixed order.
template <int Width>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
    for (int d = Width / 2; d >= 1; d /= 2) x += __shfl_xor(x, d, 64);
    return x;
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) x += __shfl_xor(x, d, 64);
    return x;
}

// Bounds of a launch: workgroups are counted in 31 bits.
constexpr long kMaxGrid = 0x7fffffffL;

}  // namespace ctp
