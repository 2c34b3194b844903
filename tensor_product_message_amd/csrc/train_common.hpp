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

// Vector v of a row of n values.  A last vector that the row does not fill is
// read from kVec values before the row's end, one access like the others, and
// shifted down afterwards (settle): the shift waits for the access, so it comes
// after all of a lane's accesses are on their way.  Rows shorter than a vector
// are read value by value.
struct Span {
    int at;         // first value read
    int shift;      // bits to shift out
    int few;        // values of a row that is shorter than a vector, else 0
};

template <class T>
__host__ __device__ __forceinline__ Span span_of(int v, int n) {
    const int at = v * kVec<T>, over = at + kVec<T> - n;
    if (n < kVec<T>) return Span{at, 0, v == 0 ? n : 0};
    return over > 0 ? Span{at - over, over * 8 * (int)sizeof(T), 0} : Span{at, 0, 0};
}

template <class T, bool Whole = false, bool Stream = false>
__device__ __forceinline__ vec_t<T> read_at(const T* at, const Span& s, int n) {
    if (Whole || n >= kVec<T>) {
        auto* x = reinterpret_cast<const typename Vec<T>::unaligned*>(at);
        return Stream ? __builtin_nontemporal_load(x) : *x;
    }
    vec_t<T> x = {};
#pragma unroll
    for (int k = 0; k < kVec<T> - 1; ++k)
        if (k < s.few) x[k] = at[k];
    return x;
}
template <class T>
__device__ __forceinline__ vec_t<T> read_span(const T* row, const Span& s, int n) {
    return read_at<T>(row + s.at, s, n);
}

// (Whole: the caller knows that rows are no shorter; Stream: see streams.)  What lies past the row's end becomes 0.
// on: the vector begins in the row.  Others are zeros that nothing was read into, and their shift is 128 bits or
// more, which is no shift.
template <class T>
__host__ __device__ __forceinline__ void settle(vec_t<T>& x, const Span& s, bool on) {
    if (on && s.shift > 0) x = __builtin_bit_cast(vec_t<T>, __builtin_bit_cast(unsigned __int128, x) >> s.shift);
}

template <class T>
__device__ __forceinline__ vec_t<T> load_vec(const T* row, int v, int n) {
    const Span s = span_of<T>(v, n);
    vec_t<T> x = read_span<T>(row, s, n);
    settle<T>(x, s, true);
    return x;
}

// Values [k, k + N) of x to where the row has room for them.
template <class T, int N>
__device__ __forceinline__ void store_part(T* row, vec_t<T> x, int k) {
    typedef T part_t __attribute__((ext_vector_type(N), aligned(alignof(T))));
    part_t y;
#pragma unroll
    for (int q = 0; q < N; ++q) {
        T z = x[q];
#pragma unroll
        for (int m = N; m + q < kVec<T>; m += N) z = k == m ? x[m + q] : z;
        y[q] = z;
    }
    *reinterpret_cast<part_t*>(row + k) = y;
}

// Around the accesses of one of two branches that differ in cache policy alone: the
// compiler would make one of them, and drop the policy.
__device__ __forceinline__ void keep_apart() { asm volatile("; a cache policy of its own" ::: "memory"); }

// x to `to`, where `left` > 0 values have room; stream: see streams_out.
template <class T>
__device__ __forceinline__ void store_left(T* to, int left, vec_t<T> x, bool stream = false) {
    if (left >= kVec<T>) {
        auto* at = reinterpret_cast<typename Vec<T>::unaligned*>(to);
        if (stream) {
            keep_apart();
            __builtin_nontemporal_store(x, at);
            keep_apart();
        } else {
            *at = x;
        }
        return;
    }
    // the row's last values, in halves of halves of a vector
    int k = 0;
    if constexpr (kVec<T> == 8)
        if (left & 4) {
            store_part<T, 4>(to, x, k);
            k += 4;
        }
    if (left & 2) {
        store_part<T, 2>(to, x, k);
        k += 2;
    }
    if (left & 1) store_part<T, 1>(to, x, k);
}

template <class T>
__device__ __forceinline__ void store_vec(T* row, int v, int n, vec_t<T> x) {
    store_left<T>(row + v * kVec<T>, n - v * kVec<T>, x);
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

// A vector that the compiler takes for a new one: what it has derived from the
// old (the fp32 values, four times the registers of bf16 pairs) is not kept
// alive for later uses but derived again.
template <class V>
__device__ __forceinline__ void forget(V& x) {
    asm volatile("" : "+v"(x));
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

// Whether a call's reads are marked non-temporal: where it moves too much for
// the 256 MB last-level cache to hold its inputs and what else a program uses,
// they would only push that out.  Norm gradients that move 805, 153 and 93 MB
// take 137, 36 and 28 us with the mark and 153, 40 and 27 without it.
constexpr long kStreamBytes = 128L << 20;
inline bool streams(long bytes) { return bytes > kStreamBytes; }

// Whether a call's outputs are written around that cache: where it would not
// hold them until their consumer.  A norm's gradient and a pass over its two
// outputs take 222 us with the mark and 238 without it for 268 MB of them, and
// 166 and 156 us for 134 MB.
constexpr long kStreamOutBytes = 192L << 20;
inline bool streams_out(long bytes) { return bytes > kStreamOutBytes; }

// Barrier of the workgroup for what it shares in LDS.  __syncthreads also waits
// until the waves' stores to memory have arrived, which costs a row of a norm
// another trip to memory at each of its reductions.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The value of another lane by a DPP control, 0 in rows of 16 lanes outside Rows.
template <int Ctrl, int Rows = 0xf>
__device__ __forceinline__ float dpp(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), Ctrl, Rows, 0xf, false));
}

// Sum over aligned groups of 16 or 64 lanes, the same bits in every lane.  All
// lanes of the wave take part.  The lanes trade in registers (DPP); through
// LDS each of the six steps would wait some 100 clocks.
template <int Width>
__device__ __forceinline__ float lane_sum(float x) {
    static_assert(Width == 16 || Width == 64);
    // both lanes of a pair add the same two values
    x += dpp<0xB1>(x);      // quad_perm 1 0 3 2
    x += dpp<0x4E>(x);      // quad_perm 2 3 0 1
    x += dpp<0x141>(x);     // row_half_mirror
    x += dpp<0x140>(x);     // row_mirror
    if constexpr (Width == 64) {
        x += dpp<0x142, 0xa>(x);    // lane 15 of rows 0 and 2 to rows 1 and 3
        x += dpp<0x143, 0xc>(x);    // lane 31 to rows 2 and 3: lane 63 has all
        x = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
    }
    return x;
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) x += __shfl_xor(x, d, 64);
    return x;
}

// Workgroups that a launch may have: its threads are counted in 32 bits, and a
// larger launch starts the remainder modulo 2^32 without an error.
constexpr long max_groups(int threads) { return 0xffffffffL / threads; }

}  // namespace ctp
