// Matrix products of the dense operators: tiles, their way through LDS, matrix
// instructions, and the way of their results back to rows.
//
//   out(m, n) = sum over k of A(m, k) B(n, k)
//
// An operand lies in memory with k contiguous ("along": rows of x or w) or
// with m or n contiguous ("across": what a gradient sums over are rows of
// storage).  Operands of 16 bits go to the matrix cores as they are.  Floats are
// taken apart into three bfloat16, x = h + m + l, each the rest rounded to
// nearest: 24 bits, so h + m + l is x (parts below 2^-126 aside).
// Of the nine products of the parts those below 2^-23 of the whole (m l, l m,
// l l) are left out; the other six are summed in fp32, which is a float
// product's accuracy at 2.7 times the rate of the fp32 matrix instructions
// (2.5 PFLOP/s over six against 157 TFLOP/s).  What comes out not finite is
// formed once more of the floats (any_beyond).
#pragma once

#include <hip/hip_runtime.h>

#include "dense_kernels.hpp"
#include "train_common.hpp"

namespace ctp {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// What the matrix cores see of an element type: parts of type E.
template <class T>
struct Parts {
    typedef T E;
    static constexpr int count = 1;
};
template <>
struct Parts<float> {
    typedef __bf16 E;
    static constexpr int count = 3;
};

template <class E>
struct Frag {
    typedef E type __attribute__((ext_vector_type(8)));
    typedef E half __attribute__((ext_vector_type(4)));
};

__device__ __forceinline__ f32x16 mfma(Frag<__bf16>::type a, Frag<__bf16>::type b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(Frag<_Float16>::type a, Frag<_Float16>::type b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// A tile of Rows values of m (or n) by Depth of k in LDS, one plane for each
// part.  Along: [row][k]; the 16-byte chunks of a row trade places by the row, so
// that the 16 rows that one clock of a b128 read takes lie in all 64 banks.
// Across: [k][row]; units of 16 values trade places by k, for the transposing
// reads, of which a clock takes two units of four values of k each.
template <class E, int Parts_, bool Along, int Rows, int Depth>
struct Tile {
    static constexpr int kPlane = Rows * Depth;     // elements
    static constexpr int kBytes = Parts_ * kPlane * 2;
    typedef typename Frag<E>::type frag_t;

    static __host__ __device__ __forceinline__ int chunk_of(int row, int c) {
        return Depth == 128 ? c ^ (row & 15) : Depth == 64 ? c ^ ((row >> 1) & 7) : c ^ ((row >> 2) & 3);
    }
    static __host__ __device__ __forceinline__ int unit_of(int k, int u) { return u ^ (Rows >= 128 ? (k & 3) << 1 : k & 2); }
    // element offset of value (row, k)
    static __device__ __forceinline__ int at(int row, int k) {
        if constexpr (Along) return row * Depth + chunk_of(row, k >> 3) * 8 + (k & 7);
        return k * Rows + (unit_of(k, row >> 4) << 4) + (row & 15);
    }
    // The fragment of 32 rows from `row` and 16 k: lane i has row i % 32, 8 values of k from k + Half (i / 32).  Which
    // k a lane has does not matter as long as both operands' lanes agree.
    template <int Half = 8>
    static __device__ __forceinline__ frag_t read(const E* plane, int row, int k, int lane) {
        if constexpr (Along) {
            return *reinterpret_cast<const frag_t*>(plane + at(row + (lane & 31), k + Half * (lane >> 5)));
        } else {
            // 16 lanes read 4 rows of 16 values, lane i the values 4 (i % 4) of row i / 4, and get the columns
            const int i = lane & 15, k0 = k + Half * (lane >> 5) + (i >> 2), r0 = row + (lane & 16) + 4 * (i & 3);
            typedef __attribute__((address_space(3))) s16x4* lds_t;
            union {
                s16x4 h[2];
                frag_t f;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(plane + at(r0, k0)));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(plane + at(r0, k0 + 4)));
            return u.f;
        }
    }
};

// f(Is<0>{}), .., f(Is<N - 1>{}): a loop that is unrolled whatever its body's size.
template <int N>
struct Is {
    static constexpr int value = N;
};
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F&& f) {
    if constexpr (I < N) {
        f(Is<I>{});
        each<N, I + 1>(f);
    }
}

// ---------------------------------------------------------------- activations

// exp(x) for x <= 0 and 1 / d for d >= 1, each off by some two roundings: the product with log2(e) is carried in
// two floats, and one Newton step follows the hardware's reciprocal.  (expf and a division are three times the
// instructions, which a layer's epilogue does not hide.)
__device__ __forceinline__ float exp_falling(float x) {
    x = x < -104.0f ? -104.0f : x;      // exp(-104) is below every float; NaN stays
    const float t = x * 1.44269502f, rest = __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, 1.44269502f, -t));
    const float y = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(y, rest * 0.693147181f, y);
}
__device__ __forceinline__ float one_over(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}

// act(z), its first and its second derivative.
template <int Act_>
__device__ __forceinline__ void activation(float z, float& f, float& d1, float& d2) {
    if constexpr (Act_ == kActRelu) {
        f = z > 0.0f ? z : (z != z ? z : 0.0f);
        d1 = z > 0.0f ? 1.0f : 0.0f;
        d2 = 0.0f;
    } else if constexpr (Act_ == kActSilu || Act_ == kActSigmoid) {
        // from exp(-|z|): nothing overflows, and sigmoid and its complement keep their relative accuracy
        const float e = exp_falling(-fabsf(z)), large = one_over(1.0f + e), small = e * large;
        const float s = z >= 0.0f ? large : small, t = large * small, u = z >= 0.0f ? small - large : large - small;
        if constexpr (Act_ == kActSigmoid) {
            f = s, d1 = t, d2 = t * u;
        } else {
            f = z * s, d1 = __builtin_fmaf(z, t, s), d2 = t * __builtin_fmaf(z, u, 2.0f);
        }
    } else if constexpr (Act_ == kActGelu) {
        // Phi(-|z|) = exp(-z^2 / 2) times a function that a polynomial in t = 1 / (1 + 0.4 |z| / sqrt(2)) follows to
        // 1.3 2^-23 of it (least squares at Chebyshev points, reweighted to even out the error), 4.4e-7 with the
        // evaluation's roundings; erfcf is four times the instructions.  Past 42 the exponential is zero anyway.
        const float near = fminf(fabsf(z), 42.0f);
        const float g = exp_falling(-0.5f * z * z), t = one_over(__builtin_fmaf(0.28284271f, near, 1.0f));
        constexpr float kPoly[9] = {0.22567586600780487f, 0.22566959261894226f, 0.20784272253513336f, 0.1685418039560318f,
                                    0.14143219590187073f, -0.005609337240457535f, 0.169087752699852f, -0.1829030066728592f,
                                    0.050262536853551865f};
        float q = kPoly[8];
#pragma unroll
        for (int k = 7; k >= 0; --k) q = __builtin_fmaf(q, t, kPoly[k]);
        q *= 0.5f * t * g;
        const float c = z < 0.0f ? q : 1.0f - q, p = 0.39894228040143268f * g;
        f = z * c, d1 = __builtin_fmaf(z, p, c);
        d2 = p * __builtin_fmaf(-near, near, 2.0f);     // z^2 may overflow where p is zero
    } else if constexpr (Act_ == kActTanh) {
        const float e = exp_falling(-2.0f * fabsf(z)), r = one_over(1.0f + e);
        f = tanhf(z);
        d1 = 4.0f * e * r * r;
        d2 = -2.0f * f * d1;
    } else {
        f = z, d1 = 1.0f, d2 = 0.0f;
    }
}

// Calls f(Is<act>{}): one branch for all values that f goes through.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case kActRelu: f(Is<kActRelu>{}); break;
        case kActSilu: f(Is<kActSilu>{}); break;
        case kActGelu: f(Is<kActGelu>{}); break;
        case kActSigmoid: f(Is<kActSigmoid>{}); break;
        case kActTanh: f(Is<kActTanh>{}); break;
        default: f(Is<kActNone>{}); break;
    }
}

// ---------------------------------------------------------------- tiles

// x = p[0] + p[1] + p[2].
struct ThreeParts {
    __bf16 p[3];
};
__device__ __forceinline__ ThreeParts take_apart(float x) {
    constexpr float kLargest = 3.3895313892515355e38f;      // of bfloat16: a value that rounds beyond it is cut instead
    ThreeParts t;
    t.p[0] = (__bf16)__builtin_amdgcn_fmed3f(x, -kLargest, kLargest);
    const float rest = x - (float)t.p[0];
    t.p[1] = (__bf16)rest;
    t.p[2] = (__bf16)(rest - (float)t.p[1]);
    return t;
}

// A tile's way from memory: 16-byte reads into registers, then into LDS as parts.
// n_rows: how many m (or n) there are, values past which are any; k_end: where k ends, zeros past it.
enum How : int { kGuarded, kWhole, kClamped };

// Whether a tile's whole steps of k may be read whole (and guarded what is left), and if not, whether clamped.
template <bool AlongA, bool AlongB>
__host__ __device__ __forceinline__ bool read_whole(bool whole_m, bool whole_n) {
    return (AlongA || whole_m) && (AlongB || whole_n);
}
template <class T, bool AlongA, bool AlongB>
__host__ __device__ __forceinline__ bool read_clamped(int m_left, int n_left, int k_end) {
    return (AlongA ? k_end : m_left) >= kVec<T> && (AlongB ? k_end : n_left) >= kVec<T>;
}

template <class T, bool Along, int Rows, int Depth, int Threads>
struct Staged {
    typedef typename Parts<T>::E E;
    typedef Tile<E, Parts<T>::count, Along, Rows, Depth> tile_t;
    static constexpr int kPerRow = (Along ? Depth : Rows) / kVec<T>;        // 16-byte vectors
    static constexpr int kVecs = Rows * Depth / kVec<T> / Threads;          // a thread's
    static_assert(kVecs * Threads * kVec<T> == Rows * Depth);
    vec_t<T> v[kVecs];

    // The tile's k from k0 on, base being the tile's first row (Along) or column and k = 0.  row_of(r): where row r of
    // the tile lies among the operand's rows (Along), which may be any permutation.  Three ways to read, of which a loop
    // takes one, so that what it waits for is known when it is compiled:
    //   kWhole    nothing of the tile lies past k_end or n_left;
    //   kClamped  reads go to the last vector and row that are there, and fix() makes of them what was meant;
    //             rows of no less than a vector (Along: k_end, Across: n_left);
    //   kGuarded  any size.
    // Row r of the tile among the operand's, and the first value that is read for the vector c of a row of `width`.
    template <int How, class F>
    static __host__ __device__ __forceinline__ long row(int r, int k0, int k_end, F&& row_of) {
        return Along ? row_of(r) : How == kClamped ? min(k0 + r, k_end - 1) : k0 + r;
    }
    template <int How>
    static __host__ __device__ __forceinline__ int value(int c, int k0, int width) {
        const int at = (Along ? k0 : 0) + c * kVec<T>;
        return How == kClamped ? min(at, width - kVec<T>) : at;
    }
    template <int How, class F>
    __device__ __forceinline__ void load(const T* base, long ld, int n_left, int k0, int k_end, F&& row_of) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int id = tid + i * Threads, r = id / kPerRow, c = id % kPerRow, width = Along ? k_end : n_left;
            const long from = row<How>(r, k0, k_end, row_of);
            const int at = value<How>(c, k0, width);
            if constexpr (How == kGuarded) {
                v[i] = vec_t<T>{};
                if (at < width && (Along || from < k_end)) v[i] = load_vec<T>(base + from * ld, at / kVec<T>, width);
            } else {
                v[i] = *reinterpret_cast<const typename Vec<T>::unaligned*>(base + from * ld + at);
            }
        }
    }
    // Zeros past k_end and n_left, the rest in its place, after a clamped load.
    __device__ __forceinline__ void fix(int n_left, int k0, int k_end) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int id = tid + i * Threads, r = id / kPerRow, c = id % kPerRow;
            const int over = (Along ? k0 : 0) + c * kVec<T> + kVec<T> - (Along ? k_end : n_left);
            const bool in = over < kVec<T> && (Along || k0 + r < k_end);
            const vec_t<T> x = __builtin_bit_cast(vec_t<T>, __builtin_bit_cast(unsigned __int128, v[i]) >> (over > 0 && in ? over * 8 * (int)sizeof(T) : 0));
            v[i] = in ? x : vec_t<T>{};
        }
    }

    // Every value times act'(z).  Summed (Across): what that is before its rounding is added to the sums of the thread's
    // columns, which are the same for all of its vectors.
    template <bool Summed>
    __device__ __forceinline__ void curve(const Staged& z, int act, float (&sum)[kVec<T>]) {
        static_assert(!Summed || (!Along && Threads % kPerRow == 0));
        with_act(act, [&](auto is) {
            float f, d1, d2;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
#pragma unroll
                for (int q = 0; q < kVec<T>; ++q) {
                    activation<decltype(is)::value>((float)z.v[i][q], f, d1, d2);
                    const float s = (float)v[i][q] * d1;
                    if constexpr (Summed) sum[q] += s;
                    v[i][q] = (T)s;
                }
        });
    }
    // Across: the values as they are, added to those sums.
    __device__ __forceinline__ void add_columns(float (&sum)[kVec<T>]) const {
        static_assert(Along || Threads % kPerRow == 0);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int q = 0; q < kVec<T>; ++q) sum[q] += (float)v[i][q];
    }

    __device__ __forceinline__ void store(E* lds) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int id = tid + i * Threads, r = id / kPerRow, c = id % kPerRow * kVec<T>;
            E* to = lds + (Along ? tile_t::at(r, c) : tile_t::at(c, r));
            if constexpr (Parts<T>::count == 1) {
                *reinterpret_cast<vec_t<T>*>(to) = v[i];
            } else {
                typename Frag<E>::half part[3];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const ThreeParts t = take_apart(v[i][q]);
#pragma unroll
                    for (int p = 0; p < 3; ++p) part[p][q] = t.p[p];
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) *reinterpret_cast<typename Frag<E>::half*>(to + p * tile_t::kPlane) = part[p];
            }
        }
    }
};

// One step of k through the matrix cores: the wave's tile of (32 MT) x (32 NT).  The matrix instruction's own rows are
// n, so that a lane's four consecutive results lie beside each other in a row of the output.
template <class TileA, class TileB, int NParts, int MT, int NT, int Depth, class E>
__device__ __forceinline__ void multiply_step(f32x16 (&acc)[NT][MT], const E* a, const E* b, int m0, int n0, int lane) {
    typedef typename Frag<E>::type frag_t;
#pragma unroll
    for (int k = 0; k < Depth; k += 16) {
        frag_t fa[MT][NParts], fb[NT][NParts];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < NParts; ++p) fa[i][p] = TileA::read(a + p * TileA::kPlane, m0 + 32 * i, k, lane);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int p = 0; p < NParts; ++p) fb[j][p] = TileB::read(b + p * TileB::kPlane, n0 + 32 * j, k, lane);
        // the parts' smallest products first
#pragma unroll
        for (int s = NParts - 1; s >= 0; --s)
#pragma unroll
            for (int p = 0; p <= s; ++p)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < MT; ++i) acc[j][i] = mfma(fb[j][s - p], fa[i][p], acc[j][i]);
    }
}

// The wave's results by rows: f(m, step, n, x, y), where x[r][0 .. V) are the values of row m + r step of the wave's
// tile in the columns n .. n + V - 1, in fp32.  slab: the wave's own piece of LDS, 32 rows of kSlab floats.
// Pairs: the halves of each 64 columns belong together, x and y for the columns n, n + 32 of them.
template <int NT>
constexpr int kSlab = 32 * NT + 4;

__device__ __forceinline__ void wave_lds_fence() {
    // LDS accesses of one wave stay in order; this keeps the compiler from moving them
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// Rows 32 i .. 32 i + 31 of the wave's tile into its slab.
template <int NT, int MT>
__device__ __forceinline__ void by_rows_block(const f32x16 (&acc)[NT][MT], int i, float* slab, int lane) {
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f32x4 x;
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = acc[j][i][4 * g + q];
            *reinterpret_cast<f32x4*>(slab + (lane & 31) * kSlab<NT> + 32 * j + 8 * g + 4 * (lane >> 5)) = x;
        }
    wave_lds_fence();
}

// Products of floats in parts give NaN where an operand is infinite (its parts are infinities of both signs) or where
// one part's product passes the range and another's does not.  Results that are not finite are formed once more, of the
// floats straight from memory.  To see that there are none costs the hidden layer of 83325 x 64 -> 64 1% of its 16 us,
// its gradients 2% of 29.
constexpr float kLargestFloat = 3.4028235e38f;

template <int MT, int NT>
__device__ __forceinline__ bool any_beyond(const f32x16 (&acc)[NT][MT]) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) t = __builtin_fmaf(acc[j][i][e], 0.0f, t);
    return __ballot(t != t) != 0;
}

// By the fp32 matrix instructions, whatever the number of terms (10^6 x 512 -> 512: d_w with an infinite row 24 ms, 5.3
// without).  read(m, n, k, a, z, b): the factors of term k of the
// wave's row m and column n, any where the output has none; curve(a, z): makes the first factors of what read gave.
template <int MT, int NT, class Read, class MakeCurve>
__device__ __forceinline__ void again_where_beyond(f32x16 (&acc)[NT][MT], int lane, int k_end, Read&& read, MakeCurve&& curve) {
    if (!any_beyond(acc)) [[likely]] return;
    forget(lane);       // what is derived from it is derived here, not before the products
    each<MT>([&](auto i) {
        constexpr int I = decltype(i)::value;
        each<NT>([&](auto j) {
            constexpr int J = decltype(j)::value, U = 4;
            f32x16 x = {};
#pragma unroll 1
            for (int k0 = 0; k0 < k_end; k0 += 2 * U) {
                float a[U] = {}, z[U] = {}, b[U] = {};
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // a lane has row and column lane % 32 and one of two k
                    const int k = k0 + 2 * u + (lane >> 5);
                    if (k < k_end) read(32 * I + (lane & 31), 32 * J + (lane & 31), k, a[u], z[u], b[u]);
                }
                curve(a, z);
#pragma unroll
                for (int u = 0; u < U; ++u) x = __builtin_amdgcn_mfma_f32_32x32x2f32(b[u], a[u], x, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[J][I][e] = fabsf(acc[J][I][e]) <= kLargestFloat ? acc[J][I][e] : x[e];
        });
    });
}

// A lane a result, for kernels that have few terms and no registers left (an infinity in each of 83325 rows of 64 -> 4352:
// 44 ms, 0.4 without).  slab: the wave's piece of LDS; there(m, n):
// whether the output has row m and column n; read as above.
template <int MT, int NT, class There, class Read>
__device__ __forceinline__ void again_by_lanes(f32x16 (&acc)[NT][MT], float* slab, int lane, int k_end, There&& there, Read&& read) {
    if (!any_beyond(acc)) [[likely]] return;
    forget(lane);
    each<MT>([&](auto i) {
        constexpr int I = decltype(i)::value;
        each<NT>([&](auto j) {
            constexpr int J = decltype(j)::value;
            float* own = slab + (lane & 31) * kSlab<1> + 4 * (lane >> 5);
            wave_lds_fence();
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int q = 0; q < 4; ++q) own[8 * g + q] = acc[J][I][4 * g + q];
            wave_lds_fence();
#pragma unroll 1
            for (int id = lane; id < 32 * 32; id += 64) {
                float* v = slab + id / 32 * kSlab<1> + id % 32;
                const int m = 32 * I + id / 32, n = 32 * J + id % 32;
                if (fabsf(*v) <= kLargestFloat || !there(m, n)) continue;
                float sum = 0.0f;
#pragma unroll 1
                for (int k = 0; k < k_end && sum == sum; ++k) {
                    float a, b;
                    read(m, n, k, a, b);
                    sum = __builtin_fmaf(a, b, sum);
                }
                *v = sum;
            }
            wave_lds_fence();
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[J][I][4 * g + q] = own[8 * g + q];
        });
    });
}

template <int V, bool Pairs, int MT, int NT, class F>
__device__ __forceinline__ void by_rows(const f32x16 (&acc)[NT][MT], float* slab, int lane, F&& f) {
    // B rows at once: one where the results themselves take half of the registers
    constexpr int kCols = 32 * NT / (Pairs ? 2 : 1), kLanes = kCols / V, kRows = 64 / kLanes, R = 32 / kRows, B = MT > 2 ? 1 : R;
    static_assert(!Pairs || NT % 2 == 0);
    const int n = lane % kLanes * V;
    each<MT>([&](auto i) {
        by_rows_block(acc, decltype(i)::value, slab, lane);
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += B) {
            float x[B][V], y[B][V];
#pragma unroll
            for (int r = 0; r < B; ++r) {
                const float* from = slab + ((r0 + r) * kRows + lane / kLanes) * kSlab<NT> + (Pairs ? n / 32 * 64 + n % 32 : n);
#pragma unroll
                for (int q = 0; q < V; q += 4) {
                    *reinterpret_cast<f32x4*>(x[r] + q) = *reinterpret_cast<const f32x4*>(from + q);
                    if constexpr (Pairs) *reinterpret_cast<f32x4*>(y[r] + q) = *reinterpret_cast<const f32x4*>(from + 32 + q);
                }
            }
            f(32 * decltype(i)::value + r0 * kRows + lane / kLanes, kRows, n, x, y);
        }
    });
}

// Row r of a tile of pairs among B's rows: 32 of them, their partners `pair` rows on, the next 32, and so on.  Rows past
// the last of `left` are the last one.
__host__ __device__ __forceinline__ long pair_row(int r, int left, long pair) {
    const int at = (r >> 6 << 5) + (r & 31);
    return (at < left ? at : left - 1) + (r >> 5 & 1) * pair;
}

// Where workgroup `id` of `total` works: the workgroups of one of the 8 XCDs, which get every eighth, take
// consecutive tiles, and those go through up to kGroup rows of tiles before the next column, so that an XCD's L2 sees
// the same operands again.
constexpr unsigned kXcds = 8, kGroup = 8;

__device__ __forceinline__ unsigned xcd_order(unsigned id, unsigned total) {
    const unsigned q = total / kXcds, r = total % kXcds, xcd = id % kXcds;
    return (xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q) + id / kXcds;
}

struct TileAt {
    unsigned m, n, outer;       // tile row, tile column, batch and split
};
__device__ __forceinline__ TileAt tile_at(unsigned id, unsigned tiles_m, unsigned tiles_n) {
    TileAt t;
    const unsigned per = tiles_m * tiles_n;
    t.outer = id / per;
    id -= t.outer * per;
    const unsigned in_group = kGroup * tiles_n, group = id / in_group, first = group * kGroup;
    const unsigned rows = min(tiles_m - first, kGroup);
    id -= group * in_group;
    t.m = first + id % rows;
    t.n = id / rows;
    return t;
}

// l of component d = l^2 .. l^2 + 2 l
__host__ __device__ __forceinline__ int degree_of(int d) { return d < 1 ? 0 : d < 4 ? 1 : d < 9 ? 2 : 3; }

}  // namespace ctp
