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
// parameter (s x and not s^3 x: the cube leaves fp32 for rows of 1e13).  A row is read once and stays in registers between the two
// reductions that it needs; memory bounds both directions.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "train_common.hpp"
#include "train_kernels.hpp"

namespace ctp {

namespace {

// Where a lane's vector i sits in the row: component, degree, vector of the component's channels.
struct Place {
    int d, l, v;
    bool on;
};

__device__ __forceinline__ int degree_of(int d) { return d < 1 ? 0 : d < 4 ? 1 : d < 9 ? 2 : 3; }

template <class T>
__device__ __forceinline__ Place place_of(int i, int nvec, int comps) {
    Place p;
    p.d = comps == 1 ? 0 : i / nvec;
    p.v = i - p.d * nvec;
    p.on = i < nvec * comps;
    p.l = degree_of(p.d);
    return p;
}

// Sums of a row's values over its lanes.  Rows of up to 64 lanes reduce in a
// wave; wider ones are a workgroup each and meet in LDS, `slot` alternating so
// that one barrier a reduction is enough.
template <int Lanes, int N>
struct RowSum {
    float (*part)[N][Lanes / 64 > 0 ? Lanes / 64 : 1];
    int slot = 0;
    __device__ __forceinline__ void operator()(float (&x)[N]) {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = lane_sum<(Lanes < 64 ? Lanes : 64)>(x[k]);
        if constexpr (Lanes > 64) {
            constexpr int kW = Lanes / 64;
            const int wave = threadIdx.x / 64;
            if (threadIdx.x % 64 == 0)
#pragma unroll
                for (int k = 0; k < N; ++k) part[slot][k][wave] = x[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kW; ++w) s += part[slot][k][w];
                x[k] = s;
            }
            slot ^= 1;
        }
    }
};

__device__ __forceinline__ float inv_root(float mean, float eps) { return 1.0f / sqrtf(mean + eps); }

// Threads of a workgroup: one row of `Lanes` lanes each, several rows where they are short.
template <int Lanes>
constexpr int kNormThreads = Lanes < 256 ? 256 : Lanes;

template <class T, int Lanes, int NV>
__global__ void __launch_bounds__(kNormThreads<Lanes>) k_norm_fwd(NormArgs a) {
    __shared__ float part[2][1][Lanes / 64 > 0 ? Lanes / 64 : 1];
    RowSum<Lanes, 1> row_sum{part};
    const int lane = threadIdx.x % Lanes;
    const long row = (long)blockIdx.x * (kNormThreads<Lanes> / Lanes) + threadIdx.x / Lanes;
    const int C = a.channels, nvec = (C + kVec<T> - 1) / kVec<T>, nl = a.lmax + 1, comps = nl * nl;
    const bool wide = a.param_dtype != a.dtype;
    const bool live = row < a.n_rows;      // rows past the end take part in the reductions with zeros
    const float inv = 1.0f / ((float)nl * (float)C);
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* r = static_cast<const T*>(a.r) + row * a.r_stride;
    const size_t psize = wide ? 4 : sizeof(T);
    Place p[NV];
    vec_t<T> hx[NV], rx[NV];
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        p[i] = place_of<T>(lane + i * Lanes, nvec, comps);
        p[i].on = p[i].on && live;
        hx[i] = rx[i] = vec_t<T>{};
        if (p[i].on) {
            rx[i] = load_vec<T>(r + p[i].d * C, p[i].v, C);
            if (a.h) hx[i] = load_vec<T>(h + p[i].d * C, p[i].v, C);
        }
    }
    Floats<T> y[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i] = widen<T>(rx[i]);
    if (a.h) {
        float s1 = 1.0f;
        if (a.w_post) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Floats<T> f = widen<T>(hx[i]);
                float q = 0.0f;
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) q = __builtin_fmaf(f.v[k], f.v[k], q);
                ss[0] = __builtin_fmaf(q, inv / (float)(2 * p[i].l + 1), ss[0]);
            }
            row_sum(ss);
            s1 = inv_root(ss[0], a.eps);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!p[i].on) continue;
            Floats<T> f = widen<T>(hx[i]);
            if (a.w_post) {
                const Floats<T> w = load_param<T>(static_cast<const char*>(a.w_post) + (size_t)p[i].l * C * psize, wide, p[i].v, C);
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) f.v[k] = f.v[k] * s1 * w.v[k];
            }
            if (a.gate != kGateNone) {
                const Floats<T> g = a.gate == kGateRow
                    ? widen<T>(load_vec<T>(static_cast<const T*>(a.gate_p) + row * a.gate_stride + (long)p[i].l * C, p[i].v, C))
                    : load_param<T>(static_cast<const char*>(a.gate_p) + (size_t)p[i].l * C * psize, wide, p[i].v, C);
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) f.v[k] *= g.v[k];
            }
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) y[i].v[k] = __builtin_fmaf(a.alpha, f.v[k], y[i].v[k]);
        }
        T* out = static_cast<T*>(a.r_out) + row * ((long)comps * C);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (p[i].on) store_vec<T>(out + p[i].d * C, p[i].v, C, narrow<T>(y[i]));
    }
    if (!a.w_pre) return;
    // u comes from r' before its rounding
    ss[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) q = __builtin_fmaf(y[i].v[k], y[i].v[k], q);
        ss[0] = __builtin_fmaf(q, inv / (float)(2 * p[i].l + 1), ss[0]);
    }
    row_sum(ss);
    const float s2 = inv_root(ss[0], a.eps);
    T* u = static_cast<T*>(a.u) + row * ((long)comps * C);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!p[i].on) continue;
        const Floats<T> w = load_param<T>(static_cast<const char*>(a.w_pre) + (size_t)p[i].l * C * psize, wide, p[i].v, C);
        Floats<T> f;
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) f.v[k] = y[i].v[k] * s2 * w.v[k];
        store_vec<T>(u + p[i].d * C, p[i].v, C, narrow<T>(f));
    }
}

// ------------------------------------------------------------ backward

// Gradients of shared parameters: every workgroup goes through rows
// blockIdx.x, + gridDim.x, .. and keeps the sums of its columns in registers;
// k_norm_join adds the workgroups' sums.
constexpr int kSums = 3;        // dw_post, dw_pre, dg
constexpr int kMaxGroups = 512;

template <class T, int Lanes, int NV>
__global__ void __launch_bounds__(kNormThreads<Lanes>) k_norm_bwd(NormArgs a) {
    constexpr int kRowsAtOnce = kNormThreads<Lanes> / Lanes;
    __shared__ float part[2][3][Lanes / 64 > 0 ? Lanes / 64 : 1];
    __shared__ float part1[2][1][Lanes / 64 > 0 ? Lanes / 64 : 1];
    extern __shared__ float row_buf[];      // a gate for every row, lmax > 0: alpha d N(h) of the rows in work
    RowSum<Lanes, 3> sum3{part};
    RowSum<Lanes, 1> sum1{part1};
    const int lane = threadIdx.x % Lanes, sub = threadIdx.x / Lanes;
    const int C = a.channels, nvec = (C + kVec<T> - 1) / kVec<T>, nl = a.lmax + 1, comps = nl * nl;
    const long W = (long)comps * C;
    const bool wide = a.param_dtype != a.dtype;
    const size_t psize = wide ? 4 : sizeof(T);
    const float inv = 1.0f / ((float)nl * (float)C);
    Place p[NV];
    float b[NV];
    Floats<T> acc_post[NV] = {}, acc_pre[NV] = {}, acc_gate[NV] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        p[i] = place_of<T>(lane + i * Lanes, nvec, comps);
        b[i] = inv / (float)(2 * p[i].l + 1);
    }
    for (long row0 = (long)blockIdx.x * kRowsAtOnce; row0 < a.n_rows; row0 += (long)gridDim.x * kRowsAtOnce) {
        const long row = row0 + sub;
        const bool live = row < a.n_rows;
        vec_t<T> hx[NV], rx[NV], grx[NV], gux[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            hx[i] = rx[i] = grx[i] = gux[i] = vec_t<T>{};
            if (!p[i].on || !live) continue;
            const long at = (long)p[i].d * C;
            if (a.w_pre) {
                rx[i] = load_vec<T>(static_cast<const T*>(a.r) + row * a.r_stride + at, p[i].v, C);
                if (a.grad_u) gux[i] = load_vec<T>(static_cast<const T*>(a.grad_u) + row * a.grad_u_stride + at, p[i].v, C);
            }
            if (a.grad_r) grx[i] = load_vec<T>(static_cast<const T*>(a.grad_r) + row * a.grad_r_stride + at, p[i].v, C);
            if (a.h) hx[i] = load_vec<T>(static_cast<const T*>(a.h) + row * a.h_stride + at, p[i].v, C);
        }
        // the squares of h and r' and <A, r'>
        float s[3] = {0.0f, 0.0f, 0.0f};
        Floats<T> A[NV] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Floats<T> h = widen<T>(hx[i]), r = widen<T>(rx[i]), gu = widen<T>(gux[i]);
            float qh = 0.0f, qr = 0.0f;
            if (a.w_pre && p[i].on) A[i] = load_param<T>(static_cast<const char*>(a.w_pre) + (size_t)p[i].l * C * psize, wide, p[i].v, C);
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                A[i].v[k] *= gu.v[k];
                qh = __builtin_fmaf(h.v[k], h.v[k], qh);
                qr = __builtin_fmaf(r.v[k], r.v[k], qr);
                s[2] = __builtin_fmaf(A[i].v[k], r.v[k], s[2]);
            }
            s[0] = __builtin_fmaf(qh, b[i], s[0]);
            s[1] = __builtin_fmaf(qr, b[i], s[1]);
        }
        sum3(s);
        const float s1 = a.w_post ? inv_root(s[0], a.eps) : 1.0f;
        const float s2 = a.w_pre ? inv_root(s[1], a.eps) : 0.0f;
        const float pull = s2 * s[2];
        float t[1] = {0.0f};
        Floats<T> B[NV] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool on = p[i].on && live;
            const Floats<T> h = widen<T>(hx[i]), r = widen<T>(rx[i]), gr = widen<T>(grx[i]), gu = widen<T>(gux[i]);
            Floats<T> d;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                const float rs = r.v[k] * s2;
                d.v[k] = __builtin_fmaf(s2, __builtin_fmaf(-pull * b[i], rs, A[i].v[k]), gr.v[k]);
                acc_pre[i].v[k] = __builtin_fmaf(gu.v[k], rs, acc_pre[i].v[k]);
            }
            if (on) store_vec<T>(static_cast<T*>(a.d_r) + row * W + (long)p[i].d * C, p[i].v, C, narrow<T>(d));
            if (!a.h) continue;
            Floats<T> w, g;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) w.v[k] = g.v[k] = 1.0f;
            if (a.w_post && on) w = load_param<T>(static_cast<const char*>(a.w_post) + (size_t)p[i].l * C * psize, wide, p[i].v, C);
            if (a.gate == kGateRow) {
                if (on) g = widen<T>(load_vec<T>(static_cast<const T*>(a.gate_p) + row * a.gate_stride + (long)p[i].l * C, p[i].v, C));
            } else if (a.gate == kGateChannel) {
                if (on) g = load_param<T>(static_cast<const char*>(a.gate_p) + (size_t)p[i].l * C * psize, wide, p[i].v, C);
            }
            Floats<T> dg;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                const float ad = a.alpha * d.v[k], hs = h.v[k] * s1, dy = ad * g.v[k];
                dg.v[k] = ad * hs * w.v[k];
                acc_post[i].v[k] = __builtin_fmaf(dy, hs, acc_post[i].v[k]);
                B[i].v[k] = dy * w.v[k];
                t[0] = __builtin_fmaf(B[i].v[k], h.v[k], t[0]);
            }
            if (a.gate == kGateChannel) {
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) acc_gate[i].v[k] += dg.v[k];
            } else if (a.gate == kGateRow) {
                if (comps == 1) {
                    if (on) store_vec<T>(static_cast<T*>(a.d_gate) + row * C, p[i].v, C, narrow<T>(dg));
                } else if (p[i].on) {
                    float* at = row_buf + ((long)sub * comps * nvec + lane + i * Lanes) * kVec<T>;
#pragma unroll
                    for (int k = 0; k < kVec<T>; ++k) at[k] = dg.v[k];
                }
            }
        }
        if (a.h) {
            float pull1 = 0.0f;
            if (a.w_post) {
                sum1(t);
                pull1 = s1 * t[0];
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!p[i].on || !live) continue;
                const Floats<T> h = widen<T>(hx[i]);
                Floats<T> dh;
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) dh.v[k] = s1 * __builtin_fmaf(-pull1 * b[i], h.v[k] * s1, B[i].v[k]);
                store_vec<T>(static_cast<T*>(a.d_h) + row * W + (long)p[i].d * C, p[i].v, C, narrow<T>(dh));
            }
            if (a.gate == kGateRow && comps > 1) {
                // the components of a degree share the row's gate
                __syncthreads();
                for (int i = lane; i < nl * nvec; i += Lanes) {
                    const int l = i / nvec, v = i - l * nvec;
                    Floats<T> g = {};
                    for (int d = l * l; d < (l + 1) * (l + 1); ++d) {
                        const float* at = row_buf + ((long)sub * comps * nvec + (long)d * nvec + v) * kVec<T>;
#pragma unroll
                        for (int k = 0; k < kVec<T>; ++k) g.v[k] += at[k];
                    }
                    if (live) store_vec<T>(static_cast<T*>(a.d_gate) + (row * nl + l) * C, v, C, narrow<T>(g));
                }
                __syncthreads();
            }
        }
    }
    // one row of fp32 sums a workgroup row and parameter: [group][sum][comps * nvec * kVec]
    const long width = (long)comps * nvec * kVec<T>;
    float* ws = static_cast<float*>(a.workspace) + ((long)blockIdx.x * kRowsAtOnce + sub) * kSums * width;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!p[i].on) continue;
        const long at = (long)(lane + i * Lanes) * kVec<T>;
#pragma unroll
        for (int k = 0; k < kVec<T>; k += 4) {
            *reinterpret_cast<float4*>(ws + at + k) = make_float4(acc_post[i].v[k], acc_post[i].v[k + 1], acc_post[i].v[k + 2], acc_post[i].v[k + 3]);
            *reinterpret_cast<float4*>(ws + width + at + k) = make_float4(acc_pre[i].v[k], acc_pre[i].v[k + 1], acc_pre[i].v[k + 2], acc_pre[i].v[k + 3]);
            if (a.gate == kGateChannel)
                *reinterpret_cast<float4*>(ws + 2 * width + at + k) = make_float4(acc_gate[i].v[k], acc_gate[i].v[k + 1], acc_gate[i].v[k + 2], acc_gate[i].v[k + 3]);
        }
    }
}

// Adds the workgroups' sums: 64 columns a workgroup, its 16 waves share the groups, then meet in LDS.
constexpr int kJoinWaves = 16;

__global__ void __launch_bounds__(64 * kJoinWaves)
k_norm_join(const float* __restrict__ ws, int groups, int nl, int channels, int padded, int out_dtype, void* d_post,
            void* d_pre, void* d_gate) {
    __shared__ float part[kJoinWaves][64];
    const int which = blockIdx.y, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    void* out = which == 0 ? d_post : which == 1 ? d_pre : d_gate;
    if (!out) return;
    const int col = blockIdx.x * 64 + lane;     // l * channels + c
    const int l = col / channels, c = col - l * channels;
    const long width = (long)nl * nl * padded;
    float x = 0.0f;
    if (l < nl)
        for (int g = wave; g < groups; g += kJoinWaves) {
            const float* row = ws + ((long)g * kSums + which) * width + c;
            for (int d = l * l; d < (l + 1) * (l + 1); ++d) x += row[(long)d * padded];
        }
    part[wave][lane] = x;
    __syncthreads();
    if (wave != 0 || l >= nl) return;
    for (int w = 1; w < kJoinWaves; ++w) x += part[w][lane];
    if (out_dtype == kBF16) static_cast<__bf16*>(out)[col] = (__bf16)x;
    else if (out_dtype == kF16) static_cast<_Float16*>(out)[col] = (_Float16)x;
    else static_cast<float*>(out)[col] = x;
}

// ------------------------------------------------------------ launches

// Calls f(lanes, vectors a lane) for the smallest shape that holds a row of n vectors.
template <class F>
auto with_shape(int n, F&& f) {
    if (n <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (n <= 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (n <= 128) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    if (n <= 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    if (n <= 512) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    if (n <= 1024) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    if (n <= 2048) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

int row_vectors(int lmax, int channels, int kvec) { return (lmax + 1) * (lmax + 1) * ((channels + kvec - 1) / kvec); }

constexpr int rows_at_once(int lanes) { return lanes < 256 ? 256 / lanes : 1; }

int bwd_grid(long n_rows, int at_once) {
    return (int)std::min<long>((n_rows + at_once - 1) / at_once, kMaxGroups);
}

}  // namespace

long norm_bwd_workspace(long n_rows, int lmax, int channels) {
    // over both vector widths
    long most = 0;
    for (int kvec : {4, 8}) {
        const int n = row_vectors(lmax, channels, kvec);
        const long groups = with_shape(n, [&](auto lanes, auto) {
            return (long)bwd_grid(n_rows, rows_at_once(lanes)) * rows_at_once(lanes);
        });
        most = std::max(most, groups * kSums * n * kvec * (long)sizeof(float));
    }
    return most;
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
    if (a.n_rows == 0) return hipSuccess;
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        return with_shape(row_vectors(a.lmax, a.channels, kVec<T>), [&](auto lanes, auto nv) {
            constexpr int kAtOnce = rows_at_once(lanes);
            k_norm_fwd<T, lanes, nv><<<(unsigned)((a.n_rows + kAtOnce - 1) / kAtOnce), kNormThreads<lanes>, 0, st>>>(a);
            return hipGetLastError();
        });
    });
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st) {
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int n = row_vectors(a.lmax, a.channels, kVec<T>);
        return with_shape(n, [&](auto lanes, auto nv) {
            constexpr int kAtOnce = rows_at_once(lanes);
            const int grid = bwd_grid(a.n_rows, kAtOnce);
            if (grid > 0) {
                const size_t lds = a.gate == kGateRow && a.lmax > 0 ? (size_t)kAtOnce * n * kVec<T> * sizeof(float) : 0;
                k_norm_bwd<T, lanes, nv><<<grid, kNormThreads<lanes>, lds, st>>>(a);
            }
            const int cols = (a.lmax + 1) * a.channels, padded = (a.channels + kVec<T> - 1) / kVec<T> * kVec<T>;
            void* d_gate = a.gate == kGateChannel ? a.d_gate : nullptr;
            if (a.d_w_post || a.d_w_pre || d_gate)
                k_norm_join<<<dim3((cols + 63) / 64, kSums), 64 * kJoinWaves, 0, st>>>(
                    static_cast<const float*>(a.workspace), grid * kAtOnce, a.lmax + 1, a.channels, padded,
                    a.param_dtype, a.d_w_post, a.d_w_pre, d_gate);
            return hipGetLastError();
        });
    });
}

}  // namespace ctp
