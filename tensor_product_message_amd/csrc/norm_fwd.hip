// Norms after and before a block, fused with its gate and residual: forward
// (formulas in norm_common.hpp).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "norm_common.hpp"

namespace ctp {

namespace {

// Memory bounds it: 8192 rows of 4096 bf16 with a gate each in 57.7 us (336 MB,
// 5.8 TB/s).  Of 1503 rows of 2048 floats (11.3 us, 49 MB, 4.4 TB/s) the GPU holds
// 1024 at once, four workgroups of 512 a CU: one and a half rounds.  Parameters
// are read with the row, so that their way from the cache is not a third wait.
// Full: h, w_post and w_pre are there and a row is no shorter than a vector,
// so that all of a lane's reads are issued in one straight line before the
// first reduction waits for them.
template <class T, int Lanes, int NV, int G, bool Full>
__global__ void __launch_bounds__(kNormThreads<Lanes>) k_norm_fwd(NormArgs a) {
    __shared__ float part[2][1][kSumWaves<Lanes>];
    RowSum<Lanes, 1> row_sum{part};
    const int lane = threadIdx.x % Lanes;
    const long row = (long)blockIdx.x * rows_at_once(Lanes) + row_in_group<Lanes>();
    const int C = a.channels, nvec = (C + kVec<T> - 1) / kVec<T>, nl = a.lmax + 1, comps = nl * nl;
    const bool live = row < a.n_rows;      // rows past the end take part in the reductions with zeros
    const bool has_h = Full || a.h, has_post = Full || a.w_post, has_pre = Full || a.w_pre;
    const float inv = 1.0f / ((float)nl * (float)C);
    const Params<T> post{a.w_post, a.param_dtype != a.dtype, C}, pre{a.w_pre, post.wide, C}, shared{a.gate_p, post.wide, C};
    Place p[NV];
    float b[NV];
    vec_t<T> hx[NV], rx[NV], gx[G == kGateRow ? NV : 1];
    Floats<T> wq[NV], wp[NV], wg[G == kGateChannel ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        p[i] = place_of<T>(lane + i * Lanes, nvec, comps, C);
        p[i].on = p[i].on && live;
        b[i] = inv / (float)(2 * p[i].l + 1);
    }
    auto read_row = [&](auto stream) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            hx[i] = rx[i] = vec_t<T>{};
            wq[i] = wp[i] = Floats<T>{};
            if constexpr (G == kGateChannel) wg[i] = Floats<T>{};
            if constexpr (G == kGateRow) gx[i] = vec_t<T>{};
            if (!p[i].on) continue;
            auto read = [&](const void* x, long stride, unsigned from) {
                return read_at<T, Full, stream>(row_of<const T>(x, row, stride) + from, p[i].span, C);
            };
            if (has_h) hx[i] = read(a.h, a.h_stride, p[i].from);
            rx[i] = read(a.r, a.r_stride, p[i].from);
            if constexpr (G == kGateRow) gx[i] = read(a.gate_p, a.gate_stride, p[i].par_from);
            if (has_post) wq[i] = post.load(p[i]);
            if constexpr (G == kGateChannel) wg[i] = shared.load(p[i]);
            if (has_pre) wp[i] = pre.load(p[i]);
        }
    };
    if (a.stream) {
        keep_apart();
        read_row(std::true_type{});
        keep_apart();
    } else {
        read_row(std::false_type{});
    }
    Floats<T> y[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (p[i].on && p[i].span.shift > 0) {
            settle<T>(hx[i], p[i].span, true), settle<T>(rx[i], p[i].span, true);
            if constexpr (G == kGateRow) settle<T>(gx[i], p[i].span, true);
        }
        y[i] = widen<T>(rx[i]);
    }
    float ss[1] = {0.0f};
    if (has_h) {
        float s1 = 1.0f;
        if (has_post) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Floats<T> f = widen<T>(hx[i]);
                float q = 0.0f;
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) q = __builtin_fmaf(f.v[k], f.v[k], q);
                ss[0] = __builtin_fmaf(q, b[i], ss[0]);
            }
            row_sum(ss);
            s1 = inv_root(ss[0], a.eps);
        }
        T* out = row_of<T>(a.r_out, row, (long)comps * C);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Floats<T> f = widen<T>(hx[i]);
            if (has_post)
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) f.v[k] = f.v[k] * s1 * wq[i].v[k];
            if constexpr (G == kGateRow) {
                const Floats<T> g = widen<T>(gx[i]);
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) f.v[k] *= g.v[k];
            }
            if constexpr (G == kGateChannel)
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) f.v[k] *= wg[i].v[k];
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) y[i].v[k] = __builtin_fmaf(a.alpha, f.v[k], y[i].v[k]);
            if (p[i].on) store_left<T>(out + p[i].to, p[i].left, narrow<T>(y[i]), a.stream_out);
        }
    }
    if (!has_pre) return;
    // u comes from r' before its rounding
    ss[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) q = __builtin_fmaf(y[i].v[k], y[i].v[k], q);
        ss[0] = __builtin_fmaf(q, b[i], ss[0]);
    }
    row_sum(ss);
    const float s2 = inv_root(ss[0], a.eps);
    T* u = row_of<T>(a.u, row, (long)comps * C);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        Floats<T> f;
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) f.v[k] = y[i].v[k] * s2 * wp[i].v[k];
        if (p[i].on) store_left<T>(u + p[i].to, p[i].left, narrow<T>(f), a.stream_out);
    }
}

// The arguments for rows [first, first + n) alone.
NormArgs rows_from(const NormArgs& all, long first, long n) {
    NormArgs a = all;
    const long nl = a.lmax + 1, row = nl * nl * a.channels, size = a.dtype == kF32 ? 4 : 2;
    auto move = [&](auto& p, long stride) {
        if (p) p = reinterpret_cast<std::decay_t<decltype(p)>>(reinterpret_cast<uintptr_t>(p) + first * stride * size);
    };
    a.n_rows = n;
    move(a.h, a.h_stride);
    move(a.r, a.r_stride);
    if (a.gate == kGateRow) move(a.gate_p, a.gate_stride);
    move(a.r_out, row);
    move(a.u, row);
    return a;
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& args, hipStream_t st) {
    if (args.n_rows == 0) return hipSuccess;
    NormArgs a = args;
    const long row = (long)(a.lmax + 1) * (a.lmax + 1) * a.channels * (a.dtype == kF32 ? 4 : 2);
    a.stream = streams(a.n_rows * (row * (2 * !!a.h + 1 + !!a.w_pre) + (a.gate == kGateRow ? row / (a.lmax + 1) : 0)));
    a.stream_out = streams_out(a.n_rows * row * (!!a.h + !!a.w_pre));
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        return with_shape(row_vectors(a.lmax, a.channels, kVec<T>), [&](auto lanes, auto nv) {
            constexpr int kAtOnce = rows_at_once(lanes);
            const bool full = a.h && a.w_post && a.w_pre && a.channels >= kVec<T>;
            auto go = [&](auto kernel) {
                // 2^28 rows of 16 lanes, 2^22 of 1024, are more than a launch takes
                constexpr long kMost = max_groups(kNormThreads<lanes>) * kAtOnce;
                for (long first = 0; first < a.n_rows; first += kMost) {
                    const NormArgs part = rows_from(a, first, std::min(kMost, a.n_rows - first));
                    kernel<<<(unsigned)((part.n_rows + kAtOnce - 1) / kAtOnce), kNormThreads<lanes>, 0, st>>>(part);
                }
            };
            auto gated = [&](auto g) {
                if (full) go(k_norm_fwd<T, lanes, nv, g, true>);
                else go(k_norm_fwd<T, lanes, nv, g, false>);
            };
            if (a.gate == kGateRow) gated(std::integral_constant<int, kGateRow>{});
            else if (a.gate == kGateChannel) gated(std::integral_constant<int, kGateChannel>{});
            else gated(std::integral_constant<int, kGateNone>{});
            return hipGetLastError();
        });
    });
}

}  // namespace ctp
