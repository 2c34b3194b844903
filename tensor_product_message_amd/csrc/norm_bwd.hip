// Gradients of the norms after and before a block (formulas in norm_common.hpp).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "norm_sums.hpp"

namespace ctp {

namespace {

// Memory bounds it: 16384 rows of 2048 floats in 139 us (805 MB, 5.8 TB/s), 8192
// rows of 4096 bf16 with a gate each in 107 us (537 MB, 5.0 TB/s); short of that,
// 5001 rows of 1003 halves in 22 us (60 MB), a row's two reductions and the
// partial sums.  Four waves a SIMD, 128 registers a lane, are what two
// workgroups of 512 a CU need.  Full: everything is there (h, both norms, both
// gradients) and a row is no shorter than a vector, so that a row's reads are
// issued in one straight line.
template <class T, int Lanes, int NV, int G, bool Full>
__global__ void __launch_bounds__(kNormThreads<Lanes>, 4) k_norm_bwd(NormArgs a) {
    constexpr int kRowsAtOnce = rows_at_once(Lanes);
    __shared__ float part[2][3][kSumWaves<Lanes>];
    __shared__ float part1[2][1][kSumWaves<Lanes>];
    extern __shared__ __align__(16) float row_buf[];    // the rows in work, in fp32, where lanes share sums
    RowSum<Lanes, 3> sum3{part};
    RowSum<Lanes, 1> sum1{part1};
    const int lane = threadIdx.x % Lanes, sub = row_in_group<Lanes>();
    const int C = a.channels, nvec = (C + kVec<T> - 1) / kVec<T>, nl = a.lmax + 1, comps = nl * nl;
    const long W = (long)comps * C;
    const bool has_h = Full || a.h, has_post = Full || a.w_post, has_pre = Full || a.w_pre;
    const bool has_gr = Full || a.grad_r, has_gu = Full || a.grad_u;
    const float inv = 1.0f / ((float)nl * (float)C);
    const Params<T> post{a.w_post, a.param_dtype != a.dtype, C}, pre{a.w_pre, post.wide, C}, shared{a.gate_p, post.wide, C};
    // With several vectors a lane their places are worked out again at each use
    // (the compiler must not see that they are the same), and one vector is
    // finished before the next: kept, they would take the registers of the rows.
    const Place p0 = place_of<T>(lane, nvec, comps, C);
    auto place = [&](int i) {
        if (NV == 1) return p0;
        __builtin_amdgcn_sched_barrier(0);
        int at = lane + i * Lanes;
        forget(at);
        return place_of<T>(at, nvec, comps, C);
    };
    auto weight = [&](const Place& p) { return inv / (float)(2 * p.l + 1); };
    const float b0 = weight(p0);
    // w_post, w_pre and the shared gate stay in registers where a lane has one vector, else they are read again
    constexpr bool kKeep = NV == 1;
    Floats<T> wq0{}, wp0{}, wg0{};
    Floats<T> acc_post[NV] = {}, acc_pre[NV] = {}, acc_gate[G == kGateChannel ? NV : 1] = {};
    if (kKeep && p0.on) {
        if (has_post) wq0 = post.load(p0);
        if (has_pre) wp0 = pre.load(p0);
        if constexpr (G == kGateChannel) wg0 = shared.load(p0);
    }
    auto w_post = [&](const Place& p) {
        if (kKeep) return wq0;
        return p.on ? post.load(p) : Floats<T>{};
    };
    auto w_pre = [&](const Place& p) {
        if (kKeep) return wp0;
        return p.on ? pre.load(p) : Floats<T>{};
    };
    for (long row0 = (long)blockIdx.x * kRowsAtOnce; row0 < a.n_rows; row0 += (long)gridDim.x * kRowsAtOnce) {
        const long row = row0 + sub;
        const bool live = is_row<Lanes>(row, a.n_rows);
        vec_t<T> hx[NV], rx[NV], grx[NV], gux[NV], gx[G == kGateRow ? NV : 1];
        auto read_row = [&](auto stream) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Place p = place(i);
                hx[i] = rx[i] = grx[i] = gux[i] = vec_t<T>{};
                if constexpr (G == kGateRow) gx[i] = vec_t<T>{};
                if (!p.on || !live) continue;
                auto read = [&](const void* x, long stride, unsigned from) {
                    return read_at<T, Full, stream>(row_of<const T>(x, row, stride) + from, p.span, C);
                };
                if (has_pre) rx[i] = read(a.r, a.r_stride, p.from);
                if (has_gu) gux[i] = read(a.grad_u, a.grad_u_stride, p.from);
                if (has_h) hx[i] = read(a.h, a.h_stride, p.from);
                if (has_gr) grx[i] = read(a.grad_r, a.grad_r_stride, p.from);
                if constexpr (G == kGateRow) gx[i] = read(a.gate_p, a.gate_stride, p.par_from);
            }
        };
        if (a.stream) {
            keep_apart();
            read_row(std::true_type{});
            keep_apart();
        } else {
            read_row(std::false_type{});
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place p = place(i);
            if (!p.on || p.span.shift <= 0) continue;
            settle<T>(rx[i], p.span, true), settle<T>(gux[i], p.span, true);
            settle<T>(hx[i], p.span, true), settle<T>(grx[i], p.span, true);
            if constexpr (G == kGateRow) settle<T>(gx[i], p.span, true);
        }
        // the squares of h and r' and <A, r'>
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Floats<T> h = widen<T>(hx[i]), r = widen<T>(rx[i]), gu = widen<T>(gux[i]);
            const Place p = place(i);
            const float b = NV == 1 ? b0 : weight(p);
            const Floats<T> w = has_pre ? w_pre(p) : Floats<T>{};
            float qh = 0.0f, qr = 0.0f;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                qh = __builtin_fmaf(h.v[k], h.v[k], qh);
                qr = __builtin_fmaf(r.v[k], r.v[k], qr);
                s[2] = __builtin_fmaf(w.v[k] * gu.v[k], r.v[k], s[2]);
            }
            s[0] = __builtin_fmaf(qh, b, s[0]);
            s[1] = __builtin_fmaf(qr, b, s[1]);
        }
        sum3(s);
#pragma unroll
        for (int i = 0; i < NV; ++i) forget(hx[i]), forget(rx[i]), forget(gux[i]);
        const float s1 = has_post ? inv_root(s[0], a.eps) : 1.0f;
        const float s2 = has_pre ? inv_root(s[1], a.eps) : 0.0f;
        const float pull = s2 * s[2];
        float t[1] = {0.0f};
        // with several vectors a lane, B waits in LDS for the second reduction, each lane's in its own places
        Floats<T> B0{};
        float* B_lds = row_buf + (G == kGateRow && comps > 1 ? comps * nvec * kVec<T> : 0) + lane * kVec<T>;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place p = place(i);
            const float b = NV == 1 ? b0 : weight(p);
            Floats<T> B{};
            const bool on = p.on && live;
            Floats<T> d = widen<T>(grx[i]);
            if (has_pre) {
                const Floats<T> r = widen<T>(rx[i]), gu = widen<T>(gux[i]);
                const Floats<T> w = w_pre(p);
                const float c = pull * b;
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k) {
                    const float rs = r.v[k] * s2;
                    d.v[k] = __builtin_fmaf(s2, __builtin_fmaf(-c, rs, w.v[k] * gu.v[k]), d.v[k]);
                    if (live) acc_pre[i].v[k] = __builtin_fmaf(gu.v[k], rs, acc_pre[i].v[k]);
                }
            }
            if (on) store_left<T>(row_of<T>(a.d_r, row, W) + p.to, p.left, narrow<T>(d), a.stream_out);
            if (!has_h) continue;
            const Floats<T> h = widen<T>(hx[i]);
            Floats<T> w, g, dg;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) w.v[k] = g.v[k] = 1.0f;
            if (has_post) w = w_post(p);
            if constexpr (G == kGateRow) g = widen<T>(gx[i]);
            if constexpr (G == kGateChannel) g = kKeep ? wg0 : p.on ? shared.load(p) : Floats<T>{};
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                const float ad = a.alpha * d.v[k], hs = h.v[k] * s1, dy = ad * g.v[k];
                dg.v[k] = ad * hs * w.v[k];
                if (live) acc_post[i].v[k] = __builtin_fmaf(dy, hs, acc_post[i].v[k]);
                B.v[k] = dy * w.v[k];
                t[0] = __builtin_fmaf(B.v[k], h.v[k], t[0]);
            }
            if constexpr (kKeep) {
                B0 = B;
            } else if (p.on) {
#pragma unroll
                for (int k = 0; k < kVec<T>; k += 4)
                    *reinterpret_cast<float4*>(B_lds + i * Lanes * kVec<T> + k) = make_float4(B.v[k], B.v[k + 1], B.v[k + 2], B.v[k + 3]);
            }
            if constexpr (G == kGateChannel) {
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k)
                    if (live) acc_gate[i].v[k] += dg.v[k];
            }
            if constexpr (G == kGateRow) {
                if (comps == 1) {
                    if (on) store_left<T>(row_of<T>(a.d_gate, row, C) + p.to, p.left, narrow<T>(dg));
                } else if (p.on) {
                    float* at = row_buf + (sub * comps * nvec + lane + i * Lanes) * kVec<T>;
#pragma unroll
                    for (int k = 0; k < kVec<T>; ++k) at[k] = dg.v[k];
                }
            }
        }
        if (!has_h) continue;
        float pull1 = 0.0f;
        if (has_post) {
            sum1(t);
            pull1 = s1 * t[0];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) forget(hx[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place p = place(i);
            const float b = NV == 1 ? b0 : weight(p);
            const Floats<T> h = widen<T>(hx[i]);
            const float c = pull1 * b;
            Floats<T> dh = B0;
            if (!kKeep && p.on) {
#pragma unroll
                for (int k = 0; k < kVec<T>; k += 4) {
                    const float4 q = *reinterpret_cast<const float4*>(B_lds + i * Lanes * kVec<T> + k);
                    dh.v[k] = q.x, dh.v[k + 1] = q.y, dh.v[k + 2] = q.z, dh.v[k + 3] = q.w;
                }
            }
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) dh.v[k] = s1 * __builtin_fmaf(-c, h.v[k] * s1, dh.v[k]);
            if (p.on && live) store_left<T>(row_of<T>(a.d_h, row, W) + p.to, p.left, narrow<T>(dh), a.stream_out);
        }
        if constexpr (G == kGateRow) {
            if (comps > 1) {
                // the components of a degree share the row's gate
                lds_barrier();
                for (int i = lane; live && i < nl * nvec; i += Lanes) {
                    const int l = i / nvec, v = i - l * nvec;
                    Floats<T> g = {};
                    for (int d = l * l; d < (l + 1) * (l + 1); ++d) {
                        const float* at = row_buf + ((sub * comps + d) * nvec + v) * kVec<T>;
#pragma unroll
                        for (int k = 0; k < kVec<T>; ++k) g.v[k] += at[k];
                    }
                    store_vec<T>(static_cast<T*>(a.d_gate) + (row * nl + l) * C, v, C, narrow<T>(g));
                }
                lds_barrier();
            }
        }
    }
    const GroupSums<T, Lanes, NV> leave{a, row_buf, lane, sub, nvec, nl};
    if (a.d_w_post) leave(0, acc_post);
    if (a.d_w_pre) leave(1, acc_pre);
    if constexpr (G == kGateChannel) leave(2, acc_gate);
}

}  // namespace

long norm_bwd_workspace(long n_rows, int lmax, int channels) {
    // over both vector widths
    long most = 0;
    for (int kvec : {4, 8}) {
        const int n = row_vectors(lmax, channels, kvec);
        const long groups = with_shape(n, [&](auto lanes, auto) { return (long)sums_grid(n_rows, lanes); });
        most = std::max(most, groups * kSums * (n / (lmax + 1)) * kvec * (long)sizeof(float));
    }
    return most;
}

hipError_t launch_norm_bwd(const NormArgs& args, hipStream_t st) {
    NormArgs a = args;
    const long row = (long)(a.lmax + 1) * (a.lmax + 1) * a.channels * (a.dtype == kF32 ? 4 : 2);
    a.stream = streams(a.n_rows * (row * (2 * !!a.h + !!a.grad_r + !!a.grad_u + !!a.w_pre + 1) +
                                   (a.gate == kGateRow ? 2 * row / (a.lmax + 1) : 0)));
    a.stream_out = streams_out(a.n_rows * row * (1 + !!a.h));
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int n = row_vectors(a.lmax, a.channels, kVec<T>);
        return with_shape(n, [&](auto lanes, auto nv) {
            hipError_t asked = hipSuccess;
            const int grid = sums_grid(a.n_rows, lanes);
            if (grid > 0) {
                constexpr int kAtOnce = rows_at_once(lanes);
                const size_t lds = sums_lds(a, n * kVec<T>, kAtOnce, nv > 1);
                auto go = [&](auto kernel) { asked = launch_sums(kernel, grid, kNormThreads<lanes>, lds, st, a); };
                const bool full = a.h && a.w_post && a.w_pre && a.grad_r && a.grad_u && a.channels >= kVec<T>;
                auto gated = [&](auto g) {
                    if (full) go(k_norm_bwd<T, lanes, nv, g, true>);
                    else go(k_norm_bwd<T, lanes, nv, g, false>);
                };
                if (a.gate == kGateRow) gated(std::integral_constant<int, kGateRow>{});
                else if (a.gate == kGateChannel) gated(std::integral_constant<int, kGateChannel>{});
                else gated(std::integral_constant<int, kGateNone>{});
            }
            if (asked != hipSuccess) return asked;
            return launch_join(a, kVec<T>, grid, st);
        });
    });
}

}  // namespace ctp
