// Second backward pass of the norms after and before a block: the gradients of
// <P, d_r> + <Q, d_h>, the outputs of the first backward pass (norm_common.hpp)
// with cotangents P and Q, in its inputs.  Training on forces needs it: they
// are first gradients, which the loss differentiates again.  In the notation
// there, with x^ = s x for h (s1) and r' (s2), per row
//
//   EB = s1 (Q - h^ <b Q, h^>)              (dL/dB; Q without w_post)
//   Ed = P + alpha g w_post EB              (dL/dd: the gradient in grad_r)
//   EA = s2 (Ed - r^ <b Ed, r^>)            (dL/dA; the gradient in grad_u is w_pre EA)
//   g_h = -s1^2 (b h^ (<Q, B> - 3 <b Q, h^> <B, h^>) + b Q <B, h^> + B <b Q, h^>)
//   g_r = -s2^2 (b r^ (<Ed, A> - 3 <b Ed, r^> <A, r^>) + b Ed <A, r^> + A <b Ed, r^>)
//   g_w_post = sum EB alpha d g,   g_w_pre = sum grad_u EA,   g_gate = sum alpha d w_post EB
//
// As in the first pass a row is read once and has two reductions: EB, d and Ed
// follow from the first four sums, everything else from the second four.
// Memory bounds it in fp32: 16384 rows of 2048 floats in 238 us (1.34 GB, 5.6
// TB/s; 308 without marks on the reads and writes, with a branch before every
// read and the parameters read at each use).  8192 rows of 4096 bf16 with a gate
// each take 192 us (805 MB, 4.2 TB/s): dozens of operations a value, which only
// two workgroups a CU hide; 215 with the registers of one.  Most 16-bit kernels
// with a gate need 8 to 88 bytes of scratch a lane beyond their 128 registers.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "norm_sums.hpp"

namespace ctp {

namespace {

// Full: everything is there, as in the first pass.
template <class T, int Lanes, int NV, int G, bool Full>
__global__ void __launch_bounds__(kNormThreads<Lanes>, 4) k_norm_bwd_bwd(NormArgs a) {
    constexpr int kRowsAtOnce = rows_at_once(Lanes);
    __shared__ float part_s[2][4][kSumWaves<Lanes>];
    __shared__ float part_t[2][4][kSumWaves<Lanes>];
    extern __shared__ __align__(16) float row_buf[];
    RowSum<Lanes, 4> sum_s{part_s}, sum_t{part_t};
    const int lane = threadIdx.x % Lanes, sub = row_in_group<Lanes>();
    const int C = a.channels, nvec = (C + kVec<T> - 1) / kVec<T>, nl = a.lmax + 1, comps = nl * nl;
    const long W = (long)comps * C;
    const bool has_h = Full || a.h, has_post = Full || a.w_post, has_pre = Full || a.w_pre;
    const float inv = 1.0f / ((float)nl * (float)C);
    const Params<T> post{a.w_post, a.param_dtype != a.dtype, C}, pre{a.w_pre, post.wide, C}, shared{a.gate_p, post.wide, C};
    // Places and parameters are kept where a lane has one vector of four values,
    // else worked out and read again: 128 registers, with which two workgroups of
    // 512 fit on a CU, do not hold eight values of each.
    constexpr bool kKeep = NV == 1 && kVec<T> == 4;
    const Place p0 = place_of<T>(lane, nvec, comps, C);
    auto place = [&](int i) {
        if (kKeep) return p0;
        __builtin_amdgcn_sched_barrier(0);
        int at = lane + i * Lanes;
        forget(at);
        return place_of<T>(at, nvec, comps, C);
    };
    Floats<T> wq0{}, wp0{}, wg0{};
    Floats<T> acc_post[NV] = {}, acc_pre[NV] = {}, acc_gate[G == kGateChannel ? NV : 1] = {};
    if (kKeep && p0.on) {
        if (has_post) wq0 = post.load(p0);
        if (has_pre) wp0 = pre.load(p0);
        if constexpr (G == kGateChannel) wg0 = shared.load(p0);
    }
    auto w_pre = [&](const Place& p) {
        if (kKeep) return wp0;
        return has_pre && p.on ? pre.load(p) : Floats<T>{};
    };
    auto ones = [] {
        Floats<T> f;
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) f.v[k] = 1.0f;
        return f;
    };
    for (long row0 = (long)blockIdx.x * kRowsAtOnce; row0 < a.n_rows; row0 += (long)gridDim.x * kRowsAtOnce) {
        const long row = row0 + sub;
        const bool live = is_row<Lanes>(row, a.n_rows);
        vec_t<T> px[NV], qx[NV], hx[NV], rx[NV], grx[NV], gux[NV], gx[G == kGateRow ? NV : 1];
        auto read_row = [&](auto stream) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Place p = place(i);
                px[i] = qx[i] = hx[i] = rx[i] = grx[i] = gux[i] = vec_t<T>{};
                if constexpr (G == kGateRow) gx[i] = vec_t<T>{};
                if (!p.on || !live) continue;
                auto read = [&](const void* x, long stride, unsigned from) {
                    return read_at<T, Full, stream>(row_of<const T>(x, row, stride) + from, p.span, C);
                };
                if (Full || a.a_d_h) qx[i] = read(a.a_d_h, W, p.from);
                if (has_pre) rx[i] = read(a.r, a.r_stride, p.from);
                if (Full || a.grad_u) gux[i] = read(a.grad_u, a.grad_u_stride, p.from);
                if (has_h) hx[i] = read(a.h, a.h_stride, p.from);
                if (Full || a.grad_r) grx[i] = read(a.grad_r, a.grad_r_stride, p.from);
                if (Full || a.a_d_r) px[i] = read(a.a_d_r, W, p.from);
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
            settle<T>(px[i], p.span, true), settle<T>(qx[i], p.span, true), settle<T>(rx[i], p.span, true);
            settle<T>(gux[i], p.span, true), settle<T>(hx[i], p.span, true), settle<T>(grx[i], p.span, true);
            if constexpr (G == kGateRow) settle<T>(gx[i], p.span, true);
        }
        float s[4] = {};        // the squares of h and r', <A, r'>, <b Q, h>
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place p = place(i);
            const Floats<T> q = widen<T>(qx[i]), h = widen<T>(hx[i]), r = widen<T>(rx[i]), gu = widen<T>(gux[i]);
            const Floats<T> w = w_pre(p);
            const float b = inv / (float)(2 * p.l + 1);
            float qh = 0.0f, qr = 0.0f, qq = 0.0f;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                qh = __builtin_fmaf(h.v[k], h.v[k], qh);
                qr = __builtin_fmaf(r.v[k], r.v[k], qr);
                qq = __builtin_fmaf(q.v[k], h.v[k], qq);
                s[2] = __builtin_fmaf(w.v[k] * gu.v[k], r.v[k], s[2]);
            }
            s[0] = __builtin_fmaf(qh, b, s[0]);
            s[1] = __builtin_fmaf(qr, b, s[1]);
            s[3] = __builtin_fmaf(qq, b, s[3]);
        }
        sum_s(s);
#pragma unroll
        for (int i = 0; i < NV; ++i) forget(qx[i]), forget(hx[i]), forget(rx[i]), forget(gux[i]);
        const float s1 = has_post ? inv_root(s[0], a.eps) : 1.0f, s2 = has_pre ? inv_root(s[1], a.eps) : 0.0f;
        const float ar = s2 * s[2], qh = has_post ? s1 * s[3] : 0.0f;      // <A, r^>, <b Q, h^>
        float t[4] = {};        // <Q, B>, <B, h>, <Ed, A>, <b Ed, r'>
        Floats<T> B[NV], Ed[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place p = place(i);
            const bool on = p.on && live;
            const float b = inv / (float)(2 * p.l + 1);
            Floats<T> w = ones(), wp{}, g = ones(), dg;
            if (has_pre) wp = w_pre(p);
            if (has_post && p.on) w = kKeep ? wq0 : post.load(p);
            if constexpr (G == kGateChannel)
                if (p.on) g = kKeep ? wg0 : shared.load(p);
            float be = 0.0f;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                if (k == 4) __builtin_amdgcn_sched_barrier(0);      // fp32 values of half a vector at a time
                const float q = (float)qx[i][k], h = (float)hx[i][k], r = (float)rx[i][k];
                const float A = wp.v[k] * (float)gux[i][k];
                const float d = __builtin_fmaf(s2, __builtin_fmaf(-ar * b, r * s2, A), (float)grx[i][k]);
                if constexpr (G == kGateRow) g.v[k] = (float)gx[i][k];
                const float EB = s1 * __builtin_fmaf(-qh, h * s1, q);
                const float ad = a.alpha * d, dy = ad * g.v[k];
                B[i].v[k] = dy * w.v[k];
                dg.v[k] = ad * w.v[k] * EB;
                Ed[i].v[k] = (float)px[i][k];
                if (has_h) {
                    if (live) acc_post[i].v[k] = __builtin_fmaf(EB, dy, acc_post[i].v[k]);
                    Ed[i].v[k] = __builtin_fmaf(a.alpha * g.v[k] * w.v[k], EB, Ed[i].v[k]);
                }
                if constexpr (G == kGateChannel)
                    if (live) acc_gate[i].v[k] += dg.v[k];
                t[0] = __builtin_fmaf(q, B[i].v[k], t[0]);
                t[1] = __builtin_fmaf(B[i].v[k], h, t[1]);
                t[2] = __builtin_fmaf(Ed[i].v[k], A, t[2]);
                be = __builtin_fmaf(Ed[i].v[k], r, be);
            }
            t[3] = __builtin_fmaf(be, b, t[3]);
            if (a.g_grad_r && on) store_left<T>(row_of<T>(a.g_grad_r, row, W) + p.to, p.left, narrow<T>(Ed[i]), a.stream_out);
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
        sum_t(t);
#pragma unroll
        for (int i = 0; i < NV; ++i) forget(qx[i]), forget(hx[i]), forget(rx[i]), forget(gux[i]);
        const float bh = s1 * t[1], er = s2 * t[3];     // <B, h^>, <b Ed, r^>
        const float along_h = t[0] - 3.0f * qh * bh, along_r = t[2] - 3.0f * er * ar;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place p = place(i);
            const bool on = p.on && live;
            const float b = inv / (float)(2 * p.l + 1);
            if (has_h) {
                const Floats<T> q = widen<T>(qx[i]), h = widen<T>(hx[i]);
                Floats<T> g;
#pragma unroll
                for (int k = 0; k < kVec<T>; ++k)
                    g.v[k] = has_post ? -s1 * s1 * (b * (h.v[k] * s1 * along_h + q.v[k] * bh) + B[i].v[k] * qh) : 0.0f;
                if (on) store_left<T>(row_of<T>(a.d_h, row, W) + p.to, p.left, narrow<T>(g), a.stream_out);
            }
            if (!has_pre) continue;
            const Floats<T> r = widen<T>(rx[i]), gu = widen<T>(gux[i]);
            const Floats<T> w = w_pre(p);
            Floats<T> g, gg;
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) {
                const float rs = r.v[k] * s2, EA = s2 * __builtin_fmaf(-er, rs, Ed[i].v[k]), A = w.v[k] * gu.v[k];
                if (live) acc_pre[i].v[k] = __builtin_fmaf(gu.v[k], EA, acc_pre[i].v[k]);
                gg.v[k] = w.v[k] * EA;
                g.v[k] = -s2 * s2 * (b * (rs * along_r + Ed[i].v[k] * ar) + A * er);
            }
            if (on) store_left<T>(row_of<T>(a.d_r, row, W) + p.to, p.left, narrow<T>(g), a.stream_out);
            if (on && a.g_grad_u) store_left<T>(row_of<T>(a.g_grad_u, row, W) + p.to, p.left, narrow<T>(gg), a.stream_out);
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

hipError_t launch_norm_bwd_bwd(const NormArgs& args, hipStream_t st) {
    NormArgs a = args;
    const long row = (long)(a.lmax + 1) * (a.lmax + 1) * a.channels * (a.dtype == kF32 ? 4 : 2);
    const long outs = !!a.h + !!a.w_pre + !!a.g_grad_r + (a.w_pre && a.g_grad_u);
    a.stream = streams(a.n_rows * (row * (outs + !!a.h + !!a.w_pre + !!a.grad_r + !!a.grad_u + !!a.a_d_r + !!a.a_d_h) +
                                   (a.gate == kGateRow ? 2 * row / (a.lmax + 1) : 0)));
    a.stream_out = streams_out(a.n_rows * row * outs);
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int n = row_vectors(a.lmax, a.channels, kVec<T>);
        return with_shape(n, [&](auto lanes, auto nv) {
            const int grid = sums_grid(a.n_rows, lanes);
            if (grid > 0) {
                const size_t lds = sums_lds(a, n * kVec<T>, rows_at_once(lanes), false);
                auto go = [&](auto kernel) { return launch_sums(kernel, grid, kNormThreads<lanes>, lds, st, a); };
                const bool full = a.h && a.w_post && a.w_pre && a.grad_r && a.grad_u && a.a_d_r && a.a_d_h && a.channels >= kVec<T>;
                auto gated = [&](auto g) {
                    return full ? go(k_norm_bwd_bwd<T, lanes, nv, g, true>) : go(k_norm_bwd_bwd<T, lanes, nv, g, false>);
                };
                const hipError_t e = a.gate == kGateRow ? gated(std::integral_constant<int, kGateRow>{})
                                     : a.gate == kGateChannel ? gated(std::integral_constant<int, kGateChannel>{})
                                                              : gated(std::integral_constant<int, kGateNone>{});
                if (e != hipSuccess) return e;
            }
            return launch_join(a, kVec<T>, grid, st);
        });
    });
}

}  // namespace ctp
