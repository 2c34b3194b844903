// Gradients of shared parameters, for the norms' first and second backward
// pass: every workgroup goes through rows blockIdx.x, + gridDim.x, .. and keeps
// the sums of its columns in registers; it leaves them in a row of its own in
// the workspace, and k_norm_join adds the workgroups' rows.
#pragma once

#include <algorithm>

#include "norm_common.hpp"

namespace ctp {

constexpr int kSums = 3;        // w_post, w_pre, the shared gate

// Threads of all workgroups together, 16 waves a CU.  More hide more of a row's
// two reductions, but each workgroup leaves a row of partial sums (16384 rows
// of 2048 floats: 182, 146 and 151 us with 512, 1024 and 2048 threads a CU).
constexpr int kTotalThreads = 1024 * 256;

inline int sums_grid(long n_rows, int lanes) {
    const int at_once = rows_at_once(lanes), threads = std::max(256, lanes);
    return (int)std::min<long>((n_rows + at_once - 1) / at_once, kTotalThreads / threads);
}

// Whether a workgroup's place has a row.  Where rows share a workgroup the last
// ones may have none: those places take part in the reductions with vectors of
// zeros, but not in the column sums, since what multiplies the zeros may not be
// finite (s without eps, a parameter of the caller's).
template <int Lanes>
__device__ __forceinline__ bool is_row(long row, long n_rows) {
    return rows_at_once(Lanes) == 1 || row < n_rows;
}

// Bytes of LDS for the rows in work, in fp32, where lanes share sums or wait
// with several vectors a lane (`waits`), and for both where they meet.
inline size_t sums_lds(const NormArgs& a, int row_values, int at_once, bool waits) {
    const size_t row = (size_t)at_once * row_values * sizeof(float);
    if (waits && a.lmax > 0 && a.gate == kGateRow) return 2 * row;
    return at_once > 1 || a.lmax > 0 || waits ? row : 0;
}

// A launch with `lds` bytes of dynamic LDS; beyond 64 KB a kernel has to ask.
template <class K>
hipError_t launch_sums(K kernel, int grid, int threads, size_t lds, hipStream_t st, const NormArgs& a) {
    if (lds > 60000)
        if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
            e != hipSuccess)
            return e;
    kernel<<<grid, threads, lds, st>>>(a);
    return hipGetLastError();
}

// Leaves a workgroup's sums: over its rows at once and over the components of a
// degree, [sum][l][padded channels].
template <class T, int Lanes, int NV>
struct GroupSums {
    const NormArgs& a;
    float* row_buf;
    int lane, sub, nvec, nl;

    __device__ __forceinline__ void operator()(int which, const Floats<T>* acc) const {
        constexpr int kRowsAtOnce = rows_at_once(Lanes);
        const int comps = nl * nl, width = nl * nvec * kVec<T>;
        float* ws = static_cast<float*>(a.workspace) + (long)blockIdx.x * kSums * width;
        const bool fold = kRowsAtOnce > 1 || comps > 1;
        float* to = fold ? row_buf + sub * comps * nvec * kVec<T> : ws + which * width;
        if (fold) lds_barrier();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * Lanes >= comps * nvec) continue;
#pragma unroll
            for (int k = 0; k < kVec<T>; k += 4)
                *reinterpret_cast<float4*>(to + (lane + i * Lanes) * kVec<T> + k) =
                    make_float4(acc[i].v[k], acc[i].v[k + 1], acc[i].v[k + 2], acc[i].v[k + 3]);
        }
        if (!fold) return;
        lds_barrier();
        for (int c = threadIdx.x; c < width; c += kNormThreads<Lanes>) {
            const int l = c / (nvec * kVec<T>), at = c - l * (nvec * kVec<T>);
            float x = 0.0f;
            for (int q = 0; q < kRowsAtOnce; ++q)
                for (int d = l * l; d < (l + 1) * (l + 1); ++d) x += row_buf[(q * comps + d) * (nvec * kVec<T>) + at];
            ws[which * width + c] = x;
        }
    }
};

namespace {

// Adds the workgroups' sums: 64 columns a workgroup, whose 16 waves share the
// groups and meet in LDS.
constexpr int kJoinWaves = 16;

__global__ void __launch_bounds__(64 * kJoinWaves)
k_norm_join(const float* __restrict__ ws, int groups, int nl, int channels, int padded, int out_dtype, void* d_post,
            void* d_pre, void* d_gate) {
    __shared__ float part[kJoinWaves][64];
    const int which = blockIdx.y, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    void* out = which == 0 ? d_post : which == 1 ? d_pre : d_gate;
    if (!out) return;
    const int width = nl * padded, col = blockIdx.x * 64 + lane;
    const int l = col / padded, c = col - l * padded;
    const bool on = col < width && c < channels;
    float x = 0.0f;
    if (on) {
        const float* at = ws + which * width + col;
#pragma unroll 8
        for (int g = wave; g < groups; g += kJoinWaves) x += at[(long)g * (kSums * width)];
    }
    part[wave][lane] = x;
    lds_barrier();
    if (wave != 0 || !on) return;
    for (int w = 1; w < kJoinWaves; ++w) x += part[w][lane];
    const long to = (long)l * channels + c;
    if (out_dtype == kBF16) static_cast<__bf16*>(out)[to] = (__bf16)x;
    else if (out_dtype == kF16) static_cast<_Float16*>(out)[to] = (_Float16)x;
    else static_cast<float*>(out)[to] = x;
}

// The parameters' gradients in `a` from the rows that `groups` workgroups left.
hipError_t launch_join(const NormArgs& a, int kvec, int groups, hipStream_t st) {
    const int padded = (a.channels + kvec - 1) / kvec * kvec, cols = (a.lmax + 1) * padded;
    void* d_gate = a.gate == kGateChannel ? a.d_gate : nullptr;
    if (!a.d_w_post && !a.d_w_pre && !d_gate) return hipSuccess;
    k_norm_join<<<dim3((cols + 63) / 64, kSums), 64 * kJoinWaves, 0, st>>>(
        static_cast<const float*>(a.workspace), groups, a.lmax + 1, a.channels, padded, a.param_dtype, a.d_w_post,
        a.d_w_pre, d_gate);
    return hipGetLastError();
}

}  // namespace

}  // namespace ctp
