// Orthogonalising matrices by Newton-Schulz products.
//
//   X = M / (|M| + eps)       |M| the root of the sum of squares
//   A = X X^T,  X <- a X + (b A + c A A) X      `steps` times
//
// which takes every singular value s of X to a s + b s^3 + c s^5 and leaves the
// singular vectors.  With a, b, c = 3.4445, -4.7750, 2.0315 (the coefficients
// published with the Muon optimiser, K. Jordan 2024) the values between
// some 0.003 and 1 are between 0.7 and 1.2 after five steps.
//
// X lies with its short side S first, [S][L]: a tall matrix is turned on its way
// in and on its way out.  Small singular values grow some 3.4 times a step, and
// the noise that a rounding of X puts beside them grows alike: with X in
// bfloat16 or float16 a matrix of few strong directions comes out wrong by 22%
// and 4%.  So X, A and b A + c A A are held in 32 bits whatever the matrix's
// type, as two float16, v 2^12 = h + l: 22 bits, and with entries below 1.3, 1.8
// and 3 nothing overflows and nothing above 2^-36 is lost.  A product is three
// of the matrix cores', h h + h l + l h (l l is below 2^-22 of it).
//
// All matrices of a call go through the same launches, three a step.
#include "dense_direct.hpp"

#include <algorithm>

namespace ctp {
namespace {

typedef _Float16 E;
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 4096.0f;
constexpr int kPad = 64;
// of k a tile: 64 where tiles are small and a product's few steps are its time, 32 where two workgroups share a CU's LDS
template <int Side>
constexpr int kDepthOf = Side == 64 ? 64 : 32;
constexpr int kMostGroups = 32;     // tensors of one launch
constexpr int kMostSums = 512;      // shares of a matrix's sum of squares
// Of the long side, a share of A's sums: as much as the short side is, at least kLeastCut, and kMostCut for short sides
// from kWideSide on (two of 8192 x 2048 and 2048 x 2048 take 4.3 ms so, which makes three shares of 8192, and 4.4 in four).
constexpr int kLeastCut = 256, kMostCut = 2688, kWideSide = 2048;
// Of one matrix no more shares than fill the card, or these: they are written and read.
constexpr int kFill = 512, kLeastShares = 16;

// One tensor: `batch` matrices.  Places are elements from the workspace's start; each matrix has two planes.
struct Group {
    const void* in;
    void* out;
    long x[2], a, b;        // X and the next X, A, b A + c A A of the first matrix
    long parts;             // shares of A, floats from the workspace's start (splits > 1)
    long sums;              // doubles from the sums' start
    int rows, cols, dtype;  // of a matrix as it is given
    int s, l;               // padded sides
    unsigned batch;
    unsigned chunks;        // shares of the sum of squares
    // A's sums are added up in shares of `cut` of the long side, in their order.  The cut goes by the matrix's sides alone,
    // so its bits do not depend on the matrices beside it.  splits: the workgroups that have the shares, one or as many.
    unsigned splits;
    int cut;
    bool tall;
};
struct Groups {
    int n;
    bool wide;              // tiles of 128, else of 64
    float eps, scale;
    E* base;
    double* sums;
    long sums_at;           // bytes from the workspace's start
    Group g[kMostGroups];
    unsigned first[kMostGroups + 1];    // of this launch's workgroups, each group's first
};

static_assert(sizeof(Groups) <= 4000);      // with a launch's other argument

// The group of a workgroup: a lane compares each group's first with it (a search would read one after the other, and
// these kernels are short).
__device__ __forceinline__ int group_of(const Groups& p, unsigned id) {
    static_assert(kMostGroups < 64);
    const int lane = threadIdx.x & 63;
    const bool behind = lane + 1 < p.n && id >= p.first[lane + 1];
    return __builtin_amdgcn_readfirstlane(__popcll(__ballot(behind)));
}

// Calls f(T{}) for an element type's code.
template <class F>
__device__ __forceinline__ void of_type(int code, F&& f) {
    if (code == kF32)
        f(float{});
    else if (code == kBF16)
        f(__bf16{});
    else
        f(_Float16{});
}

// Shares of the sums of squares, in 64 bits.
__global__ __launch_bounds__(256) void k_squares(Groups p) {
    __shared__ double part[4];
    const int k = group_of(p, blockIdx.x);
    const Group& g = p.g[k];
    const unsigned id = blockIdx.x - p.first[k], matrix = id / g.chunks, chunk = id % g.chunks;
    const long size = (long)g.rows * g.cols, per = (size + g.chunks - 1) / g.chunks;
    const long from = matrix * size, first = chunk * per, last = min(first + per, size);
    double s = 0.0;
    of_type(g.dtype, [&](auto type) {
        typedef decltype(type) T;
        const T* x = static_cast<const T*>(g.in) + from;
#pragma unroll 4
        for (long i = first + (long)threadIdx.x * kVec<T>; i < last; i += 256 * kVec<T>) {
            if (i + kVec<T> <= last) {
                const vec_t<T> v = *reinterpret_cast<const typename Vec<T>::unaligned*>(x + i);
                // squares of floats are exact in 64 bits
#pragma unroll
                for (int q = 0; q < kVec<T>; ++q) s += (double)(float)v[q] * (double)(float)v[q];
            } else {
                for (long j = i; j < last; ++j) s += (double)(float)x[j] * (double)(float)x[j];
            }
        }
    });
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) p.sums[g.sums + (long)matrix * g.chunks + chunk] = part[0] + part[1] + part[2] + part[3];
}

// 8 values at a place of two planes.
struct Eight {
    float v[8];
};
__device__ __forceinline__ Eight read_parts(const E* hi, long plane) {
    const vec_t<E> h = *reinterpret_cast<const vec_t<E>*>(hi), l = *reinterpret_cast<const vec_t<E>*>(hi + plane);
    Eight x;
#pragma unroll
    for (int q = 0; q < 8; ++q) x.v[q] = (float)h[q] + (float)l[q];
    return x;
}
__device__ __forceinline__ void write_parts(E* hi, long plane, const Eight& x) {
    vec_t<E> h, l;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        h[q] = (E)x.v[q];
        l[q] = (E)(x.v[q] - (float)h[q]);
    }
    *reinterpret_cast<vec_t<E>*>(hi) = h;
    *reinterpret_cast<vec_t<E>*>(hi + plane) = l;
}

// X 2^12 as two planes, 64 x 64 values a workgroup, turned for a tall matrix; the padding is zeros.
__global__ __launch_bounds__(256) void k_begin(Groups p) {
    __shared__ float tile[64][65];
    const int k = group_of(p, blockIdx.x);
    const Group& g = p.g[k];
    const unsigned across = g.l / 64, per = (g.s / 64) * across, id = blockIdx.x - p.first[k], matrix = id / per;
    const int s0 = id % per / across * 64, l0 = id % across * 64;
    // every wave sums the shares, in the same order
    double sum = 0.0;
    for (unsigned c = threadIdx.x & 63; c < g.chunks; c += 64) sum += p.sums[g.sums + (long)matrix * g.chunks + c];
    const double factor = (double)kScale / (sqrt(wave_sum(sum)) + (double)p.eps);
    const long size = (long)g.rows * g.cols, plane = (long)g.s * g.l;
    // the tile as it lies in the matrix: rows r0.., columns c0..
    const int r0 = g.tall ? l0 : s0, c0 = g.tall ? s0 : l0;
    of_type(g.dtype, [&](auto type) {
        typedef decltype(type) T;
        constexpr int kLanes = 64 / kVec<T>, kRows = 256 / kLanes;
        const T* in = static_cast<const T*>(g.in) + matrix * size;
        const int c = threadIdx.x % kLanes * kVec<T>;
        vec_t<T> v[64 / kRows];
#pragma unroll
        for (int i = 0; i < 64 / kRows; ++i) {
            const int r = threadIdx.x / kLanes + i * kRows;
            const T* row = in + (long)(r0 + r) * g.cols;
            v[i] = vec_t<T>{};
            if (r0 + r < g.rows && c0 + c < g.cols) v[i] = load_vec<T>(row, (c0 + c) / kVec<T>, g.cols);
        }
#pragma unroll
        for (int i = 0; i < 64 / kRows; ++i)
#pragma unroll
            for (int q = 0; q < kVec<T>; ++q)
                tile[threadIdx.x / kLanes + i * kRows][c + q] = (float)((double)(float)v[i][q] * factor);
    });
    __syncthreads();
    E* x = p.base + g.x[0] + matrix * 2 * plane;
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int r = i / 8, c = i % 8 * 8;
        Eight y;
#pragma unroll
        for (int q = 0; q < 8; ++q) y.v[q] = g.tall ? tile[c + q][r] : tile[r][c + q];
        write_parts(x + (long)(s0 + r) * g.l + l0 + c, plane, y);
    }
}

// A of the matrices whose sums are cut, from the shares in their order; 8 values a thread.
__global__ __launch_bounds__(256) void k_join_gram(Groups p) {
    const int k = group_of(p, blockIdx.x);
    const Group& g = p.g[k];
    const long plane = (long)g.s * g.s, i = ((long)(blockIdx.x - p.first[k]) * 256 + threadIdx.x) * 8, matrix = i / plane, at = i % plane;
    if (matrix >= g.batch) return;
    const float* from = reinterpret_cast<const float*>(p.base) + g.parts + matrix * g.splits * plane + at;
    Eight y{};
#pragma unroll 4
    for (unsigned s = 0; s < g.splits; ++s) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(from + s * plane), hi = *reinterpret_cast<const f32x4*>(from + s * plane + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) y.v[q] += lo[q], y.v[4 + q] += hi[q];
    }
    write_parts(p.base + g.a + matrix * 2 * plane + at, plane, y);
}

// kGramAll: kGram where a workgroup may have all shares of a sum.
enum Kind : int { kGram = 0, kPoly = 1, kStep = 2, kLast = 3, kGramAll = 4 };

__device__ __forceinline__ void write_out(void* p, int dtype, long i, float v) {
    if (dtype == kF32)
        static_cast<float*>(p)[i] = v;
    else if (dtype == kBF16)
        static_cast<__bf16*>(p)[i] = (__bf16)v;
    else
        static_cast<_Float16*>(p)[i] = (_Float16)v;
}

// Place of a triangle's tile: row m, column n <= m of them, row after row.
__device__ __forceinline__ TileAt triangle_at(unsigned id) {
    unsigned m = (unsigned)((sqrtf(8.0f * id + 1.0f) - 1.0f) * 0.5f);
    while (m * (m + 1) / 2 > id) --m;
    while ((m + 1) * (m + 2) / 2 <= id) ++m;
    return TileAt{m, id - m * (m + 1) / 2, 0};
}

// A tile of Side x Side of one of the products by 4 waves; from: which of the X buffers is X.  A and b A + c A A are
// symmetric: the tiles on and below the diagonal are computed, and blocks of 64 below it written twice (of 64 whatever the
// tile: a product's two orders of h l + l h are not the same bits).
template <int Kind_, int Side>
__global__ __launch_bounds__(256, 2) void k_product(Groups p, int from) {
    constexpr int K = Kind_ == kGramAll ? kGram : Kind_;
    constexpr int MT = Side / 64, kDepth = kDepthOf<Side>;      // MT: 32 x 32 tiles of a wave, in each direction
    constexpr bool kSymmetric = K == kGram || K == kPoly, kAlong = kSymmetric;      // kAlong: the second operand
    typedef Tile<E, 2, true, Side, kDepth> TA;
    typedef Tile<E, 2, kAlong, Side, kDepth> TB;
    constexpr int kBuffer = TA::kBytes + TB::kBytes, kSlabs = 4 * 32 * kSlab<MT> * 4;
    __shared__ __attribute__((aligned(16))) char lds[2 * kBuffer > kSlabs ? 2 * kBuffer : kSlabs];
    const int k = group_of(p, blockIdx.x);
    const Group& g = p.g[k];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave & 1) * 32 * MT, wn = (wave >> 1) * 32 * MT;
    const int width = kSymmetric ? g.s : g.l;       // of the output
    const unsigned tiles_m = (g.s + Side - 1) / Side, tiles_n = (width + Side - 1) / Side;
    const unsigned id = xcd_order(blockIdx.x - p.first[k], p.first[k + 1] - p.first[k]);
    TileAt t;
    unsigned split = 0;
    if constexpr (kSymmetric) {
        const unsigned per = tiles_m * (tiles_m + 1) / 2, splits = K == kGram ? g.splits : 1;
        t = triangle_at(id % per);
        split = id / per % splits;
        t.outer = id / per / splits;
    } else {
        t = tile_at(id, tiles_m, tiles_n);
    }
    const long x_plane = (long)g.s * g.l, a_plane = (long)g.s * g.s;
    E* x = p.base + g.x[from] + t.outer * 2 * x_plane;
    E* a = p.base + g.a + t.outer * 2 * a_plane;
    E* b = p.base + g.b + t.outer * 2 * a_plane;
    const int m0 = t.m * Side, n0 = t.n * Side;
    // the operands; rows of a tile past the matrix's last are read where the matrix's last is, and their results dropped
    const int a_ld = K == kGram ? g.l : g.s, b_ld = K == kPoly ? g.s : g.l;
    const bool all = Kind_ == kGramAll && g.splits == 1;
    const int first = K == kGram ? split * g.cut : 0, depth = K == kGram ? (all ? g.l : min(g.cut, g.l - first)) : g.s;
    const E* pa = (K == kGram ? x : K == kPoly ? a : b) + (long)m0 * a_ld + first;
    const E* pb = (K == kPoly ? a : x) + (kAlong ? (long)n0 * b_ld + first : 0);
    const long a_step = K == kGram ? x_plane : a_plane, b_step = K == kPoly ? a_plane : x_plane;
    Direct<true, Side, kDepth, 4> da;
    Direct<kAlong, Side, kDepth, 4> db;
    da.init(a_ld, [&](int r) { return (long)min(r, g.s - 1 - m0); });
    db.init(b_ld, [&](int r) { return (long)min(r, g.s - 1 - n0); });
    const unsigned base = lds_address(lds);
    auto issue = [&](int step, int buffer) {
        const int k0 = step * kDepth;
        const unsigned to = base + buffer * kBuffer;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            da.issue(buffer_at(pa + q * a_step + k0, (unsigned)kBufferBytes), to + q * TA::kPlane * 2, kDepth);
            // Across: past the last column of a row lies the next row, past the last row's the buffer's end
            const E* from_b = pb + q * b_step + (kAlong ? k0 : (long)k0 * b_ld + n0);
            const long left = kAlong ? kBufferBytes : 2 * ((long)(g.s - k0) * b_ld - n0);
            db.issue(buffer_at(from_b, (unsigned)min(left, kBufferBytes)), to + TA::kBytes + q * TB::kPlane * 2, kDepth);
        }
    };
    f32x16 acc[MT][MT] = {};
    if (Kind_ == kGramAll && all) {
        f32x16 sum[MT][MT] = {};
        const int per = g.cut / kDepth;
        int left = per;
        auto add = [&] {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) sum[j][i] += acc[j][i], acc[j][i] = f32x16{};
        };
        multiply_tiles<TA, TB, 2, MT, MT, kDepth>(acc, reinterpret_cast<const E*>(lds), depth / kDepth, wm, wn, lane, issue, [&](int) {
            if (--left == 0) add(), left = per;
        });
        add();      // a last share of fewer tiles, or zeros
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = sum[j][i];
    } else {
        multiply_tiles<TA, TB, 2, MT, MT, kDepth>(acc, reinterpret_cast<const E*>(lds), depth / kDepth, wm, wn, lane, issue, [](int) {});
    }
    tile_barrier();
    float* slab = reinterpret_cast<float*>(lds) + wave * 32 * kSlab<MT>;
    // 8 values of row m of the output, from column n on
    auto finish = [&](int m, int n, Eight y) {
#pragma unroll
        for (int q = 0; q < 8; ++q) y.v[q] *= 1.0f / kScale;
        if constexpr (K == kGram) {
            if (g.splits > 1) {
                float* to = reinterpret_cast<float*>(p.base) + g.parts + (t.outer * (long)g.splits + split) * a_plane + (long)m * g.s + n;
                *reinterpret_cast<f32x4*>(to) = f32x4{y.v[0], y.v[1], y.v[2], y.v[3]};
                *reinterpret_cast<f32x4*>(to + 4) = f32x4{y.v[4], y.v[5], y.v[6], y.v[7]};
            } else {
                write_parts(a + (long)m * g.s + n, a_plane, y);
            }
        } else if constexpr (K == kPoly) {
            const Eight z = read_parts(a + (long)m * g.s + n, a_plane);
#pragma unroll
            for (int q = 0; q < 8; ++q) y.v[q] = __builtin_fmaf(kB, z.v[q], kC * y.v[q]);
            write_parts(b + (long)m * g.s + n, a_plane, y);
        } else {
            const Eight z = read_parts(x + (long)m * g.l + n, x_plane);
#pragma unroll
            for (int q = 0; q < 8; ++q) y.v[q] = __builtin_fmaf(kA, z.v[q], y.v[q]);
            if constexpr (K == kStep) {
                write_parts(p.base + g.x[from ^ 1] + t.outer * 2 * x_plane + (long)m * g.l + n, x_plane, y);
            } else if (m < g.rows) {
                const float unscale = p.scale / kScale;
                const int some = g.cols - n;
                if (some > 0)
                    of_type(g.dtype, [&](auto type) {
                        typedef decltype(type) T;
                        T* to = static_cast<T*>(g.out) + ((long)t.outer * g.rows + m) * g.cols + n;
#pragma unroll
                        for (int h = 0; h < 8; h += kVec<T>) {
                            Floats<T> f;
#pragma unroll
                            for (int q = 0; q < kVec<T>; ++q) f.v[q] = y.v[h + q] * unscale;
                            if (some > h) store_left<T>(to + h, some - h, narrow<T>(f));
                        }
                    });
            }
        }
    };
    const bool turned = K == kLast && g.tall;       // the output's rows are the columns here
    const int block_m = (m0 + wm) / 64, block_n = (n0 + wn) / 64;
    const bool written = !kSymmetric || block_m >= block_n, twice = kSymmetric && block_m > block_n;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        by_rows_block(acc, i, slab, lane);
        constexpr int kLanes = 4 * MT, kRows = 64 / kLanes;
#pragma unroll
        for (int r = 0; r < 32; r += kRows) {
            const int mr = r + lane / kLanes, nc = lane % kLanes * 8, m = m0 + wm + 32 * i + mr, n = n0 + wn + nc;
            float* v = slab + mr * kSlab<MT> + nc;
            Eight y;
#pragma unroll
            for (int q = 0; q < 8; ++q) y.v[q] = v[q];
            if (m >= g.s || n >= width || !written) continue;
            if (turned) {
                const Eight z = read_parts(x + (long)m * g.l + n, x_plane);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = __builtin_fmaf(kA, z.v[q], y.v[q] * (1.0f / kScale));
            } else {
                finish(m, n, y);
            }
        }
        wave_lds_fence();
        if (turned || twice) {
            // columns of the tile: 4 lanes have 32 rows of one
#pragma unroll
            for (int r = 0; r < 32 * MT; r += 16) {
                const int nc = r + lane / 4, mr = lane % 4 * 8, n = n0 + wn + nc, m = m0 + wm + 32 * i + mr;
                const float* v = slab + mr * kSlab<MT> + nc;
                Eight y;
#pragma unroll
                for (int q = 0; q < 8; ++q) y.v[q] = v[q * kSlab<MT>];
                if constexpr (kSymmetric) {
                    if (m < g.s && n < g.s) finish(n, m, y);
                } else if (n < g.rows && m < g.cols) {
                    of_type(g.dtype, [&](auto type) {
                        typedef decltype(type) T;
                        T* to = static_cast<T*>(g.out) + ((long)t.outer * g.rows + n) * g.cols + m;
                        const int some = g.cols - m;
#pragma unroll
                        for (int h = 0; h < 8; h += kVec<T>) {
                            Floats<T> f;
#pragma unroll
                            for (int q = 0; q < kVec<T>; ++q) f.v[q] = y.v[h + q] * (p.scale / kScale);
                            if (some > h) store_left<T>(to + h, some - h, narrow<T>(f));
                        }
                    });
                }
            }
        }
    }
}

constexpr long align256(long bytes) { return (bytes + 255) & ~255L; }
constexpr long div_up(long a, long b) { return (a + b - 1) / b; }

// (As in dense_linear.hip: min and max without std are int's on the host.)
long triangle(long tiles) { return tiles * (tiles + 1) / 2; }

long shares_of(const Group& g) { return div_up(g.l, g.cut); }

// Places of the tensors from `first` on (at most kMostGroups) and the bytes they take.
long lay_out(Groups& p, int first, int n_tensors, const long* batch, const int* rows, const int* cols) {
    long at = 0, sums = 0;
    p.n = 0;
    for (int k = first; k < n_tensors && p.n < kMostGroups; ++k) {
        Group& g = p.g[p.n++];
        g = Group{};
        g.rows = rows[k], g.cols = cols[k];
        g.batch = (unsigned)batch[k];
        g.tall = rows[k] > cols[k];
        g.s = (int)div_up(std::min<long>(rows[k], cols[k]), kPad) * kPad;
        g.l = (int)div_up(std::max<long>(rows[k], cols[k]), kPad) * kPad;
        if (rows[k] == 0 || cols[k] == 0) g.batch = 0, g.s = g.l = kPad;      // nothing to do for it
        const long size = (long)rows[k] * cols[k];
        g.chunks = (unsigned)std::max<long>(1L, std::min<long>(kMostSums, size / 4096));
        for (long* q : {&g.x[0], &g.x[1], &g.a, &g.b}) {
            *q = at;
            at += 2 * g.batch * (long)g.s * (q < &g.a ? g.l : g.s);
        }
        g.sums = sums;
        sums += (long)g.batch * g.chunks;
    }
    // tiles of 128 where those of the smallest product fill the card
    long tiles = 0, terms = 0;
    for (int k = 0; k < p.n; ++k) tiles += p.g[k].batch * triangle(div_up(p.g[k].s, 128));
    p.wide = tiles >= 256;
    // shares go to workgroups of their own where a long side would keep few workgroups busy for long
    for (int k = 0; k < p.n; ++k) terms += p.g[k].batch * triangle(div_up(p.g[k].s, p.wide ? 128 : 64)) * p.g[k].l;
    const long most = std::max<long>(kLeastCut, div_up(terms, 1024));
    for (int k = 0; k < p.n; ++k) {
        Group& g = p.g[k];
        const long shares = std::max<long>(kFill / triangle(g.s / 64), kLeastShares);
        const long cut = std::max<long>(g.s < kWideSide ? std::max<long>(g.s, kLeastCut) : kMostCut, div_up(g.l, shares));
        g.cut = (int)div_up(div_up(g.l, std::max<long>(1, g.l / cut)), kPad) * kPad;
        g.splits = g.l / most >= 2 ? (unsigned)shares_of(g) : 1;
        g.parts = at / 2;       // a float for two E; at is a multiple of the padding's square
        if (g.splits > 1) at += 2 * g.batch * g.splits * (long)g.s * g.s;
    }
    p.sums_at = align256(2 * at);
    return align256(2 * at) + align256(8 * sums);
}

// Sets every group's first workgroup, of(g) of them each; their number.
template <class F>
unsigned place_groups(Groups& p, F&& of) {
    long total = 0;
    for (int k = 0; k < p.n; ++k) {
        p.first[k] = (unsigned)total;
        total += of(p.g[k]);
    }
    p.first[p.n] = (unsigned)total;
    return (unsigned)total;
}
// per(g) for each matrix.
template <class F>
unsigned place(Groups& p, F&& per) {
    return place_groups(p, [&](const Group& g) { return g.batch * (long)per(g); });
}

template <int K, int Side>
hipError_t product(Groups& p, int from, hipStream_t st) {
    const unsigned total = place(p, [](const Group& g) {
        if (K == kStep || K == kLast) return div_up(g.s, Side) * div_up(g.l, Side);
        return triangle(div_up(g.s, Side)) * (K == kGram || K == kGramAll ? (long)g.splits : 1);
    });
    k_product<K, Side><<<total, 256, 0, st>>>(p, from);
    return hipGetLastError();
}
template <int K>
hipError_t product(Groups& p, int from, hipStream_t st) {
    return p.wide ? product<K, 128>(p, from, st) : product<K, 64>(p, from, st);
}

#define CTP_TRY(call)                                                 \
    do {                                                              \
        if (const hipError_t e_ = (call); e_ != hipSuccess) return e_; \
    } while (0)

hipError_t run(Groups& p, int steps, hipStream_t st) {
    unsigned total = place(p, [](const Group& g) { return (long)g.chunks; });
    if (total == 0) return hipSuccess;
    k_squares<<<total, 256, 0, st>>>(p);
    CTP_TRY(hipGetLastError());
    total = place(p, [](const Group& g) { return (long)(g.s / 64) * (g.l / 64); });
    k_begin<<<total, 256, 0, st>>>(p);
    CTP_TRY(hipGetLastError());
    bool cut = false, all = false;
    for (int k = 0; k < p.n; ++k) cut |= p.g[k].batch && p.g[k].splits > 1, all |= p.g[k].batch && p.g[k].splits < shares_of(p.g[k]);
    for (int s = 0; s < steps; ++s) {
        // (a workgroup that adds shares up takes 205 registers a lane for 142)
        CTP_TRY(all ? product<kGramAll>(p, s & 1, st) : product<kGram>(p, s & 1, st));
        if (cut) {
            total = place_groups(p, [](const Group& g) {
                return g.splits > 1 ? div_up(g.batch * (long)g.s * g.s, 256 * 8) : 0L;
            });
            k_join_gram<<<total, 256, 0, st>>>(p);
            CTP_TRY(hipGetLastError());
        }
        CTP_TRY(product<kPoly>(p, s & 1, st));
        if (s + 1 < steps)
            CTP_TRY(product<kStep>(p, s & 1, st));
        else
            CTP_TRY(product<kLast>(p, s & 1, st));
    }
    return hipSuccess;
}

}  // namespace

long ortho_workspace(int n_tensors, const long* batch, const int* rows, const int* cols) {
    Groups p;
    long most = 0;
    for (int k = 0; k < n_tensors; k += kMostGroups) most = std::max<long>(most, lay_out(p, k, n_tensors, batch, rows, cols));
    return most;
}

hipError_t launch_ortho(const OrthoArgs& a, hipStream_t st) {
    for (int k = 0; k < a.n_tensors; k += kMostGroups) {
        Groups p;
        lay_out(p, k, a.n_tensors, a.batch, a.rows, a.cols);
        for (int i = 0; i < p.n; ++i) {
            Group& g = p.g[i];
            g.in = a.in[k + i];
            g.out = a.out[k + i];
            g.dtype = a.dtype[k + i];
        }
        p.eps = a.eps, p.scale = a.scale;
        p.base = static_cast<E*>(a.workspace);
        p.sums = reinterpret_cast<double*>(static_cast<char*>(a.workspace) + p.sums_at);
        CTP_TRY(run(p, a.steps, st));
    }
    return hipSuccess;
}

}  // namespace ctp
