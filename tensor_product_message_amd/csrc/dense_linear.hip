// Linear layers with their epilogue, the gated feed-forward form, and their first
// and second gradients.  One object for each element type (-DCTP_DENSE_TYPE),
// the dispatch by type in dense_dispatch.hip.
//
//   z = x W^T + b,   y = act(z) + r                or  h = act(z0) z1 (gated)
//   s = G act'(z)    d_x = s W   d_W = s^T x   d_b = sum of s
//   v = u W^T        g_G = v act'(z)   g_z = v G act''(z)
//                    g_x = g_z W   g_W = g_z^T x + s^T u   g_b = sum of g_z
//
// s, g_z (and the gated form's pairs of them) are rounded to the features' type
// before they enter a product, as the stored z is: they are operands of the
// matrix cores.  What is summed is in fp32.
#include "dense_common.hpp"
#include "dense_direct.hpp"
#include "dense_linear.hpp"

namespace ctp {
namespace {

#if CTP_DENSE_TYPE == 0
typedef float T;
#elif CTP_DENSE_TYPE == 1
typedef __bf16 T;
#else
typedef _Float16 T;
#endif
typedef Parts<T>::E E;
constexpr int kParts = Parts<T>::count, V = kVec<T>;
constexpr int kDepth = kParts == 1 ? 64 : 32;       // of k a tile: 128 bytes of a row

// ---------------------------------------------------------------- products

struct Gemm {
    const T *a, *b;
    long a_ld, b_ld;            // elements from row to row of storage
    long a_batch, b_batch;      // from batch to batch; b_batch by degree where b_degree is set
    int b_degree;
    long m, k;
    int n;                      // Pairs: columns of one half
    long pair;                  // Pairs: elements of B from a column to its partner
    long k_split;               // k of a split, a multiple of kDepth
    unsigned splits, tiles_m, tiles_n, total;
};

// V floats, the same width as a vector of T.
struct Values {
    float v[V];
};

// Whole: the vector lies in the row.
template <bool Whole>
__device__ __forceinline__ Values read_values(const T* row, int n, int width) {
    vec_t<T> r;
    if constexpr (Whole)
        r = *reinterpret_cast<const typename Vec<T>::unaligned*>(row + n);
    else
        r = load_vec<T>(row, n / V, width);
    const Floats<T> f = widen<T>(r);
    Values x;
#pragma unroll
    for (int q = 0; q < V; ++q) x.v[q] = f.v[q];
    return x;
}
template <bool Whole>
__device__ __forceinline__ void write_values(T* row, int n, int width, const float* x) {
    Floats<T> f;
#pragma unroll
    for (int q = 0; q < V; ++q) f.v[q] = x[q];
    if constexpr (Whole)
        *reinterpret_cast<typename Vec<T>::unaligned*>(row + n) = narrow<T>(f);
    else
        store_left<T>(row + n, width - n, narrow<T>(f));
}

// A wave's results through its epilogue: epi.run<Whole>(outer, batch, m, n, x, y) for V columns of a row.
template <bool Pairs, int MT, int NT, class Epi>
__device__ __forceinline__ void write_tile(const f32x16 (&acc)[NT][MT], float* slab, int lane, int wm, int wn, int m_left,
                                           int n_left, bool whole, const Epi& epi, unsigned outer, unsigned batch, long m0, int n0) {
    if (whole) {
        by_rows<V, Pairs, MT, NT>(acc, slab, lane, [&](int m, int n, const float* x, const float* y) {
            epi.template run<true>(outer, batch, m0 + wm + m, n0 + wn + n, x, y);
        });
    } else {
        by_rows<V, Pairs, MT, NT>(acc, slab, lane, [&](int m, int n, const float* x, const float* y) {
            if (wm + m < m_left && wn + n < n_left) epi.template run<false>(outer, batch, m0 + wm + m, n0 + wn + n, x, y);
        });
    }
}

// A tile of BM x BN by 4 waves, WM x (4 / WM) of them.  One buffer in LDS: the next tiles' reads are in flight in
// registers while the matrix cores work, and the workgroups that share a CU fill each other's pauses.
template <bool AlongA, bool AlongB, int BM, int BN, int WM, bool Pairs, class Epi>
__global__ __launch_bounds__(256, 2) void k_gemm(Gemm g, Epi epi) {
    constexpr int WN = 4 / WM, MT = BM / 32 / WM, NT = BN / 32 / WN;
    typedef Staged<T, AlongA, BM, kDepth, 256> SA;
    typedef Staged<T, AlongB, BN, kDepth, 256> SB;
    constexpr int kTiles = SA::tile_t::kBytes + SB::tile_t::kBytes, kSlabs = 4 * 32 * kSlab<NT> * 4;
    __shared__ __attribute__((aligned(16))) char lds[kTiles > kSlabs ? kTiles : kSlabs];
    E* la = reinterpret_cast<E*>(lds);
    E* lb = reinterpret_cast<E*>(lds + SA::tile_t::kBytes);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave % WM * 32 * MT, wn = wave / WM * 32 * NT;

    for (unsigned id = blockIdx.x; id < g.total; id += gridDim.x) {
        const TileAt t = tile_at(xcd_order(id, g.total), g.tiles_m, g.tiles_n);
        const unsigned batch = t.outer / g.splits, split = t.outer % g.splits;
        const long m0 = (long)t.m * BM, k0 = split * g.k_split;
        const int n0 = t.n * (Pairs ? BN / 2 : BN);
        const int k_end = (int)min(g.k_split, g.k - k0);    // from here on k counts from k0
        const T* a = g.a + batch * g.a_batch + (AlongA ? m0 * g.a_ld + k0 : k0 * g.a_ld + m0);
        const T* b = g.b + (g.b_degree ? degree_of(batch) : (int)batch) * g.b_batch +
                     (AlongB ? (long)n0 * g.b_ld + k0 : k0 * g.b_ld + n0);
        const int m_left = (int)min((long)BM, g.m - m0), n_left = min(g.n - n0, BN);
        // rows past the last give results that nobody stores
        auto row_a = [&](int r) { return (long)min(r, m_left - 1); };
        auto row_b = [&](int r) {
            if constexpr (Pairs) return (long)min((r >> 6 << 5) + (r & 31), n_left - 1) + (r >> 5 & 1) * g.pair;
            return (long)min(r, n_left - 1);
        };
        const bool whole_m = m_left == BM, whole_n = n_left >= (Pairs ? BN / 2 : BN);
        SA sa;
        SB sb;
        auto load = [&](int k) {
            if (k + kDepth <= k_end && (AlongA || whole_m) && (AlongB || whole_n)) {
                sa.template load<true>(a, g.a_ld, m_left, k, k_end, row_a);
                sb.template load<true>(b, g.b_ld, n_left, k, k_end, row_b);
            } else {
                sa.template load<false>(a, g.a_ld, m_left, k, k_end, row_a);
                sb.template load<false>(b, g.b_ld, n_left, k, k_end, row_b);
            }
        };
        f32x16 acc[NT][MT] = {};
        load(0);
        for (int k = 0; k < k_end; k += kDepth) {
            lds_barrier();
            sa.store(la);
            sb.store(lb);
            lds_barrier();
            if (k + kDepth < k_end) load(k + kDepth);
            multiply_step<typename SA::tile_t, typename SB::tile_t, kParts, MT, NT, kDepth>(acc, la, lb, wm, wn, lane);
        }
        lds_barrier();
        float* slab = reinterpret_cast<float*>(lds) + wave * 32 * kSlab<NT>;
        write_tile<Pairs, MT, NT>(acc, slab, lane, wm, Pairs ? wn / 2 : wn, m_left, n_left, whole_m && whole_n, epi, t.outer, batch, m0, n0);
        lds_barrier();
    }
}

// The same for operands of 16 bits whose rows begin on 16 bytes and are whole vectors long: memory to LDS without
// registers between, in two buffers, the next tiles' reads under way while the matrix cores work on these.  Side is 256
// with 8 waves (2 x 4) or 128 with 4 (2 x 2).
template <bool AlongA, bool AlongB, int Side, bool Pairs, class Epi>
__global__ __launch_bounds__(2 * Side, 2) void k_gemm_direct(Gemm g, Epi epi) {
    constexpr int Waves = Side / 32, WN = Waves / 2, MT = Side / 64, NT = Side / 32 / WN;
    typedef Tile<E, 1, AlongA, Side, kDepth> TA;
    typedef Tile<E, 1, AlongB, Side, kDepth> TB;
    constexpr int kBuffer = TA::kBytes + TB::kBytes, kSlabs = Waves * 32 * kSlab<NT> * 4;
    __shared__ __attribute__((aligned(16))) char lds[2 * kBuffer > kSlabs ? 2 * kBuffer : kSlabs];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave & 1) * 32 * MT, wn = (wave >> 1) * 32 * NT;
    const unsigned base = lds_address(lds);

    for (unsigned id = blockIdx.x; id < g.total; id += gridDim.x) {
        const TileAt t = tile_at(xcd_order(id, g.total), g.tiles_m, g.tiles_n);
        const unsigned batch = t.outer / g.splits, split = t.outer % g.splits;
        const long m0 = (long)t.m * Side, k0 = split * g.k_split;
        const int n0 = t.n * (Pairs ? Side / 2 : Side);
        const int k_end = (int)min(g.k_split, g.k - k0);    // from here on k counts from k0
        const T* a = g.a + batch * g.a_batch + (AlongA ? m0 * g.a_ld + k0 : k0 * g.a_ld + m0);
        const T* b = g.b + (g.b_degree ? degree_of(batch) : (int)batch) * g.b_batch +
                     (AlongB ? (long)n0 * g.b_ld + k0 : k0 * g.b_ld + n0);
        const int m_left = (int)min((long)Side, g.m - m0), n_left = min(g.n - n0, Side);
        Direct<AlongA, Side, kDepth, Waves> da;
        Direct<AlongB, Side, kDepth, Waves> db;
        // rows past the last give results that nobody stores
        da.init(g.a_ld, [&](int r) { return (long)min(r, m_left - 1); });
        db.init(g.b_ld, [&](int r) {
            if constexpr (Pairs) return (long)min((r >> 6 << 5) + (r & 31), n_left - 1) + (r >> 5 & 1) * g.pair;
            return (long)min(r, n_left - 1);
        });
        auto issue = [&](int step, int buffer) {
            const int k = step * kDepth;
            // Across: what lies past the last k is the buffer's end
            const long rows = min(k_end - k, kDepth) - 1;
            const long a_left = AlongA ? 0x7ffffff0L : 2 * (rows * g.a_ld + m_left);
            const long b_left = AlongB ? 0x7ffffff0L : 2 * (rows * g.b_ld + n_left);
            da.issue(buffer_at(a + (AlongA ? k : k * g.a_ld), (unsigned)min(a_left, 0x7ffffff0L)), base + buffer * kBuffer, k_end - k);
            db.issue(buffer_at(b + (AlongB ? k : k * g.b_ld), (unsigned)min(b_left, 0x7ffffff0L)),
                     base + buffer * kBuffer + TA::kBytes, k_end - k);
        };
        f32x16 acc[NT][MT] = {};
        if (k_end > 0)
            multiply_tiles<TA, TB, 1, MT, NT, kDepth>(acc, reinterpret_cast<const E*>(lds), (k_end + kDepth - 1) / kDepth, wm, wn, lane, issue);
        tile_barrier();
        float* slab = reinterpret_cast<float*>(lds) + wave * 32 * kSlab<NT>;
        write_tile<Pairs, MT, NT>(acc, slab, lane, wm, Pairs ? wn / 2 : wn, m_left, n_left,
                                  m_left == Side && n_left >= (Pairs ? Side / 2 : Side), epi, t.outer, batch, m0, n0);
        tile_barrier();
    }
}

// y = act(x + bias) + residual, z = x + bias
struct EpiLinear {
    T *y, *z;
    const T *bias, *residual;
    long row, residual_row;     // elements from row to row
    int n, act;
    template <bool Whole>
    __device__ __forceinline__ void run(unsigned, unsigned batch, long m, int at, const float* x, const float*) const {
        Values v;
#pragma unroll
        for (int q = 0; q < V; ++q) v.v[q] = x[q];
        if (bias != nullptr && batch == 0) {
            const Values b = read_values<Whole>(bias, at, n);
#pragma unroll
            for (int q = 0; q < V; ++q) v.v[q] += b.v[q];
        }
        const long to = m * row + (long)batch * n;
        if (z != nullptr) write_values<Whole>(z + to, at, n, v.v);
        with_act(act, [&](auto is) {
            float d1, d2;
#pragma unroll
            for (int q = 0; q < V; ++q) activation<decltype(is)::value>(v.v[q], v.v[q], d1, d2);
        });
        if (residual != nullptr) {
            const Values r = read_values<Whole>(residual + m * residual_row + (long)batch * n, at, n);
#pragma unroll
            for (int q = 0; q < V; ++q) v.v[q] += r.v[q];
        }
        write_values<Whole>(y + to, at, n, v.v);
    }
};

// h = act(x + bias[0]) (y + bias[1]), z the two sums
struct EpiGated {
    T *h, *z;
    const T* bias;
    int n, act;
    template <bool Whole>
    __device__ __forceinline__ void run(unsigned, unsigned, long m, int at, const float* x, const float* y) const {
        Values a, b;
#pragma unroll
        for (int q = 0; q < V; ++q) a.v[q] = x[q], b.v[q] = y[q];
        if (bias != nullptr) {
            const Values p = read_values<Whole>(bias, at, n), r = read_values<Whole>(bias + n, at, n);
#pragma unroll
            for (int q = 0; q < V; ++q) a.v[q] += p.v[q], b.v[q] += r.v[q];
        }
        if (z != nullptr) {
            write_values<Whole>(z + m * 2 * n, at, n, a.v);
            write_values<Whole>(z + m * 2 * n + n, at, n, b.v);
        }
        Values f;
        with_act(act, [&](auto is) {
            float d1, d2;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                activation<decltype(is)::value>(a.v[q], f.v[q], d1, d2);
                f.v[q] *= b.v[q];
            }
        });
        write_values<Whole>(h + m * n, at, n, f.v);
    }
};

// out = x
struct EpiPlain {
    T* out;
    long row;
    int n;
    template <bool Whole>
    __device__ __forceinline__ void run(unsigned, unsigned batch, long m, int at, const float* x, const float*) const {
        write_values<Whole>(out + m * row + (long)batch * n, at, n, x);
    }
};

// A split's share of a sum, in fp32.
struct EpiPart {
    float* parts;
    long size;      // of one part: rows n values wide
    int n;
    template <bool Whole>
    __device__ __forceinline__ void run(unsigned outer, unsigned, long m, int at, const float* x, const float*) const {
        float* to = parts + outer * size + m * n + at;
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            vec_t<float> w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = x[q + e];
            if constexpr (Whole)
                *reinterpret_cast<Vec<float>::unaligned*>(to + q) = w;
            else if (at + q < n)
                store_left<float>(to + q, n - at - q, w);
        }
    }
};

// The second backward pass's middle: v = x (gated: x and y) in, g_G, g_z and s out.
template <bool Gated>
struct EpiSecond {
    const T *grad, *z;
    T *g_grad, *g_z, *s;
    long grad_row;
    int n, act;
    template <bool Whole>
    __device__ __forceinline__ void run(unsigned, unsigned, long m, int at, const float* x, const float* y) const {
        const Values g = read_values<Whole>(grad + m * grad_row, at, n);
        const long zr = m * n * (Gated ? 2 : 1);
        const Values a = read_values<Whole>(z + zr, at, n);
        Values b{}, o, p, q, pb, qb;
        if constexpr (Gated) b = read_values<Whole>(z + zr + n, at, n);
        with_act(act, [&](auto is) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f, d1, d2;
                activation<decltype(is)::value>(a.v[i], f, d1, d2);
                if constexpr (Gated) {
                    const float gb = g.v[i] * b.v[i];
                    o.v[i] = __builtin_fmaf(x[i] * b.v[i], d1, y[i] * f);
                    p.v[i] = __builtin_fmaf(x[i] * gb, d2, y[i] * g.v[i] * d1);
                    pb.v[i] = x[i] * g.v[i] * d1;
                    q.v[i] = gb * d1;
                    qb.v[i] = g.v[i] * f;
                } else {
                    o.v[i] = x[i] * d1;
                    p.v[i] = x[i] * g.v[i] * d2;
                    q.v[i] = g.v[i] * d1;
                }
            }
        });
        if (g_grad != nullptr) write_values<Whole>(g_grad + m * n, at, n, o.v);
        if (g_z != nullptr) {
            write_values<Whole>(g_z + zr, at, n, p.v);
            if constexpr (Gated) write_values<Whole>(g_z + zr + n, at, n, pb.v);
        }
        if (s != nullptr) {
            write_values<Whole>(s + zr, at, n, q.v);
            if constexpr (Gated) write_values<Whole>(s + zr + n, at, n, qb.v);
        }
    }
};

// ---------------------------------------------------------------- few rows

// Up to 16 MB rows, where the weights' way from memory is all there is: no tile of x fills the matrix cores, and no
// weight is used twice.  Each wave takes 32 rows of w (Pairs: 16 and their partners) and one of Waves shares of k,
// straight from memory into the matrix instruction's registers, kAhead reads of each row under way at once; the
// waves' sums meet in LDS, in the waves' order.  Within 4 lanes' reads a row of w is 128 bytes in one piece: which k
// goes to which lane does not matter as long as w and x agree.
template <class U>
struct Small;
template <>
struct Small<float> {
    // fp32 matrix instructions: their rate is no limit here
    static __device__ __forceinline__ f32x4 mul(vec_t<float> w, vec_t<float> x, f32x4 c) {
#pragma unroll
        for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x4f32(w[q], x[q], c, 0, 0, 0);
        return c;
    }
};
template <>
struct Small<__bf16> {
    static __device__ __forceinline__ f32x4 mul(vec_t<__bf16> w, vec_t<__bf16> x, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
    }
};
template <>
struct Small<_Float16> {
    static __device__ __forceinline__ f32x4 mul(vec_t<_Float16> w, vec_t<_Float16> x, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, c, 0, 0, 0);
    }
};

template <int MB, int Waves, bool Pairs, class Epi>
__global__ __launch_bounds__(64 * Waves) void k_few(Gemm g, Epi epi) {
    constexpr int kStep = 8 * V, kAhead = 4 / MB, kRow = 36;
    __shared__ __attribute__((aligned(16))) float part[Waves][16 * MB][kRow];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, from = (lane >> 4) * 2 * V;
    const unsigned batch = blockIdx.y;
    const int n0 = blockIdx.x * (Pairs ? 16 : 32), k_end = (int)g.k;
    const T *a[MB], *b[2];
#pragma unroll
    for (int i = 0; i < MB; ++i) a[i] = g.a + batch * g.a_batch + min((long)(16 * i + r), g.m - 1) * g.a_ld;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const T* w = g.b + degree_of(batch) * g.b_batch + (long)min(n0 + r + (Pairs ? 0 : 16 * j), g.n - 1) * g.b_ld;
        b[j] = Pairs ? w + j * g.pair * g.b_ld : w;
    }
    f32x4 acc[2][MB] = {};
    // kAhead steps at a time, the waves in turn
    for (int k0 = wave * kAhead * kStep; k0 < k_end; k0 += Waves * kAhead * kStep) {
        vec_t<T> va[kAhead][2][MB], vb[kAhead][2][2];
        if (k0 + kAhead * kStep <= k_end) {
#pragma unroll
            for (int s = 0; s < kAhead; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = k0 + s * kStep + from + h * V;
#pragma unroll
                    for (int j = 0; j < 2; ++j) vb[s][h][j] = *reinterpret_cast<const typename Vec<T>::unaligned*>(b[j] + k);
#pragma unroll
                    for (int i = 0; i < MB; ++i) va[s][h][i] = *reinterpret_cast<const typename Vec<T>::unaligned*>(a[i] + k);
                }
        } else {
#pragma unroll
            for (int s = 0; s < kAhead; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = k0 + s * kStep + from + h * V;
                    const bool in = k < k_end;
#pragma unroll
                    for (int j = 0; j < 2; ++j) vb[s][h][j] = in ? load_vec<T>(b[j], k / V, k_end) : vec_t<T>{};
#pragma unroll
                    for (int i = 0; i < MB; ++i) va[s][h][i] = in ? load_vec<T>(a[i], k / V, k_end) : vec_t<T>{};
                }
        }
#pragma unroll
        for (int s = 0; s < kAhead; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < MB; ++i) acc[j][i] = Small<T>::mul(vb[s][h][j], va[s][h][i], acc[j][i]);
    }
    // lane: row 16 i + lane % 16 of x, columns 16 j + 4 (lane / 16) .. + 3
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) *reinterpret_cast<f32x4*>(&part[wave][16 * i + r][16 * j + 4 * (lane >> 4)]) = acc[j][i];
    lds_barrier();
    constexpr int kCols = Pairs ? 16 : 32, kLanes = kCols / V;
    for (int id = threadIdx.x; id < 16 * MB * kLanes; id += 64 * Waves) {
        const int m = id / kLanes, n = id % kLanes * V;
        if (m >= g.m || n0 + n >= g.n) continue;
        float x[V], y[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            x[q] = part[0][m][n + q];
            if constexpr (Pairs) y[q] = part[0][m][16 + n + q];
        }
        for (int w = 1; w < Waves; ++w)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                x[q] += part[w][m][n + q];
                if constexpr (Pairs) y[q] += part[w][m][16 + n + q];
            }
        epi.template run<false>(batch, batch, m, n0 + n, x, y);
    }
}

// ---------------------------------------------------------------- passes over values

// s = grad act'(z) for the products of the backward pass, and its columns' sums, a part for each chunk of rows.
// Gated: s and the sums have both halves beside each other.  A workgroup is `across` lanes wide, a vector of columns
// each, and 256 / across rows high.
struct ActBwd {
    const T *grad, *z;
    T* s;               // null: the sums alone, of grad itself
    float* sums;        // null: none; [chunk][columns]
    long grad_row, rows, chunk;
    int n, act, across;
};

// One row's vector of columns.
template <bool Gated>
struct ActRow {
    vec_t<T> g, a, b;
};

// Whole: n is whole vectors.  Rows: so many of a lane's rows are read at once.
template <bool Gated, bool Whole>
__global__ __launch_bounds__(256) void k_act_bwd(ActBwd p) {
    constexpr int H = Gated ? 2 : 1, Rows = 4;
    __shared__ float part[256 * H * V];
    const int tx = threadIdx.x % p.across, ty = threadIdx.x / p.across, high = 256 / p.across;
    const int at = (blockIdx.x * p.across + tx) * V;
    const long first = blockIdx.y * p.chunk, last = min(first + p.chunk, p.rows);
    Values sum[H] = {};
    auto read = [&](const T* row) {
        if constexpr (Whole) return (vec_t<T>)*reinterpret_cast<const typename Vec<T>::unaligned*>(row + at);
        return load_vec<T>(row, at / V, p.n);
    };
    auto values = [](vec_t<T> x) {
        const Floats<T> f = widen<T>(x);
        Values v;
#pragma unroll
        for (int q = 0; q < V; ++q) v.v[q] = f.v[q];
        return v;
    };
    for (long m0 = at < p.n ? first + ty : last; m0 < last; m0 += Rows * high) {
        ActRow<Gated> rows[Rows];
#pragma unroll
        for (int i = 0; i < Rows; ++i) {
            const long m = min(m0 + (long)i * high, last - 1);      // past the last row: the last again, not used
            rows[i].g = read(p.grad + m * p.grad_row);
            if (p.s != nullptr) {
                rows[i].a = read(p.z + m * p.n * H);
                if constexpr (Gated) rows[i].b = read(p.z + m * p.n * H + p.n);
            }
        }
#pragma unroll
        for (int i = 0; i < Rows; ++i) {
            const long m = m0 + (long)i * high;
            if (m >= last) break;
            Values g = values(rows[i].g), u{};
            if (p.s != nullptr) {
                const Values a = values(rows[i].a);
                Values b{};
                if constexpr (Gated) b = values(rows[i].b);
                with_act(p.act, [&](auto is) {
                    float f, d1, d2;
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        activation<decltype(is)::value>(a.v[q], f, d1, d2);
                        if constexpr (Gated) {
                            u.v[q] = g.v[q] * f;
                            g.v[q] = g.v[q] * b.v[q] * d1;
                        } else {
                            g.v[q] *= d1;
                        }
                    }
                });
                T* to = p.s + m * p.n * H;
                write_values<Whole>(to, at, p.n, g.v);
                if constexpr (Gated) write_values<Whole>(to + p.n, at, p.n, u.v);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) {
                sum[0].v[q] += g.v[q];
                if constexpr (Gated) sum[1].v[q] += u.v[q];
            }
        }
    }
    if (p.sums == nullptr) return;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int q = 0; q < V; ++q) part[((h * high + ty) * V + q) * p.across + tx] = sum[h].v[q];
    lds_barrier();
    // value i of the workgroup's across * V columns, summed over its rows in order
    for (int i = threadIdx.x; i < H * V * p.across; i += 256) {
        const int h = i / (V * p.across), c = i % (V * p.across), col = blockIdx.x * p.across * V + c;
        if (col >= p.n) continue;
        float s = 0.0f;
        for (int r = 0; r < high; ++r) s += part[((h * high + r) * V + c % V) * p.across + c / V];
        p.sums[(long)blockIdx.y * p.n * H + h * p.n + col] = s;
    }
}

// Parts joined: out[l][i] = sum over the parts of degree l, `ways` sums of every ways-th part first, then those.
struct Join {
    const float* parts;
    T* out;
    long size;              // of one part
    int degrees;            // part p belongs to the degree of p / per_component
    unsigned per_component;
    int ways;               // 1, 4 or 16
    unsigned groups;        // of 256 / ways values, each degree's own
};

__global__ __launch_bounds__(256) void k_join(Join first, Join second) {
    __shared__ float part[256];
    const bool is_first = blockIdx.x < first.groups * first.degrees;
    const Join j = is_first ? first : second;
    const unsigned id = is_first ? blockIdx.x : blockIdx.x - first.groups * first.degrees;
    const int wide = 256 / j.ways, c = threadIdx.x % wide, q = threadIdx.x / wide;
    const unsigned l = id / j.groups;
    const long i = (long)(id % j.groups) * wide + c;
    const unsigned p1 = (l + 1) * (l + 1) * j.per_component;
    unsigned p = l * l * j.per_component + q;
    float s = 0.0f;
    if (i < j.size) {
        // eight reads at once
        for (; p + 7 * j.ways < p1; p += 8 * j.ways) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = j.parts[(p + e * j.ways) * j.size + i];
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[e];
        }
        for (; p < p1; p += j.ways) s += j.parts[p * j.size + i];
    }
    part[threadIdx.x] = s;
    lds_barrier();
    if (q == 0 && i < j.size) {
        for (int r = 1; r < j.ways; ++r) s += part[r * wide + c];
        j.out[l * j.size + i] = (T)s;
    }
}

// ---------------------------------------------------------------- launches

constexpr long align256(long bytes) { return (bytes + 255) & ~255L; }
constexpr long div_up(long a, long b) { return (a + b - 1) / b; }

// Workgroups that fill the card: two for each of 256 CUs.
constexpr long kFill = 512;

bool set_tiles(Gemm& g, long rows, long cols, unsigned outer) {
    g.tiles_m = (unsigned)div_up(g.m, rows);
    g.tiles_n = (unsigned)div_up(g.n, cols);
    const long total = (long)g.tiles_m * g.tiles_n;
    if (total > 0xffffffffL || total * outer > 0xffffffffL) return false;
    g.total = (unsigned)(total * outer);
    return true;
}

template <bool AlongA, bool AlongB, int BM, int BN, int WM, bool Pairs, class Epi>
hipError_t run_staged(Gemm g, unsigned outer, const Epi& epi, hipStream_t st) {
    if (!set_tiles(g, BM, Pairs ? BN / 2 : BN, outer)) return hipErrorInvalidValue;
    if (g.total == 0) return hipSuccess;
    k_gemm<AlongA, AlongB, BM, BN, WM, Pairs><<<dim3((unsigned)min((long)g.total, max_groups(256))), 256, 0, st>>>(g, epi);
    return hipGetLastError();
}
template <bool AlongA, bool AlongB, int Side, bool Pairs, class Epi>
hipError_t run_direct(Gemm g, unsigned outer, const Epi& epi, hipStream_t st) {
    if (!set_tiles(g, Side, Pairs ? Side / 2 : Side, outer)) return hipErrorInvalidValue;
    if (g.total == 0) return hipSuccess;
    k_gemm_direct<AlongA, AlongB, Side, Pairs>
        <<<dim3((unsigned)min((long)g.total, max_groups(2 * Side))), 2 * Side, 0, st>>>(g, epi);
    return hipGetLastError();
}

// Whether tiles may go to LDS directly: 16-byte pieces, whole in every row.
template <bool AlongA, bool AlongB>
bool direct(const Gemm& g) {
    const auto whole = [](const T* p, long ld, long batch, long n) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % V == 0 && batch % V == 0 && n % V == 0;
    };
    return kParts == 1 && whole(g.a, g.a_ld, g.a_batch, AlongA ? g.k : g.m) && whole(g.b, g.b_ld, g.b_batch, AlongB ? g.k : (long)g.n);
}

// Tiles of 256 reuse an operand most, and are taken where they fill the card; tiles of 64 are for what has too few of
// the others.
template <bool AlongA, bool AlongB, bool Pairs, class Epi>
hipError_t run_tiles(const Gemm& g, unsigned outer, const Epi& epi, hipStream_t st) {
    const long n = Pairs ? 2L * g.n : g.n;
    if constexpr (kParts == 1) {
        if (direct<AlongA, AlongB>(g)) {
            if (div_up(g.m, 256) * div_up(n, 256) * outer >= kFill * 3 / 8) return run_direct<AlongA, AlongB, 256, Pairs>(g, outer, epi, st);
            if (div_up(g.m, 128) * div_up(n, 128) * outer >= kFill / 4) return run_direct<AlongA, AlongB, 128, Pairs>(g, outer, epi, st);
        }
    }
    if (g.m > 64 && n > 64 && g.k > 256 && div_up(g.m, 128) * div_up(n, 128) * outer >= kFill / 2)
        return run_staged<AlongA, AlongB, 128, 128, 2, Pairs>(g, outer, epi, st);
    return run_staged<AlongA, AlongB, 64, Pairs ? 128 : 64, 2, Pairs>(g, outer, epi, st);
}

template <int MB, bool Pairs, class Epi>
hipError_t run_few(const Gemm& g, unsigned batches, const Epi& epi, hipStream_t st) {
    const unsigned groups = (unsigned)div_up(g.n, Pairs ? 16 : 32);
    // more shares of k where few columns would leave the card empty
    if ((long)groups * batches < kFill / 2 && g.k >= 8 * (4 / MB) * 8 * V)
        k_few<MB, 16, Pairs><<<dim3(groups, batches), 64 * 16, 0, st>>>(g, epi);
    else
        k_few<MB, 4, Pairs><<<dim3(groups, batches), 64 * 4, 0, st>>>(g, epi);
    return hipGetLastError();
}

template <bool AlongA, bool AlongB, class Epi>
hipError_t run_gemm(Gemm g, unsigned batches, const Epi& epi, hipStream_t st) {
    if (g.m == 0) return hipSuccess;
    g.splits = 1;
    g.k_split = div_up(g.k, kDepth) * kDepth;
    if constexpr (AlongB) {
        if (g.m <= 16) return run_few<1, false>(g, batches, epi, st);
        if (g.m <= 32) return run_few<2, false>(g, batches, epi, st);
    }
    return run_tiles<AlongA, AlongB, false>(g, batches, epi, st);
}
template <class Epi>
hipError_t run_pairs(Gemm g, const Epi& epi, hipStream_t st) {
    if (g.m == 0) return hipSuccess;
    g.splits = 1;
    g.k_split = div_up(g.k, kDepth) * kDepth;
    if (g.m <= 16) return run_few<1, true>(g, 1, epi, st);
    if (g.m <= 32) return run_few<2, true>(g, 1, epi, st);
    return run_tiles<true, true, true>(g, 1, epi, st);
}

// How d_W[outer][inner] = sum over rows is cut: every component by itself, and its rows into `splits`.
struct WeightCut {
    unsigned splits;
    long k_split;
    bool direct;        // one part alone: no join
};
WeightCut weight_cut(const LinearArgs& a, bool twice) {
    const long comps = (long)(a.lmax + 1) * (a.lmax + 1), out = (long)a.outer * (a.gated ? 2 : 1);
    WeightCut c;
    // large matrices fill the card by themselves
    const bool wide = div_up(out, 128) * div_up(a.inner, 128) * comps >= kFill / 8 && a.inner > 64 && out > 64;
    const long tile = wide ? 128 : 64, tiles = div_up(out, tile) * div_up(a.inner, tile) * comps;
    long splits = max(1L, min(kFill / tiles, a.n_rows / (4 * kDepth)));
    splits = max(splits, div_up(a.n_rows, 1L << 30));       // a split's k is counted in 32 bits
    c.k_split = max(1L, div_up(div_up(a.n_rows, splits), kDepth)) * kDepth;
    c.splits = (unsigned)max(1L, div_up(a.n_rows, c.k_split));
    c.direct = c.splits == 1 && comps == 1 && !twice;
    return c;
}

struct BiasCut {
    long chunk;
    unsigned chunks;
    int across;
    unsigned groups;
};
BiasCut bias_cut(long rows, int n) {
    BiasCut c;
    c.across = 1;
    while (c.across < 64 && c.across * V < n) c.across *= 2;
    c.groups = (unsigned)div_up(n, (long)c.across * V);
    const long high = 256 / c.across;
    // enough workgroups for the card, at most 512 chunks, which are joined afterwards; a lane reads 4 rows at once
    const long most = max(1L, min(512L, div_up(4 * kFill, c.groups)));
    c.chunk = max(1L, div_up(div_up(rows, most), 4 * high)) * 4 * high;
    c.chunks = (unsigned)max(1L, div_up(rows, c.chunk));
    return c;
}

struct Layout {
    long s, g_z, sums, parts, bytes;
};
Layout layout_of(const LinearArgs& a, bool second) {
    const long z_bytes = align256(a.n_rows * a.outer * (a.gated ? 2 : 1) * (long)sizeof(T));
    const bool act = a.act != kActNone || a.gated;
    const long out = (long)a.outer * (a.gated ? 2 : 1), comps = (long)(a.lmax + 1) * (a.lmax + 1);
    const WeightCut w = weight_cut(a, second && act);
    const BiasCut b = bias_cut(a.n_rows, a.outer);
    Layout y;
    y.s = 0;
    y.g_z = act ? z_bytes : 0;
    y.sums = y.g_z + (act && second ? z_bytes : 0);
    y.parts = y.sums + align256(b.chunks * out * 4);
    y.bytes = y.parts + (w.direct ? 0 : align256(w.splits * comps * out * a.inner * 4 * (second && act ? 2 : 1)));
    return y;
}

Gemm forward_product(const LinearArgs& a, const T* x, long x_row) {
    Gemm g{};
    g.a = x;
    g.a_ld = x_row;
    g.a_batch = a.inner;
    g.b = static_cast<const T*>(a.w);
    g.b_ld = a.inner;
    g.b_degree = 1;
    g.b_batch = (long)a.outer * a.inner;
    g.m = a.n_rows;
    g.n = a.outer;
    g.k = a.inner;
    g.pair = a.outer;
    return g;
}

// out[row][inner] = s W
hipError_t input_gradient(const LinearArgs& a, const T* s, long s_row, void* out, hipStream_t st) {
    const int comps = (a.lmax + 1) * (a.lmax + 1);
    Gemm g{};
    g.a = s;
    g.a_ld = s_row;
    g.a_batch = a.outer;
    g.b = static_cast<const T*>(a.w);
    g.b_ld = a.inner;
    g.b_degree = 1;
    g.b_batch = (long)a.outer * a.inner;
    g.m = a.n_rows;
    g.n = a.inner;
    g.k = (long)a.outer * (a.gated ? 2 : 1);
    return run_gemm<true, false>(g, comps, EpiPlain{static_cast<T*>(out), (long)comps * a.inner, a.inner}, st);
}

// The parts of s^T x over the rows (direct: d_w itself).
hipError_t weight_gradient(const LinearArgs& a, const T* s, long s_row, const T* x, long x_row, const WeightCut& c,
                           float* parts, T* d_w, hipStream_t st) {
    const unsigned comps = (a.lmax + 1) * (a.lmax + 1);
    const long out = (long)a.outer * (a.gated ? 2 : 1);
    Gemm g{};
    g.a = s;
    g.a_ld = s_row;
    g.a_batch = a.outer;
    g.b = x;
    g.b_ld = x_row;
    g.b_batch = a.inner;
    g.m = out;
    g.n = a.inner;
    g.k = a.n_rows;
    g.splits = c.splits;
    g.k_split = c.k_split;
    if (c.direct) return run_tiles<false, false, false>(g, 1, EpiPlain{d_w, a.inner, a.inner}, st);
    return run_tiles<false, false, false>(g, comps * c.splits, EpiPart{parts, out * a.inner, a.inner}, st);
}

hipError_t act_bwd(const LinearArgs& a, const T* grad, long grad_row, T* s, float* sums, bool gated, int n, const BiasCut& c,
                   hipStream_t st) {
    const ActBwd p{grad, static_cast<const T*>(a.z), s, sums, grad_row, a.n_rows, c.chunk, n, a.act, c.across};
    if (a.n_rows == 0 && sums == nullptr) return hipSuccess;
    const dim3 grid(c.groups, c.chunks);
    if (n % V == 0)
        gated ? k_act_bwd<true, true><<<grid, 256, 0, st>>>(p) : k_act_bwd<false, true><<<grid, 256, 0, st>>>(p);
    else
        gated ? k_act_bwd<true, false><<<grid, 256, 0, st>>>(p) : k_act_bwd<false, false><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}

Join join_of(const float* parts, void* out, long size, int degrees, unsigned per_component) {
    const int ways = per_component <= 4 ? 1 : per_component <= 64 ? 4 : 16;
    return Join{parts, static_cast<T*>(out), size, degrees, per_component, ways, (unsigned)div_up(size, 256 / ways)};
}
hipError_t join(const Join& a, const Join& b, hipStream_t st) {
    const unsigned groups = a.groups * a.degrees + b.groups * b.degrees;
    if (groups == 0) return hipSuccess;
    k_join<<<groups, 256, 0, st>>>(a, b);
    return hipGetLastError();
}

#define CTP_TRY(call)                                                 \
    do {                                                              \
        if (const hipError_t e_ = (call); e_ != hipSuccess) return e_; \
    } while (0)

hipError_t fwd(const LinearArgs& a, hipStream_t st) {
    const int comps = (a.lmax + 1) * (a.lmax + 1);
    const Gemm g = forward_product(a, static_cast<const T*>(a.x), a.x_stride);
    if (a.gated)
        return run_pairs(g, EpiGated{static_cast<T*>(a.y), static_cast<T*>(a.z_out), static_cast<const T*>(a.bias), a.outer, a.act}, st);
    return run_gemm<true, true>(g, comps,
                                EpiLinear{static_cast<T*>(a.y), static_cast<T*>(a.z_out), static_cast<const T*>(a.bias),
                                          static_cast<const T*>(a.residual), (long)comps * a.outer, a.residual_stride,
                                          a.outer, a.act},
                                st);
}

hipError_t bwd(const LinearArgs& a, hipStream_t st) {
    const Layout y = layout_of(a, false);
    char* ws = static_cast<char*>(a.workspace);
    const bool act = a.act != kActNone || a.gated;
    const long out = (long)a.outer * (a.gated ? 2 : 1);
    float *sums = a.d_bias ? reinterpret_cast<float*>(ws + y.sums) : nullptr, *parts = reinterpret_cast<float*>(ws + y.parts);
    const BiasCut b = bias_cut(a.n_rows, a.outer);
    const T* s = static_cast<const T*>(a.grad);
    long s_row = a.grad_stride;
    if (act || sums) { CTP_TRY(act_bwd(a, s, s_row, act ? reinterpret_cast<T*>(ws + y.s) : nullptr, sums, a.gated, a.outer, b, st)); }
    if (act) s = reinterpret_cast<const T*>(ws + y.s), s_row = out;
    if (a.d_x) CTP_TRY(input_gradient(a, s, s_row, a.d_x, st));
    Join of_w{}, of_b{};
    if (a.d_w) {
        const WeightCut c = weight_cut(a, false);
        CTP_TRY(weight_gradient(a, s, s_row, static_cast<const T*>(a.x), a.x_stride, c, parts, static_cast<T*>(a.d_w), st));
        if (!c.direct) of_w = join_of(parts, a.d_w, out * a.inner, a.lmax + 1, c.splits);
    }
    if (a.d_bias) of_b = join_of(sums, a.d_bias, out, 1, b.chunks);
    return join(of_w, of_b, st);
}

hipError_t bwd_bwd(const LinearArgs& a, hipStream_t st) {
    const Layout y = layout_of(a, true);
    char* ws = static_cast<char*>(a.workspace);
    const int comps = (a.lmax + 1) * (a.lmax + 1);
    const bool act = a.act != kActNone || a.gated;
    const long out = (long)a.outer * (a.gated ? 2 : 1);
    const T *u = static_cast<const T*>(a.a_d_x), *grad = static_cast<const T*>(a.grad), *z = static_cast<const T*>(a.z);
    T *s = reinterpret_cast<T*>(ws + y.s), *g_z = reinterpret_cast<T*>(ws + y.g_z);
    float *sums = reinterpret_cast<float*>(ws + y.sums), *parts = reinterpret_cast<float*>(ws + y.parts);
    const Gemm v = forward_product(a, u, (long)comps * a.inner);
    const WeightCut c = weight_cut(a, act);
    if (!act) {
        if (a.g_grad) CTP_TRY((run_gemm<true, true>(v, comps, EpiPlain{static_cast<T*>(a.g_grad), (long)comps * a.outer, a.outer}, st)));
        if (a.g_w == nullptr) return hipSuccess;
        CTP_TRY(weight_gradient(a, grad, a.grad_stride, u, (long)comps * a.inner, c, parts, static_cast<T*>(a.g_w), st));
        return c.direct ? hipSuccess : join(join_of(parts, a.g_w, out * a.inner, a.lmax + 1, c.splits), Join{}, st);
    }
    const bool need_z = a.g_x || a.g_w || a.g_bias;
    if (a.gated)
        CTP_TRY(run_pairs(v, EpiSecond<true>{grad, z, static_cast<T*>(a.g_grad), need_z ? g_z : nullptr, a.g_w ? s : nullptr,
                                             a.grad_stride, a.outer, a.act}, st));
    else
        CTP_TRY((run_gemm<true, true>(v, 1, EpiSecond<false>{grad, z, static_cast<T*>(a.g_grad), need_z ? g_z : nullptr,
                                                            a.g_w ? s : nullptr, a.grad_stride, a.outer, a.act}, st)));
    if (a.g_x) CTP_TRY(input_gradient(a, g_z, out, a.g_x, st));
    Join of_w{}, of_b{};
    if (a.g_w) {
        CTP_TRY(weight_gradient(a, g_z, out, static_cast<const T*>(a.x), a.x_stride, c, parts, nullptr, st));
        CTP_TRY(weight_gradient(a, s, out, u, a.inner, c, parts + c.splits * out * a.inner, nullptr, st));
        of_w = join_of(parts, a.g_w, out * a.inner, 1, 2 * c.splits);
    }
    if (a.g_bias) {
        const int half = a.outer;
        const BiasCut b = bias_cut(a.n_rows, half);
        // the halves of a gated z as columns side by side: summed one half at a time
        for (int h = 0; h < (a.gated ? 2 : 1); ++h) {
            CTP_TRY(act_bwd(a, g_z + (long)h * half, out, nullptr, sums + (long)h * b.chunks * half, false, half, b, st));
            const Join of = join_of(sums + (long)h * b.chunks * half, static_cast<T*>(a.g_bias) + (long)h * half, half, 1, b.chunks);
            if (h + 1 == (a.gated ? 2 : 1))
                of_b = of;
            else
                CTP_TRY(join(of, Join{}, st));
        }
    }
    return join(of_w, of_b, st);
}

long workspace(const LinearArgs& a, bool second) { return layout_of(a, second).bytes; }

}  // namespace

template <>
const LinearOps& linear_ops<CTP_DENSE_TYPE>() {
    static constexpr LinearOps ops{fwd, bwd, bwd_bwd, workspace};
    return ops;
}

}  // namespace ctp
