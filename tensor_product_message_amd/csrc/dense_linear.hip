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
// matrix cores.  What is summed is in fp32, the biases' sums of s and g_z
// before that rounding.
#include "dense_common.hpp"
#include "dense_direct.hpp"
#include "dense_linear.hpp"

#include <algorithm>
#include <type_traits>

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
    long m_read;                // Across: values of a row of A, of B, that may be read, at least m, n
    int n_read;
    long pair;                  // Pairs: rows of B from a column's to its partner's
    long k_split;               // k of a split, a multiple of kDepth
    unsigned splits, tiles_m, tiles_n, total;
};

// Rows of V values each, of which the first `some` are there (Whole: all, and their columns too).
template <bool Whole, int R>
struct Rows {
    int some;
    int at, width;      // first column, columns of a row

    __device__ __forceinline__ vec_t<T> read(const T* row) const {
        if constexpr (Whole) return *reinterpret_cast<const typename Vec<T>::unaligned*>(row + at);
        return load_vec<T>(row, at / V, width);
    }
    // to[r step]: row r
    __device__ __forceinline__ void write(T* to, long step, const float (&x)[R][V], bool stream) const {
        if (stream) {
            keep_apart();
            write<true>(to, step, x);
            keep_apart();
        } else {
            write<false>(to, step, x);
        }
    }
    template <bool Stream>
    __device__ __forceinline__ void write(T* to, long step, const float (&x)[R][V]) const {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Floats<T> f;
#pragma unroll
            for (int q = 0; q < V; ++q) f.v[q] = x[r][q];
            const vec_t<T> v = narrow<T>(f);
            auto* place = reinterpret_cast<typename Vec<T>::unaligned*>(to + r * step + at);
            if constexpr (Whole) {
                if constexpr (Stream)
                    __builtin_nontemporal_store(v, place);
                else
                    *place = v;
            } else if (r < some) {
                store_left<T>(to + r * step + at, width - at, v);
            }
        }
    }
    // row r: what is at from[r step], zeros where there is none
    __device__ __forceinline__ void read(const T* from, long step, float (&x)[R][V]) const {
        vec_t<T> v[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v[r] = vec_t<T>{};
            if (Whole || r < some) v[r] = read(from + r * step);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < V; ++q) x[r][q] = (float)v[r][q];
    }
    // one vector added to every row
    __device__ __forceinline__ void add(const T* from, float (&x)[R][V]) const {
        const Floats<T> f = widen<T>(read(from));
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < V; ++q) x[r][q] += f.v[q];
    }
};

// A place in the output: rows m, m + step, .., of which `some` are there, and V columns from `at` on.
struct Place {
    unsigned outer, batch;
    long m;
    int step, some, at;
};

// A wave's results through its epilogue.
template <bool Pairs, int MT, int NT, class Epi>
__device__ __forceinline__ void write_tile(const f32x16 (&acc)[NT][MT], float* slab, int lane, int wm, int wn, int m_left,
                                           int n_left, bool whole, const Epi& epi, unsigned outer, unsigned batch, long m0, int n0) {
    if (whole) {
        by_rows<V, Pairs, MT, NT>(acc, slab, lane, [&](int m, int step, int n, auto& x, auto& y) {
            epi.template run<true>(Place{outer, batch, m0 + wm + m, step, 0, n0 + wn + n}, x, y);
        });
    } else {
        by_rows<V, Pairs, MT, NT>(acc, slab, lane, [&](int m, int step, int n, auto& x, auto& y) {
            const int left = wn + n < n_left ? (m_left - wm - m + step - 1) / step : 0;
            if (left > 0) epi.template run<false>(Place{outer, batch, m0 + wm + m, step, left, n0 + wn + n}, x, y);
        });
    }
}

// What a gradient's first operand is made of on its way into LDS: A times act'(z), z dense rows of z_ld values, and
// (Across) the sums of A's columns over each split's k, parts of m values.
struct Curve {
    const T* z;
    long z_ld;
    int act;
    float* sums;        // null: none
};

// Tiles of BM x BN by 4 waves, WM x (4 / WM) of them, the block-th of every `blocks`.  One buffer in LDS: the next
// tiles' reads are in flight in registers while the matrix cores work, and the workgroups that share a CU fill each
// other's pauses.
template <bool AlongA, bool AlongB, int BM, int BN, int WM>
struct StagedTiles {
    static constexpr int WN = 4 / WM, MT = BM / 32 / WM, NT = BN / 32 / WN;
    typedef Staged<T, AlongA, BM, kDepth, 256> SA;
    typedef Staged<T, AlongB, BN, kDepth, 256> SB;
    static constexpr int kTiles = SA::tile_t::kBytes + SB::tile_t::kBytes, kSlabs = 4 * 32 * kSlab<NT> * 4;
    static constexpr int kBytes = kTiles > kSlabs ? kTiles : kSlabs;
};

template <bool AlongA, bool AlongB, int BM, int BN, int WM, bool Pairs, bool Curved, bool Summed, class Epi>
__device__ __forceinline__ void staged_tiles(const Gemm& g, const Epi& epi, const Curve& c, char* lds, unsigned block, unsigned blocks) {
    typedef StagedTiles<AlongA, AlongB, BM, BN, WM> S;
    constexpr int MT = S::MT, NT = S::NT;
    typedef typename S::SA SA;
    typedef typename S::SB SB;
    E* la = reinterpret_cast<E*>(lds);
    E* lb = reinterpret_cast<E*>(lds + SA::tile_t::kBytes);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave % WM * 32 * MT, wn = wave / WM * 32 * NT;

    for (unsigned id = block; id < g.total; id += blocks) {
        const TileAt t = tile_at(xcd_order(id, g.total), g.tiles_m, g.tiles_n);
        const unsigned batch = t.outer / g.splits, split = t.outer % g.splits;
        const long m0 = (long)t.m * BM, k0 = split * g.k_split;
        const int n0 = t.n * (Pairs ? BN / 2 : BN);
        const int k_end = (int)min(g.k_split, g.k - k0);    // from here on k counts from k0
        const T* a = g.a + batch * g.a_batch + (AlongA ? m0 * g.a_ld + k0 : k0 * g.a_ld + m0);
        const T* b = g.b + (g.b_degree ? degree_of(batch) : (int)batch) * g.b_batch +
                     (AlongB ? (long)n0 * g.b_ld + k0 : k0 * g.b_ld + n0);
        const T* z = Curved ? c.z + (AlongA ? m0 * c.z_ld + k0 : k0 * c.z_ld + m0) : nullptr;
        const int m_left = (int)min((long)BM, g.m - m0), n_left = min(g.n - n0, BN);
        // rows past the last give results that nobody stores
        auto row_a = [&](int r) { return (long)min(r, m_left - 1); };
        auto row_b = [&](int r) {
            if constexpr (Pairs) return pair_row(r, n_left, g.pair);
            return (long)min(r, n_left - 1);
        };
        const bool whole_m = m_left == BM, whole_n = n_left >= (Pairs ? BN / 2 : BN);
        const bool sums = Summed && c.sums != nullptr && t.n == 0 && batch == 0;
        float sum[V] = {};
        f32x16 acc[NT][MT] = {};
        // The tiles of k from step `first` to before `last`, the next one on its way while one is multiplied.  (Two on
        // their way measured no faster: a step's own instructions are its time, not its reads.)
        auto run = [&](auto how, int first, int last) {
            constexpr int How = decltype(how)::value;
            if (first >= last) return;
            SA sa, sz;
            SB sb;
            auto load = [&](int step) {
                const int k = step * kDepth;
                sa.template load<How>(a, g.a_ld, m_left, k, k_end, row_a);
                if constexpr (Curved) sz.template load<How>(z, c.z_ld, m_left, k, k_end, row_a);
                sb.template load<How>(b, g.b_ld, n_left, k, k_end, row_b);
            };
            load(first);
            for (int step = first; step < last; ++step) {
                if constexpr (How == kClamped) {
                    sa.fix(m_left, step * kDepth, k_end);
                    if constexpr (Curved) sz.fix(m_left, step * kDepth, k_end);
                    sb.fix(n_left, step * kDepth, k_end);
                }
                if constexpr (Curved)
                    sa.template curve<Summed>(sz, c.act, sum);
                else if constexpr (Summed)
                    if (sums) sa.add_columns(sum);
                lds_barrier();
                sa.store(la);
                sb.store(lb);
                lds_barrier();
                if (step + 1 < last) load(step + 1);
                multiply_step<typename SA::tile_t, typename SB::tile_t, kParts, MT, NT, kDepth>(acc, la, lb, wm, wn, lane);
            }
        };
        const int steps = (k_end + kDepth - 1) / kDepth, whole = k_end / kDepth;
        if (read_whole<AlongA, AlongB>(whole_m, whole_n)) {
            run(Is<kWhole>{}, 0, whole);
            run(Is<kGuarded>{}, whole, steps);
        } else if (read_clamped<T, AlongA, AlongB>(m_left, n_left, k_end)) {
            run(Is<kClamped>{}, 0, steps);
        } else {
            run(Is<kGuarded>{}, 0, steps);
        }
        lds_barrier();
        float* slab = reinterpret_cast<float*>(lds) + wave * 32 * kSlab<NT>;
        if constexpr (kParts > 1)
            again_where_beyond(
                acc, lane, k_end,
                [&](int m, int n, int k, float& x, float& at, float& y) {
                    // rows past the last: the last
                    const long row = min(wm + m, m_left - 1);
                    x = (float)(AlongA ? a[row * g.a_ld + k] : a[k * g.a_ld + row]);
                    if constexpr (Curved) at = (float)(AlongA ? z[row * c.z_ld + k] : z[k * c.z_ld + row]);
                    y = (float)(AlongB ? b[row_b(wn + n) * g.b_ld + k] : b[k * g.b_ld + row_b(wn + n)]);
                },
                [&](auto& x, const auto& at) {
                    if constexpr (Curved)
                        with_act(c.act, [&](auto is) {
                            float f, d1, d2;
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                activation<decltype(is)::value>(at[u], f, d1, d2);
                                x[u] *= d1;
                            }
                        });
                });
        write_tile<Pairs, MT, NT>(acc, slab, lane, wm, Pairs ? wn / 2 : wn, m_left, n_left, whole_m && whole_n, epi, t.outer, batch, m0, n0);
        lds_barrier();
        if constexpr (Summed) {
            if (sums) {
                // the threads of a column, in their order
                constexpr int kHigh = 256 / SA::kPerRow;
                static_assert(kHigh * BM * 4 <= S::kBytes);
                float* part = reinterpret_cast<float*>(lds);
#pragma unroll
                for (int q = 0; q < V; ++q) part[threadIdx.x / SA::kPerRow * BM + threadIdx.x % SA::kPerRow * V + q] = sum[q];
                lds_barrier();
                if ((int)threadIdx.x < m_left) {
                    float s = 0.0f;
                    for (int r = 0; r < kHigh; ++r) s += part[r * BM + threadIdx.x];
                    c.sums[split * g.m + m0 + threadIdx.x] = s;
                }
                lds_barrier();
            }
        }
    }
}

template <bool AlongA, bool AlongB, int BM, int BN, int WM, bool Pairs, class Epi>
__global__ __launch_bounds__(256, 2) void k_gemm(Gemm g, Epi epi) {
    __shared__ __attribute__((aligned(16))) char lds[StagedTiles<AlongA, AlongB, BM, BN, WM>::kBytes];
    staged_tiles<AlongA, AlongB, BM, BN, WM, Pairs, false, false>(g, epi, Curve{}, lds, blockIdx.x, gridDim.x);
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
            if constexpr (Pairs) return pair_row(r, n_left, g.pair);
            return (long)min(r, n_left - 1);
        });
        auto issue = [&](int step, int buffer) {
            const int k = step * kDepth;
            // Across: what lies past the last k is the buffer's end
            const long rows = min(k_end - k, kDepth);
            const unsigned a_bytes = AlongA ? (unsigned)kBufferBytes : buffer_bytes(rows, g.a_ld, min((long)Side, g.m_read - m0));
            const unsigned b_bytes = AlongB ? (unsigned)kBufferBytes : buffer_bytes(rows, g.b_ld, min(Side, g.n_read - n0));
            da.issue(buffer_at(a + (AlongA ? k : k * g.a_ld), a_bytes), base + buffer * kBuffer, k_end - k);
            db.issue(buffer_at(b + (AlongB ? k : k * g.b_ld), b_bytes), base + buffer * kBuffer + TA::kBytes, k_end - k);
        };
        f32x16 acc[NT][MT] = {};
        if (k_end > 0)
            multiply_tiles<TA, TB, 1, MT, NT, kDepth>(acc, reinterpret_cast<const E*>(lds), (k_end + kDepth - 1) / kDepth, wm, wn, lane, issue,
                                                      [](int) {});
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
    bool stream;                // see streams_out
    template <bool Whole, int R>
    __device__ __forceinline__ void run(const Place& p, float (&x)[R][V], float (&)[R][V]) const {
        const Rows<Whole, R> rows{p.some, p.at, n};
        float r[R][V];
        if (residual != nullptr) rows.read(residual + p.m * residual_row + (long)p.batch * n, p.step * residual_row, r);
        if (bias != nullptr && p.batch == 0) rows.add(bias, x);
        const long to = p.m * row + (long)p.batch * n;
        if (z != nullptr) rows.write(z + to, p.step * row, x, stream);
        with_act(act, [&](auto is) {
            float d1, d2;
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) activation<decltype(is)::value>(x[i][q], x[i][q], d1, d2);
        });
        if (residual != nullptr)
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) x[i][q] += r[i][q];
        rows.write(y + to, p.step * row, x, stream);
    }
};

// h = act(x + bias[0]) (y + bias[1]), z the two sums.  (Not marked as streams: a wave's rows are 64 bytes of 16-bit
// values here, and half lines written around the cache are written twice, 451 MB for 403.)
struct EpiGated {
    T *h, *z;
    const T* bias;
    int n, act;
    template <bool Whole, int R>
    __device__ __forceinline__ void run(const Place& p, float (&x)[R][V], float (&y)[R][V]) const {
        const Rows<Whole, R> rows{p.some, p.at, n};
        if (bias != nullptr) {
            rows.add(bias, x);
            rows.add(bias + n, y);
        }
        if (z != nullptr) {
            rows.write(z + p.m * 2 * n, p.step * 2L * n, x, false);
            rows.write(z + p.m * 2 * n + n, p.step * 2L * n, y, false);
        }
        with_act(act, [&](auto is) {
            float d1, d2;
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    activation<decltype(is)::value>(x[i][q], x[i][q], d1, d2);
                    x[i][q] *= y[i][q];
                }
        });
        rows.write(h + p.m * n, (long)p.step * n, x, false);
    }
};

// out = x
struct EpiPlain {
    T* out;
    long row;
    int n;
    bool stream;
    template <bool Whole, int R>
    __device__ __forceinline__ void run(const Place& p, float (&x)[R][V], float (&)[R][V]) const {
        Rows<Whole, R>{p.some, p.at, n}.write(out + p.m * row + (long)p.batch * n, p.step * row, x, stream);
    }
};

// A split's share of a sum, in fp32.
struct EpiPart {
    float* parts;
    long size;      // of one part: rows n values wide
    int n;
    template <bool Whole, int R>
    __device__ __forceinline__ void run(const Place& p, float (&x)[R][V], float (&)[R][V]) const {
        float* to = parts + p.outer * size + p.m * n + p.at;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int q = 0; q < V; q += 4) {
                vec_t<float> w;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = x[i][q + e];
                if constexpr (Whole)
                    *reinterpret_cast<Vec<float>::unaligned*>(to + (long)i * p.step * n + q) = w;
                else if (i < p.some && p.at + q < n)
                    store_left<float>(to + (long)i * p.step * n + q, n - p.at - q, w);
            }
    }
};

// The second backward pass's middle: v = x (gated: x and y) in, g_G, g_z and s out.
template <bool Gated>
struct EpiSecond {
    const T *grad, *z;
    T *g_grad, *g_z, *s;
    float* exact;       // g_z before its rounding, for the bias's sums; null: not wanted
    long grad_row;
    int n, act;
    template <bool Whole>
    __device__ __forceinline__ void write_exact(float* row, int at, const float (&x)[V]) const {
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            const vec_t<float> v{x[q], x[q + 1], x[q + 2], x[q + 3]};
            if constexpr (Whole)
                *reinterpret_cast<Vec<float>::unaligned*>(row + at + q) = v;
            else if (at + q < n)
                store_left<float>(row + at + q, n - at - q, v);
        }
    }
    template <bool Whole, int R>
    __device__ __forceinline__ void run(const Place& place, float (&x)[R][V], float (&y)[R][V]) const {
        // a row at a time: its many values would not all find registers
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!Whole && i >= place.some) break;
            const Rows<Whole, 1> row{1, place.at, n};
            const long m = place.m + (long)i * place.step, zr = m * n * (Gated ? 2 : 1);
            float g[1][V], a[1][V], b[1][V], o[1][V], p[1][V], q[1][V], pb[1][V], qb[1][V];
            row.read(grad + m * grad_row, 0, g);
            row.read(z + zr, 0, a);
            if constexpr (Gated) row.read(z + zr + n, 0, b);
            with_act(act, [&](auto is) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float f, d1, d2;
                    activation<decltype(is)::value>(a[0][e], f, d1, d2);
                    const float u = x[i][e], h = g[0][e];
                    if constexpr (Gated) {
                        const float w = y[i][e], c = b[0][e], hc = h * c;
                        o[0][e] = __builtin_fmaf(u * c, d1, w * f);
                        p[0][e] = __builtin_fmaf(u * hc, d2, w * h * d1);
                        pb[0][e] = u * h * d1;
                        q[0][e] = hc * d1;
                        qb[0][e] = h * f;
                    } else {
                        o[0][e] = u * d1;
                        p[0][e] = u * h * d2;
                        q[0][e] = h * d1;
                    }
                }
            });
            if (g_grad != nullptr) row.write(g_grad + m * n, 0, o, false);
            if (exact != nullptr) {
                write_exact<Whole>(exact + zr, place.at, p[0]);
                if constexpr (Gated) write_exact<Whole>(exact + zr + n, place.at, pb[0]);
            }
            if (g_z != nullptr) {
                row.write(g_z + zr, 0, p, false);
                if constexpr (Gated) row.write(g_z + zr + n, 0, pb, false);
            }
            if (s != nullptr) {
                row.write(s + zr, 0, q, false);
                if constexpr (Gated) row.write(s + zr + n, 0, qb, false);
            }
        }
    }
};

// ---------------------------------------------------------------- small layers' gradients

// Both gradients of a layer whose matrices are small, in one launch: d_W's parts by the first workgroups, d_x by the
// others, each forming s = grad act'(z) on its way (the layer is few tiles wide, so s is not formed often), and the
// bias's sums beside d_W's.  Neither product fills the card by itself, and s is neither written nor read: the gradients
// of 83325 rows of 64 -> 64 floats take 30 us so and 44 us in four launches.
template <bool Curved>
__global__ __launch_bounds__(256, 2) void k_small_bwd(Gemm of_w, EpiPart to_w, Gemm of_x, EpiPlain to_x, Curve c) {
    typedef StagedTiles<false, false, 64, 64, 2> W;
    typedef StagedTiles<true, false, 64, 64, 2> X;
    __shared__ __attribute__((aligned(16))) char lds[W::kBytes > X::kBytes ? W::kBytes : X::kBytes];
    if (blockIdx.x < of_w.total)
        staged_tiles<false, false, 64, 64, 2, false, Curved, true>(of_w, to_w, c, lds, blockIdx.x, of_w.total);
    else
        staged_tiles<true, false, 64, 64, 2, false, Curved, false>(of_x, to_x, c, lds, blockIdx.x - of_w.total, gridDim.x - of_w.total);
}

// ---------------------------------------------------------------- long sums, few tiles

// The epilogue of a product whose k was cut: V columns of a row a thread, the parts summed in their order.  Pairs: a
// row's halves lie beside each other.
template <bool Pairs, class Epi>
__global__ __launch_bounds__(256) void k_finish(const float* parts, unsigned splits, int m, int n, unsigned batches, Epi epi) {
    const int vecs = (n + V - 1) / V, width = Pairs ? 2 * n : n;
    const long size = (long)m * width, total = (long)batches * m * vecs;
    for (long id = (long)blockIdx.x * 256 + threadIdx.x; id < total; id += 256L * gridDim.x) {
        const int at = (int)(id % vecs) * V;
        const long row = id / vecs;
        const unsigned batch = (unsigned)(row / m);
        const float* from = parts + batch * splits * size + row % m * width;
        float x[1][V] = {}, y[1][V] = {};
        auto add = [&](float (&sum)[1][V], const float* p) {
#pragma unroll
            for (int q = 0; q < V; q += 4)
                if (at + q < n) {
                    const vec_t<float> v = load_vec<float>(p, (at + q) / 4, n);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[0][q + e] += v[e];
                }
        };
#pragma unroll 4
        for (unsigned s = 0; s < splits; ++s) {
            add(x, from + s * size);
            if constexpr (Pairs) add(y, from + s * size + n);
        }
        epi.template run<false>(Place{batch, batch, row % m, 1, 1, at}, x, y);
    }
}

// ---------------------------------------------------------------- floats, short sums

#if CTP_DENSE_TYPE == 0

// Floats with at most 64 Blocks terms a sum, where taking the operands apart and what is done with the results cost
// more than the products: a wave keeps 32 rows of A in registers, taken apart once, and goes through the columns, 64
// (Pairs: 32 and their partners) at a time, whose parts the workgroup's waves share in LDS.  Results go from the matrix
// cores' registers to memory, 16 bytes a lane.
template <class Epi>
constexpr bool kIsPlain = std::is_same<Epi, EpiPlain>::value;

template <int Blocks, bool AlongB, bool Pairs, class Epi>
__global__ __launch_bounds__(256, Blocks == 2 ? (Pairs ? 1 : 2) : kIsPlain<Epi> ? 3 : 2) void k_rows(Gemm g, Epi epi, unsigned tiles_a_group) {
    constexpr int kLong = 64 * Blocks, kCols = Pairs ? 32 : 64;
    typedef Staged<T, AlongB, 64, kLong, 256> SB;
    typedef typename SB::tile_t TB;
    typedef typename Frag<E>::type frag_t;
    __shared__ __attribute__((aligned(16))) char lds[TB::kBytes];
    constexpr int kWide = kSlab<Pairs ? 2 : 1>;
    __shared__ __attribute__((aligned(16))) float slabs[4][32 * kWide];
    E* lb = reinterpret_cast<E*>(lds);
    float* slab = slabs[threadIdx.x >> 6];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const TileAt t = tile_at(xcd_order(blockIdx.x, g.total), g.tiles_m, g.tiles_n);
    const unsigned batch = t.outer;
    const long m = (long)t.m * 128 + wave * 32 + (lane & 31);
    const int k_end = (int)g.k;
    const T* row = g.a + batch * g.a_batch + min(m, g.m - 1) * g.a_ld;
    // 16 values of k a lane and 32: 64 bytes in one piece
    frag_t a[kLong / 16][kParts];
#pragma unroll
    for (int k = 0; k < kLong; k += 32) {
        vec_t<T> v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int at = k + 16 * (lane >> 5) + 4 * q;
            if (at + V <= k_end)
                v[q] = *reinterpret_cast<const typename Vec<T>::unaligned*>(row + at);
            else
                v[q] = at < k_end ? load_vec<T>(row, at / V, k_end) : vec_t<T>{};
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const ThreeParts x = take_apart(v[2 * s + q / 4][q % 4]);
#pragma unroll
                for (int p = 0; p < kParts; ++p) a[k / 16 + s][p][q] = x.p[p];
            }
    }
    const T* b = g.b + (g.b_degree ? degree_of(batch) : (int)batch) * g.b_batch;
    const int n_first = t.n * tiles_a_group * kCols, n_last = min(g.n, n_first + (int)tiles_a_group * kCols);
    SB sb;
    auto load = [&](int n0) {
        const T* from = b + (AlongB ? (long)n0 * g.b_ld : n0);
        const int n_left = g.n - n0;
        auto row_b = [&](int r) {
            if constexpr (Pairs) return (long)min(r & 31, n_left - 1) + (r >> 5) * g.pair;
            return (long)min(r, n_left - 1);
        };
        if (k_end == kLong && n_left >= kCols)
            sb.template load<kWhole>(from, g.b_ld, n_left, 0, k_end, row_b);
        else
            sb.template load<kGuarded>(from, g.b_ld, n_left, 0, k_end, row_b);
    };
    load(n_first);
    for (int n0 = n_first; n0 < n_last; n0 += kCols) {
        lds_barrier();
        sb.store(lb);
        lds_barrier();
        if (n0 + kCols < n_last) load(n0 + kCols);
        f32x16 acc[2][1] = {};
#pragma unroll
        for (int k = 0; k < kLong; k += 16) {
            frag_t f[2][kParts];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    f[j][p] = TB::template read<16>(lb + p * TB::kPlane, 32 * j, k / 32 * 32 + k % 32 / 2, lane);
            // the parts' smallest products first
#pragma unroll
            for (int s = kParts - 1; s >= 0; --s)
#pragma unroll
                for (int p = 0; p <= s; ++p)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[j][0] = mfma(f[j][s - p], a[k / 16][p], acc[j][0]);
        }
        const long m0 = (long)t.m * 128 + wave * 32;
        const auto col = [&](int n) { return n0 + (Pairs ? n & 31 : n); };
        again_by_lanes(
            acc, slab, lane, k_end, [&](int m, int n) { return m0 + m < g.m && col(n) < g.n; },
            [&](int m, int n, int k, float& x, float& y) {
                x = (g.a + batch * g.a_batch)[(m0 + m) * g.a_ld + k];
                y = AlongB ? b[(col(n) + (Pairs ? (n >> 5) * g.pair : 0L)) * g.b_ld + k] : b[(long)k * g.b_ld + col(n)];
            });
        // 32 columns at a time: a row of them is 128 bytes
        auto write = [&](auto whole) {
            constexpr bool Whole = decltype(whole)::value != 0;
            constexpr int B = kIsPlain<Epi> ? 4 : 1;       // rows of a lane at once
            const int nc = lane % 8 * 4;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (!Pairs || j == 0) wave_lds_fence();
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f32x4*>(slab + (lane & 31) * kWide + (Pairs ? 32 * j : 0) + 8 * q + 4 * (lane >> 5)) =
                        f32x4{acc[j][0][4 * q], acc[j][0][4 * q + 1], acc[j][0][4 * q + 2], acc[j][0][4 * q + 3]};
                if (Pairs && j == 0) continue;
                wave_lds_fence();
                const int n = n0 + nc + (Pairs ? 0 : 32 * j);
#pragma unroll 1
                for (int r0 = 0; r0 < 4; r0 += B) {
                    float x[B][4], y[B][4];
#pragma unroll
                    for (int r = 0; r < B; ++r) {
                        const float* from = slab + (8 * (r0 + r) + lane / 8) * kWide + nc;
                        *reinterpret_cast<f32x4*>(x[r]) = *reinterpret_cast<const f32x4*>(from);
                        if constexpr (Pairs) *reinterpret_cast<f32x4*>(y[r]) = *reinterpret_cast<const f32x4*>(from + 32);
                    }
                    const long m = m0 + 8 * r0 + lane / 8;
                    const int some = Whole || n < g.n ? (int)min((long)B, (g.m - m + 7) / 8) : 0;
                    if (Whole || some > 0) epi.template run<Whole>(Place{batch, batch, m, 8, some, n}, x, y);
                }
            }
        };
        if (n0 + kCols <= g.n && m0 + 32 <= g.m)
            write(Is<1>{});
        else
            write(Is<0>{});
    }
}
#endif

// ---------------------------------------------------------------- few rows

// Up to 16 MB rows, where the weights' way from memory is all there is: no tile of x fills the matrix cores, and no
// weight is used twice.  Each wave takes 32 rows of w (Pairs: 16 and their partners) and one of Waves shares of k,
// straight from memory into the matrix instruction's registers, kAhead reads of each row under way at once; the
// waves' sums meet in LDS, in the waves' order.  Which k goes to which lane does not matter as long as w and x agree.
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
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, from = (lane >> 4) * V;
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
                    const int k = k0 + s * kStep + h * 4 * V + from;
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
                    const int k = k0 + s * kStep + h * 4 * V + from;
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
        float x[1][V], y[1][V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            x[0][q] = part[0][m][n + q];
            if constexpr (Pairs) y[0][q] = part[0][m][16 + n + q];
        }
        for (int w = 1; w < Waves; ++w)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                x[0][q] += part[w][m][n + q];
                if constexpr (Pairs) y[0][q] += part[w][m][16 + n + q];
            }
        epi.template run<false>(Place{batch, batch, m, 1, 1, n0 + n}, x, y);
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
    long s_row;         // elements from row to row of s; above what a row has: whole vectors, zeros past its end
};

// As the members of Rows, for rows whose columns are whole vectors but whose number is `some`.
template <bool Whole, int R>
__device__ __forceinline__ void read_rows(const Rows<Whole, R>& rows, const T* from, long step, float (&x)[R][V]) {
    vec_t<T> v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        v[r] = vec_t<T>{};
        if (r < rows.some) v[r] = rows.read(from + r * step);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int q = 0; q < V; ++q) x[r][q] = (float)v[r][q];
}
template <bool Whole, int R>
__device__ __forceinline__ void write_rows(const Rows<Whole, R>& rows, T* to, long step, const float (&x)[R][V]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r < rows.some) Rows<Whole, 1>{1, rows.at, rows.width}.write(to + r * step, 0, reinterpret_cast<const float(&)[1][V]>(x[r]), false);
}

// The lanes' sums of N columns of H halves of n, `across` lanes beside each other, added over the workgroup's rows in
// their order.  part: 256 H N floats.
template <int H, int N>
__device__ __forceinline__ void put_sums(const float (&sum)[H][N], float* part, int across, int n, float* to) {
    const int tx = threadIdx.x % across, ty = threadIdx.x / across, high = 256 / across;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int q = 0; q < N; ++q) part[((h * high + ty) * N + q) * across + tx] = sum[h][q];
    lds_barrier();
    for (int i = threadIdx.x; i < H * N * across; i += 256) {
        const int h = i / (N * across), c = i % (N * across), col = blockIdx.x * across * N + c;
        if (col >= n) continue;
        float s = 0.0f;
        for (int r = 0; r < high; ++r) s += part[((h * high + r) * N + c % N) * across + c / N];
        to[h * n + col] = s;
    }
}

// Whole: n is whole vectors.
template <bool Gated, bool Whole>
__global__ __launch_bounds__(256) void k_act_bwd(ActBwd p) {
    constexpr int H = Gated ? 2 : 1, R = Gated ? 2 : 4;      // rows that a lane reads at once
    __shared__ float part[256 * H * V];
    const int tx = threadIdx.x % p.across, ty = threadIdx.x / p.across, high = 256 / p.across;
    const int at = (blockIdx.x * p.across + tx) * V;
    const long first = blockIdx.y * p.chunk, last = min(first + p.chunk, p.rows);
    float sum[H][V] = {};
    for (long m = at < p.n ? first + ty : last; m < last; m += R * high) {
        // past the chunk's last row: zeros
        const Rows<Whole, R> rows{(int)min((long)R, (last - m + high - 1) / high), at, p.n};
        float g[R][V], a[R][V], u[R][V];
        read_rows(rows, p.grad + m * p.grad_row, high * p.grad_row, g);
        if (p.s != nullptr) {
            const long zr = m * p.n * H, step = (long)high * p.n * H, sr = m * p.s_row, s_step = high * p.s_row;
            read_rows(rows, p.z + zr, step, a);
            if constexpr (Gated) read_rows(rows, p.z + zr + p.n, step, u);
            with_act(p.act, [&](auto is) {
                float f, d1, d2;
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        activation<decltype(is)::value>(a[i][q], f, d1, d2);
                        if constexpr (Gated) {
                            const float b = u[i][q];
                            u[i][q] = g[i][q] * f;
                            g[i][q] = g[i][q] * b * d1;
                        } else {
                            g[i][q] *= d1;
                        }
                    }
            });
            if (!Gated && p.s_row > p.n)
                write_rows(Rows<true, R>{rows.some, at, p.n}, p.s + sr, s_step, g);
            else
                write_rows(rows, p.s + sr, s_step, g);
            if constexpr (Gated) write_rows(rows, p.s + sr + p.n, s_step, u);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if (i >= rows.some) continue;
                sum[0][q] += g[i][q];
                if constexpr (Gated) sum[1][q] += u[i][q];
            }
    }
    if (p.sums != nullptr) put_sums(sum, part, p.across, p.n, p.sums + (long)blockIdx.y * p.n * H);
}

// Sums of the columns of dense rows of floats, a part for each chunk of rows; workgroups as k_act_bwd's.
struct ColumnSums {
    const float* from;
    float* sums;
    long rows, chunk;
    int n, across;
};

// Whole: n is whole vectors.
template <bool Whole>
__global__ __launch_bounds__(256) void k_sums(ColumnSums p) {
    constexpr int N = kVec<float>, R = 4;
    __shared__ float part[256 * N];
    const int tx = threadIdx.x % p.across, ty = threadIdx.x / p.across, high = 256 / p.across;
    const int at = (blockIdx.x * p.across + tx) * N;
    const long first = blockIdx.y * p.chunk, last = min(first + p.chunk, p.rows);
    float sum[1][N] = {};
    for (long m = at < p.n ? first + ty : last; m < last; m += R * high) {
        vec_t<float> v[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            v[i] = vec_t<float>{};
            const float* row = p.from + (m + i * high) * p.n;
            if (m + i * high < last) v[i] = Whole ? *reinterpret_cast<const Vec<float>::unaligned*>(row + at) : load_vec<float>(row, at / N, p.n);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int q = 0; q < N; ++q) sum[0][q] += v[i][q];
    }
    put_sums(sum, part, p.across, p.n, p.sums + (long)blockIdx.y * p.n);
}

// Rows laid out for 16-byte pieces: to[i][j][0 .. padded) = from[i][j][0 .. width), zeros past the width and for
// j >= there.  A few rows of which none begins on 16 bytes cost a product's tiles more than this pass: the gradients of
// 5001 rows of 1003 -> 777 float16 take 75 us with it and 140 us without.
struct Pack {
    const T* from;
    T* to;
    long n_i, from_i, from_j;   // elements from i to i and from j to j
    int n_j, there, width, padded;
};

__global__ __launch_bounds__(256) void k_pack(Pack first, Pack second, unsigned groups_first) {
    const bool is_first = blockIdx.x < groups_first;
    const Pack p = is_first ? first : second;
    const unsigned group = is_first ? blockIdx.x : blockIdx.x - groups_first, groups = is_first ? groups_first : gridDim.x - groups_first;
    const int vecs = p.padded / V;
    const long total = p.n_i * p.n_j * vecs;
    for (long id = (long)group * 256 + threadIdx.x; id < total; id += 256L * groups) {
        const long row = id / vecs, i = row / p.n_j;
        const int v = (int)(id % vecs), j = (int)(row % p.n_j);
        vec_t<T> x{};
        if (j < p.there && v * V < p.width) x = load_vec<T>(p.from + i * p.from_i + j * p.from_j, v, p.width);
        *reinterpret_cast<vec_t<T>*>(p.to + id * V) = x;
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
    const long of_first = (long)first.groups * first.degrees, total = of_first + (long)second.groups * second.degrees;
    for (long block = blockIdx.x; block < total; block += gridDim.x) {
        const bool is_first = block < of_first;
        const Join j = is_first ? first : second;
        const unsigned id = (unsigned)(is_first ? block : block - of_first);
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
        lds_barrier();
    }
}

// ---------------------------------------------------------------- launches

#define CTP_TRY(call)                                                 \
    do {                                                              \
        if (const hipError_t e_ = (call); e_ != hipSuccess) return e_; \
    } while (0)

// (Sizes here are compared by std::min and max<long>: those without std are int's on the host.)
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
    k_gemm<AlongA, AlongB, BM, BN, WM, Pairs><<<dim3((unsigned)std::min<long>(g.total, max_groups(256))), 256, 0, st>>>(g, epi);
    return hipGetLastError();
}
template <bool AlongA, bool AlongB, int Side, bool Pairs, class Epi>
hipError_t run_direct(Gemm g, unsigned outer, const Epi& epi, hipStream_t st) {
    if (!set_tiles(g, Side, Pairs ? Side / 2 : Side, outer)) return hipErrorInvalidValue;
    if (g.total == 0) return hipSuccess;
    k_gemm_direct<AlongA, AlongB, Side, Pairs>
        <<<dim3((unsigned)std::min<long>(g.total, max_groups(2 * Side))), 2 * Side, 0, st>>>(g, epi);
    return hipGetLastError();
}

// Whether tiles may go to LDS directly (a gated layer's of 2^30 values or more a matrix do not: staged tiles).
template <bool AlongA, bool AlongB, bool Pairs>
bool direct(const Gemm& g) {
    return kParts == 1 && comes_directly(g.a, g.a_ld, g.a_batch, AlongA ? g.k : g.m_read, 0) &&
           comes_directly(g.b, g.b_ld, g.b_batch, AlongB ? g.k : (long)g.n_read, Pairs ? g.pair : 0);
}

#if CTP_DENSE_TYPE == 0
template <int Blocks, bool AlongB, bool Pairs, class Epi>
hipError_t run_rows(Gemm g, unsigned batches, const Epi& epi, hipStream_t st) {
    // columns are cut into groups where the rows alone would leave the card empty
    const long cols = Pairs ? 32 : 64, tiles = div_up(g.n, cols), rows = div_up(g.m, 128) * batches;
    const long groups = std::max<long>(1L, std::min<long>(tiles, div_up(4 * kFill, rows)));
    const long per = div_up(tiles, groups);
    if (!set_tiles(g, 128, per * cols, batches)) return hipErrorInvalidValue;
    if (g.total > max_groups(256)) return hipErrorInvalidValue;
    k_rows<Blocks, AlongB, Pairs><<<dim3(g.total), 256, 0, st>>>(g, epi, (unsigned)per);
    return hipGetLastError();
}
#endif

// Tiles of 256 reuse an operand most, and are taken where they fill the card; tiles of 64 are for what has too few of
// the others.
template <bool AlongA, bool AlongB, bool Pairs, class Epi>
hipError_t run_tiles(const Gemm& g, unsigned outer, const Epi& epi, hipStream_t st) {
    const long n = Pairs ? 2L * g.n : g.n;
    if constexpr (kParts == 1) {
        if (direct<AlongA, AlongB, Pairs>(g)) {
            if (g.m > 128 && n > 128 && div_up(g.m, 256) * div_up(n, 256) * outer >= kFill * 3 / 8) return run_direct<AlongA, AlongB, 256, Pairs>(g, outer, epi, st);
            if (g.m > 64 && n > 64 && div_up(g.m, 128) * div_up(n, 128) * outer >= kFill / 4) return run_direct<AlongA, AlongB, 128, Pairs>(g, outer, epi, st);
        }
    }
#if CTP_DENSE_TYPE == 0
    if constexpr (AlongA) {
        // many columns for few terms: 83325 x 64 -> 1024 takes 94 us so and 135 us in tiles of 64, -> 256 30 and 33
        if (g.splits == 1 && div_up(g.m, 128) * outer * div_up(n, 64) >= kFill) {
            if (g.k <= 64 && n >= 256) return run_rows<1, AlongB, Pairs>(g, outer, epi, st);
            if (g.k <= 128 && n >= 512) return run_rows<2, AlongB, Pairs>(g, outer, epi, st);
        }
    }
#endif
    if (g.m > 64 && n > 64 && g.k > 256 && div_up(g.m, 128) * div_up(n, 128) * outer >= kFill / 2)
        return run_staged<AlongA, AlongB, 128, 128, 2, Pairs>(g, outer, epi, st);
    return run_staged<AlongA, AlongB, 64, Pairs ? 128 : 64, 2, Pairs>(g, outer, epi, st);
}

template <int MB, bool Pairs, class Epi>
hipError_t run_few(const Gemm& g, unsigned batches, const Epi& epi, hipStream_t st) {
    const unsigned groups = (unsigned)div_up(g.n, Pairs ? 16 : 32);
    // more shares of k where few columns would leave the card empty
    if ((long)groups * batches < kFill / 2 && g.k >= 4 * (4 / MB) * 8 * V)
        k_few<MB, 8, Pairs><<<dim3(groups, batches), 64 * 8, 0, st>>>(g, epi);
    else
        k_few<MB, 4, Pairs><<<dim3(groups, batches), 64 * 4, 0, st>>>(g, epi);
    return hipGetLastError();
}

// How many ways a product's k is cut: where its tiles leave the card empty and its sums are long.  64 rows of
// 4096 -> 4096 bf16 take 17 us cut and 36 us whole.
unsigned sum_cut(long m, long n, long k, long batches) {
    // a part's terms, and the least of a sum that is cut: 256 x 1024 -> 1024 takes 11 us cut and 8 us whole in bf16, 14
    // and 25 in floats; of few tiles shorter sums too (108 x 684 -> 29 floats 14 cut and 19 whole, 64 x 512 -> 64 11 and
    // 14, 1024 x 520 -> 200 13 and 16, 128 x 760 -> 1000 15 and 21, but 1503 x 512 -> 512 17 and 14)
    constexpr long kTerms = kParts == 1 ? 512 : 256;
    const long tiles = div_up(m, 64) * div_up(n, 64) * batches, least = kParts == 1 ? 2048 : tiles <= 64 ? 512 : 768;
    if (k < least) return 1;
    // a CU holds three workgroups of the float tiles (counted as two the gradient of 600 x 1153 -> 1200 takes 42 us for 32,
    // 200 x 3000 -> 2000 45 for 35, 400 x 900 -> 2000 27 for 26, forward 25 for 25)
    return (unsigned)std::max<long>(1L, std::min<long>((kParts == 1 ? kFill : 3 * kFill / 2) / std::max<long>(1L, tiles), k / kTerms));
}
long sum_cut_bytes(long m, long n, long k, long batches) {
    const long splits = sum_cut(m, n, k, batches);
    return splits > 1 ? align256(splits * batches * m * n * 4) : 0;
}

template <bool AlongA, bool AlongB, bool Pairs, class Epi>
hipError_t run_gemm(Gemm g, unsigned batches, const Epi& epi, float* parts, hipStream_t st) {
    if (g.m == 0) return hipSuccess;
    g.splits = 1;
    g.k_split = div_up(g.k, kDepth) * kDepth;
    if constexpr (AlongB) {
        if (g.m <= 16) return run_few<1, Pairs>(g, batches, epi, st);
        if (g.m <= 32) return run_few<2, Pairs>(g, batches, epi, st);
    }
    const int n = g.n, width = Pairs ? 2 * n : n;
    const unsigned splits = sum_cut(g.m, width, g.k, batches);
    if (splits == 1) return run_tiles<AlongA, AlongB, Pairs>(g, batches, epi, st);
    g.n = width;
    g.k_split = div_up(div_up(g.k, splits), kDepth) * kDepth;
    g.splits = (unsigned)div_up(g.k, g.k_split);
    if (const hipError_t e = run_tiles<AlongA, AlongB, false>(g, batches * g.splits, EpiPart{parts, g.m * width, width}, st)) return e;
    const long threads = batches * g.m * div_up(n, V);
    k_finish<Pairs><<<dim3((unsigned)std::min<long>(div_up(threads, 256), 4 * kFill)), 256, 0, st>>>(parts, g.splits, (int)g.m, n, batches, epi);
    return hipGetLastError();
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
    // tiles of 128 where they and the rows are enough for the card, else smaller ones in more parts
    const long most = std::max<long>(1L, a.n_rows / (4 * kDepth)), tiles128 = div_up(out, 128) * div_up(a.inner, 128) * comps;
    const bool wide = tiles128 >= 32 && tiles128 * std::min<long>(most, 16L) >= kFill / 2;
    const long tiles = wide ? tiles128 : div_up(out, 64) * div_up(a.inner, 64) * comps;
    long splits = std::max<long>(1L, std::min<long>(kFill / tiles, most));
    splits = std::max<long>(splits, div_up(a.n_rows, 1L << 30));       // a split's k is counted in 32 bits
    c.k_split = std::max<long>(1L, div_up(div_up(a.n_rows, splits), kDepth)) * kDepth;
    c.splits = (unsigned)std::max<long>(1L, div_up(a.n_rows, c.k_split));
    c.direct = c.splits == 1 && comps == 1 && !twice;
    return c;
}

// Layers whose first gradients go through k_small_bwd: few tiles wide, or few tiles at all and no long sum.
bool small_bwd(const LinearArgs& a) {
    if (a.gated) return false;
    if (a.inner <= 128 && a.outer <= 128) return true;
    const long comps = (long)(a.lmax + 1) * (a.lmax + 1);
    const long tiles = comps * (div_up(a.n_rows, 64) * div_up(a.inner, 64) + div_up(a.outer, 64) * div_up(a.inner, 64));
    return a.outer <= 512 && tiles <= kFill && sum_cut(a.n_rows, a.inner, a.outer, comps) == 1;
}

struct BiasCut {
    long chunk;
    unsigned chunks;
    int across;
    unsigned groups;
};
// vec: values of a lane's reads
BiasCut bias_cut(long rows, int n, int vec) {
    BiasCut c;
    c.across = 1;
    while (c.across < 64 && c.across * vec < n) c.across *= 2;
    c.groups = (unsigned)div_up(n, (long)c.across * vec);
    const long high = 256 / c.across;
    // enough workgroups for the card, at most 512 chunks, which are joined afterwards; a lane reads 4 rows at once
    const long most = std::max<long>(1L, std::min<long>(512L, div_up(4 * kFill, c.groups)));
    c.chunk = std::max<long>(1L, div_up(div_up(rows, most), 4 * high)) * 4 * high;
    c.chunks = (unsigned)std::max<long>(1L, div_up(rows, c.chunk));
    return c;
}

// What of a layer is laid out anew for its products: 16-bit types in rows that are not whole 16-byte pieces, where the
// products are large enough to win it back (measured in bf16: forward 8191 x 2047 -> 4099 188 us so and 249 without,
// 5001 x 1003 -> 777 33 and 31; both gradients of the latter 85 and 125, of 20000 x 301 -> 301 58 and 57).
struct Packs {
    bool x, w, grad;        // grad: without an activation, where it is s itself
    long inner, outer;      // a component's values then (outer: of s; a gated layer's two halves together)
};
Packs packs_of(const LinearArgs& a, bool bwd) {
    const long out = (long)a.outer * (a.gated ? 2 : 1), comps = (long)(a.lmax + 1) * (a.lmax + 1);
    Packs p{false, false, false, a.inner, out};
    const double flops = 2.0 * a.n_rows * comps * a.inner * out;
    if (kParts != 1 || a.n_rows <= 32 || flops < (bwd ? 6e9 : 2e10) || (bwd && (small_bwd(a) || (a.gated && out % V != 0)))) return p;
    const bool inner = a.inner % V != 0, outer = bwd && out % V != 0, curved = a.act != kActNone || a.gated;
    p.x = inner || a.x_stride % V != 0;
    p.w = inner || outer;
    p.grad = bwd && !curved && (outer || a.grad_stride % V != 0);
    p.inner = div_up(a.inner, V) * V;
    if (bwd) p.outer = div_up(out, V) * V;
    return p;
}

struct Layout {
    long x, w, s, g_z, exact, sums, parts, bytes;
};
Layout layout_of(const LinearArgs& a, bool second) {
    const long out = (long)a.outer * (a.gated ? 2 : 1), comps = (long)(a.lmax + 1) * (a.lmax + 1);
    const Packs p = second ? Packs{false, false, false, a.inner, out} : packs_of(a, true);
    const bool act = a.act != kActNone || a.gated;
    const long s_bytes = act || p.grad ? align256(a.n_rows * comps * p.outer * (long)sizeof(T)) : 0;
    const WeightCut w = weight_cut(a, second && act);
    const BiasCut b = second ? bias_cut(a.n_rows, (int)out, kVec<float>) : bias_cut(a.n_rows, a.outer, V);
    Layout y;
    y.x = 0;
    y.w = p.x ? align256(a.n_rows * comps * p.inner * (long)sizeof(T)) : 0;
    y.s = y.w + (p.w ? align256((a.lmax + 1) * p.outer * p.inner * (long)sizeof(T)) : 0);
    y.g_z = y.s + s_bytes;
    y.exact = y.g_z + (second ? s_bytes : 0);
    y.sums = y.exact + (second && act && kParts == 1 ? align256(a.n_rows * out * 4) : 0);
    y.parts = y.sums + align256(std::max<long>(b.chunks, w.splits) * out * 4);
    // one product's parts at a time
    const bool small = small_bwd(a) && !second;
    long parts = w.direct && !small ? 0 : align256(w.splits * comps * out * a.inner * 4 * (second && act ? 2 : 1));
    parts = std::max<long>(parts, sum_cut_bytes(a.n_rows, a.inner, p.outer, comps));
    if (second) parts = std::max<long>(parts, sum_cut_bytes(a.n_rows, out, a.inner, comps));
    y.bytes = y.parts + parts;
    return y;
}

Pack rows_pack(const T* from, long row, long n_rows, int comps, int width, long padded, T* to) {
    return Pack{from, to, n_rows, row, width, comps, comps, width, (int)padded};
}
// [degrees][outer][inner] to [degrees][padded outer][padded inner]
Pack weight_pack(const LinearArgs& a, long outer, long inner, T* to) {
    const int out = a.outer * (a.gated ? 2 : 1);
    return Pack{static_cast<const T*>(a.w), to, a.lmax + 1, (long)out * a.inner, a.inner, (int)outer, out, a.inner, (int)inner};
}
hipError_t pack(const Pack& a, const Pack& b, hipStream_t st) {
    const auto groups = [](const Pack& p) { return p.to ? (unsigned)std::min<long>(div_up(p.n_i * p.n_j * (p.padded / V), 256), 8 * kFill) : 0; };
    if (groups(a) + groups(b) == 0) return hipSuccess;
    k_pack<<<groups(a) + groups(b), 256, 0, st>>>(a, b, groups(a));
    return hipGetLastError();
}

// A layer's operands as a product reads them: rows of components one after the other, matrices of the degrees.
struct Operand {
    const T* p;
    long row, part;     // elements from row to row, from component to component (w: from degree to degree)
    long width;         // values of a component that may be read, zeros past those that are there
};
Operand input_of(const LinearArgs& a, const void* x, long row) { return Operand{static_cast<const T*>(x), row, a.inner, a.inner}; }
Operand weight_of(const LinearArgs& a) {
    return Operand{static_cast<const T*>(a.w), a.inner, (long)a.outer * (a.gated ? 2 : 1) * a.inner, a.inner};
}

Gemm forward_product(const LinearArgs& a, const Operand& x, const Operand& w) {
    Gemm g{};
    g.a = x.p;
    g.a_ld = x.row;
    g.a_batch = x.part;
    g.b = w.p;
    g.b_ld = w.row;
    g.b_degree = 1;
    g.b_batch = w.part;
    g.m = g.m_read = a.n_rows;
    g.n = g.n_read = a.outer;
    g.k = x.width;
    g.pair = a.outer;
    return g;
}

// out[row][inner] = s W
Gemm input_product(const LinearArgs& a, const Operand& s, const Operand& w) {
    Gemm g{};
    g.a = s.p;
    g.a_ld = s.row;
    g.a_batch = s.part;
    g.b = w.p;
    g.b_ld = w.row;
    g.b_degree = 1;
    g.b_batch = w.part;
    g.m = g.m_read = a.n_rows;
    g.n = a.inner;
    g.n_read = (int)w.width;
    g.k = s.width;
    return g;
}
EpiPlain input_epilogue(const LinearArgs& a, void* out) {
    const long row = (long)(a.lmax + 1) * (a.lmax + 1) * a.inner;
    return EpiPlain{static_cast<T*>(out), row, a.inner, streams_out(a.n_rows * row * (long)sizeof(T))};
}
hipError_t input_gradient(const LinearArgs& a, const Operand& s, const Operand& w, void* out, float* parts, hipStream_t st) {
    return run_gemm<true, false, false>(input_product(a, s, w), (a.lmax + 1) * (a.lmax + 1), input_epilogue(a, out), parts, st);
}

// s^T x over the rows, in the parts of a cut.
Gemm weight_product(const LinearArgs& a, const Operand& s, const Operand& x, const WeightCut& c) {
    Gemm g{};
    g.a = s.p;
    g.a_ld = s.row;
    g.a_batch = s.part;
    g.b = x.p;
    g.b_ld = x.row;
    g.b_batch = x.part;
    g.m = (long)a.outer * (a.gated ? 2 : 1);
    g.m_read = s.width;
    g.n = a.inner;
    g.n_read = (int)x.width;
    g.k = a.n_rows;
    g.splits = c.splits;
    g.k_split = c.k_split;
    return g;
}
EpiPart weight_epilogue(const LinearArgs& a, float* parts) {
    return EpiPart{parts, (long)a.outer * (a.gated ? 2 : 1) * a.inner, a.inner};
}
// The parts (direct: d_w itself).
hipError_t weight_gradient(const LinearArgs& a, const Operand& s, const Operand& x, const WeightCut& c, float* parts, T* d_w,
                           hipStream_t st) {
    const Gemm g = weight_product(a, s, x, c);
    if (c.direct) return run_tiles<false, false, false>(g, 1, EpiPlain{d_w, a.inner, a.inner, false}, st);
    return run_tiles<false, false, false>(g, (a.lmax + 1) * (a.lmax + 1) * c.splits, weight_epilogue(a, parts), st);
}

hipError_t act_bwd(const LinearArgs& a, const T* grad, long grad_row, T* s, long s_row, float* sums, bool gated, int n,
                   const BiasCut& c, hipStream_t st) {
    const ActBwd p{grad, static_cast<const T*>(a.z), s, sums, grad_row, a.n_rows, c.chunk, n, a.act, c.across, s_row};
    if (a.n_rows == 0 && sums == nullptr) return hipSuccess;
    const dim3 grid(c.groups, c.chunks);
    if (n % V == 0)
        gated ? k_act_bwd<true, true><<<grid, 256, 0, st>>>(p) : k_act_bwd<false, true><<<grid, 256, 0, st>>>(p);
    else
        gated ? k_act_bwd<true, false><<<grid, 256, 0, st>>>(p) : k_act_bwd<false, false><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}

Join join_of(const float* parts, void* out, long size, int degrees, unsigned per_component) {
    const int ways = per_component <= 16 ? 1 : per_component <= 64 ? 4 : 16;
    return Join{parts, static_cast<T*>(out), size, degrees, per_component, ways, (unsigned)div_up(size, 256 / ways)};
}
hipError_t join(const Join& a, const Join& b, hipStream_t st) {
    const long groups = (long)a.groups * a.degrees + (long)b.groups * b.degrees;
    if (groups == 0) return hipSuccess;
    k_join<<<dim3((unsigned)std::min<long>(groups, max_groups(256))), 256, 0, st>>>(a, b);
    return hipGetLastError();
}

struct FwdLayout {
    long x, w, parts, bytes;
};
FwdLayout fwd_layout(const LinearArgs& a) {
    const long comps = (a.lmax + 1) * (a.lmax + 1), out = (long)a.outer * (a.gated ? 2 : 1);
    const Packs p = packs_of(a, false);
    FwdLayout l{};
    if (a.n_rows <= 32) return l;       // k_few
    l.w = p.x ? align256(a.n_rows * comps * p.inner * (long)sizeof(T)) : 0;
    l.parts = l.w + (p.w ? align256((a.lmax + 1) * p.outer * p.inner * (long)sizeof(T)) : 0);
    l.bytes = l.parts + sum_cut_bytes(a.n_rows, out, p.inner, comps);
    return l;
}

hipError_t fwd(const LinearArgs& a, hipStream_t st) {
    const int comps = (a.lmax + 1) * (a.lmax + 1);
    Operand x = input_of(a, a.x, a.x_stride), w = weight_of(a);
    const Packs p = packs_of(a, false);
    const FwdLayout l = fwd_layout(a);
    char* ws = static_cast<char*>(a.workspace);
    Pack px{}, pw{};
    if (p.x) {
        px = rows_pack(x.p, x.row, a.n_rows, comps, a.inner, p.inner, reinterpret_cast<T*>(ws + l.x));
        x = Operand{px.to, comps * p.inner, p.inner, p.inner};
    }
    if (p.w) {
        pw = weight_pack(a, p.outer, p.inner, reinterpret_cast<T*>(ws + l.w));
        w = Operand{pw.to, p.inner, p.outer * p.inner, p.inner};
    }
    CTP_TRY(pack(px, pw, st));
    const Gemm g = forward_product(a, x, w);
    T *y = static_cast<T*>(a.y), *z = static_cast<T*>(a.z_out);
    const T *bias = static_cast<const T*>(a.bias), *residual = static_cast<const T*>(a.residual);
    float* parts = reinterpret_cast<float*>(ws + l.parts);
    const long row = (long)comps * a.outer;
    if (a.gated) return run_gemm<true, true, true>(g, 1, EpiGated{y, z, bias, a.outer, a.act}, parts, st);
    const bool stream = streams_out(a.n_rows * row * (long)sizeof(T) * (z ? 2 : 1));
    // without anything to do the epilogue's questions cost a layer that writes much a sixth of its time
    // (83325 x 64 -> 4352: 408 instead of 340 us)
    if (!z && !bias && !residual && a.act == kActNone)
        return run_gemm<true, true, false>(g, comps, EpiPlain{y, row, a.outer, stream}, parts, st);
    return run_gemm<true, true, false>(g, comps, EpiLinear{y, z, bias, residual, row, a.residual_stride, a.outer, a.act, stream},
                                       parts, st);
}

// k_small_bwd; the bias's sums are d_W's workgroups'.
hipError_t both_small(const LinearArgs& a, const WeightCut& c, float* sums, float* parts, hipStream_t st) {
    const unsigned comps = (a.lmax + 1) * (a.lmax + 1);
    const T* grad = static_cast<const T*>(a.grad);
    const Operand s{grad, a.grad_stride, a.outer, a.outer};
    Gemm of_w = weight_product(a, s, input_of(a, a.x, a.x_stride), c);
    Gemm of_x = input_product(a, s, weight_of(a));
    of_x.splits = 1;
    of_x.k_split = div_up(of_x.k, kDepth) * kDepth;
    if (!set_tiles(of_w, 64, 64, comps * c.splits) || !set_tiles(of_x, 64, 64, comps)) return hipErrorInvalidValue;
    if (!a.d_w && !a.d_bias) of_w.total = 0;
    if (!a.d_x) of_x.total = 0;
    const long total = (long)of_w.total + of_x.total;
    if (total == 0) return hipSuccess;
    if (of_w.total >= max_groups(256)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)std::min<long>(total, max_groups(256)));
    const Curve curve{static_cast<const T*>(a.z), a.outer, a.act, sums};
    const EpiPart to_w = weight_epilogue(a, parts);
    const EpiPlain to_x = input_epilogue(a, a.d_x);
    if (a.act != kActNone)
        k_small_bwd<true><<<grid, 256, 0, st>>>(of_w, to_w, of_x, to_x, curve);
    else
        k_small_bwd<false><<<grid, 256, 0, st>>>(of_w, to_w, of_x, to_x, curve);
    return hipGetLastError();
}

hipError_t bwd(const LinearArgs& a, hipStream_t st) {
    const Layout y = layout_of(a, false);
    char* ws = static_cast<char*>(a.workspace);
    const bool act = a.act != kActNone || a.gated;
    const long out = (long)a.outer * (a.gated ? 2 : 1);
    float *sums = a.d_bias ? reinterpret_cast<float*>(ws + y.sums) : nullptr, *parts = reinterpret_cast<float*>(ws + y.parts);
    WeightCut c = weight_cut(a, false);
    Join of_w{}, of_b{};
    if (small_bwd(a)) {
        CTP_TRY(both_small(a, c, sums, parts, st));
        if (a.d_w) of_w = join_of(parts, a.d_w, out * a.inner, a.lmax + 1, c.splits);
        if (a.d_bias) of_b = join_of(sums, a.d_bias, out, 1, c.splits);
        return join(of_w, of_b, st);
    }
    const BiasCut b = bias_cut(a.n_rows, a.outer, V);
    const int comps = (a.lmax + 1) * (a.lmax + 1);
    const Packs p = packs_of(a, true);
    const T* grad = static_cast<const T*>(a.grad);
    Operand s{grad, a.grad_stride, a.outer, a.outer}, x = input_of(a, a.x, a.x_stride), w = weight_of(a);
    T* own_s = reinterpret_cast<T*>(ws + y.s);
    Pack px{}, pw{}, ps{};
    if (p.x && a.d_w) {
        px = rows_pack(x.p, x.row, a.n_rows, comps, a.inner, p.inner, reinterpret_cast<T*>(ws + y.x));
        x = Operand{px.to, comps * p.inner, p.inner, p.inner};
    }
    if (p.w && a.d_x) {
        pw = weight_pack(a, p.outer, p.inner, reinterpret_cast<T*>(ws + y.w));
        w = Operand{pw.to, p.inner, p.outer * p.inner, p.inner};
    }
    CTP_TRY(pack(px, pw, st));
    if (act || sums) CTP_TRY(act_bwd(a, grad, a.grad_stride, act ? own_s : nullptr, p.outer, sums, a.gated, a.outer, b, st));
    if (act) s = Operand{own_s, p.outer, p.outer, p.outer};
    if (p.grad && (a.d_x || a.d_w)) {
        ps = rows_pack(grad, a.grad_stride, a.n_rows, comps, a.outer, p.outer, own_s);
        CTP_TRY(pack(ps, Pack{}, st));
        s = Operand{own_s, comps * p.outer, p.outer, p.outer};
    }
    if (a.d_x) CTP_TRY(input_gradient(a, s, w, a.d_x, parts, st));
    if (a.d_w) {
        CTP_TRY(weight_gradient(a, s, x, c, parts, static_cast<T*>(a.d_w), st));
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
    const Operand of_u = input_of(a, u, (long)comps * a.inner), of_x = input_of(a, a.x, a.x_stride), w = weight_of(a);
    const Operand of_s{s, out, out, out}, of_z{g_z, out, out, out};
    const Gemm v = forward_product(a, of_u, w);
    const WeightCut c = weight_cut(a, act);
    if (!act) {
        if (a.g_grad)
            CTP_TRY((run_gemm<true, true, false>(v, comps, EpiPlain{static_cast<T*>(a.g_grad), (long)comps * a.outer, a.outer, false}, parts, st)));
        if (a.g_w == nullptr) return hipSuccess;
        CTP_TRY(weight_gradient(a, Operand{grad, a.grad_stride, a.outer, a.outer}, of_u, c, parts, static_cast<T*>(a.g_w), st));
        return c.direct ? hipSuccess : join(join_of(parts, a.g_w, out * a.inner, a.lmax + 1, c.splits), Join{}, st);
    }
    // the bias sums what g_z is before its rounding: 16-bit types keep that beside it
    float* exact = a.g_bias ? reinterpret_cast<float*>(kParts == 1 ? ws + y.exact : ws + y.g_z) : nullptr;
    const bool need_z = a.g_x || a.g_w || (a.g_bias && kParts != 1);
    float* to_exact = kParts == 1 ? exact : nullptr;
    if (a.gated)
        CTP_TRY((run_gemm<true, true, true>(v, 1, EpiSecond<true>{grad, z, static_cast<T*>(a.g_grad), need_z ? g_z : nullptr,
                                                                  a.g_w ? s : nullptr, to_exact, a.grad_stride, a.outer, a.act}, parts, st)));
    else
        CTP_TRY((run_gemm<true, true, false>(v, 1, EpiSecond<false>{grad, z, static_cast<T*>(a.g_grad), need_z ? g_z : nullptr,
                                                                    a.g_w ? s : nullptr, to_exact, a.grad_stride, a.outer, a.act}, parts, st)));
    if (a.g_x) CTP_TRY(input_gradient(a, of_z, w, a.g_x, parts, st));
    Join of_w{}, of_b{};
    if (a.g_w) {
        CTP_TRY(weight_gradient(a, of_z, of_x, c, parts, nullptr, st));
        CTP_TRY(weight_gradient(a, of_s, of_u, c, parts + c.splits * out * a.inner, nullptr, st));
        of_w = join_of(parts, a.g_w, out * a.inner, 1, 2 * c.splits);
    }
    if (a.g_bias) {
        const BiasCut b = bias_cut(a.n_rows, (int)out, kVec<float>);
        const ColumnSums of{exact, sums, a.n_rows, b.chunk, (int)out, b.across};
        const dim3 grid(b.groups, b.chunks);
        out % kVec<float> == 0 ? k_sums<true><<<grid, 256, 0, st>>>(of) : k_sums<false><<<grid, 256, 0, st>>>(of);
        CTP_TRY(hipGetLastError());
        of_b = join_of(sums, a.g_bias, out, 1, b.chunks);
    }
    return join(of_w, of_b, st);
}

long fwd_workspace(const LinearArgs& a) { return fwd_layout(a).bytes; }
long bwd_workspace(const LinearArgs& a, bool second) { return layout_of(a, second).bytes; }

}  // namespace

template <>
const LinearOps& linear_ops<CTP_DENSE_TYPE>() {
    static constexpr LinearOps ops{fwd, bwd, bwd_bwd, fwd_workspace, bwd_workspace};
    return ops;
}

}  // namespace ctp
