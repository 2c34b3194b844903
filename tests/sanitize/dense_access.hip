// Host program under UndefinedBehaviorSanitizer, one for each element type
// (-DCTP_DENSE_TYPE): for linear layers of many sizes, strides and types of
// pass, every place that a product's tiles read (staged in each way, and
// direct) lies inside its operand, and every region of a workspace is as large
// as what is written there.  Prints the number of products and places checked.
#include <cstdio>
#include <random>
#include <vector>

#include "../../tensor_product_message_amd/csrc/dense_linear.hip"

using namespace ctp;

namespace {

long products = 0, places = 0;

// A product of a pass and the elements that its operands have from their first one on.
struct Job {
    Gemm g;
    bool along_a, along_b, pairs;
    unsigned batches;
    long size_a, size_b, size_z;    // z: read as A, rows a_ld apart (0: none)
};

bool inside(long first, long count, long size) {
    ++places;
    return first >= 0 && first + count <= size;
}

template <bool Along, int Rows, class F>
bool staged_operand(How how, long base, long ld, int n_left, int k0, int k_end, long size, F&& row_of) {
    typedef Staged<T, Along, Rows, kDepth, 256> S;
    for (int id = 0; id < Rows * kDepth / V; ++id) {
        const int r = id / S::kPerRow, c = id % S::kPerRow, width = Along ? k_end : n_left;
        const long row = how == kClamped ? S::template row<kClamped>(r, k0, k_end, row_of) : S::template row<kWhole>(r, k0, k_end, row_of);
        const int value = how == kClamped ? S::template value<kClamped>(c, k0, width) : S::template value<kWhole>(c, k0, width);
        if (how == kGuarded && !(value < width && (Along || row < k_end))) continue;
        long at = base + row * ld + value, count = V;
        if (how == kGuarded) {          // load_vec
            const Span s = span_of<T>(value / V, width);
            at = base + row * ld + s.at, count = width < V ? s.few : V;
        }
        if (!inside(at, count, size)) return false;
    }
    return true;
}

template <bool Along, int Rows, class F>
bool direct_operand(long base, long ld, int k, int k_end, long read, long size, F&& row_of) {
    typedef Direct<Along, Rows, kDepth, Rows / 32> D;
    base += Along ? k : k * ld;
    const long rows = std::min(k_end - k, kDepth), bytes = Along ? kBufferBytes : (long)buffer_bytes(rows, ld, std::min<long>(Rows, read));
    for (int chunk = 0; chunk < D::kLoads * (Rows / 32) * 64; ++chunk) {
        const long at = D::place(chunk, ld, row_of);
        if (at < 0 || at > (long)D::kNowhere) return false;
        if (Along && D::first_k(chunk) >= k_end - k) continue;
        if (at >= bytes) continue;      // gives zeros
        if (at + 16 > bytes || !inside(base + at / 2, 8, size)) return false;
    }
    return true;
}

std::vector<long> some(std::mt19937& rng, long n, long few) {
    std::vector<long> v;
    for (long k = 0; k < n; ++k)
        if (n <= few || k == 0 || k >= n - 2) v.push_back(k);
    for (long k = 0; n > few && k < few - 3; ++k) v.push_back(rng() % n);
    return v;
}

template <bool AlongA, bool AlongB, bool Pairs, int BM, int BN, bool Direct_>
bool tiles(const Job& j, std::mt19937& rng) {
    const Gemm& g = j.g;
    constexpr int kCols = Pairs ? BN / 2 : BN;
    for (const long batch : some(rng, j.batches, 3))
        for (const long split : some(rng, g.splits, 3))
            for (const long tm : some(rng, div_up(g.m, BM), 4))
                for (const long tn : some(rng, div_up(g.n, kCols), 4)) {
                    const long m0 = tm * BM, k0 = split * g.k_split;
                    const int n0 = (int)(tn * kCols), k_end = (int)std::min(g.k_split, g.k - k0);
                    const long a = batch * g.a_batch + (AlongA ? m0 * g.a_ld + k0 : k0 * g.a_ld + m0);
                    const long b = (g.b_degree ? degree_of((int)batch) : batch) * g.b_batch + (AlongB ? n0 * g.b_ld + k0 : k0 * g.b_ld + n0);
                    const int m_left = (int)std::min<long>(BM, g.m - m0), n_left = std::min(g.n - n0, BN);
                    const auto row_a = [&](int r) { return (long)std::min(r, m_left - 1); };
                    const auto row_b = [&](int r) { return Pairs ? pair_row(r, n_left, g.pair) : (long)std::min(r, n_left - 1); };
                    const int steps = (k_end + kDepth - 1) / kDepth, whole = k_end / kDepth;
                    const How edges = read_whole<AlongA, AlongB>(m_left == BM, n_left >= kCols)           ? kWhole
                                      : read_clamped<T, AlongA, AlongB>(m_left, n_left, k_end) ? kClamped
                                                                                              : kGuarded;
                    for (const long step : some(rng, steps, 5)) {
                        const int k = (int)step * kDepth;
                        if constexpr (Direct_) {
                            if (!direct_operand<AlongA, BM>(a, g.a_ld, k, k_end, g.m_read - m0, j.size_a, row_a)) return false;
                            if (!direct_operand<AlongB, BN>(b, g.b_ld, k, k_end, g.n_read - n0, j.size_b, row_b)) return false;
                        } else {
                            const How how = edges != kWhole ? edges : step < whole ? kWhole : kGuarded;
                            if (!staged_operand<AlongA, BM>(how, a, g.a_ld, m_left, k, k_end, j.size_a, row_a)) return false;
                            if (j.size_z && !staged_operand<AlongA, BM>(how, a, g.a_ld, m_left, k, k_end, j.size_z, row_a)) return false;
                            if (!staged_operand<AlongB, BN>(how, b, g.b_ld, n_left, k, k_end, j.size_b, row_b)) return false;
                        }
                    }
                }
    return true;
}

template <bool AlongA, bool AlongB, bool Pairs>
bool job(const Job& j, std::mt19937& rng) {
    ++products;
    if (!tiles<AlongA, AlongB, Pairs, 64, Pairs ? 128 : 64, false>(j, rng) || !tiles<AlongA, AlongB, Pairs, 128, 128, false>(j, rng)) return false;
    if constexpr (kParts == 1)
        if (direct<AlongA, AlongB, Pairs>(j.g))
            return tiles<AlongA, AlongB, Pairs, 128, 128, true>(j, rng) && tiles<AlongA, AlongB, Pairs, 256, 256, true>(j, rng);
    return true;
}

// A product as run_gemm makes it: cut into parts, or not.  room: bytes for the parts.
bool gemm_job(Job j, long room, std::mt19937& rng) {
    Gemm& g = j.g;
    if (g.m == 0) return true;
    g.splits = 1;
    g.k_split = div_up(g.k, kDepth) * kDepth;
    const int width = j.pairs ? 2 * g.n : g.n;
    const unsigned splits = sum_cut(g.m, width, g.k, j.batches);
    if (splits > 1 && !(j.along_b && g.m <= 32)) {
        j.pairs = false;
        g.n = width;
        g.k_split = div_up(div_up(g.k, splits), kDepth) * kDepth;
        g.splits = (unsigned)div_up(g.k, g.k_split);
        if ((long)j.batches * g.splits * g.m * width * 4 > room) return false;
    }
    if (j.pairs) return job<true, true, true>(j, rng);
    return j.along_b ? job<true, true, false>(j, rng) : job<true, false, false>(j, rng);
}

struct Layer {
    LinearArgs a;
    long x_size, grad_size, w_size, out;
    int comps;
};

const T* at(long place) { return reinterpret_cast<const T*>(place); }

// Null, or what is wrong.
const char* forward(const Layer& l, std::mt19937& rng) {
    const LinearArgs& a = l.a;
    const Packs p = packs_of(a, false);
    const FwdLayout y = fwd_layout(a);
    Operand x = input_of(a, a.x, a.x_stride), w = weight_of(a);
    long x_size = l.x_size, w_size = l.w_size;
    if (p.x) {
        x_size = a.n_rows * l.comps * p.inner;
        x = Operand{at(1 << 20), l.comps * p.inner, p.inner, p.inner};
        if (y.w - y.x < x_size * (long)sizeof(T)) return "forward x";
    }
    if (p.w) {
        w_size = (a.lmax + 1) * p.outer * p.inner;
        w = Operand{at(1 << 20), p.inner, p.outer * p.inner, p.inner};
        if (y.parts - y.w < w_size * (long)sizeof(T)) return "forward w";
    }
    if (x.width != w.width) return "forward widths";
    const Gemm g = forward_product(a, x, w);
    return gemm_job(Job{g, true, true, a.gated, (unsigned)l.comps, x_size, w_size, 0}, y.bytes - y.parts, rng) ? nullptr : "forward";
}

const char* backward(const Layer& l, std::mt19937& rng) {
    const LinearArgs& a = l.a;
    const Layout y = layout_of(a, false);
    const WeightCut c = weight_cut(a, false);
    const unsigned comps = l.comps;
    const long room = y.bytes - y.parts;
    if ((long)c.splits * c.k_split < a.n_rows || (a.n_rows && (c.splits - 1) * c.k_split >= a.n_rows) || c.k_split % kDepth) return "cut";
    if (small_bwd(a)) {
        const Operand s{at(1 << 20), a.grad_stride, a.outer, a.outer};
        const Gemm of_w = weight_product(a, s, input_of(a, a.x, a.x_stride), c);
        Gemm of_x = input_product(a, s, weight_of(a));
        of_x.splits = 1;
        of_x.k_split = div_up(of_x.k, kDepth) * kDepth;
        if ((long)c.splits * comps * l.out * a.inner * 4 > room || c.splits * l.out * 4 > y.parts - y.sums) return "small parts";
        if (!job<false, false, false>(Job{of_w, false, false, false, comps, l.grad_size, l.x_size, 0}, rng)) return "small d_w";
        if (a.n_rows && !job<true, false, false>(Job{of_x, true, false, false, comps, l.grad_size, l.w_size, 0}, rng)) return "small d_x";
        if (a.act == kActNone) return nullptr;
        // z, its rows dense
        Gemm z_w = of_w, z_x = of_x;
        z_w.a_ld = z_x.a_ld = a.outer;
        const long z_size = a.n_rows * a.outer;
        if (!job<false, false, false>(Job{z_w, false, false, false, 1, z_size, l.x_size, z_size}, rng)) return "small d_w's z";
        if (a.n_rows && !job<true, false, false>(Job{z_x, true, false, false, 1, z_size, l.w_size, z_size}, rng)) return "small d_x's z";
        return nullptr;
    }
    const Packs p = packs_of(a, true);
    const bool act = a.act != kActNone || a.gated;
    const BiasCut b = bias_cut(a.n_rows, a.outer, V);
    if (b.chunks * l.out * 4 > y.parts - y.sums || b.chunks * b.chunk < a.n_rows) return "sums";
    Operand s{at(1 << 20), a.grad_stride, a.outer, a.outer}, x = input_of(a, a.x, a.x_stride), w = weight_of(a);
    long s_size = l.grad_size, x_size = l.x_size, w_size = l.w_size;
    if (p.x) {
        x_size = a.n_rows * comps * p.inner;
        x = Operand{at(1 << 20), comps * p.inner, p.inner, p.inner};
        if (y.w - y.x < x_size * (long)sizeof(T)) return "x";
    }
    if (p.w) {
        w_size = (a.lmax + 1) * p.outer * p.inner;
        w = Operand{at(1 << 20), p.inner, p.outer * p.inner, p.inner};
        if (y.s - y.w < w_size * (long)sizeof(T)) return "w";
    }
    if (act || p.grad) {
        s_size = a.n_rows * (act ? 1 : comps) * p.outer;
        s = Operand{at(1 << 20), (act ? 1 : comps) * p.outer, p.outer, p.outer};
        if (y.g_z - y.s < s_size * (long)sizeof(T)) return "s";
    }
    if (s.width > (p.w ? p.outer : l.out) && s.width * w.row > w_size) return "widths";
    if (!gemm_job(Job{input_product(a, s, w), true, false, false, comps, s_size, w_size, 0}, room, rng)) return "d_x";
    if (!c.direct && (long)c.splits * comps * l.out * a.inner * 4 > room) return "parts";
    if (!job<false, false, false>(Job{weight_product(a, s, x, c), false, false, false, comps, s_size, x_size, 0}, rng)) return "d_w";
    return nullptr;
}

const char* second(const Layer& l, std::mt19937& rng) {
    const LinearArgs& a = l.a;
    const Layout y = layout_of(a, true);
    const bool act = a.act != kActNone || a.gated;
    const WeightCut c = weight_cut(a, act);
    const unsigned comps = l.comps;
    const long room = y.bytes - y.parts, u_size = a.n_rows * comps * a.inner, s_size = a.n_rows * l.out;
    const Operand u = input_of(a, at(1 << 20), (long)comps * a.inner), x = input_of(a, a.x, a.x_stride), w = weight_of(a);
    if (!gemm_job(Job{forward_product(a, u, w), true, true, a.gated, comps, u_size, l.w_size, 0}, room, rng)) return "v";
    if (!act) {
        if (!c.direct && (long)c.splits * comps * l.out * a.inner * 4 > room) return "second parts";
        const Gemm g = weight_product(a, Operand{at(1 << 20), a.grad_stride, a.outer, a.outer}, u, c);
        return job<false, false, false>(Job{g, false, false, false, comps, l.grad_size, u_size, 0}, rng) ? nullptr : "g_w";
    }
    const Operand s{at(1 << 20), l.out, l.out, l.out};
    if (y.g_z - y.s < s_size * (long)sizeof(T) || y.exact - y.g_z < s_size * (long)sizeof(T)) return "s, g_z";
    if (kParts == 1 && y.sums - y.exact < s_size * 4) return "exact";
    const BiasCut b = bias_cut(a.n_rows, (int)l.out, kVec<float>);
    if (b.chunks * l.out * 4 > y.parts - y.sums || b.chunks * b.chunk < a.n_rows) return "second sums";
    if (2L * c.splits * l.out * a.inner * 4 > room) return "second parts";
    if (!gemm_job(Job{input_product(a, s, w), true, false, false, 1, s_size, l.w_size, 0}, room, rng)) return "g_x";
    if (!job<false, false, false>(Job{weight_product(a, s, x, c), false, false, false, 1, s_size, l.x_size, 0}, rng)) return "g_w of x";
    if (!job<false, false, false>(Job{weight_product(a, s, u, c), false, false, false, 1, s_size, u_size, 0}, rng)) return "g_w of u";
    return nullptr;
}

}  // namespace

int main() {
    std::mt19937 rng(CTP_DENSE_TYPE + 1);
    const auto between = [&](double lo, double hi) { return (long)std::lround(std::exp(std::uniform_real_distribution<>(std::log(lo), std::log(hi))(rng))); };
    struct Size {
        long rows;
        int lmax, inner, outer, act, gated, gap;
    };
    // a water box's layers, wide odd ones, long sums of few tiles, one row, none
    std::vector<Size> sizes = {{83325, 0, 64, 64, 2, 0, 0}, {83325, 0, 64, 4352, 0, 0, 0}, {16384, 3, 128, 128, 0, 0, 0}, {1503, 3, 128, 128, 0, 0, 0},
                               {5001, 0, 1003, 777, 3, 0, 0}, {1, 0, 4096, 16384, 2, 1, 0}, {8192, 0, 2048, 8192, 2, 1, 0}, {329, 0, 1153, 3835, 2, 1, 0},
                               {108, 0, 684, 29, 0, 0, 0}, {0, 0, 100, 100, 2, 0, 0}, {0, 2, 1000, 700, 0, 0, 0}, {70, 0, 16384, 65536, 2, 1, 0},
                               {20, 1, 16384, 16384, 0, 0, 0}, {300, 0, 65536, 3, 1, 0, 5}, {300, 0, 3, 65536, 1, 0, 0}, {1L << 21, 0, 7, 5, 2, 0, 1}};
    for (int k = 0; k < 400; ++k) {
        Size s{between(1, 40000), (int)(rng() % 3 ? 0 : rng() % 4), (int)between(1, 4000), (int)between(1, 4000), (int)(rng() % 6), (int)(rng() % 3 == 0),
               (int)(rng() % 2 ? 0 : rng() % 20)};
        if (rng() % 2) s.inner = (s.inner + 7) / 8 * 8, s.outer = (s.outer + 7) / 8 * 8;
        if (s.lmax) s.act = s.gated = 0, s.inner = (s.inner + 3) / 4, s.outer = (s.outer + 3) / 4;
        sizes.push_back(s);
    }
    for (const Size& s : sizes) {
        Layer l{};
        l.comps = (s.lmax + 1) * (s.lmax + 1);
        l.out = (long)s.outer * (s.gated ? 2 : 1);
        LinearArgs& a = l.a;
        a.n_rows = s.rows, a.lmax = s.lmax, a.inner = s.inner, a.outer = s.outer, a.dtype = CTP_DENSE_TYPE, a.act = s.act, a.gated = s.gated;
        a.x_stride = (long)l.comps * s.inner + s.gap, a.grad_stride = (long)l.comps * s.outer + s.gap;
        a.x = a.w = a.grad = at(1 << 20);
        l.x_size = s.rows ? (s.rows - 1) * a.x_stride + (long)l.comps * s.inner : 0;
        l.grad_size = s.rows ? (s.rows - 1) * a.grad_stride + (long)l.comps * s.outer : 0;
        l.w_size = (s.lmax + 1) * l.out * s.inner;
        const char* wrong = forward(l, rng);
        if (!wrong) wrong = backward(l, rng);
        if (!wrong) wrong = second(l, rng);
        if (wrong) {
            std::printf("wrong: %s of %ld rows, lmax %d, %d -> %d, act %d, gated %d, gap %d\n", wrong, s.rows, s.lmax, s.inner, s.outer, s.act, s.gated, s.gap);
            return 1;
        }
    }
    std::printf("checked %ld products, %ld places\n", products, places);
    return 0;
}
