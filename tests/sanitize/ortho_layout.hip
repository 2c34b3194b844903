// Host program under AddressSanitizer and UndefinedBehaviorSanitizer: how the
// workspace of orthogonalised matrices is laid out and their work is divided
// (lay_out and place in csrc/ortho_kernels.hip), empty matrices among them, and
// that what the products' tiles read lies inside the planes.
// Prints the number of lists checked.
#include <cstdio>
#include <random>
#include <vector>

#include "../../tensor_product_message_amd/csrc/ortho_kernels.hip"

using namespace ctp;

namespace {

struct Shape {
    long batch;
    int rows, cols;
};

// Whether what the tiles of Side read of a product's operand (rows `count`, ld apart, from element `first` on; Along: its
// k from `k` on, else k are the rows) lies before element `end`.
template <bool Along, int Side>
bool operand_inside(long first, int ld, int rows, int at, int k, long end) {
    constexpr int depth = kDepthOf<Side>;
    typedef Direct<Along, Side, depth, 4> D;
    const long base = first + (Along ? (long)at * ld + k : (long)k * ld + at);
    const long bytes = Along ? kBufferBytes : std::min<long>(2 * ((long)(rows - k) * ld - at), kBufferBytes);
    for (int chunk = 0; chunk < D::kLoads * 4 * 64; ++chunk) {
        const long place = D::place(chunk, ld, [&](int r) { return (long)std::min(r, rows - 1 - at); });
        if (place < 0 || place > (long)D::kNowhere) return false;
        if (place >= bytes) continue;       // gives zeros
        if (place + 16 > bytes || base + place / 2 + 8 > end) return false;
    }
    return true;
}

// The last matrix's planes, in the places where tiles reach furthest.
template <int Side>
bool reads_inside(const Group& g) {
    const long x = g.x[1] + (g.batch - 1L) * 2 * g.s * g.l, a = g.a + (g.batch - 1L) * 2 * g.s * g.s;
    const long x_plane = (long)g.s * g.l, a_plane = (long)g.s * g.s;
    const int depth = kDepthOf<Side>, last_m = (g.s - 1) / Side * Side, last_n = (g.l - 1) / Side * Side;
    for (int q = 0; q < 2; ++q)
        for (int m : {0, last_m}) {
            const long x_end = x + (q + 1) * x_plane, a_end = a + (q + 1) * a_plane;
            for (int k : {0, g.l - depth})
                if (!operand_inside<true, Side>(x + q * x_plane, g.l, g.s, m, k, x_end)) return false;
            for (int k : {0, g.s - depth}) {
                if (!operand_inside<true, Side>(a + q * a_plane, g.s, g.s, m, k, a_end)) return false;
                for (int n : {0, last_n})
                    if (!operand_inside<false, Side>(x + q * x_plane, g.l, g.s, n, k, x_end)) return false;
            }
        }
    return true;
}

// Null, or what is wrong with a list's layout.
const char* check(const std::vector<Shape>& shapes) {
    std::vector<long> batch;
    std::vector<int> rows, cols;
    for (const Shape& s : shapes) batch.push_back(s.batch), rows.push_back(s.rows), cols.push_back(s.cols);
    const int n = (int)shapes.size();
    const long bytes = ortho_workspace(n, batch.data(), rows.data(), cols.data());
    for (int first = 0; first < n; first += kMostGroups) {
        Groups p{};
        const long size = lay_out(p, first, n, batch.data(), rows.data(), cols.data());
        if (size > bytes || size % 16 != 0 || p.n != std::min(kMostGroups, n - first)) return "size";
        long at = 0, sums = 0, work = 0;
        for (int k = 0; k < p.n; ++k) {
            const Group& g = p.g[k];
            const Shape& s = shapes[first + k];
            const bool empty = s.rows == 0 || s.cols == 0;
            if (g.batch != (empty ? 0 : s.batch)) return "batch";
            if (g.s < kPad || g.l < g.s || g.s % kPad || g.l % kPad) return "padding";
            if (!empty && (g.s < std::min(s.rows, s.cols) || g.l < std::max(s.rows, s.cols))) return "sides";
            // a share of A is whole tiles of k, and the shares are the long side; they are one workgroup's or one's each
            if (g.cut < kPad || g.cut % kPad || g.cut > g.l || g.chunks < 1) return "shares";
            if (g.splits != 1 && g.splits != shares_of(g)) return "splits";
            // and go by the matrix alone
            Groups one{};
            lay_out(one, 0, 1, &batch[first + k], &rows[first + k], &cols[first + k]);
            if (one.g[0].cut != g.cut || one.g[0].chunks != g.chunks) return "company";
            const long planes[4] = {g.x[0], g.x[1], g.a, g.b}, each[4] = {2L * g.s * g.l, 2L * g.s * g.l, 2L * g.s * g.s, 2L * g.s * g.s};
            for (int q = 0; q < 4; ++q) {
                if (planes[q] != at) return "planes";
                at += g.batch * each[q];
            }
            if (g.sums != sums) return "sums";
            sums += (long)g.batch * g.chunks;
            work += g.batch;
        }
        for (int k = 0; k < p.n; ++k)
            if (p.g[k].splits > 1) {
                if (2 * p.g[k].parts != at) return "parts";
                at += 2L * p.g[k].batch * p.g[k].splits * p.g[k].s * p.g[k].s;
            }
        if (p.sums_at < 2 * at || p.sums_at + 8 * sums > size) return "end";
        for (int k = 0; k < p.n; ++k)
            if (p.g[k].batch && !(reads_inside<64>(p.g[k]) && reads_inside<128>(p.g[k]))) return "reads";
        const unsigned total = place(p, [](const Group& g) { return (long)g.chunks; });
        if ((total == 0) != (work == 0) || total != sums) return "workgroups";
    }
    return nullptr;
}

}  // namespace

int main() {
    const std::vector<Shape> sides = {{1, 0, 0}, {1, 0, 5}, {1, 5, 0}, {2, 0, 0}, {0, 5, 5}, {0, 0, 0}, {1, 0, 1 << 17}, {1 << 16, 0, 7},
                                      {1, 1, 1}, {3, 64, 64}, {1, 4352, 64}, {1, 1 << 17, 1}, {7, 65, 200}, {1, 1024, 1 << 17}, {1 << 16, 3, 2}};
    std::vector<std::vector<Shape>> lists(1);
    for (const Shape& s : sides) lists.push_back({s});
    for (const Shape& s : sides)
        for (const Shape& t : sides) lists.push_back({s, t, s});
    lists.push_back(std::vector<Shape>(70, Shape{1, 0, 0}));
    std::mt19937 rng(1);
    for (int k = 0; k < 300; ++k) {
        std::vector<Shape> list(1 + rng() % 70);
        for (Shape& s : list) s = Shape{(long)(rng() % 4), (int)(rng() % 5 ? rng() % 2000 : 0), (int)(rng() % 5 ? rng() % 2000 : 0)};
        lists.push_back(list);
    }
    for (const auto& list : lists)
        if (const char* what = check(list)) {
            std::printf("wrong %s of %zu tensors:", what, list.size());
            for (const Shape& s : list) std::printf(" %ld x %d x %d", s.batch, s.rows, s.cols);
            std::printf("\n");
            return 1;
        }
    std::printf("checked %zu\n", lists.size());
    return 0;
}
