// Host program under UndefinedBehaviorSanitizer: the places from which tiles
// that go to LDS directly are read (csrc/dense_direct.hpp), which lanes hold in
// 32 bits.  For every operand that comes_directly lets through, all places of a
// tile lie in a buffer; rows of pairs with their partners near 2^30, 2^31 and
// 2^32 bytes on are among them.  Prints the number of tiles checked and how
// many operands were let through.
#include <cstdint>
#include <cstdio>

#include "../../tensor_product_message_amd/csrc/dense_direct.hpp"

using namespace ctp;

namespace {

const void* kPlace = reinterpret_cast<const void*>(uintptr_t(1) << 20);
long tiles = 0, direct = 0, refused = 0;

// Whether every chunk's place lies in a buffer, and is the row's and k's.
template <bool Along, int Side, int Waves, class F>
bool tile_fits(long ld, F&& row_of) {
    typedef Direct<Along, Side, 64, Waves> D;
    ++tiles;
    for (int chunk = 0; chunk < D::kLoads * Waves * 64; ++chunk) {
        const long at = D::place(chunk, ld, row_of);
        if (at < 0 || at % 16 != 0 || at + 16 > kBufferBytes) return false;
        if (Along && at != 2 * ((long)row_of(chunk / 8) * ld + D::first_k(chunk))) return false;
    }
    return true;
}

// Pairs: rows of w [2][pair][ld]; else rows ld apart.
bool check(long ld, long pair) {
    const bool pairs = comes_directly(kPlace, ld, 0, ld, pair), rows = comes_directly(kPlace, ld, 0, ld, 0);
    pairs ? ++direct : ++refused;
    if (pairs && !rows) return false;
    const int left = (int)(pair < 128 ? pair : 128);
    const auto of_pairs = [&](int r) { return pair_row(r, left, pair); };
    const auto of_rows = [](int r) { return (long)r; };
    if (pairs && !(tile_fits<true, 256, 8>(ld, of_pairs) && tile_fits<true, 128, 4>(ld, of_pairs))) return false;
    if (rows && !(tile_fits<true, 256, 8>(ld, of_rows) && tile_fits<false, 256, 8>(ld, of_rows) &&
                  tile_fits<true, 128, 4>(ld, of_rows) && tile_fits<false, 128, 4>(ld, of_rows)))
        return false;
    // what is refused has places beyond a buffer, or rows too far apart
    return pairs || ld > 1L << 21 || (pair + 256) * ld * 2 > kBufferBytes;
}

}  // namespace

int main() {
    // pair_row: 32 rows, their partners, the next 32; the last row for those past it
    if (pair_row(0, 100, 1000) != 0 || pair_row(31, 100, 1000) != 31 || pair_row(32, 100, 1000) != 1000 || pair_row(63, 100, 1000) != 1031 ||
        pair_row(64, 100, 1000) != 32 || pair_row(96, 33, 1000) != 1032 || pair_row(95, 33, 1000) != 32)
        return std::printf("wrong pairs\n"), 1;
    for (long ld = 8; ld <= 1L << 22; ld = ld < 64 ? ld + 8 : ld * 2)
        for (const long more : {0L, 8L, ld / 2 / 8 * 8}) {
            const long width = ld + more;
            for (const long bytes : {1L << 16, 1L << 30, 1L << 31, 1L << 32, 1L << 33})
                for (long by = -300; by <= 300; by += by < -2 || by >= 2 ? 149 : 1) {
                    const long pair = bytes / 2 / width + by;
                    if (pair < 1 || pair > 1L << 20) continue;
                    if (!check(width, pair)) return std::printf("wrong: rows of %ld, partners %ld rows on\n", width, pair), 1;
                }
        }
    // sizes around those where a place passes the buffer, where it wraps to 0, and ordinary ones
    const bool wide = comes_directly(kPlace, 16384, 0, 16384, 65536) || comes_directly(kPlace, 32768, 0, 32768, 65536) ||
                      comes_directly(kPlace, 32768, 0, 32768, 32768);
    const bool usual = comes_directly(kPlace, 4096, 0, 4096, 16384) && comes_directly(kPlace, 2048, 0, 2048, 8192) &&
                       comes_directly(kPlace, 16384, 0, 16384, 65000) && comes_directly(kPlace, 1L << 21, 0, 8, 0);
    if (wide || !usual) return std::printf("wrong choice: %d %d\n", wide, usual), 1;
    std::printf("checked %ld tiles, %ld direct, %ld refused\n", tiles, direct, refused);
    return direct > 100 && refused > 100 ? 0 : 1;
}
