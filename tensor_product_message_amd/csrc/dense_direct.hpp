// Tiles of 16-bit operands that go from memory to LDS without registers between.
#pragma once

#include "dense_common.hpp"

namespace ctp {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A buffer from `base` (the same in every lane): reads at or past `bytes` give zeros.
__device__ __forceinline__ i32x4 buffer_at(const void* base, unsigned bytes) {
    const unsigned long p = reinterpret_cast<unsigned long>(base);
    return i32x4{(int)__builtin_amdgcn_readfirstlane((unsigned)p),
                 (int)(__builtin_amdgcn_readfirstlane((unsigned)(p >> 32)) & 0xffff),
                 (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

// 16 bytes from each lane's offset to LDS, lane after lane from `lds` (the same in every lane).  The compiler does not
// know of the read (it would wait for all of them before any read of LDS): loads_arrived waits for it.  m0 is a
// register that it sets before each use of its own.
__device__ __forceinline__ void load_lds(const i32x4& buffer, unsigned offset, unsigned lds) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(buffer)
        : "memory");
}
template <int Left>
__device__ __forceinline__ void loads_arrived() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Left) : "memory");
}
// Behind it every wave's arrived reads and finished accesses of LDS are the others' too.
__device__ __forceinline__ void tile_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ unsigned lds_address(const void* p) {
    return (unsigned)reinterpret_cast<unsigned long>((const __attribute__((address_space(3))) void*)p);
}

// Bytes of the buffers that tiles are read from; places in them are held in 32 bits.
constexpr long kBufferBytes = 0x7ffffff0;

// Across: the buffer of `rows` rows of k, ld values apart, ends with the last one's `width` values.
__host__ __device__ __forceinline__ unsigned buffer_bytes(long rows, long ld, long width) {
    const long bytes = 2 * ((rows - 1) * ld + width);
    return (unsigned)(bytes < kBufferBytes ? bytes : kBufferBytes);
}

// Whether an operand's tiles may go this way: 16-byte pieces, whole in every row of n values, and rows so near each
// other that all places of a tile of 256 of them, and of their partners `pair` rows on, lie in a buffer.
inline bool comes_directly(const void* p, long ld, long batch, long n, long pair) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && batch % 8 == 0 && n % 8 == 0 && ld <= 1L << 21 &&
           (pair + 256) * ld * 2 <= kBufferBytes;
}

// The way of a Tile<E, NParts, Along, Rows, Depth>: each wave brings kLoads 1-KB pieces of each plane.  A lane's place in
// LDS is given, so the order of the chunks in a row (see Tile) is made by where in memory the lane reads.
template <bool Along, int Rows, int Depth, int Waves>
struct Direct {
    static constexpr int kLoads = Rows * Depth / 8 / 64 / Waves;
    static_assert(kLoads * Waves * 64 * 8 == Rows * Depth);
    typedef Tile<_Float16, 1, Along, Rows, Depth> tile_t;       // (the places are the same for any 16-bit type)
    static constexpr unsigned kNowhere = 0xfffffff0u;       // past the end of any buffer
    static constexpr int kInRow = (Along ? Depth : Rows) / 8;
    unsigned at[kLoads];        // byte offsets from the tile's first value
    int k[kLoads];              // Along: the chunk's first k

    // Along: the first k of a chunk.
    static __host__ __device__ __forceinline__ int first_k(int chunk) { return 8 * tile_t::chunk_of(chunk / kInRow, chunk % kInRow); }
    // Bytes from the tile's first value to a chunk's.  row_of(r): where row r of the tile lies among the operand's rows
    // (Along).
    template <class F>
    static __host__ __device__ __forceinline__ long place(int chunk, long ld, F&& row_of) {
        const int r = chunk / kInRow, c = chunk % kInRow;
        if constexpr (Along) return (row_of(r) * ld + first_k(chunk)) * 2;
        return (r * ld + 16 * tile_t::unit_of(r, c >> 1) + 8 * (c & 1)) * 2;
    }

    // The operand is one that comes_directly.
    template <class F>
    __device__ __forceinline__ void init(long ld, F&& row_of) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int chunk = (wave * kLoads + j) * 64 + lane;
            at[j] = (unsigned)place(chunk, ld, row_of);
            k[j] = Along ? first_k(chunk) : 0;
        }
    }
    // left: k that are there from the tile's first on (Along; Across leaves it to the buffer's end)
    __device__ __forceinline__ void issue(const i32x4& buffer, unsigned lds, int left) const {
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load_lds(buffer, !Along || k[j] < left ? at[j] : kNowhere, lds + (wave * kLoads + j) * 1024);
    }
};

// A wave's tile of (32 MT) x (32 NT) over `steps` (>= 1) tiles of k that issue(step, buffer) brings into one of two
// buffers in LDS.  The fragments of the next 16 k are read while the matrix cores work on these, and across the end of a
// tile too: its barrier stands before its last 16 k are multiplied, so that the cores have work while the first
// fragments of the next tile come.  Without that they would wait for those at each barrier, all waves at once.
// after(steps done): what is done with acc between two tiles.
template <class TA, class TB, int NParts, int MT, int NT, int Depth, class E, class Issue, class After>
__device__ __forceinline__ void multiply_tiles(f32x16 (&acc)[NT][MT], const E* lds, int steps, int wm, int wn, int lane, Issue&& issue,
                                               After&& after) {
    typedef typename Frag<E>::type frag_t;
    constexpr int kBuffer = (TA::kBytes + TB::kBytes) / 2, kParts16 = Depth / 16;       // elements; even
    frag_t fa[2][MT][NParts], fb[2][NT][NParts];
    auto read = [&](int set, const E* tile, int k) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int p = 0; p < NParts; ++p) fb[set][j][p] = TB::read(tile + TA::kBytes / 2 + p * TB::kPlane, wn + 32 * j, k, lane);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < NParts; ++p) fa[set][i][p] = TA::read(tile + p * TA::kPlane, wm + 32 * i, k, lane);
    };
    auto multiply = [&](int set) {
        // the parts' smallest products first
#pragma unroll
        for (int s = NParts - 1; s >= 0; --s)
#pragma unroll
            for (int p = 0; p <= s; ++p)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[j][i] = mfma(fb[set][j][s - p], fa[set][i][p], acc[j][i]);
    };
    issue(0, 0);
    loads_arrived<0>();
    tile_barrier();
    if (steps > 1) issue(1, 1);
    read(0, lds, 0);
    for (int step = 0; step < steps; ++step) {
        const E* tile = lds + (step & 1) * kBuffer;
#pragma unroll
        for (int q = 0; q < kParts16 - 1; ++q) {
            read((q + 1) & 1, tile, 16 * (q + 1));
            __builtin_amdgcn_sched_barrier(0);
            multiply(q & 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (step + 1 < steps) {
            // the next tile is there, and no wave reads this one any more
            loads_arrived<0>();
            tile_barrier();
            if (step + 2 < steps) issue(step + 2, step & 1);
            read(0, lds + ((step + 1) & 1) * kBuffer, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        multiply((kParts16 - 1) & 1);
        __builtin_amdgcn_sched_barrier(0);
        after(step + 1);
    }
}

}  // namespace ctp
