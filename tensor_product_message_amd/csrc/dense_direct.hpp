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
// know of the read (it would wait for all of them before any read of LDS): loads_arrived waits for it.
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

// The way of a Tile<E, NParts, Along, Rows, Depth>: each wave brings kLoads 1-KB pieces of each plane.  A lane's place in
// LDS is given, so the order of the chunks in a row (see Tile) is made by where in memory the lane reads.
template <bool Along, int Rows, int Depth, int Waves>
struct Direct {
    static constexpr int kLoads = Rows * Depth / 8 / 64 / Waves;
    static_assert(kLoads * Waves * 64 * 8 == Rows * Depth);
    static constexpr unsigned kNowhere = 0xfffffff0u;       // past the end of any buffer
    unsigned at[kLoads];        // byte offsets from the tile's first value
    int k[kLoads];              // Along: the chunk's first k

    // row_of(r): where row r of the tile lies among the operand's rows (Along).
    template <class F>
    __device__ __forceinline__ void init(long ld, F&& row_of) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int chunk = (wave * kLoads + j) * 64 + lane;
            if constexpr (Along) {
                const int row = chunk / (Depth / 8), c = chunk % (Depth / 8);
                k[j] = 8 * (Depth == 64 ? c ^ (row & 7) : c ^ ((row >> 1) & 3));
                at[j] = (unsigned)((row_of(row) * ld + k[j]) * 2);
            } else {
                const int kr = chunk / (Rows / 8), c = chunk % (Rows / 8);
                at[j] = (unsigned)((kr * ld + 8 * (c ^ ((kr & 3) << 1))) * 2);
                k[j] = 0;
            }
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

}  // namespace ctp
