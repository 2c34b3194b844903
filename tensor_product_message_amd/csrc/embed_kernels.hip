// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t, c] = scale * table[token[t], c]
//   d_table[v, c] = scale * sum over t with token[t] = v of grad_out[t, c]
//
// A token outside [0, rows) is padding: a zero row forward, no share of the
// gradient backward.  Both directions move rows and compute next to nothing,
// so memory bounds them.
//
// The gradient sums in a fixed order without atomics on values: tokens are
// sorted stably (a radix sort of ids and positions), the sorted list is cut
// into chunks of equal length, one group of lanes sums the rows of each chunk
// in order, and a run of equal tokens that spans several chunks is joined from
// the chunks' partial sums by a second kernel.  Cutting the sorted list and
// not the table's rows keeps the work even when a few tokens take most of it.
// A few tokens under a small table need no sort: one kernel (k_embed_few).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "train_common.hpp"
#include "train_kernels.hpp"

namespace ctp {

namespace {

constexpr int kThreads = 256;

// Token t as a row, or -1 where it is padding.
__device__ __forceinline__ int token_at(const void* tokens, int wide, long t, int rows) {
    const long v = wide ? static_cast<const int64_t*>(tokens)[t] : (long)static_cast<const int32_t*>(tokens)[t];
    return v >= 0 && v < rows ? (int)v : -1;
}

// ------------------------------------------------------------ forward

// A row is shared by 2^lg lanes, one 16-byte vector each at a time; every
// group of lanes looks up four rows at once so that four reads are in flight
// (one by one is no faster for few rows either).
// Memory bounds it: 32768 rows of 1024 bf16 in 23 us (134 MB at most, 5.8 TB/s).
// Stream: an output that the last-level cache does not hold is written around
// it, which leaves it to the table (262144 rows of 512 floats: 125 us, 162
// without).
constexpr int kLookups = 4;

template <class T, bool Stream>
__global__ void __launch_bounds__(kThreads)
k_embed_fwd(const T* __restrict__ table, const void* __restrict__ tokens, T* __restrict__ out, int n, int rows,
            int channels, int wide, float scale, long table_stride, long out_stride, int lg) {
    const int groups = kThreads >> lg, lane = threadIdx.x & ((1 << lg) - 1);
    const long t0 = (long)blockIdx.x * (groups * kLookups) + (threadIdx.x >> lg);
    const int nvec = (channels + kVec<T> - 1) / kVec<T>;
    int row[kLookups];
#pragma unroll
    for (int u = 0; u < kLookups; ++u) {
        const long t = t0 + u * groups;
        row[u] = t < n ? token_at(tokens, wide, t, rows) : -1;
    }
    for (int v = lane; v < nvec; v += 1 << lg) {
        const Span span = span_of<T>(v, channels);
        vec_t<T> x[kLookups];
#pragma unroll
        for (int u = 0; u < kLookups; ++u) {
            x[u] = vec_t<T>{};
            if (row[u] >= 0) x[u] = read_span<T>(table + row[u] * table_stride, span, channels);
        }
#pragma unroll
        for (int u = 0; u < kLookups; ++u) {
            const long t = t0 + u * groups;
            if (t >= n) break;
            settle<T>(x[u], span, true);
            Floats<T> f = widen<T>(x[u]);
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) f.v[k] *= scale;
            if (row[u] < 0) f = Floats<T>{};
            if (Stream && (v + 1) * kVec<T> <= channels)
                __builtin_nontemporal_store(narrow<T>(f), reinterpret_cast<typename Vec<T>::unaligned*>(out + t * out_stride + v * kVec<T>));
            else
                store_vec<T>(out + t * out_stride, v, channels, narrow<T>(f));
        }
    }
}

// ------------------------------------------------------------ gradient: places of a row

// The vector of a row that a lane works on: 2^lg lanes a row, a workgroup of
// `Threads` has Threads >> lg groups of them, blockIdx.y counts the tiles of
// 2^lg vectors.
template <int Threads>
struct Tile {
    int lane, group, groups, v, nvec;
    __device__ Tile(int lg, int channels, int kvec) {
        lane = threadIdx.x & ((1 << lg) - 1);
        group = threadIdx.x >> lg;
        groups = Threads >> lg;
        nvec = (channels + kvec - 1) / kvec;
        v = (blockIdx.y << lg) + lane;
    }
};

template <class T>
__device__ __forceinline__ void add_vec(Floats<T>& acc, const vec_t<T>& x) {
    const Floats<T> f = widen<T>(x);
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) acc.v[k] += f.v[k];
}

template <class T>
__device__ __forceinline__ void store_floats(float* p, const Floats<T>& f) {
#pragma unroll
    for (int k = 0; k < kVec<T>; k += 4) *reinterpret_cast<float4*>(p + k) = make_float4(f.v[k], f.v[k + 1], f.v[k + 2], f.v[k + 3]);
}

template <class T>
__device__ __forceinline__ void add_floats(const float* p, Floats<T>& f) {
#pragma unroll
    for (int k = 0; k < kVec<T>; k += 4) {
        const float4 q = *reinterpret_cast<const float4*>(p + k);
        f.v[k] += q.x;
        f.v[k + 1] += q.y;
        f.v[k + 2] += q.z;
        f.v[k + 3] += q.w;
    }
}

// Writes kVec<T> finished sums of vector v of a row of O.
template <class T, class O>
__device__ __forceinline__ void store_sum(O* row, int v, int n, const Floats<T>& f, float scale) {
#pragma unroll
    for (int p = 0; p < kVec<T> / kVec<O>; ++p) {
        Floats<O> g;
#pragma unroll
        for (int k = 0; k < kVec<O>; ++k) g.v[k] = f.v[p * kVec<O> + k] * scale;
        const int w = v * (kVec<T> / kVec<O>) + p;
        if (w * kVec<O> < n) store_vec<O>(row, w, n, narrow<O>(g));
    }
}

// Zeros in the same places, non-temporal: a large table's zero rows would push
// the gradients out of the last-level cache (a bf16 table of 131072 x 2048
// with 16384 tokens: 137 us, 148 without the mark).
template <class T, class O>
__device__ __forceinline__ void store_zeros(O* row, int v, int n) {
#pragma unroll
    for (int p = 0; p < kVec<T> / kVec<O>; ++p) {
        const int w = v * (kVec<T> / kVec<O>) + p, left = n - w * kVec<O>;
        if (left >= kVec<O>)
            __builtin_nontemporal_store(vec_t<O>{}, reinterpret_cast<typename Vec<O>::unaligned*>(row + w * kVec<O>));
        else if (left > 0)
            store_left<O>(row + w * kVec<O>, left, vec_t<O>{});
    }
}

// ------------------------------------------------------------ gradient: few tokens, small table

// One workgroup a table row and tile of channels goes through all tokens,
// keeps the places of its own in order and sums their rows.  Every workgroup
// reads all tokens, so this is for a few thousand of them and few rounds of
// workgroups (see few); it saves the sort's launches (100 rows of 128 floats:
// 6.5 us for the water box's 1503 tokens and 12.9 for 8000, 15.7 and 19.6 with
// the sort; 8000 tokens of one id 22.8 and 22.1, and 16000 of one id 44 and 23).
constexpr int kFewThreads = 1024;
constexpr int kFewTokens = 8192;
constexpr int kFewLanes = 3;        // log2 of the lanes of a row

template <class T, class O>
__global__ void __launch_bounds__(kFewThreads)
k_embed_few(const T* __restrict__ grad, const void* __restrict__ tokens, O* __restrict__ d_table, int n, int rows,
            int channels, int wide, float scale, long grad_stride, long table_stride) {
    __shared__ uint16_t place[kFewTokens];
    __shared__ int wave_count[kFewThreads / 64];
    __shared__ __align__(16) float part[kFewThreads / 64][(1 << kFewLanes) * kVec<T>];
    const int row = blockIdx.x, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    // a thread's tokens are consecutive, so that the places come out in order
    constexpr int kPer = kFewTokens / kFewThreads;
    const int per = (n + kFewThreads - 1) / kFewThreads;
    unsigned mine = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int t = threadIdx.x * per + k;
        if (k < per && t < n && token_at(tokens, wide, t, rows) == row) mine |= 1u << k;
    }
    const int count = __popc(mine);
    int incl = count;
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(incl, d, 64);
        if (lane >= d) incl += up;
    }
    if (lane == 63) wave_count[wave] = incl;
    __syncthreads();
    int at = incl - count, total = 0;
    for (int w = 0; w < kFewThreads / 64; ++w) {
        if (w < wave) at += wave_count[w];
        total += wave_count[w];
    }
    for (unsigned m = mine; m; m &= m - 1) place[at++] = (uint16_t)(threadIdx.x * per + __builtin_ctz(m));
    __syncthreads();
    const Tile<kFewThreads> tl(kFewLanes, channels, kVec<T>);
    const bool on = tl.v < tl.nvec;
    const Span span = span_of<T>(tl.v, channels);
    Floats<T> acc = {};
    constexpr int kAtOnce = 4;
    for (int i0 = tl.group; i0 < total; i0 += tl.groups * kAtOnce) {
        vec_t<T> x[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            const int i = i0 + q * tl.groups;
            x[q] = vec_t<T>{};
            if (on && i < total) x[q] = read_span<T>(grad + place[i] * grad_stride, span, channels);
        }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            settle<T>(x[q], span, on);
            add_vec<T>(acc, x[q]);
        }
    }
    // the wave's groups, then the waves
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k)
        for (int d = 1 << kFewLanes; d < 64; d <<= 1) acc.v[k] += __shfl_xor(acc.v[k], d, 64);
    if (lane < 1 << kFewLanes) store_floats<T>(&part[wave][lane * kVec<T>], acc);
    __syncthreads();
    if (tl.group != 0 || !on) return;
    for (int w = 1; w < kFewThreads / 64; ++w) add_floats<T>(&part[w][lane * kVec<T>], acc);
    // a row without tokens is zero whatever the scale
    store_sum<T, O>(d_table + row * table_stride, tl.v, channels, acc, total > 0 ? scale : 0.0f);
}

// ------------------------------------------------------------ gradient: sort

// Least-significant-digit radix sort of the tokens, padding as id `rows` at
// the end.  Each pass is two kernels: digit counts of every tile, then every
// tile finds where its digits begin from all tiles' counts and places its
// tokens stably.  Up to 10 bits a pass: 2 passes sort a million-row table, 1 a
// table of elements.  With one tile its own counts are all there are, and the
// first kernel is left out.  At most 64 tiles: every tile reads the counts of
// all of them, one digit a thread.  The two kernels of a pass over 131072 tokens
// take 3 and 9 us, a few memory latencies each and not bandwidth.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kDigitBits = 10;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kMaxTiles = 64;
constexpr int kTile = 2048;     // tokens of a tile, or a multiple
static_assert(kDigits <= kSortThreads);

struct SortSrc {
    const void* tokens;     // first pass: the tokens themselves
    const int32_t* keys;    // later passes: ids and positions as the pass before left them
    const int32_t* pos;
    int wide, n, rows;
};

__device__ __forceinline__ int sort_key(const SortSrc& s, int i) {
    if (s.keys) return s.keys[i];
    const int v = token_at(s.tokens, s.wide, i, s.rows);
    return v < 0 ? s.rows : v;
}

__global__ void __launch_bounds__(kSortThreads)
k_sort_count(SortSrc src, int tile, int shift, int bits, int32_t* __restrict__ counts) {
    __shared__ int32_t cnt[kDigits];
    const int digits = 1 << bits;
    if (threadIdx.x < digits) cnt[threadIdx.x] = 0;
    __syncthreads();
    const long end = min((long)src.n, (long)(blockIdx.x + 1) * tile);
    for (long i = (long)blockIdx.x * tile + threadIdx.x; i < end; i += kSortThreads)
        atomicAdd(&cnt[(sort_key(src, (int)i) >> shift) & (digits - 1)], 1);
    __syncthreads();
    if (threadIdx.x < digits) counts[(long)blockIdx.x * digits + threadIdx.x] = cnt[threadIdx.x];
}

// Lanes of the wave that hold the same digit (of `bits` bits) among those of `active`.
__device__ __forceinline__ uint64_t same_digit(int digit, int bits, uint64_t active) {
    uint64_t m = active;
    for (int b = 0; b < bits; ++b) {
        const bool set = (digit >> b) & 1;
        const uint64_t with = __ballot(set);
        m &= set ? with : ~with;
    }
    return m;
}

__global__ void __launch_bounds__(kSortThreads)
k_sort_place(SortSrc src, int tile, int n_tiles, int shift, int bits, const int32_t* __restrict__ counts,
             int32_t* __restrict__ keys_out, int32_t* __restrict__ pos_out) {
    __shared__ int32_t at[kSortWaves][kDigits];     // first counts, then the next free place of every wave and digit
    __shared__ int32_t wave_total[kSortWaves];
    const int digits = 1 << bits, mine = blockIdx.x;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    // the first 128 tokens of every wave's part of the tile, all of them in a short tile, stay in registers
    constexpr int kRounds = kTile / kSortThreads;
    const int part = tile / kSortWaves;
    const long begin = (long)mine * tile + (long)wave * part;
    const long end = min((long)src.n, begin + part);
    int key[kRounds], pos[kRounds];
    auto read = [&](long i0) {
#pragma unroll
        for (int q = 0; q < kRounds; ++q) {
            const long i = i0 + q * 64 + lane;
            key[q] = i < end ? sort_key(src, (int)i) : 0;
            pos[q] = i < end ? (src.pos ? src.pos[i] : (int)i) : 0;
        }
    };
    read(begin);
    int before = 0, total = 0;
    if (n_tiles > 1 && tid < digits) {
        constexpr int kAhead = 32;      // counts read at once
        for (int t0 = 0; t0 < n_tiles; t0 += kAhead) {
            int c[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) c[k] = t0 + k < n_tiles ? counts[(long)(t0 + k) * digits + tid] : 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                total += c[k];
                before += t0 + k < mine ? c[k] : 0;
            }
        }
    }
    for (int d = lane; d < digits; d += 64) at[wave][d] = 0;
    // every wave counts its own part
#pragma unroll
    for (int q = 0; q < kRounds; ++q)
        if (begin + q * 64 + lane < end) atomicAdd(&at[wave][(key[q] >> shift) & (digits - 1)], 1);
    for (long i = begin + 64 * kRounds + lane; i < end; i += 64)
        atomicAdd(&at[wave][(sort_key(src, (int)i) >> shift) & (digits - 1)], 1);
    __syncthreads();
    int of_wave[kSortWaves] = {};
    if (tid < digits) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) of_wave[w] = at[w][tid];
        if (n_tiles == 1)
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) total += of_wave[w];
    }
    // exclusive sum of the totals over all digits
    int incl = total;
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(incl, d, 64);
        if (lane >= d) incl += up;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    if (tid < digits) {
        int next = incl - total + before;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) next += w < wave ? wave_total[w] : 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            at[w][tid] = next;
            next += of_wave[w];
        }
    }
    __syncthreads();
    for (long i0 = begin; i0 < end; i0 += 64 * kRounds) {
        if (i0 != begin) read(i0);
#pragma unroll
        for (int q = 0; q < kRounds; ++q) {
            const bool on = i0 + q * 64 + lane < end;
            const int digit = (key[q] >> shift) & (digits - 1);
            const uint64_t same = same_digit(digit, bits, __ballot(on));
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int first = on ? at[wave][digit] : 0;
            // the wave's reads above come before its writes below, and those before the next round's reads
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (on && rank == 0) at[wave][digit] = first + __popcll(same);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (on) {
                keys_out[first + rank] = key[q];
                pos_out[first + rank] = pos[q];
            }
        }
    }
}

// ------------------------------------------------------------ gradient: sums of the sorted rows

struct Sorted {
    const int32_t* keys;    // ascending, padding (id `rows`) last
    const int32_t* pos;
    int n, rows;
    int chunk;              // rows of a chunk, a multiple of kBatch
};

constexpr int kBatch = 8;       // rows of a chunk read at once
constexpr int kZeroRows = 32;   // table rows of a workgroup that writes the zero rows
constexpr int kShortChunk = 16;
constexpr int kEntries = 4096;  // most sorted tokens of a workgroup
static_assert(kEntries >= kShortChunk * kThreads / 2);  // a chunk is never shorter than the workspace allows for

// Row j of partial sums, `nvec` whole vectors of fp32.
template <class T, class F, int Threads>
__device__ __forceinline__ F* partial_row(F* base, long j, const Tile<Threads>& t) {
    return base + (j * t.nvec + t.v) * kVec<T>;
}

// Workgroups below `chunk_wgs` sum chunks, one a group of lanes; the others write
// the zero rows of the table.  131072 rows of 128 floats under 100 ids take 15 us
// (61 MB without the padding, 4.1 TB/s), 16384 rows of 2048 bf16 under 131072 ids
// 106 us (604 MB, most of them zeros, 5.7 TB/s).
template <class T, class O>
__global__ void __launch_bounds__(kThreads)
k_embed_sum(Sorted s, const T* __restrict__ grad, O* __restrict__ d_table, int channels, float scale, long grad_stride,
            long table_stride, int lg, long chunk_wgs, float* __restrict__ heads, float* __restrict__ tails) {
    extern __shared__ int32_t sorted_lds[];     // a workgroup's ids with one neighbour on each side, then its places
    __shared__ __align__(16) float head_lds[kThreads * kVec<T>];    // each chunk's share of the run that it begins with
    const Tile<kThreads> tl(lg, channels, kVec<T>);
    if (blockIdx.x >= chunk_wgs) {
        // 32 table rows a time, and more than once where a launch has not a workgroup for all of them
        for (long v0 = (blockIdx.x - chunk_wgs) * kZeroRows; v0 < s.rows; v0 += (gridDim.x - chunk_wgs) * kZeroRows) {
            // which of them have a token: a binary search in the sorted ids, one row a lane
            const int row = (int)min(v0 + (threadIdx.x & (kZeroRows - 1)), (long)s.rows - 1);
            int lo = 0, hi = s.n;
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if (s.keys[mid] < row) lo = mid + 1;
                else hi = mid;
            }
            const uint64_t present = __ballot(lo < s.n && s.keys[lo] == row);
            for (int k = tl.group; k < kZeroRows && v0 + k < s.rows; k += tl.groups)
                if (tl.v < tl.nvec && !(present >> k & 1))
                    store_zeros<T, O>(d_table + (v0 + k) * table_stride, tl.v, channels);
        }
        return;
    }
    const long wg_begin = (long)blockIdx.x * tl.groups * s.chunk;
    const int entries = tl.groups * s.chunk;
    int32_t *skey = sorted_lds, *spos = sorted_lds + entries + 2;
    for (int k = threadIdx.x; k < entries + 2; k += kThreads) {
        const long i = wg_begin + k - 1;
        skey[k] = i < 0 ? -1 : i < s.n ? s.keys[i] : s.rows;
        if (k < entries && i + 1 < s.n) spos[k] = s.pos[i + 1];
    }
    __syncthreads();
    const int at = tl.group * s.chunk;      // the chunk's first entry
    const int32_t* key = skey + 1 + at;
    const int32_t* pos = spos + at;
    int cur = key[0];
    const bool on = cur != s.rows && tl.v < tl.nvec;
    bool head = key[-1] == cur;                 // the run began in an earlier chunk
    const Span span = span_of<T>(tl.v, channels);
    Floats<T> acc = {};
    auto read = [&](vec_t<T> (&x)[kBatch], int k0) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            x[q] = vec_t<T>{};
            if (on && k0 < s.chunk && key[k0 + q] != s.rows)
                x[q] = read_span<T>(grad + pos[k0 + q] * grad_stride, span, channels);
        }
    };
    float* mine = head_lds + threadIdx.x * kVec<T>;
    if (on) {
        vec_t<T> x[kBatch], y[kBatch];
        read(x, 0);
        for (int k0 = 0; k0 < s.chunk; k0 += kBatch) {
            read(y, k0 + kBatch);       // on their way while the rows before them are added
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int now = key[k0 + q];
                if (now != cur) {
                    if (cur != s.rows) {
                        if (head) store_floats<T>(mine, acc);
                        else store_sum<T, O>(d_table + cur * table_stride, tl.v, channels, acc, scale);
                    }
                    cur = now;
                    head = false;
                    acc = Floats<T>{};
                }
                settle<T>(x[q], span, true);
                add_vec<T>(acc, x[q]);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) x[q] = y[q];
        }
        if (cur != s.rows && head) store_floats<T>(mine, acc);
    }
    // what the run at the chunk's end goes on to; `tail`: it began in this chunk
    const bool leaves = key[s.chunk] == cur, tail = on && cur != s.rows && !head;
    if (tail && !leaves) store_sum<T, O>(d_table + cur * table_stride, tl.v, channels, acc, scale);
    __syncthreads();
    // Runs inside the workgroup's chunks: the chunk where one begins adds the
    // heads of the next ones.  A run that enters the workgroup's first chunk or
    // leaves its last one is left to k_embed_join.
    auto add_heads = [&](int id, int g) {       // from group g on; the first group that the run does not reach
        for (; g < tl.groups && skey[1 + g * s.chunk] == id; ++g)
            add_floats<T>(head_lds + ((g << lg) + tl.lane) * kVec<T>, acc);
        return g;
    };
    if (tail && leaves) {
        const int g = add_heads(cur, tl.group + 1);
        if (g == tl.groups && key[(g - tl.group) * s.chunk] == cur)
            store_floats<T>(partial_row<T>(tails, blockIdx.x, tl), acc);
        else
            store_sum<T, O>(d_table + cur * table_stride, tl.v, channels, acc, scale);
    }
    if (on && tl.group == 0 && key[-1] == key[0]) {
        acc = Floats<T>{};
        add_heads(key[0], 0);
        store_floats<T>(partial_row<T>(heads, blockIdx.x, tl), acc);
    }
}

// What is left are the spans of k_embed_sum's workgroups (`s.chunk` tokens here,
// one row of heads and tails each).  Where a run begins in a span and leaves
// it, its sum is the span's tail plus the heads of the spans that the run
// reaches, which are those that begin with its id.  Every group of lanes looks
// at one span and joins a run over a few of them by itself; longer runs (hot
// tokens) are then joined by the whole workgroup one after the other, since
// the longest decides how long the kernel takes (6.6 us for 131072 tokens of 100
// ids and 128 floats).
constexpr int kJoinThreads = 1024;
constexpr int kShortRun = 8;        // chunks that a short run reaches beyond its own

template <class T, class O>
__global__ void __launch_bounds__(kJoinThreads)
k_embed_join(Sorted s, O* __restrict__ d_table, int channels, float scale, long table_stride, int lg, long chunks,
             const float* __restrict__ heads, const float* __restrict__ tails) {
    __shared__ __align__(16) float part[kJoinThreads * kVec<T>];
    __shared__ int32_t long_run[kJoinThreads / 2];      // id of the long run that begins in each group's chunk, else `rows`
    const Tile<kJoinThreads> tl(lg, channels, kVec<T>);
    const int lane = threadIdx.x & 63;
    const long j = (long)blockIdx.x * tl.groups + tl.group, end = (j + 1) * s.chunk;
    // the ids around the span's end, and all first ones that a short run may reach, are read at once
    int id = s.rows;
    int32_t next[kShortRun + 1];
    if (end < s.n) {
        const int first = j > 0 ? s.keys[j * s.chunk - 1] : -1, last = s.keys[end - 1];
#pragma unroll
        for (int k = 0; k <= kShortRun; ++k) next[k] = j + 1 + k < chunks ? s.keys[(j + 1 + k) * s.chunk] : s.rows;
        // else no run leaves, or it began in an earlier span
        if (last == next[0] && first != last) id = last;
    }
    bool is_long = false;
    if (id != s.rows) {
        is_long = next[kShortRun] == id;
        if (!is_long && tl.v < tl.nvec) {
            Floats<T> acc = {};
            add_floats<T>(partial_row<T>(tails, j, tl), acc);
#pragma unroll
            for (int k = 0; k < kShortRun; ++k)
                if (next[k] == id) add_floats<T>(partial_row<T>(heads, j + 1 + k, tl), acc);
            store_sum<T, O>(d_table + id * table_stride, tl.v, channels, acc, scale);
        }
    }
    if (tl.lane == 0) long_run[tl.group] = is_long ? id : s.rows;
    __syncthreads();
    for (int g0 = 0; g0 < tl.groups; g0 += 64) {
        const int mine = g0 + lane < tl.groups ? long_run[g0 + lane] : s.rows;
        for (uint64_t found = __ballot(mine != s.rows); found; found &= found - 1) {
            const int which = __builtin_ctzll(found);
            const long first = (long)blockIdx.x * tl.groups + g0 + which;
            const int cur = __builtin_amdgcn_readlane(mine, which);
            // the last chunk that the run reaches, before `beyond`: a search by 64 probes at a time
            long last = first;
            for (long beyond = chunks; beyond - last > 1;) {
                const long step = (beyond - last + 63) / 64, k = last + (lane + 1) * step;
                last += step * __popcll(__ballot(k < beyond && s.keys[k * s.chunk] == cur));
                beyond = min(beyond, last + step);
            }
            Floats<T> acc = {};
            if (tl.v < tl.nvec) {
                if (tl.group == 0) add_floats<T>(partial_row<T>(tails, first, tl), acc);
#pragma unroll 8
                for (long k = first + 1 + tl.group; k <= last; k += tl.groups) add_floats<T>(partial_row<T>(heads, k, tl), acc);
            }
            // groups' sums by halves: `used` of them have any
            int used = (int)min((long)tl.groups, last - first);
            while (used > 1) {
                const int half = (used + 1) / 2;
                if (tl.group >= half && tl.group < used) store_floats<T>(part + threadIdx.x * kVec<T>, acc);
                __syncthreads();
                if (tl.group + half < used) add_floats<T>(part + (threadIdx.x + (half << lg)) * kVec<T>, acc);
                __syncthreads();
                used = half;
            }
            if (tl.group == 0 && tl.v < tl.nvec) store_sum<T, O>(d_table + cur * table_stride, tl.v, channels, acc, scale);
        }
    }
}

// ------------------------------------------------------------ plans

int log2_up(long x) {
    int b = 0;
    while ((1L << b) < x) ++b;
    return b;
}

// Lanes of a row: enough for all of its vectors, from 2 up to a workgroup.
int lanes_log2(int channels, int kvec) { return std::clamp(log2_up((channels + kvec - 1) / kvec), 1, 8); }

int few_tiles(int channels, int kvec) { return ((channels + kvec - 1) / kvec + (1 << kFewLanes) - 1) >> kFewLanes; }

// Whether k_embed_few takes a call: where its workgroups, of which a CU holds
// two with the registers of fp32 and one with those of 16-bit types, all get
// their turn in four rounds, or in two with more than half of its tokens.
// Uniform ids, us here and with the sort: 512 tokens of 128 floats 6 and 15 in
// one round, 14 and 16 in four, 26 and 19 in eight; 8192 tokens 13 and 20 in one,
// 21 and 20 in two, 37 and 21 in four.  Of 256 bf16 channels: 512 tokens 13 and
// 16 in four, 23 and 17 in eight; 8192 tokens 16 and 20 in two, 28 and 21 in four.
bool few(long n, long rows, int channels, int kvec) {
    const long at_once = kvec == 4 ? 512 : 256, rounds = n > kFewTokens / 2 ? 2 : 4;
    return n <= kFewTokens && rows * few_tiles(channels, kvec) <= rounds * at_once;
}

struct Plan {
    int passes, bits, tile, tiles;
    long keys, counts, partials, total;    // byte sizes: of one id array, the digit counts, one partial array; all
};

long up256(long b) { return (b + 255) / 256 * 256; }

Plan plan_of(long n, long rows, int channels) {
    Plan p{};
    const int bits = std::max(1, log2_up(rows + 1));
    p.passes = (bits + kDigitBits - 1) / kDigitBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.tile = kTile * (int)std::max(1L, (n + (long)kTile * kMaxTiles - 1) / ((long)kTile * kMaxTiles));
    p.tiles = (int)((n + p.tile - 1) / p.tile);
    p.keys = up256(4 * n);
    p.counts = up256(4L * p.tiles << p.bits);
    // a row a span; spans are shortest where rows take the most lanes, in float32
    const long span = (long)kShortChunk * (kThreads >> lanes_log2(channels, kVec<float>));
    p.partials = up256((n + span - 1) / span * ((channels + 7L) / 8 * 8) * 4);
    p.total = 4 * p.keys + p.counts + 2 * p.partials;
    return p;
}

template <class T, class O>
hipError_t sum_and_join(const EmbedArgs& a, const int32_t* keys, const int32_t* pos, float* heads, float* tails,
                        hipStream_t st) {
    const int lg = lanes_log2(a.channels, kVec<T>), groups = kThreads >> lg;
    const int nvec = (a.channels + kVec<T> - 1) / kVec<T>;
    // Chunks of 16 rows keep the GPU busy where there are few vectors; longer ones, as these grow in number, leave
    // fewer partial sums.  With chunks of 16, 32 and 64 (100 ids, us): 1 M vectors, 131072 rows of 32 floats, 30, 33
    // and 40; 2 M, 65536 of 128, 27.9, 27.9 and 34.5; 4 M, 131072 of 128, 34.7, 33.6 and 37.5; 8 M, 262144 of 128,
    // 50, 51 and 50, and 16384 of 2048, 50, 43 and 40; 34 M, 65536 of 2048, 173, 141 and 131.
    const long vectors = a.n_tokens * nvec;
    int chunk = vectors < 1L << 21 ? kShortChunk : vectors < 1L << 23 ? 2 * kShortChunk : 4 * kShortChunk;
    chunk = std::min(chunk, kEntries / groups);
    const Sorted s{keys, pos, (int)a.n_tokens, (int)a.n_rows, chunk};
    const unsigned tiles = (unsigned)((nvec + (1 << lg) - 1) >> lg);
    const long chunks = (a.n_tokens + chunk - 1) / chunk;
    const long chunk_wgs = (chunks + groups - 1) / groups;     // spans too
    const long zero_wgs = std::min((a.n_rows + kZeroRows - 1) / kZeroRows, max_groups(kThreads) - chunk_wgs);
    if (chunk_wgs + zero_wgs > 0)
        k_embed_sum<T, O><<<dim3((unsigned)(chunk_wgs + zero_wgs), tiles), kThreads, (2 * groups * chunk + 2) * sizeof(int32_t), st>>>(
            s, static_cast<const T*>(a.src), static_cast<O*>(a.dst), a.channels, a.scale, a.src_stride, a.dst_stride,
            lg, chunk_wgs, heads, tails);
    if (chunk_wgs > 1) {
        Sorted spans = s;
        spans.chunk = chunk * groups;
        const long at_once = kJoinThreads >> lg;
        k_embed_join<T, O><<<dim3((unsigned)((chunk_wgs + at_once - 1) / at_once), tiles), kJoinThreads, 0, st>>>(
            spans, static_cast<O*>(a.dst), a.channels, a.scale, a.dst_stride, lg, chunk_wgs, heads, tails);
    }
    return hipGetLastError();
}

template <class T, class O>
hipError_t embed_bwd(const EmbedArgs& a, hipStream_t st) {
    if (few(a.n_tokens, a.n_rows, a.channels, kVec<T>)) {
        k_embed_few<T, O><<<dim3((unsigned)a.n_rows, few_tiles(a.channels, kVec<T>)), kFewThreads, 0, st>>>(
            static_cast<const T*>(a.src), a.tokens, static_cast<O*>(a.dst), (int)a.n_tokens, (int)a.n_rows, a.channels,
            a.wide_index, a.scale, a.src_stride, a.dst_stride);
        return hipGetLastError();
    }
    const Plan p = plan_of(a.n_tokens, a.n_rows, a.channels);
    char* ws = static_cast<char*>(a.workspace);
    int32_t* ids[2] = {reinterpret_cast<int32_t*>(ws), reinterpret_cast<int32_t*>(ws + p.keys)};
    int32_t* pos[2] = {reinterpret_cast<int32_t*>(ws + 2 * p.keys), reinterpret_cast<int32_t*>(ws + 3 * p.keys)};
    int32_t* counts = reinterpret_cast<int32_t*>(ws + 4 * p.keys);
    float* heads = reinterpret_cast<float*>(ws + 4 * p.keys + p.counts);
    float* tails = reinterpret_cast<float*>(ws + 4 * p.keys + p.counts + p.partials);
    int to = 0;
    for (int k = 0; k < p.passes && a.n_tokens > 0; ++k, to ^= 1) {
        SortSrc src{a.tokens, k ? ids[to ^ 1] : nullptr, k ? pos[to ^ 1] : nullptr, a.wide_index, (int)a.n_tokens,
                    (int)a.n_rows};
        if (p.tiles > 1) k_sort_count<<<p.tiles, kSortThreads, 0, st>>>(src, p.tile, k * p.bits, p.bits, counts);
        k_sort_place<<<p.tiles, kSortThreads, 0, st>>>(src, p.tile, p.tiles, k * p.bits, p.bits, counts, ids[to], pos[to]);
    }
    return sum_and_join<T, O>(a, ids[to ^ 1], pos[to ^ 1], heads, tails, st);
}

}  // namespace

long embed_bwd_workspace(long n_tokens, long n_rows, int channels) {
    return plan_of(n_tokens, n_rows, channels).total;
}

hipError_t launch_embed_fwd(const EmbedArgs& a, hipStream_t st) {
    if (a.n_tokens == 0) return hipSuccess;
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        const int lg = lanes_log2(a.channels, kVec<T>), groups = kThreads >> lg;
        auto* kernel = streams_out(a.n_tokens * a.channels * (long)sizeof(T)) ? k_embed_fwd<T, true> : k_embed_fwd<T, false>;
        // 2^26 tokens of 256 lanes are more than a launch takes (a lane looks up four)
        const long at_once = groups * kLookups, most = max_groups(kThreads) * at_once;
        for (long first = 0; first < a.n_tokens; first += most) {
            const long n = std::min(most, a.n_tokens - first);
            kernel<<<(unsigned)((n + at_once - 1) / at_once), kThreads, 0, st>>>(
                static_cast<const T*>(a.src), static_cast<const char*>(a.tokens) + first * (a.wide_index ? 8 : 4),
                static_cast<T*>(a.dst) + first * a.dst_stride, (int)n, (int)a.n_rows, a.channels, a.wide_index, a.scale,
                a.src_stride, a.dst_stride, lg);
        }
        return hipGetLastError();
    });
}

hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t st) {
    if (a.n_rows == 0) return hipSuccess;
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        return a.out_dtype == a.dtype ? embed_bwd<T, T>(a, st) : embed_bwd<T, float>(a, st);
    });
}

}  // namespace ctp
