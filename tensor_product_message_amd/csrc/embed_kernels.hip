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
// group of lanes looks up U rows at once so that U reads are in flight.
template <class T, int U>
__global__ void __launch_bounds__(kThreads)
k_embed_fwd(const T* __restrict__ table, const void* __restrict__ tokens, T* __restrict__ out, int n, int rows,
            int channels, int wide, float scale, long table_stride, long out_stride, int lg) {
    const int groups = kThreads >> lg, lane = threadIdx.x & ((1 << lg) - 1);
    const long t0 = (long)blockIdx.x * (groups * U) + (threadIdx.x >> lg);
    const int nvec = (channels + kVec<T> - 1) / kVec<T>;
    int row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long t = t0 + u * groups;
        row[u] = t < n ? token_at(tokens, wide, t, rows) : -1;
    }
    for (int v = lane; v < nvec; v += 1 << lg) {
        const Span span = span_of<T>(v, channels);
        vec_t<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = vec_t<T>{};
            if (row[u] >= 0) x[u] = read_span<T>(table + row[u] * table_stride, span, channels);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long t = t0 + u * groups;
            if (t >= n) break;
            settle<T>(x[u], span);
            Floats<T> f = widen<T>(x[u]);
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) f.v[k] *= scale;
            if (row[u] < 0) f = Floats<T>{};
            store_vec<T>(out + t * out_stride, v, channels, narrow<T>(f));
        }
    }
}

// ------------------------------------------------------------ sort

// Least-significant-digit radix sort of the tokens, padding as id `rows` at
// the end.  Each pass is two kernels: digit counts of every tile, then every
// tile finds where its digits begin from all tiles' counts and places its
// tokens stably.  Up to 10 bits a pass: 2 passes sort a million-row table, 1 a
// table of elements.
constexpr int kDigitBits = 10;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kMaxTiles = 128;
constexpr int kTile = 1024;     // tokens of a tile, or a multiple
constexpr int kWaves = kThreads / 64;
constexpr int kRounds = kTile / kThreads;    // rounds of 64 tokens a wave has of each 1024

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

__global__ void __launch_bounds__(kThreads)
k_sort_count(SortSrc src, int tile, int shift, int bits, int32_t* __restrict__ counts) {
    __shared__ int32_t cnt[kDigits];
    const int digits = 1 << bits;
    for (int d = threadIdx.x; d < digits; d += kThreads) cnt[d] = 0;
    __syncthreads();
    const long end = min((long)src.n, (long)(blockIdx.x + 1) * tile);
    for (long i = (long)blockIdx.x * tile + threadIdx.x; i < end; i += kThreads)
        atomicAdd(&cnt[(sort_key(src, (int)i) >> shift) & (digits - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kThreads) counts[(long)blockIdx.x * digits + d] = cnt[d];
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

__global__ void __launch_bounds__(kThreads)
k_sort_place(SortSrc src, int tile, int n_tiles, int shift, int bits, const int32_t* __restrict__ counts,
             int32_t* __restrict__ keys_out, int32_t* __restrict__ pos_out) {
    __shared__ int32_t at[kWaves][kDigits];     // first counts, then the next free place of every wave and digit
    __shared__ int32_t wave_total[kWaves];
    const int digits = 1 << bits, mine = blockIdx.x;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    constexpr int kPer = kDigits / kThreads;    // digits tid * kPer .. of this thread
    int before[kPer] = {}, total[kPer] = {};
    for (int t = 0; t < n_tiles; ++t) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int d = tid * kPer + j;
            const int c = d < digits ? counts[(long)t * digits + d] : 0;
            total[j] += c;
            if (t < mine) before[j] += c;
        }
    }
    for (int d = tid; d < kWaves * kDigits; d += kThreads) (&at[0][0])[d] = 0;
    // exclusive sum of the totals over all digits
    int sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += total[j];
    int incl = sum;
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(incl, d, 64);
        if (lane >= d) incl += up;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    int base = incl - sum;
    for (int w = 0; w < wave; ++w) base += wave_total[w];
    // every wave counts its own part of the tile
    const long tile_begin = (long)mine * tile;
    const int part = tile / kWaves;
    const long begin = tile_begin + (long)wave * part;
    const long end = min((long)src.n, begin + part);
    for (long i = begin + lane; i < end; i += 64)
        atomicAdd(&at[wave][(sort_key(src, (int)i) >> shift) & (digits - 1)], 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = tid * kPer + j;
        if (d < digits) {
            int next = base + before[j];
            for (int w = 0; w < kWaves; ++w) {
                const int c = at[w][d];
                at[w][d] = next;
                next += c;
            }
        }
        base += total[j];
    }
    __syncthreads();
    for (long i0 = begin; i0 < end; i0 += 64 * kRounds) {
        int key[kRounds], pos[kRounds];
#pragma unroll
        for (int q = 0; q < kRounds; ++q) {
            const long i = i0 + q * 64 + lane;
            key[q] = i < end ? sort_key(src, (int)i) : 0;
            pos[q] = i < end ? (src.pos ? src.pos[i] : (int)i) : 0;
        }
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

// ------------------------------------------------------------ sums of the sorted rows

struct Sorted {
    const int32_t* keys;    // ascending, padding (id `rows`) last
    const int32_t* pos;
    int n, rows;
    int chunk;              // rows of a chunk, a multiple of kBatch
};

constexpr int kBatch = 8;       // rows of a chunk read at once
constexpr int kZeroRows = 64;   // table rows of a workgroup that writes the zero rows

// Places of the channel tile a lane works on.
struct Tile {
    int lane, group, groups, v, nvec;
    __device__ Tile(int lg, int channels, int kvec) {
        lane = threadIdx.x & ((1 << lg) - 1);
        group = threadIdx.x >> lg;
        groups = kThreads >> lg;
        nvec = (channels + kvec - 1) / kvec;
        v = (blockIdx.y << lg) + lane;
    }
};

// Row of a partial sum: `nvec` whole vectors of fp32.
template <class T, class F>
__device__ __forceinline__ F* partial_row(F* base, long j, const Tile& t) {
    return base + (j * t.nvec + t.v) * kVec<T>;
}

template <class T>
__device__ __forceinline__ void store_partial(float* p, const Floats<T>& f) {
#pragma unroll
    for (int k = 0; k < kVec<T>; k += 4) *reinterpret_cast<float4*>(p + k) = make_float4(f.v[k], f.v[k + 1], f.v[k + 2], f.v[k + 3]);
}

template <class T>
__device__ __forceinline__ void add_partial(const float* p, Floats<T>& f) {
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

// Workgroups below `chunk_wgs` sum chunks, one a group of lanes; the others write the zero rows of the table.
template <class T, class O>
__global__ void __launch_bounds__(kThreads)
k_embed_sum(Sorted s, const T* __restrict__ grad, O* __restrict__ d_table, int channels, float scale, long grad_stride,
            long table_stride, int lg, long chunk_wgs, float* __restrict__ heads, float* __restrict__ tails) {
    const Tile tl(lg, channels, kVec<T>);
    if (blockIdx.x >= chunk_wgs) {
        // which of 64 table rows have a token: a binary search in the sorted ids, one row a lane
        const long v0 = (blockIdx.x - chunk_wgs) * kZeroRows;
        const int row = (int)min(v0 + (threadIdx.x & 63), (long)s.rows - 1);
        int lo = 0, hi = s.n;
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (s.keys[mid] < row) lo = mid + 1;
            else hi = mid;
        }
        const uint64_t present = __ballot(lo < s.n && s.keys[lo] == row);
        if (tl.v >= tl.nvec) return;
        for (int k = tl.group; k < kZeroRows && v0 + k < s.rows; k += tl.groups)
            if (!(present >> k & 1)) store_sum<T, O>(d_table + (v0 + k) * table_stride, tl.v, channels, Floats<T>{}, 0.0f);
        return;
    }
    const long j = (long)blockIdx.x * tl.groups + tl.group;
    const long begin = j * s.chunk;
    if (begin >= s.n || tl.v >= tl.nvec) return;
    const long end = min((long)s.n, begin + s.chunk);
    int cur = s.keys[begin];
    bool head = begin > 0 && s.keys[begin - 1] == cur;      // the run began in an earlier chunk
    const int next = end < s.n ? s.keys[end] : s.rows;
    const Span span = span_of<T>(tl.v, channels);
    Floats<T> acc = {};
    for (long i0 = begin; i0 < end && cur != s.rows; i0 += kBatch) {
        int key[kBatch];
        vec_t<T> x[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) key[q] = i0 + q < end ? s.keys[i0 + q] : s.rows;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            x[q] = vec_t<T>{};
            if (key[q] != s.rows) x[q] = read_span<T>(grad + s.pos[i0 + q] * grad_stride, span, channels);
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if (i0 + q >= end) break;
            if (key[q] != cur) {
                if (head) store_partial<T>(partial_row<T>(heads, j, tl), acc);
                else store_sum<T, O>(d_table + cur * table_stride, tl.v, channels, acc, scale);
                cur = key[q];
                head = false;
                acc = Floats<T>{};
                if (cur == s.rows) break;
            }
            settle<T>(x[q], span);
            const Floats<T> f = widen<T>(x[q]);
#pragma unroll
            for (int k = 0; k < kVec<T>; ++k) acc.v[k] += f.v[k];
        }
    }
    if (cur == s.rows) return;
    if (head) store_partial<T>(partial_row<T>(heads, j, tl), acc);
    else if (next == cur) store_partial<T>(partial_row<T>(tails, j, tl), acc);
    else store_sum<T, O>(d_table + cur * table_stride, tl.v, channels, acc, scale);
}

// One workgroup a chunk: where a run begins in the chunk and leaves it, its
// sum is the chunk's tail plus the heads of the chunks that the run reaches.
template <class T, class O>
__global__ void __launch_bounds__(kThreads)
k_embed_join(Sorted s, O* __restrict__ d_table, int channels, float scale, long table_stride, int lg,
             const float* heads, const float* tails) {
    __shared__ float part[kThreads * kVec<T>];
    const Tile tl(lg, channels, kVec<T>);
    const long j = blockIdx.x, begin = j * s.chunk, end = begin + s.chunk;
    if (end >= s.n) return;
    const int cur = s.keys[end];
    if (cur == s.rows || s.keys[end - 1] != cur) return;
    if (begin > 0 && s.keys[begin - 1] == cur) return;      // it began in an earlier chunk
    int lo = (int)end, hi = s.n;                            // one past the run's last token
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (s.keys[mid] <= cur) lo = mid + 1;
        else hi = mid;
    }
    const long last = (lo - 1) / s.chunk;
    Floats<T> acc = {};
    if (tl.v < tl.nvec) {
        if (tl.group == 0) add_partial<T>(partial_row<T>(tails, j, tl), acc);
#pragma unroll 4
        for (long k = j + 1 + tl.group; k <= last; k += tl.groups)
            add_partial<T>(partial_row<T>(heads, k, tl), acc);
    }
    store_partial<T>(part + threadIdx.x * kVec<T>, acc);
    __syncthreads();
    if (tl.group != 0 || tl.v >= tl.nvec) return;
    for (int g = 1; g < tl.groups; ++g) add_partial<T>(part + ((g << lg) + tl.lane) * kVec<T>, acc);
    store_sum<T, O>(d_table + cur * table_stride, tl.v, channels, acc, scale);
}

// ------------------------------------------------------------ plans

int log2_up(long x) {
    int b = 0;
    while ((1L << b) < x) ++b;
    return b;
}

// Lanes of a row: enough for all of its vectors, up to a workgroup.
int lanes_log2(int channels, int kvec) { return std::min(8, log2_up((channels + kvec - 1) / kvec)); }

struct Plan {
    int passes, bits, tile, tiles, chunk;
    long chunks;
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
    // chunks of 16 rows keep a few thousand groups busy; longer ones, as n grows, leave fewer partial sums
    p.chunk = n <= 65536 ? 16 : n <= 262144 ? 32 : 64;
    p.chunks = (n + p.chunk - 1) / p.chunk;
    p.keys = up256(4 * n);
    p.counts = up256(4L * p.tiles << p.bits);
    p.partials = up256(p.chunks * ((channels + 7L) / 8 * 8) * 4);
    p.total = 4 * p.keys + p.counts + 2 * p.partials;
    return p;
}

template <class T, class O>
hipError_t sum_and_join(const EmbedArgs& a, const Plan& p, const int32_t* keys, const int32_t* pos, float* heads,
                        float* tails, hipStream_t st) {
    const Sorted s{keys, pos, (int)a.n_tokens, (int)a.n_rows, p.chunk};
    const int lg = lanes_log2(a.channels, kVec<T>), groups = kThreads >> lg;
    const int nvec = (a.channels + kVec<T> - 1) / kVec<T>;
    const unsigned tiles = (unsigned)((nvec + (1 << lg) - 1) >> lg);
    const long chunk_wgs = (p.chunks + groups - 1) / groups, zero_wgs = (a.n_rows + kZeroRows - 1) / kZeroRows;
    k_embed_sum<T, O><<<dim3((unsigned)(chunk_wgs + zero_wgs), tiles), kThreads, 0, st>>>(
        s, static_cast<const T*>(a.src), static_cast<O*>(a.dst), a.channels, a.scale, a.src_stride, a.dst_stride, lg,
        chunk_wgs, heads, tails);
    if (p.chunks > 1)
        k_embed_join<T, O><<<dim3((unsigned)p.chunks, tiles), kThreads, 0, st>>>(
            s, static_cast<O*>(a.dst), a.channels, a.scale, a.dst_stride, lg, heads, tails);
    return hipGetLastError();
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
        const int n = (int)a.n_tokens;
        auto go = [&](auto kernel, int unroll) {
            const unsigned grid = (unsigned)((a.n_tokens + groups * unroll - 1) / (groups * unroll));
            kernel<<<grid, kThreads, 0, st>>>(static_cast<const T*>(a.src), a.tokens, static_cast<T*>(a.dst), n,
                                              (int)a.n_rows, a.channels, a.wide_index, a.scale, a.src_stride,
                                              a.dst_stride, lg);
        };
        // one row a group until the GPU is full, then four
        if (a.n_tokens <= 1024L * groups) go(k_embed_fwd<T, 1>, 1);
        else go(k_embed_fwd<T, 4>, 4);
        return hipGetLastError();
    });
}

hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t st) {
    if (a.n_rows == 0) return hipSuccess;
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
        k_sort_count<<<p.tiles, kThreads, 0, st>>>(src, p.tile, k * p.bits, p.bits, counts);
        k_sort_place<<<p.tiles, kThreads, 0, st>>>(src, p.tile, p.tiles, k * p.bits, p.bits, counts, ids[to], pos[to]);
    }
    const int32_t* keys_sorted = ids[to ^ 1];
    const int32_t* pos_sorted = pos[to ^ 1];
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        if (a.out_dtype == a.dtype) return sum_and_join<T, T>(a, p, keys_sorted, pos_sorted, heads, tails, st);
        return sum_and_join<T, float>(a, p, keys_sorted, pos_sorted, heads, tails, st);
    });
}

}  // namespace ctp
