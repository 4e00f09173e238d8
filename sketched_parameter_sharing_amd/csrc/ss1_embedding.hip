// Token embedding with scaling, and the table's gradient by sorted tokens
// (ss1_embedding_forward, ss1_embedding_backward).
//
// Backward: dE[v] is a sum over the tokens of row v, so the tokens are brought
// into the order of their rows first, and then every row is written once.
//
// Sort.  Block b of NB (a power of two) owns the rows v with v % NB == b, so
// the frequent rows, which have low numbers in most vocabularies, lie in
// different blocks.  Every block reads all M ids (from L2): it counts the ones
// that blocks before it own, which is where its own tokens begin in the sorted
// order, and its own by row; a prefix sum over its rows and a second pass over
// the ids give every token its place.  Each of the 16 waves takes a run of the
// ids and has counters of its own, and lanes of one row take their rank from a
// ballot for each bit of the row number, so the order is stable, nothing is
// atomic in global memory, and one launch sorts.  From kDealTokens on the ids
// are dealt to their blocks first (in tables of up to 262144 rows), and few tokens
// go in one launch altogether.
//
// Sum.  A wave takes T consecutive places of the sorted order and 64 lanes'
// worth of columns, so a row with many tokens is shared by many waves.  A row
// whose tokens all lie in the T is written at once; the others leave partial
// sums (at most two a wave: its first and its last row), which a last launch
// adds in order.  Rows without tokens are zeroed by further blocks of the
// sum's launch.
//
// Bound by memory where the table or the batch is large: 8192 x 1280 bf16 into
// 50000 rows of bf16 (149 MB) 35 to 41 us a call, of which sort and the first zeros
// 16, sum and the other zeros 15, join 4; 2048 tokens into 128256 x 4096 float32
// (2.1 GB) 392 us, 5.4 TB/s.  333 tokens of 1283 into 2003 rows: 8.9 us, one
// launch.  One row with all the tokens is the worst: 131072 of them, 768 wide, 238
// us for 109, since one block sorts and joins them.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "ss1_model_ops.h"

namespace ss1 {

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortRows = 512;   // rows of a sorting block at most
constexpr int kSortKeep = 16;    // steps whose ids a lane keeps between the two passes
constexpr int kMinBlocks = 256;  // sorting blocks at least (one a compute unit)
constexpr int kTile = 16;        // tokens of a summing wave, up to kMaxTiles waves a column slice
constexpr int kMaxTiles = 1024;
constexpr int kZeroVecs = 4 * kSortThreads;  // 16-byte vectors that a block of the sort's launch clears
constexpr int64_t kZeroFirst = int64_t(64) << 20;  // what the sort's launch clears beside its own work: 10 us
constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / 64;
constexpr int kZeroRows = 16;    // rows of a zeroing wave

// ------------------------------------------------------------ element access
// VEC consecutive columns of a row (16 bytes of the type that is read most), of
// which n > 0 are left; rows of an odd width start anywhere, so the vectors are
// not aligned (one instruction all the same, at full speed where the address
// is).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any2 __attribute__((aligned(2)));
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));
typedef u32x2 u32x2_any2 __attribute__((aligned(2)));

template <typename T, int VEC>
struct Raw {
    static constexpr int kWords = VEC * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p, int n) {
        if (n >= VEC) {
            if constexpr (kWords == 2) {
                const u32x2 a = *reinterpret_cast<const u32x2_any2*>(p);
                w[0] = a[0];
                w[1] = a[1];
            } else {
#pragma unroll
                for (int i = 0; i < kWords; i += 4) {
                    using V = typename std::conditional<sizeof(T) == 2, u32x4_any2, u32x4_any4>::type;
                    const u32x4 a = *reinterpret_cast<const V*>(p + i * 4 / static_cast<int>(sizeof(T)));
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[i + j] = a[j];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
            for (int i = 0; i < VEC - 1; ++i)
                if (i < n) {
                    if constexpr (sizeof(T) == 2) w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
                    else w[i] = __float_as_uint(p[i]);
                }
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        else return __uint_as_float(w[i]);
    }
};

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
template <int VEC>
__device__ __forceinline__ void store_row(float* p, const float (&v)[VEC], int n) {
    if (n >= VEC) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<u32x4_any4*>(p + i) = u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]),
                                                          __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])};
    } else {
#pragma unroll
        for (int i = 0; i < VEC - 1; ++i)
            if (i < n) p[i] = v[i];
    }
}
template <int VEC>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[VEC], int n) {
    if (n >= VEC) {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) w[i] = bf16_bits(v[2 * i]) | bf16_bits(v[2 * i + 1]) << 16;
        if constexpr (VEC == 8) *reinterpret_cast<u32x4_any2*>(p) = u32x4{w[0], w[1], w[2], w[3]};
        else *reinterpret_cast<u32x2_any2*>(p) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
        for (int i = 0; i < VEC - 1; ++i)
            if (i < n) p[i] = static_cast<uint16_t>(bf16_bits(v[i]));
    }
}

// -------------------------------------------------------------------- forward
// A wave takes one token and a run of kSlices * 64 * VEC columns, all its loads
// in flight together.  Bound by memory: 16384 rows of 4096 bf16 (190 MB with the
// rows that are read twice counted once) 41.6 us, 4.6 TB/s; 64 rows 7.9 us, the
// host's time for a call.
constexpr int kSlices = 4;

// Columns of a lane, and of a wave.
template <typename T>
constexpr int kVecOf = 16 / static_cast<int>(sizeof(T));
template <typename T>
constexpr int kSliceOf = 64 * kVecOf<T>;

template <typename I, typename TE, typename TY>
__global__ __launch_bounds__(kSumThreads) void embedding_forward_kernel(const I* __restrict__ ids, int64_t M, int64_t V,
                                                                        int K, int runs, float scale,
                                                                        const TE* __restrict__ E,
                                                                        TY* __restrict__ y) {
    constexpr int kVec = kVecOf<TE>, kSlice = kSliceOf<TE>;
    const int lane = threadIdx.x & 63;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kSumWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m = unit / runs;
    if (m >= M) return;
    const int c0 = static_cast<int>(unit % runs) * kSlices * kSlice + lane * kVec;
    const int64_t id = static_cast<int64_t>(ids[m]);
    const bool real = id >= 0 && id < V;
    Raw<TE, kVec> r[kSlices];
#pragma unroll
    for (int i = 0; i < kSlices; ++i) {
        const int c = c0 + i * kSlice;
        if (real && c < K) r[i].load(E + id * K + c, K - c);
    }
#pragma unroll
    for (int i = 0; i < kSlices; ++i) {
        const int c = c0 + i * kSlice;
        if (c >= K) break;
        float v[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = real ? r[i].at(j) * scale : 0.0f;
        store_row<kVec>(y + m * K + c, v, K - c);
    }
}

// ----------------------------------------------------------------------- sort
// How the rows lie in the sorted order: row v has place (v % NB) * rows + v / NB.
struct RowOrder {
    int32_t log2_blocks;
    int32_t rows;  // of a block
};

__device__ __forceinline__ int64_t place_of(const RowOrder& o, int64_t v) {
    return (v & ((int64_t(1) << o.log2_blocks) - 1)) * o.rows + (v >> o.log2_blocks);
}

// A token's row among the block's own, or -1 for another block's or none; and
// whether a block before this one owns it.
struct Own {
    int row;
    bool before;
};
template <typename I>
__device__ __forceinline__ bool is_row(I id, int64_t V) {
    return static_cast<uint64_t>(static_cast<int64_t>(id)) < static_cast<uint64_t>(V);
}
template <typename I>
__device__ __forceinline__ Own own_row(I id, int64_t V, const RowOrder& o, uint32_t block) {
    const bool real = is_row(id, V);
    const uint32_t v = static_cast<uint32_t>(id);  // V < 2^29
    const uint32_t owner = v & ((1u << o.log2_blocks) - 1);
    Own r;
    r.row = real && owner == block ? static_cast<int>(v >> o.log2_blocks) : -1;
    r.before = real && owner < block;
    return r;
}

// Counts the wave's keys (-1: none) in LDS; the lanes that share the first one's
// make one addition, since the additions to one address follow each other.
__device__ __forceinline__ void count_keys(int32_t* hist, int key) {
    const uint64_t some = __ballot(key >= 0);
    if (some == 0) return;
    const int lane = threadIdx.x & 63, first = __builtin_ctzll(some);
    const uint64_t same = __ballot(key == __builtin_amdgcn_readlane(key, first));
    if (lane == first) atomicAdd(&hist[key], static_cast<int>(__popcll(same)));
    else if (key >= 0 && !(same >> lane & 1)) atomicAdd(&hist[key], 1);
}

// Place of each lane's key among the wave's, next[key] being the first free one:
// the lanes of one key take consecutive places.
__device__ __forceinline__ int take_place(int32_t* next, int key, int bits) {
    const int lane = threadIdx.x & 63;
    uint64_t same = __ballot(key >= 0);
    int p = 0;
    if (same == 0) return p;
    for (int b = 0; b < bits; ++b) {
        const bool bit = (key >> b) & 1;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
    }
    if (key >= 0) {
        p = next[key] + __popcll(same & ((uint64_t(1) << lane) - 1));
        // the key's last lane of the step, after every lane's read
        if ((same >> lane) == 1) next[key] = p + 1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return p;
}

// The sum over the block's threads before this one (kSortThreads of them).
__device__ __forceinline__ int scan_before(int mine, int32_t* sums) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int scan = mine;
    for (int off = 1; off < 64; off <<= 1) {
        const int t = __shfl_up(scan, off);
        if (lane >= off) scan += t;
    }
    if (lane == 63) sums[wave] = scan;
    __syncthreads();
    int at = scan - mine;
    for (int w = 0; w < wave; ++w) at += sums[w];
    return at;
}

// ------------------------------------------------------------- many tokens
// With many tokens, every block's reading of all ids is the time (256 blocks x
// 131072 ids: 91 us of the sort), so they are first handed out to the blocks
// that own them (up to kOwners of them, which 262144 rows have; a larger table's
// blocks still read all ids: 131072 tokens, 64 wide, into 262144 rows 89 us and into
// 262145 317, 768 wide 176 and 418; 8192 tokens, 64 wide, 31 and 40): chunk c of the ids counts them by owner, and then puts them,
// in order, behind those of the chunks before it.  Every chunk adds up the
// counts for itself.
constexpr int kOwners = 512;   // owners at most
constexpr int kChunks = 128;   // chunks at most

struct Token {
    int32_t row;  // among the owner's
    int32_t m;
};

template <typename I>
__global__ __launch_bounds__(kSortThreads) void embedding_count_kernel(const I* __restrict__ ids, int M, int64_t V,
                                                                       RowOrder o, int chunk,
                                                                       int32_t* __restrict__ counts) {
    __shared__ int32_t hist[kOwners];
    const int tid = threadIdx.x, owners = 1 << o.log2_blocks;
    for (int i = tid; i < owners; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    const int begin = blockIdx.x * chunk, end = min(begin + chunk, M);
    for (int i = begin; i < end; i += kSortThreads) {
        const I id = i + tid < end ? ids[i + tid] : static_cast<I>(-1);
        count_keys(hist, is_row(id, V) ? static_cast<int>(static_cast<uint32_t>(id) & (owners - 1)) : -1);
    }
    __syncthreads();
    for (int i = tid; i < owners; i += kSortThreads) counts[blockIdx.x * owners + i] = hist[i];
}

template <typename I>
__global__ __launch_bounds__(kSortThreads) void embedding_deal_kernel(const I* __restrict__ ids, int M, int64_t V,
                                                                      RowOrder o, int chunk, int chunks,
                                                                      const int32_t* __restrict__ counts,
                                                                      int32_t* __restrict__ first,
                                                                      Token* __restrict__ tokens) {
    __shared__ int32_t hist[kSortWaves][kOwners];
    __shared__ int32_t total[2][kSortThreads];
    __shared__ int32_t sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int owners = 1 << o.log2_blocks;
    for (int i = tid; i < kSortWaves * owners; i += kSortThreads) hist[i >> o.log2_blocks][i & (owners - 1)] = 0;
    // an owner's tokens, of all chunks and of those before this one: the threads
    // of an owner take every (kSortThreads / owners)-th chunk
    int all = 0, before = 0;
    for (int c = tid >> o.log2_blocks; c < chunks; c += kSortThreads >> o.log2_blocks) {
        const int n = counts[c * owners + (tid & (owners - 1))];
        all += n;
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
    }
    total[0][tid] = all;
    total[1][tid] = before;
    __syncthreads();

    const int begin = blockIdx.x * chunk, end = min(begin + chunk, M);
    const int run = chunk / kSortWaves;  // of a wave: whole steps of 64
    const int from = begin + wave * run;
    auto owner_at = [&](int i) {
        const I id = i < end ? ids[i] : static_cast<I>(-1);
        return is_row(id, V) ? static_cast<int>(static_cast<uint32_t>(id) & (owners - 1)) : -1;
    };
    for (int i = 0; i < run; i += 64) count_keys(hist[wave], owner_at(from + i + lane));
    __syncthreads();

    all = before = 0;
    if (tid < owners)
        for (int i = tid; i < kSortThreads; i += owners) {
            all += total[0][i];
            before += total[1][i];
        }
    const int base = scan_before(all, sums);
    if (blockIdx.x == 0 && tid < owners) first[tid] = base;
    if (blockIdx.x == 0 && tid == owners - 1) first[owners] = base + all;
    if (tid < owners) {
        int at = base + before;
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = hist[w][tid];
            hist[w][tid] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int i = 0; i < run; i += 64) {
        const int m = from + i + lane;
        const int owner = owner_at(m);
        const int p = take_place(hist[wave], owner, o.log2_blocks);
        if (owner >= 0) tokens[p] = {static_cast<int32_t>(static_cast<uint32_t>(ids[m]) >> o.log2_blocks), m};
    }
}

// Writes start[place of row] (where the row's tokens begin in the sorted order)
// for the block's rows, the last block also the end of the last row, and
// order[] (the tokens by row, ascending within a row).  Blocks from `blocks` on
// clear the first zero_vecs 16-byte vectors of dE meanwhile.
//
// I is the type of the ids, or Token: then the block's own tokens are dealt
// already, from place first[block] on.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void embedding_sort_kernel(const I* __restrict__ ids, int M, int64_t V,
                                                                      RowOrder o, const int32_t* __restrict__ first,
                                                                      int32_t* __restrict__ start,
                                                                      int32_t* __restrict__ order,
                                                                      u32x4* __restrict__ dE, int64_t zero_vecs) {
    constexpr bool DEALT = __is_same(I, Token);
    __shared__ int32_t hist[kSortWaves][kSortRows];
    __shared__ int32_t sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int blocks = 1 << o.log2_blocks;
    if (static_cast<int>(blockIdx.x) >= blocks) {
        const int64_t at = static_cast<int64_t>(blockIdx.x - blocks) * kZeroVecs + tid;
#pragma unroll
        for (int i = 0; i < kZeroVecs / kSortThreads; ++i)
            if (at + i * kSortThreads < zero_vecs) dE[at + i * kSortThreads] = u32x4{0, 0, 0, 0};
        return;
    }
    for (int r = tid & 511; r < o.rows; r += 512)
        for (int w = tid >> 9; w < kSortWaves; w += kSortThreads >> 9) hist[w][r] = 0;
    const int begin = DEALT ? first[blockIdx.x] : 0, n = DEALT ? first[blockIdx.x + 1] - begin : M;
    __syncthreads();

    // the wave's run of the tokens: whole steps of 64
    const int steps = (n + kSortThreads - 1) / kSortThreads;
    const int64_t run = begin + static_cast<int64_t>(wave) * steps * 64, end = begin + static_cast<int64_t>(n);
    struct Key {
        int row, m;
        bool before;
    };
    auto fetch = [&](int s) {
        const int64_t i = run + s * 64 + lane;
        if constexpr (DEALT) return i < end ? ids[i] : Token{-1, 0};
        else return i < end ? ids[i] : static_cast<I>(-1);
    };
    auto key_of = [&](I t, int s) {
        if constexpr (DEALT) {
            return Key{t.row, t.m, false};
        } else {
            const Own w = own_row(t, V, o, blockIdx.x);
            return Key{w.row, static_cast<int>(run) + s * 64 + lane, w.before};
        }
    };
    I keep[kSortKeep];
#pragma unroll
    for (int s = 0; s < kSortKeep; ++s)
        if (s < steps) keep[s] = fetch(s);
    int before = 0;
    auto count = [&](I t, int s) {
        const Key k = key_of(t, s);
        count_keys(hist[wave], k.row);
        if constexpr (!DEALT) before += __popcll(__ballot(k.before));
    };
#pragma unroll
    for (int s = 0; s < kSortKeep; ++s)
        if (s < steps) count(keep[s], s);
    for (int s = kSortKeep; s < steps; ++s) count(fetch(s), s);
    int base = begin;
    if constexpr (!DEALT) {
        if (lane == 0) sums[wave] = before;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) base += sums[w];
    }
    __syncthreads();

    // prefix sum over the rows (thread r has row r), the waves of a row in turn
    int mine = 0, own[kSortWaves];
    if (tid < o.rows)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) mine += own[w] = hist[w][tid];
    int at = base + scan_before(mine, sums);
    if (tid < o.rows) start[static_cast<int64_t>(blockIdx.x) * o.rows + tid] = at;
    if (static_cast<int>(blockIdx.x) == blocks - 1 && tid == o.rows - 1)
        start[static_cast<int64_t>(blocks) * o.rows] = at + mine;
    if (tid < o.rows)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            hist[w][tid] = at;
            at += own[w];
        }
    __syncthreads();

    const int bits = 32 - __builtin_clz(o.rows);
    auto put = [&](I t, int s) {
        const Key k = key_of(t, s);
        const int p = take_place(hist[wave], k.row, bits);
        if (k.row >= 0) order[p] = k.m;
    };
#pragma unroll
    for (int s = 0; s < kSortKeep; ++s)
        if (s < steps) put(keep[s], s);
    for (int s = kSortKeep; s < steps; ++s) put(fetch(s), s);
}

// ------------------------------------------------------------------------ sum
// dE at p from the sum of a row's tokens (n columns left).
template <typename T, int kVec>
__device__ __forceinline__ void write_row(T* p, int n, const float (&sum)[kVec], float scale, bool accumulate) {
    float v[kVec];
    if (accumulate) {
        Raw<T, kVec> r;
        r.load(p, n);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = r.at(j) + sum[j] * scale;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = sum[j] * scale;
    }
    store_row<kVec>(p, v, n);
}

// Zeros in columns [from, to) of a row by one wave, 16 bytes a lane side by side.
template <typename T>
__device__ __forceinline__ void zero_row(T* p, int from, int to, int lane) {
    const float zero[kVecOf<T>] = {};
    for (int c = from + lane * kVecOf<T>; c < to; c += kSliceOf<T>) store_row<kVecOf<T>>(p + c, zero, to - c);
}

struct SumArgs {
    const int32_t* start;
    const int32_t* order;
    float* partial;    // [tiles][2][K]: the share of the first row, of the last row
    int64_t V;
    int64_t zeroed;      // rows that the sort's launch has cleared
    int32_t tiles;
    int32_t sum_blocks;  // blocks from here on zero rows
    int32_t T;
    int32_t K;
    int32_t slices;
    int32_t accumulate;
    RowOrder o;
    float scale;
};

__device__ __forceinline__ int tokens_of(const SumArgs& a) {
    return a.start[(int64_t(1) << a.o.log2_blocks) * a.o.rows];
}

// The rows of the places first, first + 1, ... (lane l the l-th of 64), -1
// outside [0, total).
template <typename I>
__device__ __forceinline__ int row_at(const I* ids, const int32_t* order, int place, int total) {
    return place >= 0 && place < total ? static_cast<int>(ids[order[place]]) : -1;
}

constexpr int kBatch = 8;  // rows of dy, or shares, whose loads are in flight together

template <typename I, typename TD, typename TE>
__global__ __launch_bounds__(kSumThreads) void embedding_sum_kernel(const I* __restrict__ ids, const TD* __restrict__ dy,
                                                                    TE* __restrict__ dE, SumArgs a) {
    constexpr int kVec = kVecOf<TD>, kSlice = kSliceOf<TD>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = a.K;
    if (static_cast<int>(blockIdx.x) >= a.sum_blocks) {  // rows without tokens
        const int64_t v0 = a.zeroed + (static_cast<int64_t>(blockIdx.x - a.sum_blocks) * kSumWaves + wave) * kZeroRows;
        bool empty = false;
        if (lane < kZeroRows && v0 + lane < a.V) {
            const int64_t p = place_of(a.o, v0 + lane);
            empty = a.start[p] == a.start[p + 1];
        }
        uint64_t rows = __ballot(empty);
        while (rows) {
            const int r = __builtin_ctzll(rows);
            rows &= rows - 1;
            zero_row(dE + (v0 + r) * K, 0, K, lane);
        }
        return;
    }
    const int unit = static_cast<int>(blockIdx.x) * kSumWaves + wave;
    const int tile = unit / a.slices;
    if (tile >= a.tiles) return;
    const int c = unit % a.slices * kSlice + lane * kVec;
    const int left = K - c;
    const int total = tokens_of(a);
    const int begin = min(tile * a.T, total), end = min(begin + a.T, total);
    if (begin == end) return;
    const int before = row_at(ids, a.order, begin - 1, total), behind = row_at(ids, a.order, end, total);
    float sum[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
    int row = -1;
    bool first = true;
    auto flush = [&](bool last) {
        if (left > 0) {
            if (first && row == before)
                store_row<kVec>(a.partial + static_cast<int64_t>(tile) * 2 * K + c, sum, left);
            else if (last && row == behind)
                store_row<kVec>(a.partial + (static_cast<int64_t>(tile) * 2 + 1) * K + c, sum, left);
            else
                write_row(dE + static_cast<int64_t>(row) * K + c, left, sum, a.scale, a.accumulate);
        }
        first = false;
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
    };
    for (int i0 = begin; i0 < end; i0 += 64) {
        const int mine = i0 + lane < end ? a.order[i0 + lane] : 0;
        const int rows = i0 + lane < end ? static_cast<int>(ids[mine]) : -1;
        for (int b = 0; b < 64 && i0 + b < end; b += kBatch) {
            Raw<TD, kVec> r[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int m = __builtin_amdgcn_readlane(mine, b + i);
                if (left > 0 && i0 + b + i < end) r[i].load(dy + static_cast<int64_t>(m) * K + c, left);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i0 + b + i >= end) break;
                const int v = __builtin_amdgcn_readlane(rows, b + i);
                if (v != row) {
                    if (row >= 0) flush(false);
                    row = v;
                }
                if (left > 0) {
#pragma unroll
                    for (int j = 0; j < kVec; ++j) sum[j] += r[i].at(j);
                }
            }
        }
    }
    flush(true);
}

// Rows whose tokens lie in several tiles: a block for the tile where the row
// begins.  Its waves add a run of the shares each, in order, then the first
// adds theirs.
template <typename I, typename TD, typename TE>
__global__ __launch_bounds__(kSumThreads) void embedding_join_kernel(const I* __restrict__ ids, TE* __restrict__ dE,
                                                                     SumArgs a) {
    constexpr int kVec = kVecOf<TD>, kSlice = kSliceOf<TD>;
    __shared__ float part[kSumWaves - 1][kVec][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = blockIdx.x / a.slices;
    const int K = a.K;
    const int total = tokens_of(a);
    const int begin = tile * a.T, end = begin + a.T;
    if (end >= total) return;
    const int row = row_at(ids, a.order, end, total);
    if (row != row_at(ids, a.order, end - 1, total)) return;  // no row goes on behind the tile
    const int64_t p = place_of(a.o, row);
    const int from = a.start[p], to = a.start[p + 1];
    if (from < begin) return;  // it began in an earlier tile
    // the shares: of the tile's last row, then of the first row of the next tiles
    const int n = (to - 1) / a.T - tile + 1;
    const int w0 = n * wave / kSumWaves, w1 = n * (wave + 1) / kSumWaves;
    const int c = static_cast<int>(blockIdx.x % a.slices) * kSlice + lane * kVec;
    const int left = K - c;
    float sum[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
    for (int i0 = w0; i0 < w1; i0 += kBatch) {
        Raw<float, kVec> r[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t t = i0 + i == 0 ? tile * 2LL + 1 : (tile + i0 + i) * 2LL;
            if (left > 0 && i0 + i < w1) r[i].load(a.partial + t * K + c, left);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i0 + i < w1) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) sum[j] += r[i].at(j);
            }
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) part[wave - 1][j][lane] = sum[j];
    }
    __syncthreads();
    if (wave > 0 || left <= 0) return;
#pragma unroll
    for (int w = 0; w < kSumWaves - 1; ++w)
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum[j] += part[w][j][lane];
    write_row(dE + static_cast<int64_t>(row) * K + c, left, sum, a.scale, a.accumulate);
}

// ---------------------------------------------------------------- few tokens
constexpr int kFewTokens = 512;
constexpr int kFewBatch = 16;                        // rows of dy whose loads are in flight together
constexpr int kFewShared = 64;                       // more tokens: a row that the waves share
constexpr int kFewHot = kFewTokens / kFewShared;     // such rows at most

// Up to kFewTokens tokens in one launch: a block keeps the tokens of its rows in
// LDS, one a thread and in order, ranks each by counting the ones that come
// before it (a smaller row, or the same row earlier), and then its waves sum
// and write the rows, or zeros, in columns of 64 lanes.  A row with many tokens
// is shared by all waves of its block.
template <typename I, typename TD, typename TE>
__global__ __launch_bounds__(kSortThreads) void embedding_few_kernel(const I* __restrict__ ids,
                                                                     const TD* __restrict__ dy, TE* __restrict__ dE,
                                                                     int M, int64_t V, int K, RowOrder o, float scale,
                                                                     int accumulate) {
    constexpr int kVec = kVecOf<TD>, kSlice = kSliceOf<TD>;
    __shared__ __attribute__((aligned(16))) int32_t list[kFewTokens];  // row * kFewTokens + place, as found
    __shared__ int32_t list_m[kFewTokens], sorted_m[kFewTokens], sorted_row[kFewTokens];
    __shared__ int32_t begin[kSortRows + 1];
    __shared__ int32_t sums[kSortWaves];
    __shared__ int32_t hot[kFewHot], hot_count;
    __shared__ float part[kSortWaves][kVec][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = tid < M ? own_row(ids[tid], V, o, blockIdx.x).row : -1;
    const uint64_t found = __ballot(row >= 0);
    if (lane == 0) sums[wave] = __popcll(found);
    for (int r = tid; r <= o.rows; r += kSortThreads) begin[r] = 0;
    __syncthreads();
    int at = __popcll(found & ((uint64_t(1) << lane) - 1)), n = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) at += sums[w];
        n += sums[w];
    }
    if (row >= 0) {
        list[at] = row * kFewTokens + at;
        list_m[at] = tid;
    }
    if (tid < 4 && n + tid < kFewTokens) list[n + tid] = 0x7FFFFFFF;  // the last four are read whole
    __syncthreads();
    int rank = 0;
    if (tid < n) {
        const int mine = list[tid];
        for (int i = 0; i < n; i += 4) {
            const int4 k = *reinterpret_cast<const int4*>(list + i);
            rank += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
        }
        sorted_m[rank] = list_m[tid];
        sorted_row[rank] = mine / kFewTokens;
    }
    __syncthreads();
    if (tid < n) {  // where a row ends
        const int r = sorted_row[tid];
        if (tid + 1 == n || sorted_row[tid + 1] != r) begin[r + 1] = tid + 1;
    }
    __syncthreads();
    // rows without tokens end where the row before ends; a wave scans 64 at a time
    if (wave == 0) {
        int carry = 0, many = 0;
        for (int r0 = 1; r0 <= o.rows; r0 += 64) {
            int e = r0 + lane <= o.rows ? begin[r0 + lane] : 0;
            for (int off = 1; off < 64; off <<= 1) {
                const int t = __shfl_up(e, off);
                if (lane >= off) e = max(e, t);
            }
            e = max(e, carry);
            if (r0 + lane <= o.rows) begin[r0 + lane] = e;
            const int up = __shfl_up(e, 1);
            const bool is_hot = r0 + lane <= o.rows && e - (lane ? up : carry) > kFewShared;
            const uint64_t hots = __ballot(is_hot);
            if (is_hot) hot[many + __popcll(hots & ((uint64_t(1) << lane) - 1))] = r0 + lane - 1;
            many += __popcll(hots);
            carry = __builtin_amdgcn_readlane(e, 63);
        }
        if (lane == 0) hot_count = many;
    }
    __syncthreads();
    const int slices = (K + kSlice - 1) / kSlice;
    auto add = [&](float (&sum)[kVec], int from, int to, int c) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
        if (c >= K) return;
        for (int i0 = from; i0 < to; i0 += kFewBatch) {
            Raw<TD, kVec> d[kFewBatch];
#pragma unroll
            for (int i = 0; i < kFewBatch; ++i)
                if (i0 + i < to) d[i].load(dy + static_cast<int64_t>(sorted_m[i0 + i]) * K + c, K - c);
#pragma unroll
            for (int i = 0; i < kFewBatch; ++i) {
                if (i0 + i < to) {
#pragma unroll
                    for (int j = 0; j < kVec; ++j) sum[j] += d[i].at(j);
                }
            }
        }
    };
    for (int u = wave; u < o.rows * slices; u += kSortWaves) {
        const int r = u / slices;
        const int64_t v = (static_cast<int64_t>(r) << o.log2_blocks) + blockIdx.x;
        if (v >= V) break;
        const int from = __builtin_amdgcn_readfirstlane(begin[r]), to = __builtin_amdgcn_readfirstlane(begin[r + 1]);
        if (to - from > kFewShared) continue;
        const int c0 = (u - r * slices) * kSlice, c = c0 + lane * kVec;
        if (from == to) {
            if (!accumulate) zero_row(dE + v * K, c0, min(c0 + kSlice, K), lane);
            continue;
        }
        if (c >= K) continue;
        float sum[kVec];
        add(sum, from, to, c);
        write_row(dE + v * K + c, K - c, sum, scale, accumulate);
    }
    const int shared = __builtin_amdgcn_readfirstlane(hot_count) * slices;
    for (int u = 0; u < shared; ++u) {
        const int r = __builtin_amdgcn_readfirstlane(hot[u / slices]);
        const int from = __builtin_amdgcn_readfirstlane(begin[r]);
        const int n = __builtin_amdgcn_readfirstlane(begin[r + 1]) - from;
        const int c = u % slices * kSlice + lane * kVec;
        float sum[kVec];
        add(sum, from + n * wave / kSortWaves, from + n * (wave + 1) / kSortWaves, c);
        if (u > 0) __syncthreads();  // the shares before are read
#pragma unroll
        for (int j = 0; j < kVec; ++j) part[wave][j][lane] = sum[j];
        __syncthreads();
        if (wave == u % kSortWaves && c < K) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                sum[j] = part[0][j][lane];
                for (int w = 1; w < kSortWaves; ++w) sum[j] += part[w][j][lane];
            }
            write_row(dE + ((static_cast<int64_t>(r) << o.log2_blocks) + blockIdx.x) * K + c, K - c, sum, scale, accumulate);
        }
    }
}

// -------------------------------------------------------------------- sizes
RowOrder row_order(int64_t V) {
    RowOrder o{0, 1};
    while ((int64_t(1) << o.log2_blocks) < kMinBlocks || (V + (int64_t(1) << o.log2_blocks) - 1) >> o.log2_blocks > kSortRows)
        ++o.log2_blocks;
    const int64_t nb = int64_t(1) << o.log2_blocks;
    o.rows = static_cast<int32_t>((V + nb - 1) >> o.log2_blocks);
    if (o.rows < 1) o.rows = 1;
    return o;
}

int32_t tile_tokens(int64_t M) {
    int64_t T = kTile;
    while ((M + T - 1) / T > kMaxTiles) T *= 2;
    return static_cast<int32_t>(T);
}

// Whether one launch does it all.  A frequent row's tokens all go through one
// compute unit there, so M * K is bounded: the bound weighs what tokens of text gain
// against what tokens of one row lose.  us that way and by sort, sum and join, into
// 2003 rows:
//   tokens x width     text           all apart      all one row
//   512 x  256          8.0   14.8     4.4   14.2    16.6   12.4
//   333 x 1283          9.1   16.7     7.7   15.9    39.8   14.1
//   512 x 1024          9.3   16.4     6.5   15.3    36.4   13.5   the bound
//   512 x 2048         12.2   17.9     9.3   16.8    61.4   15.3
//   128 x 8192         18.8   23.8    19.3   23.0    79.2   23.6
// Into 50000 rows, where the zeros are the time, 511 x 768 takes 29.5 and 30.6, all
// one row 52.5 and 29.9.  Tables beyond 2^27 elements took 20% longer with rows
// zeroed 256 apart.
constexpr int64_t kFewElements = int64_t(1) << 19, kFewTable = int64_t(1) << 27;
bool few_tokens(int64_t M, int64_t V, int64_t K) {
    return M <= kFewTokens && M * K <= kFewElements && V * K <= kFewTable;
}

// Chunks of the ids that are dealt out before the sort, 0 where they are not: two
// more launches.  Tokens into 50000 x 768 without and with: 8192 31.0 and 34.1 us,
// 12000 36.0 and 38.5, 16384 39.6 and 39.9, 24000 55.6 and 48.1, 131072 215 and 112;
// into 2003 x 1280: 12000 27.9 and 29.7, 16384 32.3 and 31.6, 24000 41.4 and 35.6.
constexpr int64_t kDealTokens = 16384;
int64_t chunk_tokens(int64_t M) { return up_to((M + kChunks - 1) / kChunks, kSortThreads); }
int32_t deal_chunks(int64_t M, const RowOrder& o) {
    if (M < kDealTokens || (1 << o.log2_blocks) > kOwners) return 0;
    return static_cast<int32_t>((M + chunk_tokens(M) - 1) / chunk_tokens(M));
}
size_t deal_bytes(int64_t M, const RowOrder& o) {
    const int64_t chunks = deal_chunks(M, o), owners = int64_t(1) << o.log2_blocks;
    return chunks == 0 ? 0 : static_cast<size_t>(M * 8 + up_to((owners + 1) * 4, 16) + chunks * owners * 4);
}

size_t start_bytes(const RowOrder& o) {
    return static_cast<size_t>(up_to(((int64_t(1) << o.log2_blocks) * o.rows + 1) * 4, 16));
}

template <typename I, typename TE, typename TY>
ss1_status forward_t(const EmbeddingArgs& a) {
    constexpr int kRun = kSlices * kSliceOf<TE>;
    const int runs = (a.K + kRun - 1) / kRun;
    // a grid's threads are numbered in 32 bits
    const int64_t most = ((int64_t(1) << 24) - 1) / runs * kSumWaves;
    for (int64_t at = 0; at < a.M; at += most) {
        const int64_t m = a.M - at < most ? a.M - at : most;
        hipLaunchKernelGGL((embedding_forward_kernel<I, TE, TY>),
                           dim3(static_cast<unsigned>((m * runs + kSumWaves - 1) / kSumWaves)), dim3(kSumThreads), 0,
                           static_cast<hipStream_t>(a.stream), static_cast<const I*>(a.ids) + at, m, a.V, a.K, runs,
                           a.scale, static_cast<const TE*>(a.E), static_cast<TY*>(a.y) + at * a.K);
    }
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

template <typename I, typename TD, typename TE>
ss1_status backward_t(const EmbeddingArgs& a) {
    const RowOrder o = row_order(a.V);
    const hipStream_t stream = static_cast<hipStream_t>(a.stream);
    const I* ids = static_cast<const I*>(a.ids);
    const TD* dy = static_cast<const TD*>(a.dy);
    TE* dE = static_cast<TE*>(a.dE);
    const unsigned blocks = 1u << o.log2_blocks;
    const int slices = (a.K + kSliceOf<TD> - 1) / kSliceOf<TD>;
    if (few_tokens(a.M, a.V, a.K)) {
        hipLaunchKernelGGL((embedding_few_kernel<I, TD, TE>), dim3(blocks), dim3(kSortThreads), 0, stream, ids,
                           dy, dE, static_cast<int>(a.M), a.V, a.K, o, a.scale, a.accumulate);
        return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
    }
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    SumArgs s{};
    int32_t* start = reinterpret_cast<int32_t*>(ws);
    int32_t* order = reinterpret_cast<int32_t*>(ws + start_bytes(o));
    s.start = start;
    s.order = order;
    s.partial = reinterpret_cast<float*>(ws + start_bytes(o) + up_to(a.M * 4, 16));
    s.V = a.V;
    s.T = tile_tokens(a.M);
    s.tiles = static_cast<int32_t>((a.M + s.T - 1) / s.T);
    s.K = a.K;
    s.accumulate = a.accumulate;
    s.o = o;
    s.scale = a.scale;
    s.slices = slices;
    s.sum_blocks = (s.tiles * s.slices + kSumWaves - 1) / kSumWaves;
    // rows that the sort's launch clears: whole 16-byte vectors, but for the
    // rows at the table's end
    int64_t zero_vecs = 0, zero_blocks = 0;
    if (!a.accumulate) {
        const int64_t row = static_cast<int64_t>(a.K) * sizeof(TE);
        s.zeroed = kZeroFirst / row < a.V ? kZeroFirst / row / 8 * 8 : a.V / 8 * 8;
        zero_vecs = s.zeroed * row / 16;
        zero_blocks = (a.V - s.zeroed + kZeroRows * kSumWaves - 1) / (kZeroRows * kSumWaves);
    }
    const dim3 sort_grid(blocks + static_cast<unsigned>((zero_vecs + kZeroVecs - 1) / kZeroVecs));
    const int M = static_cast<int>(a.M);
    u32x4* zeros = reinterpret_cast<u32x4*>(dE);
    if (const int chunks = deal_chunks(a.M, o)) {
        const int chunk = static_cast<int>(chunk_tokens(a.M));
        Token* tokens = reinterpret_cast<Token*>(s.partial + static_cast<int64_t>(s.tiles) * 2 * a.K);
        int32_t* first = reinterpret_cast<int32_t*>(tokens + a.M);
        int32_t* counts = first + up_to(static_cast<int64_t>(blocks) + 1, 4);
        hipLaunchKernelGGL((embedding_count_kernel<I>), dim3(chunks), dim3(kSortThreads), 0, stream, ids, M, a.V, o,
                           chunk, counts);
        hipLaunchKernelGGL((embedding_deal_kernel<I>), dim3(chunks), dim3(kSortThreads), 0, stream, ids, M, a.V, o,
                           chunk, chunks, counts, first, tokens);
        hipLaunchKernelGGL((embedding_sort_kernel<Token>), sort_grid, dim3(kSortThreads), 0, stream, tokens, M, a.V, o,
                           first, start, order, zeros, zero_vecs);
    } else {
        hipLaunchKernelGGL((embedding_sort_kernel<I>), sort_grid, dim3(kSortThreads), 0, stream, ids, M, a.V, o,
                           static_cast<const int32_t*>(nullptr), start, order, zeros, zero_vecs);
    }
    hipLaunchKernelGGL((embedding_sum_kernel<I, TD, TE>), dim3(static_cast<unsigned>(s.sum_blocks + zero_blocks)),
                       dim3(kSumThreads), 0, stream, ids, dy, dE, s);
    if (s.tiles > 0)
        hipLaunchKernelGGL((embedding_join_kernel<I, TD, TE>), dim3(static_cast<unsigned>(s.tiles * s.slices)),
                           dim3(kSumThreads), 0, stream, ids, dE, s);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

template <typename I>
ss1_status forward_i(const EmbeddingArgs& a) {
    if (a.table_dtype == SS1_BF16)
        return a.row_dtype == SS1_BF16 ? forward_t<I, uint16_t, uint16_t>(a) : forward_t<I, uint16_t, float>(a);
    return a.row_dtype == SS1_BF16 ? forward_t<I, float, uint16_t>(a) : forward_t<I, float, float>(a);
}

template <typename I>
ss1_status backward_i(const EmbeddingArgs& a) {
    if (a.table_dtype == SS1_BF16)
        return a.row_dtype == SS1_BF16 ? backward_t<I, uint16_t, uint16_t>(a) : backward_t<I, float, uint16_t>(a);
    return a.row_dtype == SS1_BF16 ? backward_t<I, uint16_t, float>(a) : backward_t<I, float, float>(a);
}

}  // namespace

ss1_status launch_embedding_forward(const EmbeddingArgs& a) {
    return a.id_bytes == 4 ? forward_i<int32_t>(a) : forward_i<int64_t>(a);
}

size_t embedding_backward_workspace(int64_t M, int64_t V, int32_t K) {
    if (few_tokens(M, V, K)) return 0;
    const RowOrder o = row_order(V);
    const int64_t T = tile_tokens(M), tiles = (M + T - 1) / T;
    return start_bytes(o) + static_cast<size_t>(up_to(M * 4, 16)) + static_cast<size_t>(tiles) * 2 * K * 4 +
           deal_bytes(M, o);
}

ss1_status launch_embedding_backward(const EmbeddingArgs& a) {
    return a.id_bytes == 4 ? backward_i<int32_t>(a) : backward_i<int64_t>(a);
}

}  // namespace ss1
