// Token embedding with scaling, and the table's gradient by sorted tokens
// (ss1_embedding_forward, ss1_embedding_backward).
//
// Backward: dE[v] is a sum over the tokens of row v, so the tokens are brought
// into the order of their rows first, and then every row is written once.
//
// Sort.  Block b of NB (a power of two) owns the rows v with v % NB == b, so
// the frequent rows, which have low numbers in most vocabularies, lie in
// different blocks.  Every block reads all M ids (a few KB to a few hundred,
// from L2): it counts the ones that blocks before it own, which is where its
// own tokens begin in the sorted order, and its own by row; a prefix sum over
// its rows and a second pass over the ids give every token its place.  Each of
// the 16 waves takes a run of the ids and has counters of its own, and lanes of
// one row take their rank from a ballot for each bit of the row number, so the
// order is stable, nothing is atomic in global memory, and one launch sorts.
//
// Sum.  A wave takes T consecutive places of the sorted order and 64 lanes'
// worth of columns, so a row with many tokens is shared by many waves.  A row
// whose tokens all lie in the T is written at once; the others leave partial
// sums (at most two a wave: its first and its last row), which a last launch
// adds in order.  Rows without tokens are zeroed by further blocks of the
// sum's launch.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_model_ops.h"

namespace ss1 {

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortRows = 512;   // rows of a sorting block at most
constexpr int kSortKeep = 16;    // steps whose ids a lane keeps between the two passes
constexpr int kMinBlocks = 256;  // sorting blocks at least (one a compute unit)
constexpr int kTile = 16;        // tokens of a summing wave, up to kMaxTiles waves a column slice
constexpr int kMaxTiles = 4096;
constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / 64;
constexpr int kZeroRows = 16;    // rows of a zeroing wave

// ------------------------------------------------------------ element access
template <int VEC>
__device__ __forceinline__ void load_row(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        v[0] = __uint_as_float(static_cast<uint32_t>(*p) << 16);
    }
}
__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
template <int VEC>
__device__ __forceinline__ void store_row(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}
template <int VEC>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        uint4 o;
        o.x = bf16_bits(v[0]) | bf16_bits(v[1]) << 16;
        o.y = bf16_bits(v[2]) | bf16_bits(v[3]) << 16;
        o.z = bf16_bits(v[4]) | bf16_bits(v[5]) << 16;
        o.w = bf16_bits(v[6]) | bf16_bits(v[7]) << 16;
        *reinterpret_cast<uint4*>(p) = o;
    } else {
        *p = static_cast<uint16_t>(bf16_bits(v[0]));
    }
}

// -------------------------------------------------------------------- forward
// A wave takes one token and a run of kSlices * 64 * VEC columns.
constexpr int kSlices = 4;

template <typename I, typename TE, typename TY, int VEC>
__global__ __launch_bounds__(kSumThreads) void embedding_forward_kernel(const I* __restrict__ ids, int64_t M, int64_t V,
                                                                        int K, int runs, float scale,
                                                                        const TE* __restrict__ E,
                                                                        TY* __restrict__ y) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kSumWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m = unit / runs;
    if (m >= M) return;
    const int c0 = static_cast<int>(unit % runs) * kSlices * 64 * VEC + lane * VEC;
    const int64_t id = static_cast<int64_t>(ids[m]);
    const bool real = id >= 0 && id < V;
    float v[kSlices][VEC];
#pragma unroll
    for (int i = 0; i < kSlices; ++i) {
        const int c = c0 + i * 64 * VEC;
        if (real && c < K) {
            load_row<VEC>(E + id * K + c, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < kSlices; ++i) {
        const int c = c0 + i * 64 * VEC;
        if (c >= K) break;
        if (real) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] *= scale;
        }
        store_row<VEC>(y + m * K + c, v[i]);
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
__device__ __forceinline__ Own own_row(I id, int64_t V, const RowOrder& o) {
    const int64_t v = static_cast<int64_t>(id);
    const bool real = v >= 0 && v < V;
    const int owner = static_cast<int>(v & ((int64_t(1) << o.log2_blocks) - 1));
    Own r;
    r.row = real && owner == static_cast<int>(blockIdx.x) ? static_cast<int>(v >> o.log2_blocks) : -1;
    r.before = real && owner < static_cast<int>(blockIdx.x);
    return r;
}

// Writes start[place of row] (where the row's tokens begin in the sorted order)
// for the block's rows, the last block also the end of the last row, and
// order[] (the tokens by row, ascending within a row).
template <typename I>
__global__ __launch_bounds__(kSortThreads) void embedding_sort_kernel(const I* __restrict__ ids, int M, int64_t V,
                                                                      RowOrder o, int32_t* __restrict__ start,
                                                                      int32_t* __restrict__ order) {
    __shared__ int32_t hist[kSortWaves][kSortRows];
    __shared__ int32_t sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int r = tid; r < kSortWaves * kSortRows; r += kSortThreads) hist[r / kSortRows][r % kSortRows] = 0;
    __syncthreads();

    // the wave's run of ids: whole steps of 64
    const int steps = (M + kSortThreads - 1) / kSortThreads;
    const int64_t first = static_cast<int64_t>(wave) * steps * 64;
    const I none = static_cast<I>(-1);
    I keep[kSortKeep];
#pragma unroll
    for (int s = 0; s < kSortKeep; ++s) {
        const int64_t m = first + s * 64 + lane;
        keep[s] = s < steps && m < M ? ids[m] : none;
    }
    int before = 0;
    auto count = [&](I id) {
        const Own w = own_row(id, V, o);
        if (w.row >= 0) atomicAdd(&hist[wave][w.row], 1);
        before += __popcll(__ballot(w.before));
    };
#pragma unroll
    for (int s = 0; s < kSortKeep; ++s)
        if (s < steps) count(keep[s]);
    for (int s = kSortKeep; s < steps; ++s) {
        const int64_t m = first + s * 64 + lane;
        count(m < M ? ids[m] : none);
    }
    if (lane == 0) sums[wave] = before;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) base += sums[w];
    __syncthreads();

    // prefix sum over the rows (thread r has row r), the waves of a row in turn
    int mine = 0;
    if (tid < kSortRows)
        for (int w = 0; w < kSortWaves; ++w) mine += hist[w][tid];
    int scan = mine;
    for (int off = 1; off < 64; off <<= 1) {
        const int t = __shfl_up(scan, off);
        if (lane >= off) scan += t;
    }
    if (lane == 63) sums[wave] = scan;
    __syncthreads();
    int at = base + scan - mine;
    for (int w = 0; w < wave; ++w) at += sums[w];
    if (tid < o.rows) start[static_cast<int64_t>(blockIdx.x) * o.rows + tid] = at;
    if (blockIdx.x == gridDim.x - 1 && tid == o.rows - 1) start[static_cast<int64_t>(gridDim.x) * o.rows] = at + mine;
    if (tid < kSortRows)
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = hist[w][tid];
            hist[w][tid] = at;
            at += n;
        }
    __syncthreads();

    // places: the lanes of one row in a step take consecutive ones
    const int bits = 32 - __builtin_clz(o.rows);
    auto put = [&](I id, int64_t m) {
        const int row = own_row(id, V, o).row;
        uint64_t same = __ballot(row >= 0);
        if (same == 0) return;
        for (int b = 0; b < bits; ++b) {
            const bool bit = (row >> b) & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        if (row >= 0) {
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int p = hist[wave][row] + rank;
            order[p] = static_cast<int32_t>(m);
            // the row's last lane of the step, after every lane's read
            if ((same >> lane) == 1) hist[wave][row] = p + 1;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
#pragma unroll
    for (int s = 0; s < kSortKeep; ++s)
        if (s < steps) put(keep[s], first + s * 64 + lane);
    for (int s = kSortKeep; s < steps; ++s) {
        const int64_t m = first + s * 64 + lane;
        put(m < M ? ids[m] : none, m);
    }
}

// ------------------------------------------------------------------------ sum
template <typename T, int VEC>
__device__ __forceinline__ void write_row(T* dE, int64_t at, const float (&sum)[VEC], float scale, bool accumulate) {
    float v[VEC];
    if (accumulate) {
        load_row<VEC>(dE + at, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += sum[j] * scale;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = sum[j] * scale;
    }
    store_row<VEC>(dE + at, v);
}

// A tile of the sorted order: its places [begin, end), and whether its first
// row began before it and its last row goes on behind it.
struct Tile {
    int begin, end;
    bool open_front, open_back;
};
template <typename I>
__device__ __forceinline__ Tile tile_of(int64_t tile, int T, int total, const I* ids, const int32_t* order) {
    Tile t;
    const int64_t b = tile * T;
    t.begin = b < total ? static_cast<int>(b) : total;
    t.end = b + T < total ? static_cast<int>(b) + T : total;
    t.open_front = t.begin < t.end && t.begin > 0 && ids[order[t.begin - 1]] == ids[order[t.begin]];
    t.open_back = t.begin < t.end && t.end < total && ids[order[t.end]] == ids[order[t.end - 1]];
    return t;
}

struct SumArgs {
    const int32_t* start;
    const int32_t* order;
    float* partial;    // [tiles][2][K]: the share of the first row, of the last row
    int64_t V;
    int64_t tiles;
    int64_t sum_blocks;  // blocks from here on zero rows
    int32_t T;
    int32_t K;
    int32_t slices;
    int32_t accumulate;
    RowOrder o;
    float scale;
};

template <typename I, typename TD, typename TE, int VEC>
__global__ __launch_bounds__(kSumThreads) void embedding_sum_kernel(const I* __restrict__ ids, const TD* __restrict__ dy,
                                                                    TE* __restrict__ dE, SumArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = a.K;
    if (blockIdx.x >= a.sum_blocks) {  // rows without tokens
        const int64_t v0 = ((blockIdx.x - a.sum_blocks) * kSumWaves + wave) * kZeroRows;
        bool empty = false;
        if (lane < kZeroRows && v0 + lane < a.V) {
            const int64_t p = place_of(a.o, v0 + lane);
            empty = a.start[p] == a.start[p + 1];
        }
        uint64_t rows = __ballot(empty);
        float zero[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) zero[j] = 0.0f;
        while (rows) {
            const int r = __builtin_ctzll(rows);
            rows &= rows - 1;
            for (int c = lane * VEC; c < K; c += 64 * VEC) store_row<VEC>(dE + (v0 + r) * K + c, zero);
        }
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kSumWaves + wave;
    const int64_t tile = unit / a.slices;
    if (tile >= a.tiles) return;
    const int c = static_cast<int>(unit % a.slices) * 64 * VEC + lane * VEC;
    const int total = a.start[(int64_t(1) << a.o.log2_blocks) * a.o.rows];
    const Tile t = tile_of(tile, a.T, total, ids, a.order);
    const bool in = c < K;
    float sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
    int64_t row = -1;
    bool first = true;
    auto flush = [&](bool last) {
        if (in) {
            if (first && t.open_front)
                store_row<VEC>(a.partial + (tile * 2) * K + c, sum);
            else if (last && t.open_back)
                store_row<VEC>(a.partial + (tile * 2 + 1) * K + c, sum);
            else
                write_row<TE, VEC>(dE, row * K + c, sum, a.scale, a.accumulate);
        }
        first = false;
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
    };
    for (int i = t.begin; i < t.end; ++i) {
        const int m = a.order[i];
        const int64_t v = static_cast<int64_t>(ids[m]);
        if (v != row) {
            if (row >= 0) flush(false);
            row = v;
        }
        if (in) {
            float d[VEC];
            load_row<VEC>(dy + static_cast<int64_t>(m) * K + c, d);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum[j] += d[j];
        }
    }
    if (row >= 0) flush(true);
}

// Rows whose tokens lie in several tiles: the wave of the tile where the row
// begins adds the shares in order.
template <typename I, typename TE, int VEC>
__global__ __launch_bounds__(kSumThreads) void embedding_join_kernel(const I* __restrict__ ids, TE* __restrict__ dE,
                                                                     SumArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kSumWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tile = unit / a.slices;
    if (tile >= a.tiles) return;
    const int c = static_cast<int>(unit % a.slices) * 64 * VEC + lane * VEC;
    const int K = a.K;
    const int total = a.start[(int64_t(1) << a.o.log2_blocks) * a.o.rows];
    const Tile t = tile_of(tile, a.T, total, ids, a.order);
    if (!t.open_back || c >= K) return;
    const int64_t row = static_cast<int64_t>(ids[a.order[t.end - 1]]);
    const int64_t p = place_of(a.o, row);
    if (a.start[p] < t.begin) return;  // it began in an earlier tile
    const int64_t last = (a.start[p + 1] - 1) / a.T;
    float sum[VEC];
    load_row<VEC>(a.partial + (tile * 2 + 1) * K + c, sum);
    for (int64_t i = tile + 1; i <= last; ++i) {
        float d[VEC];
        load_row<VEC>(a.partial + (i * 2) * K + c, d);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] += d[j];
    }
    write_row<TE, VEC>(dE, row * K + c, sum, a.scale, a.accumulate);
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

size_t start_bytes(const RowOrder& o) {
    return static_cast<size_t>(up_to(((int64_t(1) << o.log2_blocks) * o.rows + 1) * 4, 16));
}

template <typename I, typename TE, typename TY>
ss1_status forward_t(const EmbeddingArgs& a) {
    const int vec = a.K % 8 == 0 ? 8 : 1;
    const int runs = (a.K + kSlices * 64 * vec - 1) / (kSlices * 64 * vec);
    // a grid's threads are numbered in 32 bits
    const int64_t most = ((int64_t(1) << 24) - 1) / runs * kSumWaves;
    auto kern = vec == 8 ? &embedding_forward_kernel<I, TE, TY, 8> : &embedding_forward_kernel<I, TE, TY, 1>;
    for (int64_t at = 0; at < a.M; at += most) {
        const int64_t m = a.M - at < most ? a.M - at : most;
        hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((m * runs + kSumWaves - 1) / kSumWaves)),
                           dim3(kSumThreads), 0, static_cast<hipStream_t>(a.stream),
                           static_cast<const I*>(a.ids) + at, m, a.V, a.K, runs, a.scale,
                           static_cast<const TE*>(a.E), static_cast<TY*>(a.y) + at * a.K);
    }
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

template <typename I, typename TD, typename TE>
ss1_status backward_t(const EmbeddingArgs& a) {
    const RowOrder o = row_order(a.V);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    SumArgs s{};
    int32_t* start = reinterpret_cast<int32_t*>(ws);
    int32_t* order = reinterpret_cast<int32_t*>(ws + start_bytes(o));
    s.start = start;
    s.order = order;
    s.partial = reinterpret_cast<float*>(ws + start_bytes(o) + up_to(a.M * 4, 16));
    s.V = a.V;
    s.T = tile_tokens(a.M);
    s.tiles = (a.M + s.T - 1) / s.T;
    s.K = a.K;
    s.accumulate = a.accumulate;
    s.o = o;
    s.scale = a.scale;
    const int vec = a.K % 8 == 0 ? 8 : 1;
    s.slices = (a.K + 64 * vec - 1) / (64 * vec);
    s.sum_blocks = (s.tiles * s.slices + kSumWaves - 1) / kSumWaves;
    const int64_t zero_blocks = a.accumulate ? 0 : (a.V + kZeroRows * kSumWaves - 1) / (kZeroRows * kSumWaves);
    const hipStream_t stream = static_cast<hipStream_t>(a.stream);
    const I* ids = static_cast<const I*>(a.ids);
    TE* dE = static_cast<TE*>(a.dE);
    hipLaunchKernelGGL((embedding_sort_kernel<I>), dim3(1u << o.log2_blocks), dim3(kSortThreads), 0, stream, ids,
                       static_cast<int>(a.M), a.V, o, start, order);
    auto sum = vec == 8 ? &embedding_sum_kernel<I, TD, TE, 8> : &embedding_sum_kernel<I, TD, TE, 1>;
    if (s.sum_blocks + zero_blocks > 0)
        hipLaunchKernelGGL(sum, dim3(static_cast<unsigned>(s.sum_blocks + zero_blocks)), dim3(kSumThreads), 0, stream,
                           ids, static_cast<const TD*>(a.dy), dE, s);
    auto join = vec == 8 ? &embedding_join_kernel<I, TE, 8> : &embedding_join_kernel<I, TE, 1>;
    if (s.tiles > 1)
        hipLaunchKernelGGL(join, dim3(static_cast<unsigned>(s.sum_blocks)), dim3(kSumThreads), 0, stream, ids, dE, s);
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
    const RowOrder o = row_order(V);
    const int64_t T = tile_tokens(M), tiles = (M + T - 1) / T;
    return start_bytes(o) + static_cast<size_t>(up_to(M * 4, 16)) + static_cast<size_t>(tiles) * 2 * K * 4;
}

ss1_status launch_embedding_backward(const EmbeddingArgs& a) {
    return a.id_bytes == 4 ? backward_i<int32_t>(a) : backward_i<int64_t>(a);
}

}  // namespace ss1
