// Low-rank adapters of many requests beside a shared projection
// (ss1_adapter_forward, _backward).
//
// With both factors stored rank-major the two directions are the same three
// products:
//   shrink  v[m][j]  = sum_k x[m][k] A[j][k]           (and dv from dy and B)
//   expand  y[m][n]  = base[m][n] + sum_j v[m][j] B[j][n]   (and dx from dv and A)
//   outer   dA[j][k] = sum_m dv[m][j] x[m][k]          (and dB from v and dy)
// All run on 16x16 matrix tiles with float32 accumulators.  bf16: 16x16x32
// MFMAs; v stays float32 in memory and enters the second product as the sum
// of two bf16 values (an error of 2^-17 of v), so that it costs no precision
// beside the last rounding.  float32: 16x16x4 MFMAs (exact products).
//
// The tokens are cut into pieces that lie in one segment and in one tile of
// TM tokens; a block takes a piece.  Every array is read through a buffer
// descriptor that ends with its piece or adapter: rows past the end read as
// zero and stores past it are dropped, so ragged lengths and ranks cost no
// branch, and nothing of another request can enter a sum.
//
// What bounds them: the bytes of x, base and y on large batches, the latency of
// a few dependent reads on small ones; never the products (2 R multiply-adds an
// element of x or y).  So there are as few launches as the dependences allow
// (shrink; expand; the outer products; their join where tokens are split), v and
// dv are the only arrays between them, and each is R float32 values a token.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "ss1_adapter_list.h"
#include "ss1_device.h"
#include "ss1_dma.h"
#include "ss1_ops.h"

namespace ss1 {

namespace {

using dev::bf16x2;
using dev::bf16x8;
using dev::buf_load16;
using dev::f32x4;
using dev::make_rsrc;
using dev::pair_lane_mask;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int64_t kMaxBlocks = int64_t(1) << 22;  // items beyond that loop
constexpr uint32_t kOutside = 0x80000000u;        // past every descriptor (2^31 bytes at most)

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__device__ __forceinline__ void buf_store16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint4 v) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    // non-temporal: nothing in this call reads it again (117 MB of y, the expand 66
    // -> 63 us; smaller outputs, and what a next reader of y pays, were not measured)
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{v.x, v.y, v.z, v.w}, r, voff, 0, 2);
}

// A value that the whole wave reads at one index: a scalar load.  The scalar
// cache is not swept by the tensors that stream through the vector caches, so
// the few dependent reads at the start of a block take a fraction of what they
// do behind a queue of vector loads.
template <typename T>
__device__ __forceinline__ T uniform_load(const T* p, int i) {
    typedef const __attribute__((address_space(4))) T* scalar_ptr;
    return reinterpret_cast<scalar_ptr>(reinterpret_cast<uintptr_t>(p))[__builtin_amdgcn_readfirstlane(i)];
}

// First row and rank of adapter e, inside [0, R) whatever the arrays hold.
__device__ __forceinline__ int rows_of(const AdapterView& ad, int e, int* first) {
    const int r0 = clampi(uniform_load(ad.row, e), 0, ad.R), r1 = clampi(uniform_load(ad.row, e + 1), r0, ad.R);
    *first = r0;
    return min(r1 - r0, ad.max_rank);
}

struct Piece {
    int begin, n;     // tokens
    int first, rank;  // adapter rows; rank 0: no adapter
    float scale;
};

// Piece p of the batch: with F(s) = s + offset[s] / TM, segment s has pieces
// F(s) .. F(s+1) - 1, one for each tile of TM tokens that it touches (the last
// may be empty), so no prefix sum over the segments is needed: a binary search
// of p in F finds the segment.
__device__ __forceinline__ Piece find_piece(const AdapterView& ad, int TM, int p) {
    Piece out{0, 0, 0, 0, 0.0f};
    int s = 0, b = 0, t = ad.M, e = -1;
    if (ad.S > 0) {
        int hi = ad.S;
        while (hi - s > 1) {
            const int mid = s + (hi - s) / 2;
            if (mid + clampi(uniform_load(ad.seg, mid), 0, ad.M) / TM <= p) s = mid; else hi = mid;
        }
        e = uniform_load(ad.seg_adapter, s);
        b = clampi(uniform_load(ad.seg, s), 0, ad.M);
        t = clampi(uniform_load(ad.seg, s + 1), b, ad.M);
    }
    const int64_t tile = static_cast<int64_t>(p) - s;
    const int64_t from = max(int64_t(b), tile * TM), to = min(int64_t(t), (tile + 1) * TM);
    if (to <= from) return out;
    out.begin = static_cast<int>(from);
    out.n = static_cast<int>(to - from);
    if (e >= 0 && e < ad.E) {
        out.rank = rows_of(ad, e, &out.first);
        out.scale = uniform_load(ad.scale, e);
    }
    return out;
}

int64_t pieces_of(int64_t M, int64_t S, int TM) { return M / TM + (S > 0 ? S : 1); }

// ------------------------------------------------------------ matrix operands
// An operand lane holds 16 bytes of one row of a [rows][k] matrix: 8 bf16 of
// 32 k, or 4 floats of 16 k (four 16x16x4 products, the i-th of the floats i).
__device__ __forceinline__ f32x4 mma(const __bf16*, uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x4 mma(const float*, uint4 a, uint4 b, f32x4 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
}

// Two loads of 8 rows x 128 bytes -> two operands of 16 rows x 64 bytes.
__device__ __forceinline__ void pair_operands(uint4 a, uint4 b, uint32_t lo8, uint4& t0, uint4& t1) {
    dev::pair_operands(a, b, lo8, t0, t1);
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// Eight rows of 8 bf16 columns -> for each column its 8 rows (an operand).
__device__ __forceinline__ void transpose8(const uint4 (&r)[8], uint4 (&f)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t a = (&r[2 * q].x)[d], b = (&r[2 * q + 1].x)[d];
            lo[q] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            hi[q] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        }
        f[2 * d] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        f[2 * d + 1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

// A lane's float32 values of v as operands: hi and lo (bf16), or themselves.
__device__ __forceinline__ void rank_operands(const __bf16*, const float (&v)[8], uint4 (&f)[2]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * j], v[2 * j + 1]}, bf16x2));
        const float a = v[2 * j] - __uint_as_float(hi[j] << 16);
        const float b = v[2 * j + 1] - __uint_as_float(hi[j] & 0xFFFF0000u);
        lo[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
        // a value whose hi is infinite has no rest (inf - inf would make it a NaN)
        const uint32_t full = hi[j] & 0x7F807F80u;
        if ((full & 0x7F80u) == 0x7F80u) lo[j] &= 0xFFFF0000u;
        if ((full >> 16) == 0x7F80u) lo[j] &= 0x0000FFFFu;
    }
    f[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    f[1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}
__device__ __forceinline__ void rank_operands(const float*, const float (&v)[4], uint4 (&f)[1]) {
    f[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// Rows of v of a piece copied to rows of `stride` floats: the outer products
// gather 16 bytes at a time, which rows of any other length would let run past
// the end of the array.
struct Repack {
    const float* from;  // [M][cols]; null: nothing to do
    float* to;          // [M][stride]
    int cols, stride;
};

__device__ __forceinline__ void repack_rows(const Repack& v, int begin, int n) {
    for (int i = threadIdx.x; i < n * v.stride; i += kThreads) {
        const size_t m = static_cast<size_t>(begin) + i / v.stride;
        const int j = i % v.stride;
        v.to[m * v.stride + j] = j < v.cols ? v.from[m * v.cols + j] : 0.0f;
    }
}

__global__ __launch_bounds__(kThreads) void repack_kernel(Repack v, int M) {
    for (int64_t m = static_cast<int64_t>(blockIdx.x) * 16; m < M; m += static_cast<int64_t>(gridDim.x) * 16)
        repack_rows(v, static_cast<int>(m), static_cast<int>(min(int64_t(16), M - m)));
}

// The outer products' work list.  Requests share the adapters unevenly, so the
// tokens of each adapter are cut into parts of P: part i of adapter e is entry
// {e, i P, end, slot}, where parts of an adapter that has several go to slots of
// a partial buffer (slot -1: straight to the gradient).  multi[0].x counts the
// adapters with several parts, multi[1 + i] = {e, parts, first slot}.
struct OuterPlan {
    int4* table;  // [most]; null: every adapter is one part (M <= P)
    int4* multi;  // [E + 1]
    int P, most, slots;
};

__device__ __forceinline__ int4 block_scan(int4 v, int4* sums, int4* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int x = __shfl_up(v.x, off), y = __shfl_up(v.y, off), z = __shfl_up(v.z, off);
        if (lane >= off) v = make_int4(v.x + x, v.y + y, v.z + z, 0);
    }
    __syncthreads();
    if (lane == 63) sums[wave] = v;
    __syncthreads();
    *total = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int4 o = sums[w];
        if (w < wave) v = make_int4(v.x + o.x, v.y + o.y, v.z + o.z, 0);
        *total = make_int4(total->x + o.x, total->y + o.y, total->z + o.z, 0);
    }
    return v;
}

// Written by one block (an extra one of the shrink's launch); `lds` holds
// 1024 + 64 bytes.
__device__ void plan_outer(const AdapterView& ad, const OuterPlan& plan, int* lds) {
    int4* sums = reinterpret_cast<int4*>(lds + kThreads);
    PlanSums done{0, 0, 0};
    for (int e0 = 0; e0 < ad.E; e0 += kThreads) {
        __syncthreads();
        lds[threadIdx.x] = 0;
        __syncthreads();
        for (int s = threadIdx.x; s < ad.S; s += kThreads) {
            const int e = ad.seg_adapter[s] - e0, b = clampi(ad.seg[s], 0, ad.M), n = clampi(ad.seg[s + 1], b, ad.M) - b;
            if (e >= 0 && e < kThreads && e0 + e < ad.E && n > 0) atomicAdd(lds + e, n);
        }
        __syncthreads();
        const int e = e0 + threadIdx.x, tokens = clampi(lds[threadIdx.x], 0, ad.M);
        const int parts = e < ad.E ? parts_of(tokens, plan.P) : 0;
        int4 total;
        const int4 in = make_int4(parts, parts > 1 ? parts : 0, parts > 1, 0), end = block_scan(in, sums, &total);
        const int q = done.entries + end.x - in.x, slot = done.slots + end.y - in.y, c = done.several + end.z - in.z;
        // (there is room for all of them unless the offsets are out of order)
        const bool several = parts > 1 && slot + parts <= plan.slots;
        for (int i = 0; i < parts; ++i)
            if (q + i < plan.most)
                plan.table[q + i] = several ? make_int4(e, i * plan.P, part_end(tokens, plan.P, i), slot + i)
                                            : make_int4(i == 0 ? e : -1, 0, tokens, -1);
        if (parts > 1) plan.multi[1 + c] = several ? make_int4(e, parts, slot, 0) : make_int4(e, 0, 0, 0);
        done = plan_add(done, {total.x, total.y, total.z}, plan.most, plan.slots);
    }
    for (int q = done.entries + threadIdx.x; q < plan.most; q += kThreads) plan.table[q] = make_int4(-1, 0, 0, -1);
    if (threadIdx.x == 0) plan.multi[0] = make_int4(done.several, 0, 0, 0);
}

__global__ __launch_bounds__(kThreads) void plan_outer_kernel(AdapterView ad, OuterPlan plan) {
    __shared__ __align__(16) int lds[kThreads + 16];
    plan_outer(ad, plan, lds);
}

// ---------------------------------------------------------------------- shrink
// One block: a piece of up to 16 tokens and a slice q of K; its waves split the
// slice, their tiles are added in LDS.  A wave's operands come straight from
// global memory in whole 128-byte lines.  part[q][m][stride], columns past the
// rank 0.
// Bound by A and the chain of dependent reads (64 requests of ranks up to 64, K =
// 4096, bf16: 15 MB of factors, mostly from cache, in 9.4 us with launch and
// lookup), hence the slices: the more blocks read a factor, the shorter each one's
// chain.
// ROWS: rows of x that may be there, 8 or 16.
template <typename T, int RT, int UN = 1, int ROWS = 16>
__device__ __forceinline__ void shrink_body(const Piece& pc, const T* x, const T* A, float* out, int K, int Q, int q,
                                            int stride, float scale, f32x4* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t Kb = static_cast<uint32_t>(K) * sizeof(T);
    const int units = static_cast<int>((Kb + 127) / 128);
    // the slice's units go to the waves in turn, so that the block reads each
    // row in one run of memory
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * q / Q);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (q + 1) / Q);
    const auto rx = make_rsrc(x + static_cast<size_t>(pc.begin) * K, static_cast<uint32_t>(pc.n) * Kb);
    const auto ra = make_rsrc(A + static_cast<size_t>(pc.first) * K, static_cast<uint32_t>(pc.rank) * Kb);
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0, 0, 0, 0};
    // a load covers 8 rows x 128 bytes; pair_operands makes two operands of
    // 16 rows x 64 bytes from two loads
    const uint32_t piece = 16u * ((lane >> 4) + 4 * ((lane >> 3) & 1)), lo8 = pair_lane_mask(lane);
    const uint32_t lane_off = (lane & 7) * Kb + piece;
    // UN units' loads are in flight together (past the wave's share or the row:
    // zeros); beside other blocks on the compute unit 1, 2 and 3 measure the same
    for (int ub = u0 + wave * UN; ub < u1; ub += UN * kWaves) {
        uint4 xf[UN][2], af[UN][RT][2];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const uint32_t at = 128u * (ub + u);
            const uint32_t off = ub + u < u1 && at + piece < Kb ? lane_off + at : kOutside;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                xf[u][h] = 8 * h < ROWS ? buf_load16(rx, off + h * 8 * Kb, 0) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 2 * RT; ++r) af[u][r / 2][r % 2] = buf_load16(ra, off + r * 8 * Kb, 0);
        }
        __builtin_amdgcn_sched_barrier(0);  // or each load sinks to its first use
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            pair_operands(xf[u][0], xf[u][1], lo8, xf[u][0], xf[u][1]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                pair_operands(af[u][r][0], af[u][r][1], lo8, af[u][r][0], af[u][r][1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) acc[r] = mma(x, xf[u][h], af[u][r][h], acc[r]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r) red[(wave * RT + r) * 64 + lane] = acc[r];
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 64; i += kThreads) {
        f32x4 s = red[i];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += red[w * RT * 64 + i];
        const int j = 16 * (i >> 6) + (i & 15), m = 4 * ((i >> 4) & 3);
        if (j < stride)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (m + k < pc.n) out[static_cast<size_t>(m + k) * stride + j] = j < pc.rank ? s[k] * scale : 0.0f;
    }
    const int rest = stride - 16 * RT;  // columns past the tiles are zero
    if (rest > 0)
        for (int i = threadIdx.x; i < pc.n * rest; i += kThreads)
            out[static_cast<size_t>(i / rest) * stride + 16 * RT + i % rest] = 0.0f;
}

template <typename T, int RT>
__global__ __launch_bounds__(kThreads) void shrink_kernel(AdapterView ad, const T* __restrict__ x,
                                                          const T* __restrict__ A, float* __restrict__ part, int stride,
                                                          int K, int Q, int scaled, Repack v, OuterPlan plan, int64_t items) {
    __shared__ f32x4 red[kWaves * RT * 64 + 64];
    if (plan.table && blockIdx.x == gridDim.x - 1) {
        plan_outer(ad, plan, reinterpret_cast<int*>(red));
        return;
    }
    const int64_t step = gridDim.x - (plan.table != nullptr);
    for (int64_t item = blockIdx.x; item < items; item += step) {
        const int q = static_cast<int>(item % Q);
        const Piece pc = find_piece(ad, 16, static_cast<int>(item / Q));
        if (pc.n == 0) continue;
        if (v.from && q == 0) repack_rows(v, pc.begin, pc.n);
        float* out = part + (static_cast<size_t>(q) * ad.M + pc.begin) * stride;
        const float scale = scaled ? pc.scale : 1.0f;
        if (pc.rank == 0) {
            for (int i = threadIdx.x; i < pc.n * stride; i += kThreads) out[i] = 0.0f;
            continue;
        }
        // tiles for the rank of this adapter, not for the largest
        if (RT == 1 || pc.rank <= 16)
            shrink_body<T, 1>(pc, x, A, out, K, Q, q, stride, scale, red);
        else if (RT == 2 || pc.rank <= 32)
            shrink_body<T, RT < 2 ? RT : 2>(pc, x, A, out, K, Q, q, stride, scale, red);
        else if (RT == 4 || pc.rank <= 64)
            shrink_body<T, RT < 4 ? RT : 4>(pc, x, A, out, K, Q, q, stride, scale, red);
        else
            shrink_body<T, RT>(pc, x, A, out, K, Q, q, stride, scale, red);
    }
}

// The shrink of long segments: 64 tokens and a slice of K a block, in stages
// of 128 bytes of every row of x and A.  Each stage goes from global memory
// straight to LDS (whole lines, no registers), a ring of kStages of them deep;
// wave w takes tokens 16 w .. 16 w + 15 of the tile and all ranks, so nothing
// has to be added across the waves.  A is read once a 64 tokens and comes from
// cache; x sets the time: 8192 x 5120 bf16 (84 MB) and rank 64 in 25.8 us, 3.3
// TB/s; 4096 x 4096 in 13.9.
// Stages: 2 / 3 / 4 in us of the whole call: forward of 4096 tokens 4096 -> 14336
// 82.0 / 80.3 / 80.6, gradients of 8192 tokens 1280 -> 5120 103.2 / 98.8 / 99.5.
constexpr int kStages = 3;

// Wave-wide loads (8 rows x 128 bytes) of a stage, the same number a wave;
// rows of A past the rank read as zero.
constexpr int stage_loads(int RT) { return (8 + 2 * RT + kWaves - 1) / kWaves; }

template <typename T, int RT>
__device__ __forceinline__ void shrink_tile_body(const Piece& pc, const T* x, const T* A, float* out, int K, int Q,
                                                 int q, int stride, float scale, uint8_t* ring) {
    constexpr int L = stage_loads(RT), BYTES = L * kWaves * 1024;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t Kb = static_cast<uint32_t>(K) * sizeof(T);
    const int units = static_cast<int>((Kb + 127) / 128);
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * q / Q);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (q + 1) / Q);
    const auto rx = dev::dma_rsrc(x + static_cast<size_t>(pc.begin) * K, static_cast<uint32_t>(pc.n) * Kb);
    const auto ra = dev::dma_rsrc(A + static_cast<size_t>(pc.first) * K, static_cast<uint32_t>(pc.rank) * Kb);
    const uint32_t lds = dev::lds_address(ring);
    // row p of a stage holds piece i of its 128 bytes at slot i ^ key(p)
    const auto issue = [&](int u, int buffer) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int group = i * kWaves + wave, row = 8 * group + (lane >> 3);
            const uint32_t at = 128u * u + 16 * ((lane & 7) ^ dev::swz_key<128>(row));
            const bool in = u < u1 && at < Kb;
            const uint32_t to = lds + buffer * BYTES + group * 1024;
            if (group < 8)
                dev::lds_dma16(rx, to, in ? row * Kb + at : kOutside, 0);
            else
                dev::lds_dma16(ra, to, in ? (row - 64) * Kb + at : kOutside, 0);
        }
    };
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0, 0, 0, 0};
    __syncthreads();  // the ring's last readers
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(u0 + s, s);
    const int m = 16 * wave + (lane & 15), g = lane >> 4;
    int buffer = 0;
    for (int u = u0; u < u1; ++u) {
        // this stage has landed, and everyone is done with the one before it,
        // whose place the next stage takes
        dev::dma_stage_barrier<L*(kStages - 2)>();
        issue(u + kStages - 1, buffer == 0 ? kStages - 1 : buffer - 1);
        const uint8_t* stage = ring + buffer * BYTES;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 xf = *reinterpret_cast<const uint4*>(stage + m * 128 + 16 * ((4 * h + g) ^ dev::swz_key<128>(m)));
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = 64 + 16 * r + (lane & 15);
                const uint4 af =
                    *reinterpret_cast<const uint4*>(stage + row * 128 + 16 * ((4 * h + g) ^ dev::swz_key<128>(row)));
                acc[r] = mma(x, xf, af, acc[r]);
            }
        }
        buffer = buffer + 1 == kStages ? 0 : buffer + 1;
    }
    dev::dma_stage_barrier<0>();  // nothing in flight into the ring
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int j = 16 * r + (lane & 15);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = 16 * wave + 4 * g + k;
            if (j < stride && t < pc.n) out[static_cast<size_t>(t) * stride + j] = j < pc.rank ? acc[r][k] * scale : 0.0f;
        }
    }
    const int rest = stride - 16 * RT;  // columns past the tiles are zero
    if (rest > 0)
        for (int i = threadIdx.x; i < pc.n * rest; i += kThreads)
            out[static_cast<size_t>(i / rest) * stride + 16 * RT + i % rest] = 0.0f;
}

template <typename T, int RT>
__global__ __launch_bounds__(kThreads) void shrink_tile_kernel(AdapterView ad, const T* __restrict__ x,
                                                               const T* __restrict__ A, float* __restrict__ part,
                                                               int stride, int K, int Q, int scaled, Repack v,
                                                               OuterPlan plan, int64_t items) {
    __shared__ __align__(1024) uint8_t ring[kStages * stage_loads(RT) * kWaves * 1024];
    if (plan.table && blockIdx.x == gridDim.x - 1) {
        plan_outer(ad, plan, reinterpret_cast<int*>(ring));
        return;
    }
    const int64_t step = gridDim.x - (plan.table != nullptr);
    for (int64_t item = blockIdx.x; item < items; item += step) {
        const int q = static_cast<int>(item % Q);
        const Piece pc = find_piece(ad, 64, static_cast<int>(item / Q));
        if (pc.n == 0) continue;
        if (v.from && q == 0) repack_rows(v, pc.begin, pc.n);
        float* out = part + (static_cast<size_t>(q) * ad.M + pc.begin) * stride;
        const float scale = scaled ? pc.scale : 1.0f;
        if (pc.rank == 0) {
            for (int i = threadIdx.x; i < pc.n * stride; i += kThreads) out[i] = 0.0f;
            continue;
        }
        if (RT == 1 || pc.rank <= 16)
            shrink_tile_body<T, 1>(pc, x, A, out, K, Q, q, stride, scale, ring);
        else if (RT == 2 || pc.rank <= 32)
            shrink_tile_body<T, RT < 2 ? RT : 2>(pc, x, A, out, K, Q, q, stride, scale, ring);
        else if (RT == 4 || pc.rank <= 64)
            shrink_tile_body<T, RT < 4 ? RT : 4>(pc, x, A, out, K, Q, q, stride, scale, ring);
        else
            shrink_tile_body<T, RT>(pc, x, A, out, K, Q, q, stride, scale, ring);
    }
}

// ---------------------------------------------------------------------- expand
// Tokens in the rows of the product, columns in its columns: an operand of B is 16
// columns of a rank unit, 16 bytes of each of its rows turned in registers, and
// a lane's sums are 16 bytes of four rows of y.
//
// expand_kernel, short segments.  One block: a piece of up to 16 tokens and a few
// column tiles of kWaves * 16 vectors of 16 bytes.  The piece's v (its Q partial
// sums added in order) goes to LDS as operands; each wave then takes 16 vectors
// of every tile, and the rows of B and base of the next tile are in flight while
// it multiplies this one.
// Bound by B, base and y (64 requests, N = 14336, ranks up to 64: 55 MB of which
// B, 51 MB, comes partly from cache, in 15.0 us).
// Rank units: 32 (bf16: one product each of hi and lo) or 16 (float32).
template <int N>
struct Int {
    static constexpr int value = N;
};
template <typename T>
struct Unit;
template <>
struct Unit<__bf16> {
    static constexpr int kRanks = 32, kLoads = 8, kCols = 8, kFrags = 2;
};
template <>
struct Unit<float> {
    static constexpr int kRanks = 16, kLoads = 4, kCols = 4, kFrags = 1;
};

// Rows (of B: ranks; of x: tokens) of this lane's 16 bytes of columns -> one
// operand a column.
__device__ __forceinline__ void column_operands(const __bf16*, const uint4 (&t)[8], uint4 (&f)[8]) {
    transpose8(t, f);
}
__device__ __forceinline__ void column_operands(const float*, const uint4 (&t)[4], uint4 (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = make_uint4((&t[0].x)[j], (&t[1].x)[j], (&t[2].x)[j], (&t[3].x)[j]);
}

// 16 bytes of a row of base into element i of the column accumulators, and back.
__device__ __forceinline__ void unpack(const __bf16*, uint4 w, int i, f32x4 (&acc)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        acc[2 * d][i] = __uint_as_float((&w.x)[d] << 16);
        acc[2 * d + 1][i] = __uint_as_float((&w.x)[d] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const float*, uint4 w, int i, f32x4 (&acc)[4]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) acc[d][i] = __uint_as_float((&w.x)[d]);
}
__device__ __forceinline__ uint4 pack(const __bf16*, const f32x4 (&acc)[8], int i) {
    uint32_t w[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] = bf16_bits(acc[2 * d][i]) | bf16_bits(acc[2 * d + 1][i]) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float*, const f32x4 (&acc)[4], int i) {
    return make_uint4(__float_as_uint(acc[0][i]), __float_as_uint(acc[1][i]), __float_as_uint(acc[2][i]),
                      __float_as_uint(acc[3][i]));
}

// Where the sums of a tile start.  bf16: at base, whose share of the roundings of up
// to 128 products is far below the last one.  float32: at zero, and base is added to
// the finished sum; rounding every partial sum at base's size cost three of float32's
// bits where base is large beside the adapter's share.
__device__ __forceinline__ void start_sums(const __bf16* t, const uint4 (&old)[4], f32x4 (&acc)[8], f32x4 (&)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack(t, old[i], i, acc);
}
__device__ __forceinline__ void start_sums(const float* t, const uint4 (&old)[4], f32x4 (&acc)[4], f32x4 (&last)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unpack(t, old[i], i, last);
        acc[i] = f32x4{0, 0, 0, 0};
    }
}
__device__ __forceinline__ void end_sums(const __bf16*, f32x4 (&)[8], const f32x4 (&)[8]) {}
__device__ __forceinline__ void end_sums(const float*, f32x4 (&acc)[4], const f32x4 (&last)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += last[j];
}

// First of the column tiles of block cg of `columns` (at most one a tile): shares
// that differ by one tile at most (10 tiles in 3: 20.2 us, as 4 + 4 + 2 21.7).
__device__ __forceinline__ int first_tile(int cg, int tiles, int columns) {
    return static_cast<int>(static_cast<int64_t>(tiles) * cg / columns);
}

// Tokens without an adapter: y = base (zeros without one) in `wide` 16-byte
// columns from c0 on, and v = 0.
template <typename T>
__device__ __forceinline__ void without_adapter(const Piece& pc, const T* base, T* y, float* v_out, int v_stride,
                                                int v_cols, int N, int c0, int wide) {
    if (v_out)
        for (int i = threadIdx.x; i < pc.n * v_cols; i += kThreads)
            v_out[static_cast<size_t>(pc.begin + i / v_cols) * v_stride + i % v_cols] = 0.0f;
    if (base == y) return;
    const int row = static_cast<int>(static_cast<uint32_t>(N) * sizeof(T) / 16);
    wide = min(wide, row - c0);
    const size_t at = static_cast<size_t>(pc.begin) * N;
    for (int i = threadIdx.x; i < pc.n * wide; i += kThreads) {
        const size_t o = static_cast<size_t>(i / wide) * row + c0 + i % wide;
        reinterpret_cast<uint4*>(y + at)[o] =
            base ? reinterpret_cast<const uint4*>(base + at)[o] : make_uint4(0, 0, 0, 0);
    }
}

// `part`: the piece's rows of v, complete when make_v() returns (called with the
// first tile's loads in flight).
template <typename T, int KU, typename F>
__device__ __forceinline__ void expand_body(const Piece& pc, const float* part, size_t slice, int Q, int stride,
                                            int v_stride, int v_cols, const T* B, const T* base, T* y, float* v_out,
                                            int N, int tile0, int tiles, float scale, uint4* frags, F make_v) {
    using U = Unit<T>;
    constexpr int GROUP = U::kRanks / 4;  // ranks of one operand lane
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const uint32_t Nb = static_cast<uint32_t>(N) * sizeof(T);
    const auto rb = make_rsrc(B + static_cast<size_t>(pc.first) * N, static_cast<uint32_t>(pc.rank) * Nb);
    const auto ry = make_rsrc(y + static_cast<size_t>(pc.begin) * N, static_cast<uint32_t>(pc.n) * Nb);
    const auto rs = make_rsrc((base ? base : y) + static_cast<size_t>(pc.begin) * N,
                              base ? static_cast<uint32_t>(pc.n) * Nb : 0u);
    const auto column = [&](int tile) {  // (a row's offset is under 2^31, so kOutside plus it stays outside)
        const uint32_t col = 16u * (static_cast<uint32_t>(tile) * (kThreads / 4) + wave * 16 + c);
        return tile < tile0 + tiles && col < Nb ? col : kOutside;
    };
    // rows of B and of base (tokens 4 g + i) in this lane's columns
    uint4 rows[KU][U::kLoads], old[4];
    const auto fetch = [&](uint32_t col) {
        // opaque, or the compiler keeps every row's offset in a register
        uint32_t wide = Nb;
        asm volatile("" : "+s"(wide));
        uint32_t at = GROUP * g * wide + col;
#pragma unroll
        for (int k = 0; k < KU; ++k) {
#pragma unroll
            for (int i = 0; i < U::kLoads; ++i) {
                rows[k][i] = buf_load16(rb, at, 0);
                at += wide;
            }
            at += (U::kRanks - U::kLoads) * wide;
        }
        at = 4 * g * wide + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            old[i] = buf_load16(rs, at, 0);
            at += wide;
        }
    };
    fetch(column(tile0));  // in flight while v is made and staged
    make_v();
    __syncthreads();  // the last piece's readers of frags
    // v of the piece, summed over the slices of K in order (columns past the
    // rank are zero there; the stride is a multiple of 8)
#pragma unroll 1
    for (int i = threadIdx.x; i < 16 * KU * 4; i += kThreads) {
        const int m = i / (KU * 4), unit = i % (KU * 4) / 4, gi = i % 4, r = unit * U::kRanks + GROUP * gi;
        f32x4 v[GROUP / 4];
#pragma unroll
        for (int j = 0; j < GROUP / 4; ++j) v[j] = f32x4{0, 0, 0, 0};
        if (m < pc.n && r < stride) {
            const f32x4* from = reinterpret_cast<const f32x4*>(part + static_cast<size_t>(m) * stride + r);
            for (int q0 = 0; q0 < Q; q0 += 4) {  // four slices' loads together
                f32x4 w[4][GROUP / 4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < GROUP / 4; ++j) w[q][j] = from[min(q0 + q, Q - 1) * (slice / 4) + j];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < GROUP / 4; ++j)
                        if (q0 + q < Q) v[j] += w[q][j];
            }
            if (v_out)
                for (int j = 0; j < GROUP; ++j)
                    if (r + j < v_cols)
                        v_out[static_cast<size_t>(pc.begin + m) * v_stride + r + j] = v[j / 4][j % 4];
        }
        float scaled[GROUP];
#pragma unroll
        for (int j = 0; j < GROUP; ++j) scaled[j] = v[j / 4][j % 4] * scale;
        uint4 f[U::kFrags];
        rank_operands(B, scaled, f);
#pragma unroll
        for (int h = 0; h < U::kFrags; ++h) frags[(unit * U::kFrags + h) * 64 + m + 16 * gi] = f[h];
    }
    const int past = KU * U::kRanks;  // columns that no unit covers are zero
    if (v_out && past < v_cols)
        for (int i = threadIdx.x; i < pc.n * (v_cols - past); i += kThreads)
            v_out[static_cast<size_t>(pc.begin + i / (v_cols - past)) * v_stride + past + i % (v_cols - past)] = 0.0f;
    __syncthreads();
#pragma unroll 1
    for (int tile = tile0; tile < tile0 + tiles; ++tile) {
        f32x4 acc[U::kCols], last[U::kCols];
        start_sums(B, old, acc, last);
        uint4 f[KU][U::kCols];
#pragma unroll
        for (int k = 0; k < KU; ++k) {
            column_operands(B, rows[k], f[k]);
            __builtin_amdgcn_sched_barrier(0);  // one unit's rows at a time
        }
        fetch(column(tile + 1));
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
            for (int h = 0; h < U::kFrags; ++h) {
                const uint4 a = frags[(k * U::kFrags + h) * 64 + lane];
#pragma unroll
                for (int j = 0; j < U::kCols; ++j) acc[j] = mma(B, a, f[k][j], acc[j]);
            }
        end_sums(B, acc, last);
        uint32_t at = 4 * g * Nb + column(tile);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            buf_store16(ry, at, pack(B, acc, i));
            at += Nb;
        }
    }
}

template <typename T, int KU>
__global__ __launch_bounds__(kThreads, 2) void expand_kernel(AdapterView ad, const float* __restrict__ part, int stride,
                                                             int Q, const T* __restrict__ B, const T* base, T* y,
                                                             float* __restrict__ v_out, int v_stride, int v_cols,
                                                             int N, int scaled, int columns, int tiles,
                                                             int64_t items) {
    __shared__ uint4 frags[KU * Unit<T>::kFrags * 64];
    const size_t slice = static_cast<size_t>(ad.M) * stride;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int cg = static_cast<int>(item % columns);
        const Piece pc = find_piece(ad, 16, static_cast<int>(item / columns));
        if (pc.n == 0) continue;
        const int tile0 = first_tile(cg, tiles, columns), count = first_tile(cg + 1, tiles, columns) - tile0;
        float* vo = cg == 0 ? v_out : nullptr;
        if (pc.rank == 0) {
            without_adapter(pc, base, y, vo, v_stride, v_cols, N, tile0 * kThreads / 4, count * kThreads / 4);
            continue;
        }
        const float scale = scaled ? pc.scale : 1.0f;
        const float* rows = part + static_cast<size_t>(pc.begin) * stride;
        constexpr int R = Unit<T>::kRanks;
        if (KU == 1 || pc.rank <= R)
            expand_body<T, 1>(pc, rows, slice, Q, stride, v_stride, v_cols, B, base, y, vo, N, tile0,
                              count, scale, frags, [] {});
        else if (KU == 2 || pc.rank <= 2 * R)
            expand_body<T, KU < 2 ? KU : 2>(pc, rows, slice, Q, stride, v_stride, v_cols, B, base, y, vo, N, tile0,
                                            count, scale, frags, [] {});
        else if (KU == 4 || pc.rank <= 4 * R)
            expand_body<T, KU < 4 ? KU : 4>(pc, rows, slice, Q, stride, v_stride, v_cols, B, base, y, vo, N, tile0,
                                            count, scale, frags, [] {});
        else
            expand_body<T, KU>(pc, rows, slice, Q, stride, v_stride, v_cols, B, base, y, vo, N, tile0,
                               count, scale, frags, [] {});
    }
}

// Shrink and expand of small batches in one launch: a block makes v of its piece
// for itself, in LDS, and goes on to its columns, so there is one launch in place
// of two (a call of one token is bound by the host) and no v in memory between
// them.  Every block of a piece reads the whole of its adapter's A, at about 25
// bytes a ns, which sets where this holds: the rate of its four waves with four units
// in flight each (blocks of more waves were not tried).  One token of rank 16, 4096 ->
// 14336: 9.3 us, the lookup, four rounds over A, B and the stores one after the other.
template <typename T, int KU>
__global__ __launch_bounds__(kThreads, 2) void one_kernel(
    AdapterView ad, const T* __restrict__ x, const T* __restrict__ A, const T* __restrict__ B, const T* base, T* y,
    float* __restrict__ v_out, int v_stride, int v_cols, int stride, int K, int N, int scaled_v, int scaled_y, Repack v,
    int columns, int tiles, int64_t items) {
    using U = Unit<T>;
    constexpr int MOST = KU * U::kRanks / 16;  // rank tiles, 1 or 2
    __shared__ f32x4 red[kWaves * MOST * 64];
    __shared__ __align__(16) float rows[16 * 16 * MOST];
    __shared__ uint4 frags[KU * U::kFrags * 64];
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int cg = static_cast<int>(item % columns);
        const Piece pc = find_piece(ad, 16, static_cast<int>(item / columns));
        if (pc.n == 0) continue;
        const int tile0 = first_tile(cg, tiles, columns), count = first_tile(cg + 1, tiles, columns) - tile0;
        float* vo = cg == 0 ? v_out : nullptr;
        if (v.from && cg == 0) repack_rows(v, pc.begin, pc.n);
        if (pc.rank == 0) {
            without_adapter(pc, base, y, vo, v_stride, v_cols, N, tile0 * kThreads / 4, count * kThreads / 4);
            continue;
        }
        const float vs = scaled_v ? pc.scale : 1.0f, ys = scaled_y ? pc.scale : 1.0f;
        // MANY units of K in flight, and half the loads of x for up to 8 tokens
        const auto run = [&](auto rt, auto ku) {
            constexpr int RT = decltype(rt)::value, MANY = 4 / RT;
            expand_body<T, decltype(ku)::value>(pc, rows, 0, 1, stride, v_stride, v_cols, B, base, y, vo, N, tile0,
                                                count, ys, frags, [&] {
                                                    if (pc.n <= 8)
                                                        shrink_body<T, RT, MANY, 8>(pc, x, A, rows, K, 1, 0, stride, vs,
                                                                                    red);
                                                    else
                                                        shrink_body<T, RT, MANY, 16>(pc, x, A, rows, K, 1, 0, stride,
                                                                                     vs, red);
                                                });
        };
        if (MOST == 1 || pc.rank <= 16)
            run(Int<1>{}, Int<1>{});
        else
            run(Int<2>{}, Int<KU>{});
    }
}

// OWN of the rows of one rank unit (from `row0` on, in this lane's columns) into
// their places in the operands of the unit's columns, 64 operands apart in LDS.
template <int OWN>
__device__ __forceinline__ void stage_columns(const __bf16*, const uint4 (&rows)[OWN], uint4* unit, int row0) {
    static_assert(OWN % 2 == 0 && OWN <= 8, "whole row pairs of one unit");
    constexpr int P = OWN / 2;
    typedef uint32_t part __attribute__((ext_vector_type(P), aligned(4 * P)));
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t lo[P], hi[P];
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const uint32_t a = (&rows[2 * q].x)[d], b = (&rows[2 * q + 1].x)[d];
            lo[q] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            hi[q] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        }
        uint32_t* l = reinterpret_cast<uint32_t*>(unit + 2 * d * 64) + row0 / 2;
        uint32_t* h = reinterpret_cast<uint32_t*>(unit + (2 * d + 1) * 64) + row0 / 2;
        *reinterpret_cast<part*>(l) = __builtin_bit_cast(part, lo);
        *reinterpret_cast<part*>(h) = __builtin_bit_cast(part, hi);
    }
}
template <int OWN>
__device__ __forceinline__ void stage_columns(const float*, const uint4 (&rows)[OWN], uint4* unit, int row0) {
    constexpr int P = OWN < 4 ? OWN : 4;
    typedef uint32_t part __attribute__((ext_vector_type(P), aligned(4 * P)));
#pragma unroll
    for (int o = 0; o < OWN; o += P)  // OWN = 8: two units
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[P];
#pragma unroll
            for (int q = 0; q < P; ++q) w[q] = (&rows[o + q].x)[j];
            *reinterpret_cast<part*>(reinterpret_cast<uint32_t*>(unit + (o / 4 * 4 + j) * 64) + row0) =
                __builtin_bit_cast(part, w);
        }
}

// The expand of long segments.  One block: 64 tokens, wave w the tokens
// 16 w .. 16 w + 15 with their v in registers, and `tiles` column tiles of 16
// vectors one after the other.  A tile's operands of B are made once for the
// four waves, in LDS, a quarter of its rows by each, while the rows of B of the
// tile after it and the base of the next are in flight: one barrier a tile,
// and registers for four blocks a compute unit.
// Bound by base and y: 4096 tokens, N = 14336, bf16, 235 MB and the factors in 63
// to 65 us, 3.7 TB/s (a copy of the same rows and tiles: 44 to 46).  186 MB are read
// where base, B and the six slices of v are 134: the 14 blocks of a piece lie on all
// eight XCDs, and each XCD fetches the slices for itself.  Beside that the blocks'
// start (v of the piece, the first rows of B) and pieces that a segment's end cuts
// short; deeper prefetch, 8 vectors a tile and other numbers of tiles a block all
// measured within 5%.
template <typename T, int KU>
__device__ __forceinline__ void expand_tile_body(const Piece& pc, const float* part, size_t slice, int Q, int stride,
                                                 const T* B, const T* base, T* y, float* v_out, int v_stride,
                                                 int v_cols, int N, int tile0, int tiles, float scale, uint4* bt) {
    using U = Unit<T>;
    constexpr int GROUP = U::kRanks / 4, BUF = KU * U::kCols * 64;
    constexpr int OWN = KU * U::kLoads / kWaves;  // rows of B that this wave stages
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const uint32_t Nb = static_cast<uint32_t>(N) * sizeof(T);
    const auto rb = make_rsrc(B + static_cast<size_t>(pc.first) * N, static_cast<uint32_t>(pc.rank) * Nb);
    const auto ry = make_rsrc(y + static_cast<size_t>(pc.begin) * N, static_cast<uint32_t>(pc.n) * Nb);
    const auto rs = make_rsrc((base ? base : y) + static_cast<size_t>(pc.begin) * N,
                              base ? static_cast<uint32_t>(pc.n) * Nb : 0u);
    const auto column = [&](int tile) {  // (a row's offset is under 2^31, so kOutside plus it stays outside)
        const uint32_t col = 16u * (static_cast<uint32_t>(tile) * 16 + c);
        return tile < tile0 + tiles && col < Nb ? col : kOutside;
    };
    uint4 rows[OWN], old[4];
    const auto fetch_rows = [&](uint32_t col) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int row = wave * OWN + i;  // of the KU * kLoads that a lane group has
            const int rank = row / U::kLoads * U::kRanks + GROUP * g + row % U::kLoads;
            rows[i] = buf_load16(rb, rank * Nb + col, 0);
        }
    };
    const auto stage_rows = [&](uint4* to) {
        uint4* unit = to + wave * OWN / U::kLoads * U::kCols * 64 + lane;
        stage_columns(B, rows, unit, wave * OWN % U::kLoads);
    };
    const auto fetch_base = [&](uint32_t col, uint4 (&to)[4]) {
        uint32_t at = (16 * wave + 4 * g) * Nb + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            to[i] = buf_load16(rs, at, 0);
            at += Nb;
        }
    };
    fetch_rows(column(tile0));
    fetch_base(column(tile0), old);
    // v of this lane's token, summed over the slices of K in order (columns
    // past the rank are zero there; the stride is a multiple of 8)
    uint4 va[KU][U::kFrags];
    const int m = 16 * wave + c;
    f32x4 v[KU][GROUP / 4];
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int j = 0; j < GROUP / 4; ++j) v[k][j] = f32x4{0, 0, 0, 0};
    const f32x4* from =
        reinterpret_cast<const f32x4*>(part + static_cast<size_t>(pc.begin + min(m, pc.n - 1)) * stride);
    for (int q0 = 0; q0 < Q; q0 += 2) {  // two slices' loads together
        f32x4 w[2][KU][GROUP / 4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int k = 0; k < KU; ++k)
#pragma unroll
                for (int j = 0; j < GROUP / 4; ++j)
                    w[q][k][j] = from[min(q0 + q, Q - 1) * (slice / 4) +
                                      min(k * U::kRanks + GROUP * g, stride - GROUP) / 4 + j];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int k = 0; k < KU; ++k)
#pragma unroll
                for (int j = 0; j < GROUP / 4; ++j)
                    if (q0 + q < Q) v[k][j] += w[q][k][j];
    }
#pragma unroll
    for (int k = 0; k < KU; ++k) {
        const int r = k * U::kRanks + GROUP * g;
        const bool real = m < pc.n && r < stride;
        if (v_out && real)
            for (int j = 0; j < GROUP; ++j)
                if (r + j < v_cols) v_out[static_cast<size_t>(pc.begin + m) * v_stride + r + j] = v[k][j / 4][j % 4];
        float scaled[GROUP];
#pragma unroll
        for (int j = 0; j < GROUP; ++j) scaled[j] = real ? v[k][j / 4][j % 4] * scale : 0.0f;
        rank_operands(B, scaled, va[k]);
    }
    const int past = KU * U::kRanks;  // columns that no unit covers are zero
    if (v_out && past < v_cols)
        for (int i = threadIdx.x; i < pc.n * (v_cols - past); i += kThreads)
            v_out[static_cast<size_t>(pc.begin + i / (v_cols - past)) * v_stride + past + i % (v_cols - past)] = 0.0f;
    __syncthreads();  // the last piece's readers of bt
    stage_rows(bt);
    fetch_rows(column(tile0 + 1));
    int cur = 0;
#pragma unroll 1
    for (int tile = tile0; tile < tile0 + tiles; ++tile) {
        const uint32_t col = column(tile);
        // this tile's operands are in LDS and the other half is free (LDS
        // only: the loads stay in flight across the barrier)
        dev::lds_barrier();
        stage_rows(bt + (cur ^ 1) * BUF);  // rows that had a whole tile's time to come
        fetch_rows(column(tile + 2));
        uint4 next[4];
        fetch_base(column(tile + 1), next);
        f32x4 acc[U::kCols], last[U::kCols];
        start_sums(B, old, acc, last);
        const uint4* bc = bt + cur * BUF + lane;
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
            for (int j = 0; j < U::kCols; ++j) {
                const uint4 f = bc[(k * U::kCols + j) * 64];
#pragma unroll
                for (int h = 0; h < U::kFrags; ++h) acc[j] = mma(B, va[k][h], f, acc[j]);
            }
        end_sums(B, acc, last);
        uint32_t at = (16 * wave + 4 * g) * Nb + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            buf_store16(ry, at, pack(B, acc, i));
            old[i] = next[i];
            at += Nb;
        }
        cur ^= 1;
    }
}

template <typename T, int KU>
__global__ __launch_bounds__(kThreads, KU <= 2 ? 4 : 2) void expand_tile_kernel(
    AdapterView ad, const float* __restrict__ part, int stride, int Q, const T* __restrict__ B, const T* base, T* y,
    float* __restrict__ v_out, int v_stride, int v_cols, int N, int scaled, int columns, int tiles,
    int64_t items) {
    __shared__ uint4 bt[2 * KU * Unit<T>::kCols * 64];
    const size_t slice = static_cast<size_t>(ad.M) * stride;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int cg = static_cast<int>(item % columns);
        const Piece pc = find_piece(ad, 64, static_cast<int>(item / columns));
        if (pc.n == 0) continue;
        const int tile0 = first_tile(cg, tiles, columns), count = first_tile(cg + 1, tiles, columns) - tile0;
        float* vo = cg == 0 ? v_out : nullptr;
        if (pc.rank == 0) {
            without_adapter(pc, base, y, vo, v_stride, v_cols, N, tile0 * 16, count * 16);
            continue;
        }
        const float scale = scaled ? pc.scale : 1.0f;
        constexpr int R = Unit<T>::kRanks;
        if (KU == 1 || pc.rank <= R)
            expand_tile_body<T, 1>(pc, part, slice, Q, stride, B, base, y, vo, v_stride, v_cols, N, tile0,
                                   count, scale, bt);
        else if (KU == 2 || pc.rank <= 2 * R)
            expand_tile_body<T, KU < 2 ? KU : 2>(pc, part, slice, Q, stride, B, base, y, vo, v_stride, v_cols, N, tile0,
                                                 count, scale, bt);
        else if (KU == 4 || pc.rank <= 4 * R)
            expand_tile_body<T, KU < 4 ? KU : 4>(pc, part, slice, Q, stride, B, base, y, vo, v_stride, v_cols, N, tile0,
                                                 count, scale, bt);
        else
            expand_tile_body<T, KU>(pc, part, slice, Q, stride, B, base, y, vo, v_stride, v_cols, N, tile0,
                                    count, scale, bt);
    }
}

// The slices of a shrink joined in order, where no expand does it.
__global__ __launch_bounds__(kThreads) void join_slices_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                               size_t n, int Q) {
    for (size_t i = (static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x) * 4; i < n;
         i += static_cast<size_t>(gridDim.x) * kThreads * 4) {
        f32x4 s = *reinterpret_cast<const f32x4*>(part + i);
        for (int q = 1; q < Q; ++q) s += *reinterpret_cast<const f32x4*>(part + q * n + i);
        *reinterpret_cast<f32x4*>(out + i) = s;
    }
}

// ----------------------------------------------------------------------- outer
// dA and dB in one launch.  A block: one part of an adapter's tokens, up to
// 16 RT of its ranks, 256 bytes of columns.  It lists the adapter's tokens window
// by window in LDS (they may lie in many segments) and gathers their rows of x
// and v, 32 tokens a stage, straight into a ring in LDS.  Wave w turns rank
// tile w of a stage's v into operands, in place and one stage ahead, and takes
// 64 bytes of the columns with all ranks: nothing is added across the waves.
// 8192 tokens of six adapters of ranks up to 64, K = 1280, N = 5120, bf16: 105 MB
// of x and dy in 44 us.  Bound by each block's chain (lookup, listing, first
// gather, stages, stores): the compute units are busy for 31 us of it, in 1.5
// rounds of blocks, the vector instructions for 13.  Blocks of 512 bytes of
// columns, one a compute unit, took 55 with four waves and 47.6 with eight; parts
// cut evenly over all adapters' tokens with several adapters a block 41 here but
// 5 to 18% more with many adapters.
struct OuterJob {
    const float* v;  // [M][v_stride]
    const void* x;
    void* out;       // the gradient, or
    float* partial;  // [slots][max_rank][cols]
    int cols;
    int v_stride;
    int scaled;
    int64_t first_item;
};

constexpr int kWindow = 1024;    // tokens listed at a time, four a thread
constexpr int kOuterStages = 4;  // two blocks' rings, of at most 72 KB with the list, share a compute unit's LDS

template <typename T, int RT>
struct Outer {
    using U = Unit<T>;
    static constexpr int ROWS = U::kLoads;               // tokens of one operand lane
    static constexpr int VT = RT < 2 ? 2 : RT;           // rank tiles staged (whole loads for every wave)
    static constexpr int CT = 4 / sizeof(T);             // column tiles of a wave
    static constexpr int XBYTES = 32 * 256, VBYTES = 32 * 64 * VT, BYTES = XBYTES + VBYTES;
    static constexpr int LX = XBYTES / 1024 / kWaves, LV = VBYTES / 1024 / kWaves, L = LX + LV;

    // LDS places: piece i (16 bytes) of row t is stored at i ^ key, so that the
    // four lane groups of an operand read (rows ROWS apart) and consecutive
    // rows both fall on different banks.
    static __device__ __forceinline__ int x_key(int t) { return 4 * ((t / ROWS) & 3); }
    static __device__ __forceinline__ int v_key(int t) { return 4 * ((t / ROWS + t) & (VT - 1)); }

    // Eight (or twice four) tokens of this lane's rank as operands, in the bytes
    // that they came from: the tile's 128 pieces hold operand h of lane l at
    // number 64 h + l.
    static __device__ __forceinline__ uint4* operand(uint8_t* v, int r, int h, int lane) {
        const int q = 64 * h + lane, t = q >> 2;
        return reinterpret_cast<uint4*>(v + t * 64 * VT + 16 * ((4 * r + (q & 3)) ^ v_key(t)));
    }
    static __device__ __forceinline__ float raw(const uint8_t* v, int r, int t, int c) {
        return *reinterpret_cast<const float*>(v + t * 64 * VT + 16 * ((4 * r + (c >> 2)) ^ v_key(t)) + 4 * (c & 3));
    }
    static __device__ __forceinline__ uint32_t x_word(const uint8_t* x, int t, int w) {
        return *reinterpret_cast<const uint32_t*>(x + t * 256 + 16 * ((w >> 2) ^ x_key(t)) + 4 * (w & 3));
    }
};

// A lane's i-th of the 32 tokens of a stage: 8 in a row (bf16: one product of
// 32), or 4 of each half (float32: two of 16).
template <typename T>
__device__ __forceinline__ int stage_token(int g, int i) {
    return sizeof(T) == 2 ? 8 * g + i : 16 * (i / 4) + 4 * g + i % 4;
}

// v of this lane's rank over its eight tokens -> the two operands of the rank
// tile: hi and lo of all of them (bf16), or the halves as they are (float32).
__device__ __forceinline__ void stage_operands(const __bf16* t, const float (&f)[8], uint4 (&a)[2]) {
    rank_operands(t, f, a);
}
__device__ __forceinline__ void stage_operands(const float*, const float (&f)[8], uint4 (&a)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        a[h] = make_uint4(__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]), __float_as_uint(f[4 * h + 2]),
                          __float_as_uint(f[4 * h + 3]));
}

// One stage into a wave's accumulators: w holds this lane's eight tokens' 4
// bytes of x (two bf16 columns, or one float32), a the rank operands.
template <int RT>
__device__ __forceinline__ void stage_products(const __bf16* t, const uint32_t (&w)[8], const uint4 (&a)[RT][2],
                                               int rank, f32x4 (&acc)[RT][2]) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        lo[q] = __builtin_amdgcn_perm(w[2 * q + 1], w[2 * q], 0x05040100u);
        hi[q] = __builtin_amdgcn_perm(w[2 * q + 1], w[2 * q], 0x07060302u);
    }
    const uint4 f0 = make_uint4(lo[0], lo[1], lo[2], lo[3]), f1 = make_uint4(hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        if (16 * r >= rank) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            acc[r][0] = mma(t, a[r][h], f0, acc[r][0]);
            acc[r][1] = mma(t, a[r][h], f1, acc[r][1]);
        }
    }
}
template <int RT>
__device__ __forceinline__ void stage_products(const float* t, const uint32_t (&w)[8], const uint4 (&a)[RT][2],
                                               int rank, f32x4 (&acc)[RT][1]) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        if (16 * r >= rank) break;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            acc[r][0] = mma(t, a[r][h], make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]), acc[r][0]);
    }
}

template <typename T, int RT>
__global__ __launch_bounds__(kThreads, 2) void outer_kernel(AdapterView ad, OuterJob job0, OuterJob job1,
                                                            int rank_groups, OuterPlan plan, int64_t items) {
    using O = Outer<T, RT>;
    __shared__ __align__(1024) uint8_t ring[kOuterStages * O::BYTES];
    __shared__ int4 tokens[kWindow / 4];
    __shared__ int ends[kThreads], starts[kThreads], wave_sum[kWaves], window_base;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int* token_at = reinterpret_cast<const int*>(tokens);
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const OuterJob& job = it >= job1.first_item ? job1 : job0;
        int64_t item = it - job.first_item;
        const uint32_t row_bytes = static_cast<uint32_t>(job.cols) * sizeof(T), v_bytes = job.v_stride * 4u;
        const int tiles = static_cast<int>((row_bytes + 255) / 256);
        const int tile = static_cast<int>(item % tiles);
        item /= tiles;
        const int r0 = static_cast<int>(item % rank_groups) * 16 * RT;
        const int q = static_cast<int>(item / rank_groups);
        int e = q, part_from = 0, part_to = ad.M, slot = -1;
        if (plan.table) {
            const int* entry = reinterpret_cast<const int*>(plan.table + q);
            e = uniform_load(entry, 0);
            part_from = uniform_load(entry, 1);
            part_to = uniform_load(entry, 2);
            slot = uniform_load(entry, 3);
        }
        if (e < 0) continue;
        int first = 0;
        const int rank = rows_of(ad, e, &first) - r0;
        if (rank <= 0) continue;
        first += r0;
        int listed = 0;  // tokens of the adapter in the segments so far
        // tokens of a window lie within this many rows of its first, so that
        // 32-bit offsets from there reach all of them
        const int reach = static_cast<int>((kOutside - 32) / max(row_bytes, v_bytes));
        f32x4 acc[RT][O::CT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < O::CT; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
        // the adapter's tokens, 256 segments at a time
        for (int s0 = 0; s0 < ad.S; s0 += kThreads) {
            const int s = s0 + threadIdx.x;
            int b = 0, n = 0;
            if (s < ad.S) {
                const int o0 = ad.seg[s], o1 = ad.seg[s + 1], a = ad.seg_adapter[s];
                b = clampi(o0, 0, ad.M);
                n = a == e ? clampi(o1, b, ad.M) - b : 0;
            }
            int sum = n;  // inclusive prefix sum over the block
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int o = __shfl_up(sum, off);
                if (lane >= off) sum = add_capped(sum, o, ad.M);
            }
            const int up = __shfl_up(sum, 1);
            __syncthreads();
            if (lane == 63) wave_sum[wave] = sum;
            __syncthreads();
            int before = 0, total = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (w < wave) before = add_capped(before, wave_sum[w], ad.M);
                total = add_capped(total, wave_sum[w], ad.M);
            }
            const ListRun run = list_run(b, n, add_capped(before, lane > 0 ? up : 0, ad.M), ad.M);
            ends[threadIdx.x] = run.end;
            starts[threadIdx.x] = run.start;
            total = __builtin_amdgcn_readfirstlane(total);
            const int from = max(0, part_from - listed), to = min(total, part_to - listed);
            listed = add_capped(listed, total, ad.M);
            for (int w0 = from; w0 < to;) {
                __syncthreads();
                const int skip = 4 * threadIdx.x, left = to - w0 - skip;
                int t[4] = {-1, -1, -1, -1};
                if (left > 0) {
                    const int at = w0 + skip;
                    int lo = 0, hi = kThreads - 1;  // the first segment whose end is past `at`
                    while (lo < hi) {
                        const int mid = (lo + hi) / 2;
                        if (ends[mid] > at) hi = mid; else lo = mid + 1;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < left) {
                            while (ends[lo] <= at + i) ++lo;  // to <= ends[kThreads - 1]
                            t[i] = starts[lo] + at + i;
                        }
                }
                if (threadIdx.x == 0) window_base = t[0];
                __syncthreads();
                const int base = __builtin_amdgcn_readfirstlane(window_base);
                int have = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    t[i] = t[i] >= base && t[i] - base < reach ? t[i] - base : -1;
                    have += t[i] >= 0;
                }
                tokens[threadIdx.x] = make_int4(t[0], t[1], t[2], t[3]);
#pragma unroll
                for (int off = 32; off > 0; off >>= 1) have += __shfl_xor(have, off);
                if (lane == 0) wave_sum[wave] = have;
                __syncthreads();
                const int count = __builtin_amdgcn_readfirstlane(wave_sum[0] + wave_sum[1] + wave_sum[2] + wave_sum[3]);
                const int64_t rows_left = ad.M - base;
                const auto rx = dev::dma_rsrc(static_cast<const T*>(job.x) + static_cast<size_t>(base) * job.cols,
                                              static_cast<uint32_t>(min(rows_left * row_bytes, int64_t(kOutside) - 16)));
                const auto rv = dev::dma_rsrc(job.v + static_cast<size_t>(base) * job.v_stride,
                                              static_cast<uint32_t>(min(rows_left * v_bytes, int64_t(kOutside) - 16)));
                const uint32_t lds = dev::lds_address(ring);
                constexpr int PIECES = 4 * O::VT;  // of a row of v
                const auto list = [&](int stage, int (&tok)[O::L]) {
#pragma unroll
                    for (int i = 0; i < O::L; ++i) {
                        const int row = i < O::LX ? 4 * (i * kWaves + wave) + (lane >> 4)
                                                  : 64 / PIECES * ((i - O::LX) * kWaves + wave) + lane / PIECES;
                        const int at = 32 * stage + row;
                        tok[i] = at < kWindow ? token_at[at] : -1;
                    }
                };
                const auto issue = [&](const int (&tok)[O::L], int buffer) {
                    const uint32_t xl = lds + buffer * O::BYTES, vl = xl + O::XBYTES;
#pragma unroll
                    for (int i = 0; i < O::LX; ++i) {
                        const int group = i * kWaves + wave, row = 4 * group + (lane >> 4);
                        const uint32_t col = 256u * tile + 16 * ((lane & 15) ^ O::x_key(row));
                        dev::lds_dma16(rx, xl + group * 1024,
                                       tok[i] < 0 || col >= row_bytes ? kOutside : tok[i] * row_bytes + col, 0);
                    }
#pragma unroll
                    for (int i = 0; i < O::LV; ++i) {
                        const int group = i * kWaves + wave, row = 64 / PIECES * group + lane / PIECES;
                        const uint32_t col = 4u * r0 + 16 * ((lane & (PIECES - 1)) ^ O::v_key(row));
                        dev::lds_dma16(rv, vl + group * 1024,
                                       tok[O::LX + i] < 0 ? kOutside : tok[O::LX + i] * v_bytes + col, 0);
                    }
                };
                // raw v of this wave's rank tile, and its operands in its place
                const auto read_v = [&](const uint8_t* v, float (&f)[8]) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = O::raw(v, wave, stage_token<T>(lane >> 4, i), lane & 15);
                };
                const auto write_v = [&](uint8_t* v, float (&f)[8]) {
                    if (16 * wave + (lane & 15) >= rank)
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
                    uint4 a[2];
                    stage_operands(static_cast<const T*>(nullptr), f, a);
                    *O::operand(v, wave, 0, lane) = a[0];
                    *O::operand(v, wave, 1, lane) = a[1];
                };
                const int steps = (min(count, kWindow) + 31) / 32;
                int tok[O::L];
#pragma unroll
                for (int s = 0; s < kOuterStages - 1; ++s) {
                    list(s, tok);
                    issue(tok, s);
                }
                list(kOuterStages - 1, tok);
                dev::dma_stage_barrier<O::L*(kOuterStages - 2)>();
                float f[8];
                if (wave < RT) {
                    read_v(ring + O::XBYTES, f);
                    __builtin_amdgcn_wave_barrier();
                    write_v(ring + O::XBYTES, f);
                }
                // one turn of the ring unrolled: its places are constants (45.0 us,
                // 46.0 with remainders)
                for (int turn = 0; turn < steps; turn += kOuterStages) {
#pragma unroll
                    for (int place = 0; place < kOuterStages; ++place) {
                        const int st = turn + place;
                        if (st >= steps) break;
                        // the next stage has landed and this one's operands are made;
                        // the place of the one before is free
                        dev::dma_stage_barrier<O::L*(kOuterStages - 3)>();
                        const uint8_t* now = ring + place * O::BYTES;
                        uint8_t* ahead = ring + (place + 1) % kOuterStages * O::BYTES + O::XBYTES;
                        // every LDS read of the stage before the loads are issued
                        // (which keep memory accesses on their side)
                        uint32_t w[8];
                        uint4 a[RT][2];
                        if (wave < RT) read_v(ahead, f);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = O::x_word(now, stage_token<T>(lane >> 4, i), 16 * wave + (lane & 15));
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                a[r][h] = *O::operand(const_cast<uint8_t*>(now) + O::XBYTES, r, h, lane);
                        int next[O::L];
                        list(st + kOuterStages, next);
                        issue(tok, (place + kOuterStages - 1) % kOuterStages);
#pragma unroll
                        for (int i = 0; i < O::L; ++i) tok[i] = next[i];
                        if (wave < RT) write_v(ahead, f);
                        stage_products<RT>(static_cast<const T*>(nullptr), w, a, rank, acc);
                    }
                }
                dev::dma_stage_barrier<0>();  // nothing in flight into the ring
                w0 += max(count, 1);
            }
        }
        const float scale = job.scaled ? uniform_load(ad.scale, e) : 1.0f;
        const int c = lane & 15, g = lane >> 4;
        const int col = (256 * tile + 64 * wave) / static_cast<int>(sizeof(T)) + O::CT * c;
        if (col >= job.cols) continue;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 16 * r + 4 * g + i;
                if (j >= rank) continue;
                const size_t at = static_cast<size_t>(first + j) * job.cols + col;
                float* o = job.partial + (static_cast<size_t>(max(slot, 0)) * ad.max_rank + r0 + j) * job.cols + col;
                if constexpr (O::CT == 2) {
                    const float a = acc[r][0][i] * scale, b = acc[r][1][i] * scale;
                    if (slot >= 0)
                        *reinterpret_cast<float2*>(o) = make_float2(a, b);
                    else
                        *reinterpret_cast<uint32_t*>(static_cast<T*>(job.out) + at) = bf16_bits(a) | bf16_bits(b) << 16;
                } else {
                    *(slot >= 0 ? o : static_cast<float*>(job.out) + at) = acc[r][0][i] * scale;
                }
            }
    }
}

// The parts of the adapters that have several joined in order, both gradients,
// four columns a thread.
template <typename T>
__global__ __launch_bounds__(kThreads) void join_parts_kernel(AdapterView ad, OuterJob job0, OuterJob job1,
                                                              OuterPlan plan) {
    const int count = uniform_load(reinterpret_cast<const int*>(plan.multi), 0);
    const int64_t colsA = job0.out ? job0.cols : 0, colsB = job1.out ? job1.cols : 0, quads = (colsA + colsB) / 4;
    const int64_t most = static_cast<int64_t>(count) * ad.max_rank * quads;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; k < most;
         k += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t row = k / quads;
        const int4 m = plan.multi[1 + row / ad.max_rank];
        const int j = static_cast<int>(row % ad.max_rank);
        const int r0 = clampi(ad.row[m.x], 0, ad.R), r1 = clampi(ad.row[m.x + 1], r0, ad.R);
        if (j >= r1 - r0 || m.y == 0) continue;
        const int64_t c = k % quads * 4;
        const bool second = c >= colsA;
        const OuterJob& job = second ? job1 : job0;
        const int64_t col = second ? c - colsA : c;
        const size_t slice = static_cast<size_t>(ad.max_rank) * job.cols;
        const float* part = job.partial + m.z * slice + static_cast<size_t>(j) * job.cols + col;
        T* out = static_cast<T*>(job.out) + static_cast<size_t>(r0 + j) * job.cols + col;
        f32x4 s = *reinterpret_cast<const f32x4*>(part);
        for (int z = 1; z < m.y; ++z) s += *reinterpret_cast<const f32x4*>(part + z * slice);
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<f32x4*>(out) = s;
        else
            *reinterpret_cast<uint2*>(out) =
                make_uint2(bf16_bits(s[0]) | bf16_bits(s[1]) << 16, bf16_bits(s[2]) | bf16_bits(s[3]) << 16);
    }
}

// Zero gradients for a set without adapters.
__global__ __launch_bounds__(kThreads) void zero_kernel(uint4* out, size_t n) {
    for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<size_t>(gridDim.x) * kThreads)
        out[i] = make_uint4(0, 0, 0, 0);
}

// -------------------------------------------------------------------- launches
// Blocks that fill the card (two a compute unit).  A shrink's slices for 512 or
// 1024 blocks, the call in us: 64 requests 26.9 or 28.0, 4096 tokens 80.3 or 82.5,
// gradients of 8192 tokens 98.8 or 103.4 (more partial sums).
constexpr int64_t kFill = 512;

// Tokens up to which the outer products take an adapter whole, without a work
// list, and shrink and expand may be one launch.
constexpr int64_t kWhole = 256;

int esize(int32_t dtype) { return dtype == SS1_BF16 ? 2 : 4; }

// Most slices of a shrink (the workspace's) over `cols` inputs: at least 8 units
// of 128 bytes a block, 8 slices, and no more than fill the card.  At most 4 / 8 /
// 16 (with 4 units), bf16, the call in us: one token 4096 -> 14336 20.4 / 17.8 /
// 17.0, one 14336 -> 4096 13.1 / 12.4 / 13.3, 64 requests 28.2 / 26.9 / 27.0, 512
// tokens 17.9 / 17.3 / 20.5, their gradients 34.6 / 33.8 / 36.3.
int most_slices(int64_t M, int32_t cols, int32_t dtype) {
    const int64_t units = (static_cast<int64_t>(cols) * esize(dtype) + 127) / 128;
    int64_t q = units / 8;
    const int64_t fill = kFill / ((M + 63) / 64 > 0 ? (M + 63) / 64 : 1);
    if (q > fill) q = fill;
    if (q > 8) q = 8;
    return static_cast<int>(q < 1 ? 1 : q);
}

// Whether the batch takes the kernels of 64-token tiles, or those of 16, by the
// mean length of a segment.  2048 tokens of 16 adapters of rank up to 32, K = N =
// 4096, bf16, 16- against 64-token tiles, forward / backward in us: mean length
// 8: 38.8 / 72.8 against 51.9 / 85.6; 16: 29.1 / 59.6 against 32.9 / 64.0; 24:
// 28.5 / 57.0 against 26.8 / 56.7; 96: 25.5 / 55.3 against 23.5 / 54.4.
bool long_segments(int64_t M, int64_t S) { return M > 20 * std::max(S, int64_t(1)); }

// Floats of one token's row of v in the workspace: 16-byte loads of 8 ranks.
int stride_of(int32_t max_rank) { return (max_rank + 7) / 8 * 8; }

unsigned grid_of(int64_t items) { return static_cast<unsigned>(items < kMaxBlocks ? items : kMaxBlocks); }

// Slices of a call's shrink, at most most_slices(): enough blocks to fill the
// card.
int slices_of(const AdapterArgs& a, int K) {
    const int64_t pieces = pieces_of(a.ad.M, a.ad.S, long_segments(a.ad.M, a.ad.S) ? 64 : 16);
    const int64_t Q = kFill / pieces, most = most_slices(a.ad.M, K, a.dtype);
    return static_cast<int>(std::max(int64_t(1), std::min(Q, most)));
}

template <typename T>
int launch_shrink(const AdapterArgs& a, const void* x, const void* A, float* part, int stride, int K, int scaled,
                  const Repack& v, const OuterPlan& plan, hipStream_t s) {
    const bool tile64 = long_segments(a.ad.M, a.ad.S);
    const int Q = slices_of(a, K), rt = (a.ad.max_rank + 15) / 16;
    const int64_t items = pieces_of(a.ad.M, a.ad.S, tile64 ? 64 : 16) * Q;
    auto k = !tile64 ? (rt <= 1 ? shrink_kernel<T, 1> : rt <= 2 ? shrink_kernel<T, 2>
                        : rt <= 4 ? shrink_kernel<T, 4> : shrink_kernel<T, 8>)
                     : (rt <= 1 ? shrink_tile_kernel<T, 1> : rt <= 2 ? shrink_tile_kernel<T, 2>
                        : rt <= 4 ? shrink_tile_kernel<T, 4> : shrink_tile_kernel<T, 8>);
    hipLaunchKernelGGL(k, dim3(grid_of(items) + (plan.table != nullptr)), dim3(kThreads), 0, s, a.ad,
                       static_cast<const T*>(x), static_cast<const T*>(A), part, stride, K, Q, scaled, v, plan, items);
    return Q;
}

// v_out: where the summed v goes too (v_cols columns, rows v_stride apart), or
// null.
template <typename T>
void launch_expand(const AdapterArgs& a, const float* part, int stride, int Q, const void* B, void* y, float* v_out,
                   int v_stride, int v_cols, int N, int scaled, hipStream_t s) {
    const bool tile64 = long_segments(a.ad.M, a.ad.S);
    const int64_t pieces = pieces_of(a.ad.M, a.ad.S, tile64 ? 64 : 16);
    const int wide = (tile64 ? 16 : 64) * Unit<T>::kCols, tiles = (N + wide - 1) / wide;
    // a block takes several column tiles (v is read once) while the card stays
    // full: four at least where that leaves a block a compute unit (gradients of
    // 8192 tokens at K = 1280: 25.8 us with one, 20.7 with two)
    const int64_t work = pieces * tiles;
    const int64_t several = std::max(work / (2 * kFill), std::min(int64_t(4), work / (kFill / 2)));
    const int64_t per = std::max(int64_t(1), std::min(int64_t(tiles), several));
    const int columns = static_cast<int>((tiles + per - 1) / per);
    const int ku = (a.ad.max_rank + Unit<T>::kRanks - 1) / Unit<T>::kRanks;
    constexpr int MOST = sizeof(T) == 2 ? 4 : 8;
    auto k = tile64 ? (ku <= 1 ? expand_tile_kernel<T, 1> : ku <= 2 ? expand_tile_kernel<T, 2>
                       : ku <= 4 ? expand_tile_kernel<T, 4> : expand_tile_kernel<T, MOST>)
                    : (ku <= 1 ? expand_kernel<T, 1> : ku <= 2 ? expand_kernel<T, 2>
                       : ku <= 4 ? expand_kernel<T, 4> : expand_kernel<T, MOST>);
    hipLaunchKernelGGL(k, dim3(grid_of(pieces * columns)), dim3(kThreads), 0, s, a.ad, part, stride, Q,
                       static_cast<const T*>(B), static_cast<const T*>(a.base), static_cast<T*>(y), v_out, v_stride,
                       v_cols, N, scaled, columns, tiles, pieces * columns);
}

// How a call in one launch is split over blocks.
struct OneSplit {
    int64_t pieces;
    int tiles, columns;  // column tiles, and the blocks that share them
};

OneSplit one_split(const AdapterArgs& a, int N) {
    OneSplit o;
    const int wide = kThreads / 4 * 16 / esize(a.dtype);
    o.pieces = pieces_of(a.ad.M, a.ad.S, 16);
    o.tiles = (N + wide - 1) / wide;
    const int64_t per = std::max(int64_t(1), std::min(int64_t(o.tiles), o.pieces * o.tiles / kFill));
    o.columns = static_cast<int>((o.tiles + per - 1) / per);
    return o;
}

// Whether shrink and expand are one launch: an adapter's A is at most 128 KB (bf16;
// float32, whose products take four instructions, 64), which a block's four waves
// read in 5 us, and all blocks' reads of A at most 40 MB.  The host takes 14.1 us for
// a call of one token against 16.7.  On the device alone, one launch against two
// in us, bf16 unless noted: 1 token of rank 8 1024 -> 4096 8.8 / 10.0, 64 tokens of
// rank 32 1280 -> 5120 10.5 / 13.1, 256 requests of rank 16 2048 -> 2048 15.8 /
// 20.7, at 128 KB of A 16 requests of rank 16 4096 -> 4096 11.5 / 11.2 and 8 of rank
// 32 2048 -> 2048 11.3 / 11.1.  Beyond: 256 KB, 1 token of rank 16 8192 -> 8192 15.7
// / 11.0; 70 MB, 64 requests of rank 16 4096 -> 4096 18.5 / 14.9; float32 at 128 KB,
// 256 tokens of rank 16 2048 -> 2048 16.5 / 13.8.
bool one_launch(const AdapterArgs& a, int K, int N) {
    const int64_t factor = static_cast<int64_t>((a.ad.max_rank + 15) / 16 * 16) * K * esize(a.dtype);
    const OneSplit o = one_split(a, N);
    return a.ad.M <= kWhole && a.ad.max_rank <= 32 && factor <= (a.dtype == SS1_BF16 ? 128 : 64) * 1024 &&
           factor * o.pieces * o.columns <= int64_t(40) << 20;
}

template <typename T>
void launch_one(const AdapterArgs& a, const void* x, const void* A, const void* B, void* y, float* v_out, int v_stride,
                int v_cols, int K, int N, int scaled_v, int scaled_y, const Repack& v, hipStream_t s) {
    const OneSplit o = one_split(a, N);
    constexpr int R = Unit<T>::kRanks;
    auto k = a.ad.max_rank <= R ? one_kernel<T, 1> : one_kernel<T, 32 / R>;
    hipLaunchKernelGGL(k, dim3(grid_of(o.pieces * o.columns)), dim3(kThreads), 0, s, a.ad, static_cast<const T*>(x),
                       static_cast<const T*>(A), static_cast<const T*>(B), static_cast<const T*>(a.base),
                       static_cast<T*>(y), v_out, v_stride, v_cols, stride_of(a.ad.max_rank), K, N, scaled_v, scaled_y,
                       v, o.columns, o.tiles, o.pieces * o.columns);
}

template <typename T>
void forward(const AdapterArgs& a, hipStream_t s) {
    float* part = static_cast<float*>(a.workspace);
    const int stride = stride_of(a.ad.max_rank);
    int Q = 1;
    if (a.ad.max_rank > 0 && one_launch(a, a.K, a.N)) {
        launch_one<T>(a, a.x, a.A, a.B, a.y, a.v, a.ad.max_rank, a.ad.max_rank, a.K, a.N, 0, 1, Repack{}, s);
        return;
    }
    if (a.ad.max_rank > 0) {
        // a single slice with rows of v's own length writes v itself
        if (a.v && stride == a.ad.max_rank && slices_of(a, a.K) == 1) part = a.v;
        Q = launch_shrink<T>(a, a.x, a.A, part, stride, a.K, 0, Repack{}, OuterPlan{}, s);
    }
    launch_expand<T>(a, part, stride, Q, a.B, a.y, part == a.v ? nullptr : a.v, a.ad.max_rank, a.ad.max_rank, a.N, 1, s);
}

// How the outer products are split.
struct OuterSplit {
    int RT, rank_groups;
    int P;       // tokens of a part
    int slots;   // partial results at most: every adapter with several parts has under 2 / P of its tokens
    bool table;  // whether some adapter may have several
};

OuterSplit outer_split(int64_t M, int32_t K, int32_t N, int32_t max_rank, int32_t dtype) {
    OuterSplit o;
    const int rt = (max_rank + 15) / 16;
    o.RT = rt <= 1 ? 1 : rt <= 2 ? 2 : 4;
    o.rank_groups = std::max(1, (rt + o.RT - 1) / o.RT);
    // parts enough that all tokens' would fill the card (for 256 / 384 / 512 / 640
    // blocks: 56.8 / 44.6 / 45.0 / 48.4 us at 8192 tokens), of 256 tokens at least
    // (128 / 256 / 512: gradients of 512 tokens 33.5 / 33.8 / 32.4 us, of one
    // adapter 31.6 / 30.6 / 31.6, of 2048 tokens 45.7 / 45.6 / 46.5)
    const int wide = 256 / esize(dtype);
    const int64_t tiles = (K + wide - 1) / wide + (N + wide - 1) / wide;
    const int64_t parts = std::max(int64_t(1), kFill / (tiles * o.rank_groups));
    o.P = static_cast<int>(std::max(kWhole, (M / parts + 31) / 32 * 32));
    o.table = M > o.P;
    o.slots = o.table ? static_cast<int>(2 * M / o.P) : 0;
    return o;
}

// Entries of the work list.
int64_t outer_entries(const OuterSplit& o, int64_t M, int32_t E) { return o.table ? E + M / o.P : E; }

template <typename T>
void zero(void* p, size_t elements, hipStream_t s) {
    const size_t n = elements * sizeof(T) / 16;
    if (n > 0)
        hipLaunchKernelGGL(zero_kernel, dim3(static_cast<unsigned>(n / kThreads < 4096 ? n / kThreads + 1 : 4096)),
                           dim3(kThreads), 0, s, static_cast<uint4*>(p), n);
}

template <typename T>
void launch_outer(const AdapterArgs& a, const OuterSplit& o, const OuterPlan& plan, const float* dv, int dv_stride,
                  const float* v, int v_stride, float* partial, hipStream_t s) {
    if (a.ad.E == 0) {
        if (a.dA) zero<T>(a.dA, static_cast<size_t>(a.ad.R) * a.K, s);
        if (a.dB) zero<T>(a.dB, static_cast<size_t>(a.ad.R) * a.N, s);
        return;
    }
    const auto count = [&](int cols) {
        const int64_t tiles = (static_cast<int64_t>(cols) * sizeof(T) + 255) / 256;
        return tiles * o.rank_groups * outer_entries(o, a.ad.M, a.ad.E);
    };
    const int64_t itemsA = a.dA ? count(a.K) : 0, itemsB = a.dB ? count(a.N) : 0;
    const OuterJob jobA{dv, a.x, a.dA, partial, a.K, dv_stride, 0, 0};
    const OuterJob jobB{v, a.dy, a.dB, partial + static_cast<size_t>(o.slots) * a.ad.max_rank * a.K, a.N, v_stride, 1,
                        itemsA};
    auto k = o.RT == 1 ? outer_kernel<T, 1> : o.RT == 2 ? outer_kernel<T, 2> : outer_kernel<T, 4>;
    hipLaunchKernelGGL(k, dim3(grid_of(itemsA + itemsB)), dim3(kThreads), 0, s, a.ad, jobA, jobB, o.rank_groups, plan,
                       itemsA + itemsB);
    if (o.table)
        hipLaunchKernelGGL((join_parts_kernel<T>), dim3(2048), dim3(kThreads), 0, s, a.ad, jobA, jobB, plan);
}

// Whether v's rows are whole 16-byte pieces.
bool v_in_pieces(int32_t max_rank) { return max_rank % 4 == 0; }

template <typename T>
void backward(const AdapterArgs& a, hipStream_t s) {
    const int stride = stride_of(a.ad.max_rank);
    const size_t rows = static_cast<size_t>(a.ad.M) * stride;
    const int most = most_slices(a.ad.M, a.N, a.dtype);
    const OuterSplit o = outer_split(a.ad.M, a.K, a.N, a.ad.max_rank, a.dtype);
    const int64_t entries = o.table ? outer_entries(o, a.ad.M, a.ad.E) : 0;
    // workspace: the work list, the slices of dv, their sum, v in rows of the
    // stride, the parts of the gradients
    int4* table = static_cast<int4*>(a.workspace);
    float* part = reinterpret_cast<float*>(table + (o.table ? entries + a.ad.E + 1 : 0));
    float* joined = most > 1 ? part + most * rows : part;
    float* packed = joined + rows;
    float* partial = v_in_pieces(a.ad.max_rank) ? packed : packed + rows;
    const bool repack = a.dB && !v_in_pieces(a.ad.max_rank);
    const Repack v{repack ? a.v : nullptr, packed, a.ad.max_rank, stride};
    const bool list = o.table && a.ad.E > 0 && (a.dA || a.dB);
    const OuterPlan plan{list ? table : nullptr, table + entries, o.P, static_cast<int>(entries), o.slots};
    int Q = 1;
    const bool any = a.ad.max_rank > 0 && a.ad.M > 0;
    if (a.dx && any && !list && one_launch(a, a.N, a.K)) {
        launch_one<T>(a, a.dy, a.B, a.A, a.dx, a.dA ? part : nullptr, stride, stride, a.N, a.K, 1, 0, v, s);
        if (a.dA || a.dB)
            launch_outer<T>(a, o, plan, part, stride, repack ? packed : a.v, repack ? stride : a.ad.max_rank, partial, s);
        return;
    }
    if ((a.dx || a.dA) && any) {
        Q = launch_shrink<T>(a, a.dy, a.B, part, stride, a.N, 1, v, plan, s);
    } else if (any) {
        if (repack)
            hipLaunchKernelGGL(repack_kernel, dim3(grid_of((static_cast<int64_t>(a.ad.M) + 15) / 16)), dim3(kThreads),
                               0, s, v, a.ad.M);
        if (list) hipLaunchKernelGGL(plan_outer_kernel, dim3(1), dim3(kThreads), 0, s, a.ad, plan);
    }
    if (a.dx)  // leaves the sum of dv's slices for the outer products
        launch_expand<T>(a, part, stride, Q, a.A, a.dx, Q > 1 && a.dA ? joined : nullptr, stride, stride, a.K, 0, s);
    else if (a.dA && Q > 1)
        hipLaunchKernelGGL(join_slices_kernel,
                           dim3(static_cast<unsigned>(rows / 1024 < 4096 ? rows / 1024 + 1 : 4096)), dim3(kThreads), 0,
                           s, part, joined, rows, Q);
    if (a.dA || a.dB)
        launch_outer<T>(a, o, plan, Q > 1 ? joined : part, stride, repack ? packed : a.v,
                        repack ? stride : a.ad.max_rank, partial, s);
}

}  // namespace

size_t adapter_forward_workspace(int64_t M, int32_t K, int32_t, int32_t, int32_t, int32_t max_rank, int32_t dtype) {
    return static_cast<size_t>(M) * stride_of(max_rank) * sizeof(float) * most_slices(M, K, dtype);
}

size_t adapter_backward_workspace(int64_t M, int32_t K, int32_t N, int32_t E, int32_t, int32_t max_rank,
                                  int32_t dtype) {
    const size_t rows = static_cast<size_t>(M) * stride_of(max_rank) * sizeof(float);
    const int most = most_slices(M, N, dtype);
    const OuterSplit o = outer_split(M, K, N, max_rank, dtype);
    size_t n = rows * ((most > 1 ? most + 1 : 1) + (v_in_pieces(max_rank) ? 0 : 1));
    if (o.table)
        n += static_cast<size_t>(outer_entries(o, M, E) + E + 1) * sizeof(int4) +
             static_cast<size_t>(o.slots) * max_rank * (static_cast<size_t>(K) + N) * sizeof(float);
    return n;
}

ss1_status launch_adapter_forward(const AdapterArgs& a) {
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    if (a.dtype == SS1_F32) forward<float>(a, s); else forward<__bf16>(a, s);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

ss1_status launch_adapter_backward(const AdapterArgs& a) {
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    if (a.dtype == SS1_F32) backward<float>(a, s); else backward<__bf16>(a, s);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace ss1
