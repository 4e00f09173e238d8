// Quantisation to block-scaled E4M3 (ss1_quantize_fp8_blocks): a power-of-two
// scale for 128 elements of a row or for a tile of 128 x 128, along the rows of
// x, along its columns, or both in one pass.
//
// With a power-of-two scale the quotient x / scale is exact, so a code is one
// rounding of its value, and the matrix instructions apply the scale by
// themselves.  The format loses nothing against a free scale: E4M3 keeps the
// same three mantissa bits over 2^-6 .. 448, and the scaled maximum lies in
// (224, 448].
//
// A block takes 128 x 128 elements.  Each 16 lanes hold a row of 128 in
// registers (8 elements a lane), so a row's maximum is four lane exchanges and
// its codes leave as whole 128-byte lines.  For the transposed codes the values
// also go to LDS, from where a thread takes two neighbouring columns and 16
// rows; the codes go back there, so that they too leave as whole lines (44 us of
// kernel for 51 with each thread's bytes stored at once, at the size below).
// Eight waves a block: four took 43.4 us for 41.0 there, and 7.0 for 5.4 where
// there are fewer blocks than compute units (333 x 768 float32); sixteen 45.5.
//
// Bound by memory where x is large: 14336 x 4096 bf16, both ways in tiles (235
// MB), 48 us a call, 4.9 TB/s.  1111 x 1283 float32, both ways, is 6.2 us of
// kernel and 12.0 of the host's time.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_blocks.h"
#include "ss1_model_ops.h"

namespace ss1 {

namespace {

using namespace blocks;

constexpr int kB = SS1_FP8_BLOCK;
constexpr int kThreads = 512;
constexpr int kRowsAPass = kThreads / 16;
constexpr int kPasses = kB / kRowsAPass;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = kB / kWaves;  // of a wave's columns, for the transposed codes
// blocks of a launch: a grid's threads are numbered in 32 bits
constexpr int64_t kMostBlocks = ((int64_t(1) << 32) - 1) / kThreads;

// The scale bytes of a row from its last block to the row's end are 127.
__device__ __forceinline__ void pad_scales(uint8_t* row, int64_t block, int64_t blocks, int64_t cols) {
    if (block == blocks - 1)
        for (int64_t j = blocks; j < cols; ++j) row[j] = 127;
}

// A thread's columns 2p and 2p + 1 of the tile in LDS, kRows rows of them: row i as
// the bits of the two values.
template <typename T>
struct Pairs;

template <>
struct Pairs<uint16_t> {
    uint32_t w[kRows];
    __device__ __forceinline__ void load(const uint16_t* p, int pitch) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + i * pitch);
    }
    __device__ __forceinline__ uint32_t bits(int i, int h) const { return h ? w[i] & 0xFFFF0000u : w[i] << 16; }
    __device__ __forceinline__ void tops(uint32_t (&t)[2]) const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) m = max_halves(m, w[i]);
        t[0] = m << 16;
        t[1] = m & 0xFFFF0000u;
    }
    // codes of rows 4j .. 4j + 3 of column h
    __device__ __forceinline__ uint32_t codes(int j, int h, float scale) const {
        const uint32_t sel = h ? 0x07060302u : 0x05040100u;  // the halves h of two words
        const uint32_t lo = __builtin_amdgcn_perm(w[4 * j + 1], w[4 * j], sel);
        const uint32_t hi = __builtin_amdgcn_perm(w[4 * j + 3], w[4 * j + 2], sel);
        return codes2(hi, scale, codes2(lo, scale, 0, false), true);
    }
};

template <>
struct Pairs<float> {
    uint32_t w[2][kRows];
    __device__ __forceinline__ void load(const float* p, int pitch) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const uint2 v = *reinterpret_cast<const uint2*>(p + i * pitch);
            w[0][i] = v.x;
            w[1][i] = v.y;
        }
    }
    __device__ __forceinline__ uint32_t bits(int i, int h) const { return w[h][i]; }
    __device__ __forceinline__ void tops(uint32_t (&t)[2]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            t[h] = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) t[h] = larger(t[h], w[h][i] & 0x7FFFFFFFu);
        }
    }
    __device__ __forceinline__ uint32_t codes(int j, int h, float scale) const {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[h][4 * j + i]);
        return codes2(v[2], v[3], scale, codes2(v[0], v[1], scale, 0, false), true);
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_blocks_kernel(const T* __restrict__ x, int64_t R, int64_t C,
                                                                   uint32_t col_blocks, uint32_t first, BlocksView q,
                                                                   BlocksView qt) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    T* tile = reinterpret_cast<T*>(smem);  // [128][kPitch], only with qt
    constexpr int kPitch = kB + 16 / static_cast<int>(sizeof(T));
    constexpr int kCodePitch = kB + 16;  // bytes; in the same place
    static_assert(kCodePitch <= kPitch * sizeof(T), "the codes fit into the tile");
    __shared__ uint32_t s_top[kWaves][kB];
    __shared__ uint32_t s_wave[kWaves];
    const int tid = threadIdx.x, l16 = tid & 15;
    const uint32_t block = first + blockIdx.x;
    const int64_t bc = block % col_blocks, br = block / col_blocks;
    const int64_t r0 = br * kB, c0 = bc * kB;

    Eight<T> v[kPasses];
    uint32_t top[kPasses];
    bool special[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t r = r0 + p * kRowsAPass + (tid >> 4);
        v[p].clear();
        if (r < R) v[p].load(x + r * C, c0 + l16 * 8, C);
    }
    uint32_t all = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        top[p] = max16(finite_top(v[p], special[p]));
        all = larger(all, top[p]);
        if (qt.codes) v[p].put(tile + (p * kRowsAPass + (tid >> 4)) * kPitch + l16 * 8);
    }
    const bool whole = q.shift || qt.shift;
    if (whole) {  // the tile's maximum: over the wave's four rows, then the waves
        for (int off = 16; off < 64; off <<= 1)
            all = larger(all, static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), off)));
        if ((tid & 63) == 0) s_wave[tid >> 6] = all;
    }
    if (whole || qt.codes) __syncthreads();
    if (whole) {
        all = s_wave[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) all = larger(all, s_wave[w]);
    }
    if (q.codes) {
        const int64_t blocks = q.code_cols / kB;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int64_t r = r0 + p * kRowsAPass + (tid >> 4);
            if (r >= R) continue;
            const uint32_t byte = scale_byte(q.shift ? all : top[p]);
            *reinterpret_cast<uint2*>(q.codes + r * q.code_cols + c0 + l16 * 8) =
                codes_of(v[p], scale_of(byte), special[p]);
            if (l16 == 0 && (q.shift == 0 || r == r0)) {
                uint8_t* srow = q.scale + (r >> q.shift) * q.scale_cols;
                srow[bc] = static_cast<uint8_t>(byte);
                pad_scales(srow, bc, blocks, q.scale_cols);
            }
        }
    }
    if (!qt.codes) return;
    // columns 2 * pair and 2 * pair + 1, rows kRows * part ..
    const int pair = tid & 63, part = tid >> 6;
    Pairs<T> t;
    t.load(tile + part * kRows * kPitch + 2 * pair, kPitch);
    uint32_t tops[2];
    t.tops(tops);
    const bool odd = larger(tops[0], tops[1]) >= kInf;
    if (odd) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            tops[h] = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) tops[h] = larger(tops[h], finite_size(t.bits(i, h)));
        }
    }
    if (!qt.shift) {
        s_top[part][2 * pair] = tops[0];
        s_top[part][2 * pair + 1] = tops[1];
    }
    __syncthreads();  // the tile is read: the transposed codes take its place
    const int64_t blocks = qt.code_cols / kB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int col = 2 * pair + h;
        const int64_t c = c0 + col;
        uint32_t m = all;
        if (!qt.shift) {
            m = s_top[0][col];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) m = larger(m, s_top[w][col]);
        }
        const uint32_t byte = scale_byte(m);
        const float scale = scale_of(byte);
        uint32_t w[kRows / 4];
#pragma unroll
        for (int j = 0; j < kRows / 4; ++j) w[j] = t.codes(j, h, scale);
        if (odd) {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if ((t.bits(i, h) & 0x7FFFFFFFu) >= kInf) w[i / 4] |= 0x7Fu << (8 * (i & 3));
        }
        uint4* out = reinterpret_cast<uint4*>(smem + col * kCodePitch + part * kRows);
#pragma unroll
        for (int i = 0; i < kRows / 16; ++i) out[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        if (c < C && part == 0 && (qt.shift == 0 || col == 0)) {
            uint8_t* srow = qt.scale + (c >> qt.shift) * qt.scale_cols;
            srow[br] = static_cast<uint8_t>(byte);
            pad_scales(srow, br, blocks, qt.scale_cols);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kB * 8 / kThreads; ++i) {  // 8 lanes a column: whole lines
        const int col = (i * kThreads + tid) >> 3, piece = tid & 7;
        if (c0 + col < C)
            *reinterpret_cast<uint4*>(qt.codes + (c0 + col) * qt.code_cols + r0 + piece * 16) =
                *reinterpret_cast<const uint4*>(smem + col * kCodePitch + piece * 16);
    }
}

template <typename T>
ss1_status launch_t(const QuantizeBlocksArgs& a) {
    const size_t pitch = kB + 16 / sizeof(T);
    const size_t lds = a.qt.codes ? kB * pitch * sizeof(T) : 0;
    auto kern = &quantize_blocks_kernel<T>;
    if (lds > 48 * 1024 && hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                               hipFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(lds)) != hipSuccess)
        return SS1_ERR_HIP;
    const int64_t bc = (a.C + kB - 1) / kB;
    const int64_t br = (a.R + kB - 1) / kB;
    for (int64_t at = 0; at < bc * br; at += kMostBlocks) {
        const int64_t n = bc * br - at < kMostBlocks ? bc * br - at : kMostBlocks;
        hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(n)), dim3(kThreads), lds,
                           static_cast<hipStream_t>(a.stream), static_cast<const T*>(a.x), a.R, a.C,
                           static_cast<uint32_t>(bc), static_cast<uint32_t>(at), a.q, a.qt);
    }
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace

ss1_status launch_quantize_blocks(const QuantizeBlocksArgs& a) {
    return a.dtype == SS1_BF16 ? launch_t<uint16_t>(a) : launch_t<float>(a);
}

}  // namespace ss1
