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
// also go to LDS, from where a thread takes two neighbouring columns and 32
// rows.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_blocks.h"
#include "ss1_model_ops.h"

namespace ss1 {

namespace {

using namespace blocks;

constexpr int kB = SS1_FP8_BLOCK;
constexpr int kThreads = 256;
constexpr int kRowsAPass = kThreads / 16;
constexpr int kPasses = kB / kRowsAPass;
// The scale bytes of a row from its last block to the row's end are 127.
__device__ __forceinline__ void pad_scales(uint8_t* row, int64_t block, int64_t blocks, int64_t cols) {
    if (block == blocks - 1)
        for (int64_t j = blocks; j < cols; ++j) row[j] = 127;
}

template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void quantize_blocks_kernel(const T* __restrict__ x, int64_t R, int64_t C,
                                                                   uint32_t col_blocks, BlocksView q, BlocksView qt) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    T* tile = reinterpret_cast<T*>(smem);  // [128][128 + pad], only with qt
    constexpr int kPitch = kB + 16 / static_cast<int>(sizeof(T));
    __shared__ uint32_t s_top[4][kB];
    __shared__ uint32_t s_wave[kThreads / 64];
    const int tid = threadIdx.x, l16 = tid & 15;
    const int64_t bc = blockIdx.x % col_blocks, br = blockIdx.x / col_blocks;
    const int64_t r0 = br * kB, c0 = bc * kB;

    float v[kPasses][8];
    uint32_t top[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t r = r0 + p * kRowsAPass + (tid >> 4);
        if (r < R) {
            load8<VEC>(x + r * C, c0 + l16 * 8, C, v[p]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
        }
    }
    uint32_t all = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        uint32_t u = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t f = finite_size(v[p][i]);
            u = u > f ? u : f;
        }
        top[p] = max16(u);
        all = all > top[p] ? all : top[p];
    }
    if (qt.codes) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            T* t = tile + (p * kRowsAPass + (tid >> 4)) * kPitch + l16 * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (sizeof(T) == 2)
                    t[i] = static_cast<uint16_t>(__float_as_uint(v[p][i]) >> 16);
                else
                    t[i] = v[p][i];
            }
        }
    }
    if (q.shift || qt.shift) {  // the tile's maximum: over the wave's four rows, then the waves
        for (int off = 16; off < 64; off <<= 1) {
            const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), off));
            all = all > o ? all : o;
        }
        if ((tid & 63) == 0) s_wave[tid >> 6] = all;
    }
    __syncthreads();
    if (q.shift || qt.shift) {
        all = s_wave[0];
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) all = all > s_wave[w] ? all : s_wave[w];
    }
    const int64_t blocks = q.codes ? q.code_cols / kB : 0;
    if (q.codes) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int64_t r = r0 + p * kRowsAPass + (tid >> 4);
            if (r >= R) continue;
            const uint32_t byte = scale_byte(q.shift ? all : top[p]);
            const float inv = inverse_scale(byte);
            uint2 w;
            w.x = codes4(v[p][0], v[p][1], v[p][2], v[p][3], inv);
            w.y = codes4(v[p][4], v[p][5], v[p][6], v[p][7], inv);
            *reinterpret_cast<uint2*>(q.codes + r * q.code_cols + c0 + l16 * 8) = w;
            if (l16 == 0 && (q.shift == 0 || r == r0)) {
                uint8_t* srow = q.scale + (r >> q.shift) * q.scale_cols;
                srow[bc] = static_cast<uint8_t>(byte);
                pad_scales(srow, bc, blocks, q.scale_cols);
            }
        }
    }
    if (!qt.codes) return;
    // columns 2 * pair and 2 * pair + 1, rows 32 * part ..
    const int pair = tid & 63, part = tid >> 6;
    float lo[32], hi[32];
    uint32_t tl = 0, th = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const T* t = tile + (part * 32 + i) * kPitch + 2 * pair;
        if constexpr (sizeof(T) == 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(t);
            lo[i] = __uint_as_float(w << 16);
            hi[i] = __uint_as_float(w & 0xFFFF0000u);
        } else {
            const float2 w = *reinterpret_cast<const float2*>(t);
            lo[i] = w.x;
            hi[i] = w.y;
        }
        const uint32_t a = finite_size(lo[i]), b = finite_size(hi[i]);
        tl = tl > a ? tl : a;
        th = th > b ? th : b;
    }
    s_top[part][2 * pair] = tl;
    s_top[part][2 * pair + 1] = th;
    __syncthreads();
    const int64_t tblocks = qt.code_cols / kB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int col = 2 * pair + h;
        const int64_t c = c0 + col;
        if (c >= C) continue;
        uint32_t t = all;
        if (!qt.shift) {
            t = s_top[0][col];
#pragma unroll
            for (int w = 1; w < 4; ++w) t = t > s_top[w][col] ? t : s_top[w][col];
        }
        const uint32_t byte = scale_byte(t);
        const float inv = inverse_scale(byte);
        uint4 w[2];
        uint32_t* o = reinterpret_cast<uint32_t*>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = h ? codes4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3], inv)
                     : codes4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3], inv);
        uint4* out = reinterpret_cast<uint4*>(qt.codes + c * qt.code_cols + r0 + part * 32);
        out[0] = w[0];
        out[1] = w[1];
        if (part == 0 && (qt.shift == 0 || col == 0)) {
            uint8_t* srow = qt.scale + (c >> qt.shift) * qt.scale_cols;
            srow[br] = static_cast<uint8_t>(byte);
            pad_scales(srow, br, tblocks, qt.scale_cols);
        }
    }
}

template <typename T>
ss1_status launch_t(const QuantizeBlocksArgs& a) {
    const size_t pitch = kB + 16 / sizeof(T);
    const size_t lds = a.qt.codes ? kB * pitch * sizeof(T) : 0;
    auto kern = a.C % 8 == 0 ? &quantize_blocks_kernel<T, true> : &quantize_blocks_kernel<T, false>;
    if (lds > 48 * 1024 && hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                               hipFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(lds)) != hipSuccess)
        return SS1_ERR_HIP;
    const int64_t bc = (a.C + kB - 1) / kB;
    const int64_t br = (a.R + kB - 1) / kB;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(bc * br)), dim3(kThreads), lds,
                       static_cast<hipStream_t>(a.stream), static_cast<const T*>(a.x), a.R, a.C,
                       static_cast<uint32_t>(bc), a.q, a.qt);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace

ss1_status launch_quantize_blocks(const QuantizeBlocksArgs& a) {
    return a.dtype == SS1_BF16 ? launch_t<uint16_t>(a) : launch_t<float>(a);
}

}  // namespace ss1
