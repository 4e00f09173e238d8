// Device-side building blocks of block-scaled E4M3: reading 8 values of a row,
// the scale of a block and its codes.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace ss1 {
namespace blocks {

constexpr uint32_t kInf = 0x7F800000u;

__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }

// Elements [c, c + 8) of a row that has n; elements from n on are 0.
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* row, int64_t c, int64_t n, float (&v)[8]) {
    if (VEC) {  // n % 8 == 0
        const uint4 r = c < n ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < n ? widen(row[c + i]) : 0.0f;
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int64_t c, int64_t n, float (&v)[8]) {
    if (VEC) {
        const float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4 a = c < n ? *reinterpret_cast<const float4*>(row + c) : z;
        const float4 b = c < n ? *reinterpret_cast<const float4*>(row + c + 4) : z;
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < n ? row[c + i] : 0.0f;
    }
}

// |v| as bits, 0 where it is not finite.
__device__ __forceinline__ uint32_t finite_size(float v) {
    const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
    return u < kInf ? u : 0u;
}

// Scale byte of a block with this largest finite |x| (its bits): the exponent
// of the smallest power of two that brings it to 448 = 1.75 * 2^8 or below.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int b = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return top == 0 ? 127u : static_cast<uint32_t>(b < 1 ? 1 : b);
}
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four values as four codes; an infinity or a NaN as NaN.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    uint32_t w = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, lo, true));
    const float v[4] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((__float_as_uint(v[i]) & 0x7FFFFFFFu) >= kInf) w |= 0x7Fu << (8 * i);
    return w;
}

__device__ __forceinline__ uint32_t max16(uint32_t u) {  // over 16 lanes
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
        const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(u), off));
        u = u > o ? u : o;
    }
    return u;
}

}  // namespace blocks
}  // namespace ss1
