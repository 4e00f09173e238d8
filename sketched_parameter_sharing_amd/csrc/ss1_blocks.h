// Device-side building blocks of block-scaled E4M3: eight values of a row as
// they lie in memory, the scale of a block, and codes.
//
// A block's largest |x| is found on the bits (they order like the values), and a
// code is one conversion that takes the block's scale, two values an
// instruction.  Infinities and NaN lie above every finite value in that order,
// so a thread knows from its maximum whether it holds any; only then are they
// left out of the maximum and their codes set to NaN one by one.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace ss1 {
namespace blocks {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any2 __attribute__((aligned(2)));
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kInf = 0x7F800000u;

// max |v| of two bf16 pairs, by halves.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    const u16x2 m = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a & 0x7FFF7FFFu),
                                              __builtin_bit_cast(u16x2, b & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, m);
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
// |v| as bits of float32, 0 where it is not finite.
__device__ __forceinline__ uint32_t finite_size(uint32_t bits) {
    const uint32_t u = bits & 0x7FFFFFFFu;
    return u < kInf ? u : 0u;
}

// Two values over the scale as codes in the low or high half of `to`.
__device__ __forceinline__ uint32_t codes2(uint32_t pair, float scale, uint32_t to, bool high) {
    const s16x2 o = __builtin_bit_cast(s16x2, to);
    const bf16x2 v = __builtin_bit_cast(bf16x2, pair);
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, scale, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, scale, false));
}
__device__ __forceinline__ uint32_t codes2(float a, float b, float scale, uint32_t to, bool high) {
    const s16x2 o = __builtin_bit_cast(s16x2, to);
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, false));
}

// Scale byte of a block with this largest finite |x| (bits of float32): the
// exponent of the smallest power of two that brings it to 448 = 1.75 * 2^8 or
// below; and the scale itself.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const int b = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return top == 0 ? 127u : static_cast<uint32_t>(b < 1 ? 1 : b);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// The maximum over 16 lanes, in each of them (row rotations by 8, 4, 2, 1).
__device__ __forceinline__ uint32_t max16(uint32_t u) {
    u = larger(u, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(u), 0x128, 0xF, 0xF, true)));
    u = larger(u, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(u), 0x124, 0xF, 0xF, true)));
    u = larger(u, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(u), 0x122, 0xF, 0xF, true)));
    u = larger(u, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(u), 0x121, 0xF, 0xF, true)));
    return u;
}

// Columns [c, c + 8) of a row that has n; columns from n on are 0.  Rows of an
// odd width start anywhere: the vectors are not aligned.
template <typename T>
struct Eight;

template <>
struct Eight<uint16_t> {
    u32x4 a;
    __device__ __forceinline__ void load(const uint16_t* row, int64_t c, int64_t n) {
        a = u32x4{0, 0, 0, 0};
        if (c + 8 <= n) {
            a = *reinterpret_cast<const u32x4_any2*>(row + c);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (c + i < n) a[i / 2] |= static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
        }
    }
    __device__ __forceinline__ void clear() { a = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void put(uint16_t* p) const { *reinterpret_cast<u32x4*>(p) = a; }
    __device__ __forceinline__ uint32_t bits(int i) const { return i & 1 ? a[i / 2] & 0xFFFF0000u : a[i / 2] << 16; }
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t m = max_halves(max_halves(a[0], a[1]), max_halves(a[2], a[3]));
        return larger(m & 0xFFFF0000u, m << 16);
    }
    __device__ __forceinline__ uint2 codes(float scale) const {
        return make_uint2(codes2(a[1], scale, codes2(a[0], scale, 0, false), true),
                          codes2(a[3], scale, codes2(a[2], scale, 0, false), true));
    }
};

template <>
struct Eight<float> {
    u32x4 a, b;
    __device__ __forceinline__ void load(const float* row, int64_t c, int64_t n) {
        a = b = u32x4{0, 0, 0, 0};
        if (c + 8 <= n) {
            a = *reinterpret_cast<const u32x4_any4*>(row + c);
            b = *reinterpret_cast<const u32x4_any4*>(row + c + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c + i < n) a[i] = __float_as_uint(row[c + i]);
                if (c + i + 4 < n) b[i] = __float_as_uint(row[c + i + 4]);
            }
        }
    }
    __device__ __forceinline__ void clear() { a = b = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void put(float* p) const {
        *reinterpret_cast<u32x4*>(p) = a;
        *reinterpret_cast<u32x4*>(p + 4) = b;
    }
    __device__ __forceinline__ uint32_t bits(int i) const { return i < 4 ? a[i] : b[i - 4]; }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = larger(m, bits(i) & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ uint2 codes(float scale) const {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(bits(i));
        return make_uint2(codes2(v[2], v[3], scale, codes2(v[0], v[1], scale, 0, false), true),
                          codes2(v[6], v[7], scale, codes2(v[4], v[5], scale, 0, false), true));
    }
};

// The largest finite |v| of eight, and whether any is not finite.
template <typename T>
__device__ __forceinline__ uint32_t finite_top(const Eight<T>& e, bool& special) {
    uint32_t m = e.top();
    special = m >= kInf;
    if (special) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = larger(m, finite_size(e.bits(i)));
    }
    return m;
}
template <typename T>
__device__ __forceinline__ uint2 codes_of(const Eight<T>& e, float scale, bool special) {
    uint2 w = e.codes(scale);
    if (special) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((e.bits(i) & 0x7FFFFFFFu) >= kInf) (i < 4 ? w.x : w.y) |= 0x7Fu << (8 * (i & 3));
    }
    return w;
}

}  // namespace blocks
}  // namespace ss1
