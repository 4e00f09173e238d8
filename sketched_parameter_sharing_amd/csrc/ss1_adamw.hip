// AdamW over many tensors in one launch (ss1_adamw_step).
//
// Each work item is a run of kAdamWChunk elements of one tensor; the tensors'
// addresses come from a table in device memory, so a step over hundreds of
// small tensors is one launch.  A thread takes 8 consecutive elements at a
// time (16-byte loads of bf16 and float, 8-byte loads of codes), so the 256
// elements that share a scale of an 8-bit state are 32 lanes of one wave and
// their maximum is 5 lane exchanges, with no LDS and no barrier.
//
// The step is one pass over the data, bound by HBM: 118M bf16 elements with
// float32 masters, float32 states 28 bytes an element in 665 us (4.97 TB/s, a
// large copy's rate), 8-bit states 16 bytes in 350 us (5.4 TB/s; the vector
// instructions, 85 an element, take about 270).  bf16 elements without masters:
// 22 bytes with float32 states in 497 us (5.2 TB/s), 10 bytes with 8-bit states in
// 295 (4.0 TB/s: the instructions of the two roundings).  400 tensors of 1.5M elements together take
// 12 us, of which about 8 are their 39 MB and the rest one chain of reads: item,
// entry, data.  A block passes once over a chunk: with chunks of 2048 / 4096 /
// 8192 elements the three took 673 / 671 / 699, 459 / 469 / 471 (in the slower
// form with a division an element) and 17.5 / 20.6 / 20.4 us in one process.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_ops.h"

namespace ss1 {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;
static_assert(SS1_ADAMW_BLOCK == 32 * kVec, "32 lanes hold the elements of one scale");
static_assert(kAdamWChunk % (kThreads * kVec) == 0, "a chunk is whole passes of the block");

// SplitMix64: the state of a counter (the next counter's is kGolden further),
// and the output for a state.
constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
__device__ __forceinline__ uint64_t random_state(uint64_t seed, uint64_t counter) {
    return seed + (counter + 1) * kGolden;
}
__device__ __forceinline__ uint64_t random_bits(uint64_t z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// 0 <= a <= 448 (up to a rounding) as an E4M3 value, up or down with the
// probability of its distance (448 for a NaN: quantize8 puts it back).  In the normal range (3 mantissa bits: 20 are
// dropped) adding 16 random bits below the last kept bit and cutting off does
// that; below 2^-6 the quantum is 2^-9.
__device__ __forceinline__ float e4m3_normal(float a, uint32_t u16) {
    return fminf(__uint_as_float((__float_as_uint(a) + (u16 << 4)) & 0xFFF00000u), 448.0f);
}
__device__ __forceinline__ float e4m3_small(float a, uint32_t u16) {
    return floorf(a * 512.0f + static_cast<float>(u16) * 0x1p-16f) * 0x1p-9f;
}

// Elements [i, i + 8) of a tensor as float32; elements from `n` on are 0.
__device__ __forceinline__ void load8(const float* p, int64_t i, int n, float (&v)[kVec]) {
    if (n >= kVec) {
        const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = j < n ? p[i + j] : 0.0f;
    }
}
__device__ __forceinline__ void load8(const uint16_t* p, int64_t i, int n, float (&v)[kVec]) {
    if (n >= kVec) {
        const uint4 r = *reinterpret_cast<const uint4*>(p + i);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = j < n ? __uint_as_float(uint32_t(p[i + j]) << 16) : 0.0f;
    }
}
__device__ __forceinline__ void load8(const uint8_t* p, int64_t i, int n, float (&v)[kVec]) {
    uint32_t w[2] = {0, 0};
    if (n >= kVec) {
        const uint2 r = *reinterpret_cast<const uint2*>(p + i);
        w[0] = r.x;
        w[1] = r.y;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) w[j / 4] |= uint32_t(p[i + j]) << (8 * (j & 3));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v[4 * h] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w[h]), 0);
        v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w[h]), 1);
        v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w[h]), 2);
        v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w[h]), 3);
    }
}

__device__ __forceinline__ void store8(float* p, int64_t i, int n, const float (&v)[kVec]) {
    if (n >= kVec) {
        *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[i + j] = v[j];
    }
}
// 16-bit patterns of 8 values.
__device__ __forceinline__ void store8(uint16_t* p, int64_t i, int n, const uint32_t (&h)[kVec]) {
    if (n >= kVec) {
        *reinterpret_cast<uint4*>(p + i) =
            make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[i + j] = static_cast<uint16_t>(h[j]);
    }
}
// E4M3 codes of 8 values that E4M3 holds exactly.
__device__ __forceinline__ void store8(uint8_t* p, int64_t i, int n, const float (&v)[kVec]) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
        w[h] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], lo, true));
    }
    if (n >= kVec) {
        *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[i + j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j & 3)));
    }
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// The value of lane (l + N) % 16 of the 16-lane row (DPP row_ror, a VALU
// operand modifier).
template <int N>
__device__ __forceinline__ float rotate(float v) {
    return __uint_as_float(static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(__float_as_uint(v)), 0x120 + N, 0xF, 0xF, true)));
}

// The larger one, a NaN where either is (v_maximum3_f32, whose price is v_max3's).
__device__ __forceinline__ float nan_max(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// max over the 32 lanes that share a scale (the half wave): rotations inside
// the 16-lane rows, and one lane exchange between the two rows.
__device__ __forceinline__ float half_wave_max(float v) {
    v = nan_max(v, rotate<8>(v));
    v = nan_max(v, rotate<4>(v));
    v = nan_max(v, rotate<2>(v));
    v = nan_max(v, rotate<1>(v));
    return nan_max(v, __shfl_xor(v, 16));
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// t / scale rounded to nearest, from y = 1 / scale rounded to nearest: the
// remainder of the first quotient is exact, and adding its share rounds as the
// division does (Markstein 1990), while nothing leaves the normal range.
__device__ __forceinline__ float quotient(float t, float scale, float y) {
    const float q = t * y;
    return fmaf(fmaf(-q, scale, t), y, q);
}

// The state's codes of 8 values of this lane, and the new scale of their block:
// max |t| times 1/448 as a float (1 for a block of zeros), the quotients as IEEE
// division gives them.  u[j] holds the random bits of element j.  ROOT: the
// values are square roots, and a nonzero one keeps at least the smallest code.
// E4M3 has a NaN and no infinity: a value that is either becomes its NaN and
// stays out of the maximum, so the rest of the block keeps its scale and codes.
template <bool ROOT>
__device__ __forceinline__ void quantize8(uint8_t* codes, float* scales, int64_t i, int n, const float (&t)[kVec],
                                          const uint32_t (&u)[kVec]) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) top = nan_max(top, fabsf(t[j]));
    top = half_wave_max(top);
    const bool special = !finite(top);  // the same in the 32 lanes
    if (special) {
        top = 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) top = nan_max(top, finite(t[j]) ? fabsf(t[j]) : 0.0f);
        top = half_wave_max(top);
    }
    const float scale = top > 0.0f ? top * (1.0f / 448.0f) : 1.0f;
    if (n > 0 && (threadIdx.x & 31) == 0) scales[i / SS1_ADAMW_BLOCK] = scale;
    float q[kVec];
    // one reciprocal for the 8 values, where their remainders cannot leave the
    // normal range (a value under 2^-25 of the scale rounds to the same code
    // whatever its last bit).  118M elements, in one process: 440 to 456 us with
    // a division each, whose instructions then bound the step, 372 to 401 so
    if (scale >= 0x1p-76f && scale <= 0x1p76f) {
        const float y = __fdiv_rn(1.0f, scale);
#pragma unroll
        for (int j = 0; j < kVec; ++j) q[j] = quotient(t[j], scale, y);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) q[j] = __fdiv_rn(t[j], scale);
    }
    // values under 2^-6 (of 448 at the block's largest) are rare
    bool small = false;
    float r[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const float a = ROOT ? q[j] : fabsf(q[j]);
        small |= a < 0x1p-6f;
        r[j] = e4m3_normal(a, u[j]);
    }
    if (small)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const float a = ROOT ? q[j] : fabsf(q[j]);
            if (a < 0x1p-6f) r[j] = e4m3_small(a, u[j]);
            if (ROOT && t[j] > 0.0f) r[j] = fmaxf(r[j], 0x1p-9f);
        }
    if (special)
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (!finite(t[j])) r[j] = NAN;
    if (!ROOT)
#pragma unroll
        for (int j = 0; j < kVec; ++j) r[j] = copysignf(r[j], t[j]);  // (the short quotient of -0 is +0)
    store8(codes, i, n, r);
}

// sqrt(v) rounded to nearest for 2^-96 <= v < 2^120: one Goldschmidt step on the
// reciprocal root, then the exact remainder (Markstein 1990).  The general form
// also scales v into this range and picks out zeros and infinities.
__device__ __forceinline__ float short_sqrt(float v) {
    const float y = __builtin_amdgcn_rsqf(v);
    float s = v * y, h = 0.5f * y;
    const float e = fmaf(-h, s, 0.5f);
    h = fmaf(h, e, h);
    s = fmaf(s, e, s);
    return fmaf(fmaf(-s, s, v), h, s);
}

// a / b rounded to nearest while b and the quotient are far inside the normal
// range: a Newton step on the reciprocal and two exact remainders.
__device__ __forceinline__ float short_div(float a, float b) {
    float y = __builtin_amdgcn_rcpf(b);
    y = fmaf(fmaf(-b, y, 1.0f), y, y);
    float q = a * y;
    q = fmaf(fmaf(-b, q, a), y, q);
    return fmaf(fmaf(-b, q, a), y, q);
}

enum class Param { F32, Bf16Master, Bf16 };

// One chunk of a tensor.  Products and sums are rounded one by one (no fused
// multiply-add): an 8-bit state turns a last bit of difference into another
// code now and then, and this keeps the codes those of the formula.
template <Param P, typename G, bool EIGHT>
__device__ __forceinline__ void adamw_chunk(const ss1_adamw_entry& e, int item, int64_t begin, const AdamWCoef& c,
                                            float keep, float gs) {
#pragma clang fp contract(off)
    const uint64_t stream = static_cast<uint64_t>(item) << 40;
    // 8-bit states are bound by their instructions; the denominator and the
    // quotient of the short forms stay within 2^-40 and 2^120
    const bool short_forms = c.eps >= 0x1p-40f && c.eps <= 0x1p16f && c.inv_sqrt_c2 <= 0x1p16f && c.step_size <= 0x1p16f;
    const int64_t end = min(begin + kAdamWChunk, e.numel);
    for (int64_t at = begin; at < end; at += kThreads * kVec) {
        const int64_t i = at + kVec * threadIdx.x;
        // elements of this thread; a thread past the end keeps its place in
        // the exchanges of the wave with zeros
        const int n = static_cast<int>(max(int64_t(0), min(int64_t(kVec), end - i)));
        float p[kVec], g[kVec], m[kVec], v[kVec], r[kVec];
        load8(static_cast<const G*>(e.grad), i, n, g);
        if constexpr (P == Param::Bf16Master)
            load8(static_cast<const float*>(e.master), i, n, p);
        else if constexpr (P == Param::F32)
            load8(static_cast<const float*>(e.param), i, n, p);
        else
            load8(static_cast<const uint16_t*>(e.param), i, n, p);
        if constexpr (EIGHT) {
            load8(static_cast<const uint8_t*>(e.m), i, n, m);
            load8(static_cast<const uint8_t*>(e.v), i, n, v);
            const float ms = n > 0 ? e.m_scale[i / SS1_ADAMW_BLOCK] : 0.0f;
            const float vs = n > 0 ? e.v_scale[i / SS1_ADAMW_BLOCK] : 0.0f;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                m[j] *= ms;
                v[j] *= vs;
                v[j] *= v[j];
            }
        } else {
            load8(static_cast<const float*>(e.m), i, n, m);
            load8(static_cast<const float*>(e.v), i, n, v);
        }
        float low = INFINITY, high = 0.0f, most = 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            g[j] *= gs;
            m[j] = c.beta1 * m[j] + c.one_minus_beta1 * g[j];
            v[j] = c.beta2 * v[j] + c.one_minus_beta2 * g[j] * g[j];
            low = fminf(low, v[j]);
            high = fmaxf(high, v[j]);
            most = fmaxf(most, fabsf(m[j]));
        }
        // Short forms of the same bits (every mantissa of both exponent parities
        // for the root, 2^29 drawn quotients, at six exponents each): 118M elements
        // 393 to 418 us without, 366 to 384 with, together with the rare path of
        // small codes.  A NaN leaves the bounds as they are and comes out of
        // either form.
        if (EIGHT && short_forms && low >= 0x1p-96f && high < 0x1p120f && most < 0x1p60f) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                r[j] = short_sqrt(v[j]);
                p[j] = p[j] * keep - short_div(c.step_size * m[j], r[j] * c.inv_sqrt_c2 + c.eps);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                r[j] = sqrtf(v[j]);
                p[j] = p[j] * keep - c.step_size * m[j] / (r[j] * c.inv_sqrt_c2 + c.eps);
            }
        }
        if constexpr (EIGHT) {
            uint32_t um[kVec], uv[kVec];
            uint64_t state = random_state(c.seed, stream + static_cast<uint64_t>(i >> 1));
#pragma unroll
            for (int j = 0; j < kVec; j += 2) {
                const uint64_t z = random_bits(state);
                state += kGolden;
                um[j] = static_cast<uint32_t>(z) & 0xFFFF;
                uv[j] = static_cast<uint32_t>(z) >> 16;
                um[j + 1] = static_cast<uint32_t>(z >> 32) & 0xFFFF;
                uv[j + 1] = static_cast<uint32_t>(z >> 48);
            }
            quantize8<false>(static_cast<uint8_t*>(e.m), e.m_scale, i, n, m, um);
            quantize8<true>(static_cast<uint8_t*>(e.v), e.v_scale, i, n, r, uv);
        } else {
            store8(static_cast<float*>(e.m), i, n, m);
            store8(static_cast<float*>(e.v), i, n, v);
        }
        if constexpr (P == Param::F32) {
            store8(static_cast<float*>(e.param), i, n, p);
        } else {
            uint32_t h[kVec];
            if constexpr (P == Param::Bf16Master) {
                store8(e.master, i, n, p);
#pragma unroll
                for (int j = 0; j < kVec; ++j) h[j] = bf16_bits(p[j]);
            } else {
                uint64_t state = random_state(c.seed, stream + (uint64_t(1) << 39) + static_cast<uint64_t>(i >> 2));
#pragma unroll
                for (int j = 0; j < kVec; j += 4) {
                    const uint64_t z = random_bits(state);
                    state += kGolden;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t bits = __float_as_uint(p[j + q]);
                        // adding to an infinity or a NaN would change what it is
                        const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
                        h[j + q] = finite ? (bits + (static_cast<uint32_t>(z >> (16 * q)) & 0xFFFF)) >> 16
                                          : bf16_bits(p[j + q]);
                    }
                }
            }
            store8(static_cast<uint16_t*>(e.param), i, n, h);
        }
    }
}

__global__ __launch_bounds__(kThreads) void adamw_kernel(const ss1_adamw_entry* __restrict__ entries, int count,
                                                         const int32_t* __restrict__ map, AdamWCoef c) {
    const int item = map[2 * static_cast<size_t>(blockIdx.x)];
    const int64_t part = map[2 * static_cast<size_t>(blockIdx.x) + 1];
    if (item < 0 || item >= count || part < 0) return;
    const ss1_adamw_entry e = entries[item];
    const float keep = static_cast<float>(1.0 - c.lr * static_cast<double>(e.weight_decay));
    const float gs = c.grad_scale_dev ? c.grad_scale * *c.grad_scale_dev : c.grad_scale;
    const int64_t begin = part * kAdamWChunk;
    // one branch a block: every format of a plan in the same launch
    const bool gf = e.grad_dtype == SS1_F32, eight = e.state_dtype == SS1_FP8_E4M3;
#define SS1_CHUNK(P)                                                                     \
    do {                                                                                 \
        if (gf && eight) adamw_chunk<P, float, true>(e, item, begin, c, keep, gs);       \
        else if (gf) adamw_chunk<P, float, false>(e, item, begin, c, keep, gs);          \
        else if (eight) adamw_chunk<P, uint16_t, true>(e, item, begin, c, keep, gs);     \
        else adamw_chunk<P, uint16_t, false>(e, item, begin, c, keep, gs);               \
    } while (0)
    if (e.param_dtype == SS1_F32)
        SS1_CHUNK(Param::F32);
    else if (e.master)
        SS1_CHUNK(Param::Bf16Master);
    else
        SS1_CHUNK(Param::Bf16);
#undef SS1_CHUNK
}

}  // namespace

ss1_status launch_adamw(const ss1_adamw_entry* entries, int32_t count, const int32_t* map, int64_t chunks,
                        const AdamWCoef& coef, void* stream) {
    // the grid's x extent times 256 threads stays under 2^32
    const int64_t most = int64_t(1) << 23;
    for (int64_t at = 0; at < chunks; at += most) {
        const int64_t n = chunks - at < most ? chunks - at : most;
        hipLaunchKernelGGL(adamw_kernel, dim3(static_cast<unsigned>(n)), dim3(kThreads), 0,
                           static_cast<hipStream_t>(stream), entries, count, map + 2 * at, coef);
    }
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace ss1
