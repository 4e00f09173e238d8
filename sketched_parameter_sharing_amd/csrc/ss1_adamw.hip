// AdamW over many tensors in one launch (ss1_adamw_step).  Each work item is
// a run of kAdamWChunk elements of one tensor; the tensors' addresses come
// from a table in device memory, so the number of tensors costs nothing.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_ops.h"

namespace ss1 {

namespace {

static_assert(SS1_ADAMW_BLOCK == 256 && kAdamWChunk % SS1_ADAMW_BLOCK == 0, "a block of threads takes a scale block");

// SplitMix64's output for state seed + (counter + 1) golden.
__device__ __forceinline__ uint64_t random_bits(uint64_t seed, uint64_t counter) {
    uint64_t z = seed + (counter + 1) * 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

__device__ __forceinline__ float e4m3_value(uint8_t code) {
    return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(code), 0);
}

// |q| <= 448 (up to a rounding) as an E4M3 value, up or down with the
// probability of its distance: adding 16 random bits below the last kept bit
// and cutting off does that for the normal range (3 mantissa bits: 20 are
// dropped); below 2^-6 the quantum is 2^-9.
__device__ __forceinline__ float e4m3_round(float q, uint32_t u16) {
    const float a = fabsf(q);
    const float high = __uint_as_float((__float_as_uint(a) + (u16 << 4)) & 0xFFF00000u);
    const float low = floorf(__fadd_rn(a * 512.0f, static_cast<float>(u16) * 0x1p-16f)) * 0x1p-9f;
    return copysignf(a < 0x1p-6f ? low : fminf(high, 448.0f), q);
}

__device__ __forceinline__ uint8_t e4m3_code(float v) {
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xFF);
}

__device__ __forceinline__ float block_max(float v, float* red) {
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

__global__ __launch_bounds__(256) void adamw_kernel(const ss1_adamw_entry* __restrict__ entries, int count,
                                                    const int32_t* __restrict__ map, AdamWCoef c) {
    __shared__ float red[4];
    const int item = map[2 * static_cast<size_t>(blockIdx.x)];
    const int64_t part = map[2 * static_cast<size_t>(blockIdx.x) + 1];
    if (item < 0 || item >= count || part < 0) return;
    const ss1_adamw_entry e = entries[item];
    const float keep = static_cast<float>(1.0 - c.lr * static_cast<double>(e.weight_decay));
    const float gs = c.grad_scale_dev ? c.grad_scale * *c.grad_scale_dev : c.grad_scale;
    const bool eight = e.state_dtype == SS1_FP8_E4M3;
    const uint64_t stream = static_cast<uint64_t>(item) << 40;
    const int64_t end = min((part + 1) * kAdamWChunk, e.numel);
    for (int64_t at = part * kAdamWChunk; at < end; at += 256) {
        const int64_t i = at + threadIdx.x;
        const bool in = i < end;
        float g = 0.0f, p = 0.0f, m = 0.0f, v = 0.0f;
        if (in) {
            g = e.grad_dtype == SS1_F32 ? static_cast<const float*>(e.grad)[i]
                                        : static_cast<float>(static_cast<const __bf16*>(e.grad)[i]);
            p = e.master ? e.master[i]
                         : e.param_dtype == SS1_F32 ? static_cast<float*>(e.param)[i]
                                                    : static_cast<float>(static_cast<__bf16*>(e.param)[i]);
            if (eight) {
                m = e4m3_value(static_cast<uint8_t*>(e.m)[i]) * e.m_scale[i / SS1_ADAMW_BLOCK];
                const float r = e4m3_value(static_cast<uint8_t*>(e.v)[i]) * e.v_scale[i / SS1_ADAMW_BLOCK];
                v = r * r;
            } else {
                m = static_cast<float*>(e.m)[i];
                v = static_cast<float*>(e.v)[i];
            }
        }
        g *= gs;
        m = c.beta1 * m + c.one_minus_beta1 * g;
        v = c.beta2 * v + c.one_minus_beta2 * g * g;
        const float r = sqrtf(v);
        p = p * keep - c.step_size * m / (r * c.inv_sqrt_c2 + c.eps);
        if (eight) {
            // the old scales of this block are read by every thread before
            // the first barrier of block_max, and written after it
            const float mt = block_max(fabsf(m), red), rt = block_max(r, red);
            const float ms = mt > 0.0f ? __fdiv_rn(mt, 448.0f) : 1.0f, rs = rt > 0.0f ? __fdiv_rn(rt, 448.0f) : 1.0f;
            if (threadIdx.x == 0) {
                e.m_scale[at / SS1_ADAMW_BLOCK] = ms;
                e.v_scale[at / SS1_ADAMW_BLOCK] = rs;
            }
            if (in) {
                const uint64_t z = random_bits(c.seed, stream + static_cast<uint64_t>(i >> 1)) >> ((i & 1) * 32);
                static_cast<uint8_t*>(e.m)[i] = e4m3_code(e4m3_round(__fdiv_rn(m, ms), z & 0xFFFF));
                float q = e4m3_round(__fdiv_rn(r, rs), (z >> 16) & 0xFFFF);
                if (r > 0.0f) q = fmaxf(q, 0x1p-9f);
                static_cast<uint8_t*>(e.v)[i] = e4m3_code(q);
            }
        } else if (in) {
            static_cast<float*>(e.m)[i] = m;
            static_cast<float*>(e.v)[i] = v;
        }
        if (!in) continue;
        if (e.master) {
            e.master[i] = p;
            static_cast<__bf16*>(e.param)[i] = static_cast<__bf16>(p);
        } else if (e.param_dtype == SS1_F32) {
            static_cast<float*>(e.param)[i] = p;
        } else {
            const uint64_t z = random_bits(c.seed, stream + (uint64_t(1) << 39) + static_cast<uint64_t>(i >> 2)) >>
                               ((i & 3) * 16);
            const uint32_t bits = __float_as_uint(p);
            // adding to an infinity or a NaN would change what it is
            const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
            static_cast<uint16_t*>(e.param)[i] =
                finite ? static_cast<uint16_t>((bits + static_cast<uint32_t>(z & 0xFFFF)) >> 16)
                       : __builtin_bit_cast(uint16_t, static_cast<__bf16>(p));
        }
    }
}

}  // namespace

ss1_status launch_adamw(const ss1_adamw_entry* entries, int32_t count, const int32_t* map, int64_t chunks,
                        const AdamWCoef& coef, void* stream) {
    hipLaunchKernelGGL(adamw_kernel, dim3(static_cast<unsigned>(chunks)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), entries, count, map, coef);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace ss1
