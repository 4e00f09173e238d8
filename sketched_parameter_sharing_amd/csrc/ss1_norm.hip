// Layer norm, forward and backward (ss1_layernorm_forward, _backward).
//
// Forward of a row: mean, then the variance from the differences to it, then
// (x - mean) rstd gamma + beta.  Backward, xh = (x - mean) rstd and
// g = dy gamma: dx = rstd (g - mean(g) - xh mean(g xh)), and column sums of
// dy xh (dgamma) and dy (dbeta).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_ops.h"

namespace ss1 {

namespace {

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __bf16* p) { return static_cast<float>(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__bf16* p, float v) { *p = static_cast<__bf16>(v); }

__device__ __forceinline__ float block_sum(float s, float* red) {
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// One block of 256 threads per row.
template <typename T, typename G>
__global__ __launch_bounds__(256) void layernorm_forward_kernel(const T* __restrict__ x, const G* __restrict__ gamma,
                                                                const G* __restrict__ beta, T* y,
                                                                float* __restrict__ mean, float* __restrict__ rstd,
                                                                int K, float eps) {
    __shared__ float red[4];
    const size_t base = static_cast<size_t>(blockIdx.x) * K;
    float s = 0.0f;
    for (int k = threadIdx.x; k < K; k += 256) s += load_f(x + base + k);
    const float mu = block_sum(s, red) / K;
    float q = 0.0f;
    for (int k = threadIdx.x; k < K; k += 256) {
        const float d = load_f(x + base + k) - mu;
        q += d * d;
    }
    const float rs = 1.0f / sqrtf(block_sum(q, red) / K + eps);
    if (threadIdx.x == 0) {
        if (mean) mean[blockIdx.x] = mu;
        if (rstd) rstd[blockIdx.x] = rs;
    }
    for (int k = threadIdx.x; k < K; k += 256) {
        const float b = beta ? load_f(beta + k) : 0.0f;
        store_f(y + base + k, (load_f(x + base + k) - mu) * rs * load_f(gamma + k) + b);
    }
}

template <typename T, typename G>
__global__ __launch_bounds__(256) void layernorm_dx_kernel(const T* dy, const T* __restrict__ x,
                                                           const G* __restrict__ gamma,
                                                           const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, T* dx, int K) {
    __shared__ float red[4];
    const size_t base = static_cast<size_t>(blockIdx.x) * K;
    const float mu = mean[blockIdx.x], rs = rstd[blockIdx.x];
    float s1 = 0.0f, s2 = 0.0f;
    for (int k = threadIdx.x; k < K; k += 256) {
        const float g = load_f(dy + base + k) * load_f(gamma + k);
        s1 += g;
        s2 += g * ((load_f(x + base + k) - mu) * rs);
    }
    s1 = block_sum(s1, red) / K;
    s2 = block_sum(s2, red) / K;
    for (int k = threadIdx.x; k < K; k += 256) {
        const float g = load_f(dy + base + k) * load_f(gamma + k);
        const float xh = (load_f(x + base + k) - mu) * rs;
        store_f(dx + base + k, rs * (g - s1 - xh * s2));
    }
}

// Partial column sums of one group of rows: partial[group][0][k] of dy xh,
// partial[group][1][k] of dy.
template <typename T>
__global__ __launch_bounds__(256) void layernorm_columns_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                                const float* __restrict__ mean,
                                                                const float* __restrict__ rstd,
                                                                float* __restrict__ partial, int64_t M, int K) {
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= K) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        const size_t at = static_cast<size_t>(m) * K + k;
        const float d = load_f(dy + at);
        dg += d * ((load_f(x + at) - mean[m]) * rstd[m]);
        db += d;
    }
    partial[(static_cast<size_t>(blockIdx.y) * 2) * K + k] = dg;
    partial[(static_cast<size_t>(blockIdx.y) * 2 + 1) * K + k] = db;
}

// The groups' sums joined in order.
template <typename G>
__global__ __launch_bounds__(256) void layernorm_join_kernel(const float* __restrict__ partial, G* __restrict__ dgamma,
                                                             G* __restrict__ dbeta, int groups, int K) {
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= K) return;
    float dg = 0.0f, db = 0.0f;
    for (int p = 0; p < groups; ++p) {
        dg += partial[(static_cast<size_t>(p) * 2) * K + k];
        db += partial[(static_cast<size_t>(p) * 2 + 1) * K + k];
    }
    if (dgamma) store_f(dgamma + k, dg);
    if (dbeta) store_f(dbeta + k, db);
}

int row_groups(int64_t M) { return M < 256 ? static_cast<int>(M) : 256; }

template <typename T, typename G>
void forward(const NormArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((layernorm_forward_kernel<T, G>), dim3(static_cast<unsigned>(a.M)), dim3(256), 0, s,
                       static_cast<const T*>(a.x), static_cast<const G*>(a.gamma), static_cast<const G*>(a.beta),
                       static_cast<T*>(a.y), a.mean, a.rstd, a.K, a.eps);
}

template <typename T, typename G>
void backward(const NormArgs& a, hipStream_t s) {
    const unsigned kb = static_cast<unsigned>((a.K + 255) / 256);
    const int groups = row_groups(a.M);
    // the column sums first: dx may be dy itself
    if (a.dgamma || a.dbeta) {
        if (groups > 0)
            hipLaunchKernelGGL((layernorm_columns_kernel<T>), dim3(kb, static_cast<unsigned>(groups)), dim3(256), 0, s,
                               static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.mean_in, a.rstd_in,
                               a.partial, a.M, a.K);
        hipLaunchKernelGGL((layernorm_join_kernel<G>), dim3(kb), dim3(256), 0, s, a.partial,
                           static_cast<G*>(a.dgamma), static_cast<G*>(a.dbeta), groups, a.K);
    }
    if (a.dx && a.M > 0)
        hipLaunchKernelGGL((layernorm_dx_kernel<T, G>), dim3(static_cast<unsigned>(a.M)), dim3(256), 0, s,
                           static_cast<const T*>(a.dy), static_cast<const T*>(a.x), static_cast<const G*>(a.gamma),
                           a.mean_in, a.rstd_in, static_cast<T*>(a.dx), a.K);
}

}  // namespace

size_t layernorm_backward_workspace(int64_t M, int32_t K) {
    return static_cast<size_t>(row_groups(M)) * 2 * static_cast<size_t>(K) * sizeof(float);
}

ss1_status launch_layernorm_forward(const NormArgs& a) {
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    if (a.dtype == SS1_F32)
        forward<float, float>(a, s);
    else if (a.affine_dtype == SS1_F32)
        forward<__bf16, float>(a, s);
    else
        forward<__bf16, __bf16>(a, s);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

ss1_status launch_layernorm_backward(const NormArgs& a) {
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    if (a.dtype == SS1_F32)
        backward<float, float>(a, s);
    else if (a.affine_dtype == SS1_F32)
        backward<__bf16, float>(a, s);
    else
        backward<__bf16, __bf16>(a, s);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace ss1
