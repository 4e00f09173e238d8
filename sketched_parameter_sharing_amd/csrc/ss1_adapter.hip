// Low-rank adapters of many requests beside a shared projection
// (ss1_adapter_forward, _backward).  With both factors stored rank-major the
// two directions are the same three products: the shrink v = x A^T (and
// dv = dy B^T), the expand y = base + s v B (and dx = dx_base + dv A), and
// the outer product dA = dv^T x (and dB = s v^T dy).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_ops.h"

namespace ss1 {

namespace {

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __bf16* p) { return static_cast<float>(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__bf16* p, float v) { *p = static_cast<__bf16>(v); }

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Largest i in [0, n) with a[i] <= t, for ascending a; -1 when there is none.
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int t) {
    int lo = -1, hi = n;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (a[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// First row and rank of adapter e, inside [0, R) whatever the arrays hold.
__device__ __forceinline__ int rows_of(const AdapterView& ad, int e, int* first) {
    const int r0 = clampi(ad.row[e], 0, ad.R), r1 = clampi(ad.row[e + 1], r0, ad.R);
    *first = r0;
    return min(r1 - r0, ad.max_rank);
}

// The adapter of a token, or -1.
__device__ __forceinline__ int adapter_of(const AdapterView& ad, int m) {
    if (ad.E == 0) return -1;
    const int s = last_at_most(ad.seg, ad.S + 1, m);
    if (s < 0 || s >= ad.S) return -1;
    const int e = ad.seg_adapter[s];
    return e >= 0 && e < ad.E ? e : -1;
}

// One wave per (token, rank row): v[m][j] = x[m] . A[row + j].
template <typename T>
__global__ __launch_bounds__(64) void shrink_kernel(AdapterView ad, const T* __restrict__ x, const T* __restrict__ A,
                                                    float* __restrict__ v, int K, int scaled) {
    const int m = blockIdx.x, j = blockIdx.y;
    const int e = adapter_of(ad, m);
    int first = 0;
    const int rank = e < 0 ? 0 : rows_of(ad, e, &first);
    float s = 0.0f;
    if (j < rank) {
        const size_t xb = static_cast<size_t>(m) * K, ab = static_cast<size_t>(first + j) * K;
        for (int k = threadIdx.x; k < K; k += 64) s += load_f(x + xb + k) * load_f(A + ab + k);
        for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
        if (scaled) s *= ad.scale[e];
    }
    if (threadIdx.x == 0) v[static_cast<size_t>(m) * ad.max_rank + j] = s;
}

// One thread per output: y[m][n] = base[m][n] + s sum_j v[m][j] B[row + j][n].
template <typename T>
__global__ __launch_bounds__(256) void expand_kernel(AdapterView ad, const float* __restrict__ v,
                                                     const T* __restrict__ B, const T* base, T* y, int N,
                                                     int scaled) {
    const int m = blockIdx.x, n = blockIdx.y * 256 + threadIdx.x;
    if (n >= N) return;
    const int e = adapter_of(ad, m);
    int first = 0;
    const int rank = e < 0 ? 0 : rows_of(ad, e, &first);
    float s = 0.0f;
    for (int j = 0; j < rank; ++j)
        s += v[static_cast<size_t>(m) * ad.max_rank + j] * load_f(B + static_cast<size_t>(first + j) * N + n);
    if (scaled && e >= 0) s *= ad.scale[e];
    const size_t at = static_cast<size_t>(m) * N + n;
    store_f(y + at, (base ? load_f(base + at) : 0.0f) + s);
}

// One thread per output: dA[r][k] = sum over the tokens of r's adapter of
// v[m][r - first] x[m][k].
template <typename T>
__global__ __launch_bounds__(256) void outer_kernel(AdapterView ad, const float* __restrict__ v,
                                                    const T* __restrict__ x, T* __restrict__ dA, int K, int scaled) {
    const int r = blockIdx.x, k = blockIdx.y * 256 + threadIdx.x;
    if (k >= K) return;
    float s = 0.0f;
    const int e = ad.E > 0 ? last_at_most(ad.row, ad.E + 1, r) : -1;
    if (e >= 0 && e < ad.E) {
        int first = 0;
        const int rank = rows_of(ad, e, &first);
        if (r - first < rank) {
            for (int i = 0; i < ad.S; ++i) {
                if (ad.seg_adapter[i] != e) continue;
                const int b = clampi(ad.seg[i], 0, ad.M), t = clampi(ad.seg[i + 1], b, ad.M);
                for (int m = b; m < t; ++m)
                    s += v[static_cast<size_t>(m) * ad.max_rank + (r - first)] *
                         load_f(x + static_cast<size_t>(m) * K + k);
            }
            if (scaled) s *= ad.scale[e];
        }
    }
    store_f(dA + static_cast<size_t>(r) * K + k, s);
}

template <typename T>
void forward(const AdapterArgs& a, hipStream_t s) {
    const unsigned M = static_cast<unsigned>(a.ad.M);
    float* v = a.v ? a.v : static_cast<float*>(a.workspace);
    if (a.ad.max_rank > 0)
        hipLaunchKernelGGL((shrink_kernel<T>), dim3(M, static_cast<unsigned>(a.ad.max_rank)), dim3(64), 0, s, a.ad,
                           static_cast<const T*>(a.x), static_cast<const T*>(a.A), v, a.K, 0);
    hipLaunchKernelGGL((expand_kernel<T>), dim3(M, static_cast<unsigned>((a.N + 255) / 256)), dim3(256), 0, s, a.ad,
                       v, static_cast<const T*>(a.B), static_cast<const T*>(a.base), static_cast<T*>(a.y), a.N, 1);
}

template <typename T>
void backward(const AdapterArgs& a, hipStream_t s) {
    const unsigned M = static_cast<unsigned>(a.ad.M), R = static_cast<unsigned>(a.ad.R);
    const unsigned kb = static_cast<unsigned>((a.K + 255) / 256), nb = static_cast<unsigned>((a.N + 255) / 256);
    float* dv = static_cast<float*>(a.workspace);
    if ((a.dx || a.dA) && a.ad.max_rank > 0 && M > 0)
        hipLaunchKernelGGL((shrink_kernel<T>), dim3(M, static_cast<unsigned>(a.ad.max_rank)), dim3(64), 0, s, a.ad,
                           static_cast<const T*>(a.dy), static_cast<const T*>(a.B), dv, a.N, 1);
    if (a.dx)
        hipLaunchKernelGGL((expand_kernel<T>), dim3(M, kb), dim3(256), 0, s, a.ad, dv, static_cast<const T*>(a.A),
                           static_cast<const T*>(a.base), static_cast<T*>(a.dx), a.K, 0);
    if (a.dA)
        hipLaunchKernelGGL((outer_kernel<T>), dim3(R, kb), dim3(256), 0, s, a.ad, dv, static_cast<const T*>(a.x),
                           static_cast<T*>(a.dA), a.K, 0);
    if (a.dB)
        hipLaunchKernelGGL((outer_kernel<T>), dim3(R, nb), dim3(256), 0, s, a.ad, a.v, static_cast<const T*>(a.dy),
                           static_cast<T*>(a.dB), a.N, 1);
}

}  // namespace

size_t adapter_forward_workspace(int64_t M, int32_t, int32_t, int32_t, int32_t max_rank, int32_t) {
    return static_cast<size_t>(M) * static_cast<size_t>(max_rank) * sizeof(float);
}

size_t adapter_backward_workspace(int64_t M, int32_t K, int32_t N, int32_t R, int32_t max_rank, int32_t dtype) {
    return adapter_forward_workspace(M, K, N, R, max_rank, dtype);
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
