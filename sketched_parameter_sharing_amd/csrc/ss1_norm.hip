// Layer norm, forward and backward (ss1_layernorm_forward, _backward).
//
// Forward of a row: mean, then the variance from the differences to it, then
// (x - mean) rstd gamma + beta.  Backward, xh = (x - mean) rstd and
// g = dy gamma: dx = rstd (g - mean(g) - xh mean(g xh)), and column sums of
// dy xh (dgamma) and dy (dbeta).
//
// Both are one pass over the data, bound by HBM: a row lives in the registers
// of T threads (NV vectors of 8 elements each) between its loads and its
// stores.  The backward pass keeps each thread's columns of dgamma and dbeta
// in registers too while a block walks over its rows, so the column sums cost
// no second read of dy and x: every block writes one partial row, and a small
// second launch adds those in order.  Small inputs take one launch instead, which
// reads dy and x twice.
//
// 16384 x 4096 bf16: forward 55.9 us (269 MB, 4.8 TB/s), backward 79.6 + 4.9 us
// for the join (403 MB, 5.1 TB/s in the first launch), a large copy 5.0 to 5.3.
// float32: 107 us and, in both launches together, 162 (5.0 TB/s).
// 16 x 4096 forward 3.7 us and 1111 x 1283 float32 backward 11.6 us in one launch,
// both below what the host takes for the calls.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_ops.h"

namespace ss1 {

namespace {

constexpr int kVec = 8;

// 16-byte accesses at the alignment of one element: rows of an odd K start
// anywhere, and global memory takes dword accesses of any alignment.
typedef uint32_t u32x4_any2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// Elements [0, n) of p as float32, the rest 0; n is kVec unless TAIL.
template <bool TAIL>
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[kVec]) {
    if (!TAIL || n >= kVec) {
        const f32x4_any a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = j < n ? p[j] : 0.0f;
    }
}
template <bool TAIL>
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&v)[kVec]) {
    if (!TAIL || n >= kVec) {
        const u32x4_any2 r = *reinterpret_cast<const u32x4_any2*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(r[j] << 16);
            v[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = j < n ? __uint_as_float(uint32_t(p[j]) << 16) : 0.0f;
    }
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

template <bool TAIL>
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[kVec]) {
    if (!TAIL || n >= kVec) {
        *reinterpret_cast<f32x4_any*>(p) = f32x4_any{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4_any*>(p + 4) = f32x4_any{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[j] = v[j];
    }
}
template <bool TAIL>
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&v)[kVec]) {
    if (!TAIL || n >= kVec) {
        u32x4_any2 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = bf16_bits(v[2 * j]) | bf16_bits(v[2 * j + 1]) << 16;
        *reinterpret_cast<u32x4_any2*>(p) = r;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (j < n) p[j] = static_cast<uint16_t>(bf16_bits(v[j]));
    }
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(bf16_bits(v)); }

// The value of lane (l + N) % 16 of the 16-lane row (DPP row_ror, a VALU
// operand modifier).
template <int N>
__device__ __forceinline__ float rotate(float v) {
    return __uint_as_float(static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(__float_as_uint(v)), 0x120 + N, 0xF, 0xF, true)));
}

// Sum over the wave, the same bits in every lane (each step adds the same pairs
// in either order): four rotations inside the 16-lane rows and four lane reads,
// no LDS.  With LDS lane exchanges for all six steps the forward of 16384 x 768
// bf16 took 17.1 us instead of 15.9.
__device__ __forceinline__ float wave_sum(float v) {
    v += rotate<8>(v);
    v += rotate<4>(v);
    v += rotate<2>(v);
    v += rotate<1>(v);
    const int w = static_cast<int>(__float_as_uint(v));
    const float a = __uint_as_float(__builtin_amdgcn_readlane(w, 0)), b = __uint_as_float(__builtin_amdgcn_readlane(w, 16));
    const float c = __uint_as_float(__builtin_amdgcn_readlane(w, 32)), d = __uint_as_float(__builtin_amdgcn_readlane(w, 48));
    return (a + b) + (c + d);
}

// Sums over the T threads of a row (T a multiple of 64; a wave or several) of
// one or two values.  Rows of one wave need no LDS.  With several waves every
// thread of the block calls this together; `red` holds one pair a wave and
// alternates between two halves from call to call, so one barrier a call is
// enough: a half is written again only after the barrier of the call between.
template <int T, int BLOCK, bool TWO>
__device__ __forceinline__ float2 row_sums(float2 s, float2* red, int& phase) {
    s.x = wave_sum(s.x);
    if (TWO) s.y = wave_sum(s.y);
    if constexpr (T == 64) return s;
    float2* half = red + phase * (BLOCK / 64);
    phase ^= 1;
    if ((threadIdx.x & 63) == 0) half[threadIdx.x / 64] = s;
    __syncthreads();
    const int first = threadIdx.x / T * (T / 64);
    float2 t = half[first];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) {
        t.x += half[first + w].x;
        if (TWO) t.y += half[first + w].y;
    }
    return t;
}

// ------------------------------------------------------------------- forward
// Elements of this thread's vector i of a row; > 0 when it has any.
__device__ __forceinline__ int count_of(int K, int at) { return min(kVec, K - at); }

// BLOCK / T rows at a time, a row in the registers of T threads.  With KEEP a
// block keeps gamma and beta in registers too, over all of its rows: in float32
// they are twice the bytes of a bf16 row (16384 x 4096 bf16: 60.7 us reading
// them for each row, 55.9 keeping them).
template <typename X, typename G, int T, int NV, int BLOCK, bool TAIL>
__global__ __launch_bounds__(BLOCK) void layernorm_forward_kernel(const X* x, const G* __restrict__ gamma,
                                                                  const G* __restrict__ beta, X* y,
                                                                  float* __restrict__ mean, float* __restrict__ rstd,
                                                                  int64_t M, int K, float eps) {
    __shared__ float2 red[2 * BLOCK / 64];
    constexpr int ROWS = BLOCK / T;
    constexpr bool KEEP = T < 1024;
    const int t = threadIdx.x % T;
    int phase = 0;
    float w[NV][kVec], b[NV][kVec];
    const auto affine = [&](int i) {
        const int at = (i * T + t) * kVec, n = count_of(K, at);
#pragma unroll
        for (int j = 0; j < kVec; ++j) b[i][j] = 0.0f;
        if (n > 0) {
            load8<TAIL>(gamma + at, n, w[i]);
            if (beta) load8<TAIL>(beta + at, n, b[i]);
        }
    };
    if (KEEP)
#pragma unroll
        for (int i = 0; i < NV; ++i) affine(i);
    for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * ROWS; m0 < M; m0 += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t m = m0 + threadIdx.x / T;
        const bool row = m < M;
        const size_t base = static_cast<size_t>(m) * K;
        float v[NV][kVec];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * T + t) * kVec;
            const int n = row ? count_of(K, at) : 0;
            if (n > 0) {
                load8<TAIL>(x + base + at, n, v[i]);
#pragma unroll
                for (int j = 0; j < kVec; ++j) s += v[i][j];
            }
        }
        const float mu = row_sums<T, BLOCK, false>(make_float2(s, 0.0f), red, phase).x / K;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * T + t) * kVec;
            const int n = row ? count_of(K, at) : 0;
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    v[i][j] = !TAIL || j < n ? v[i][j] - mu : 0.0f;
                    q += v[i][j] * v[i][j];
                }
            }
        }
        const float rs = 1.0f / sqrtf(row_sums<T, BLOCK, false>(make_float2(q, 0.0f), red, phase).x / K + eps);
        if (row && t == 0) {
            if (mean) mean[m] = mu;
            if (rstd) rstd[m] = rs;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * T + t) * kVec;
            const int n = row ? count_of(K, at) : 0;
            if (!KEEP) affine(i);
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[i][j] = v[i][j] * rs * w[i][j] + b[i][j];
                store8<TAIL>(y + base + at, n, v[i]);
            }
        }
    }
}

// Rows too long for registers (forward over 32768 elements, backward over 16384):
// one block a row, three passes over it (the later ones from cache), single
// elements.  A rare size, kept simple.
constexpr int kLong = 512;
template <typename X, typename G>
__global__ __launch_bounds__(kLong) void layernorm_forward_long(const X* x, const G* __restrict__ gamma,
                                                                const G* __restrict__ beta, X* y,
                                                                float* __restrict__ mean, float* __restrict__ rstd,
                                                                int64_t M, int K, float eps) {
    __shared__ float2 red[2 * kLong / 64];
    int phase = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const size_t base = static_cast<size_t>(m) * K;
        float s = 0.0f;
        for (int k = threadIdx.x; k < K; k += kLong) s += load1(x + base + k);
        const float mu = row_sums<kLong, kLong, false>(make_float2(s, 0.0f), red, phase).x / K;
        float q = 0.0f;
        for (int k = threadIdx.x; k < K; k += kLong) {
            const float d = load1(x + base + k) - mu;
            q += d * d;
        }
        const float rs = 1.0f / sqrtf(row_sums<kLong, kLong, false>(make_float2(q, 0.0f), red, phase).x / K + eps);
        if (threadIdx.x == 0) {
            if (mean) mean[m] = mu;
            if (rstd) rstd[m] = rs;
        }
        for (int k = threadIdx.x; k < K; k += kLong) {
            const float b = beta ? load1(beta + k) : 0.0f;
            store1(y + base + k, (load1(x + base + k) - mu) * rs * load1(gamma + k) + b);
        }
    }
}

// ------------------------------------------------------------------ backward
// dx of the rows m0 + (thread / T), m0 from `first` on by `step`, and with SUMS
// each thread's sums of dy xh and dy over its rows for its columns.
template <typename X, typename G, int T, int NV, int BLOCK, bool TAIL, bool SUMS>
__device__ __forceinline__ void backward_rows_of(const X* dy, const X* __restrict__ x, const G* __restrict__ gamma,
                                                 const float* __restrict__ mean, const float* __restrict__ rstd, X* dx,
                                                 int64_t M, int K, int64_t first, int64_t step, float2* red,
                                                 float2 (&sum)[NV][kVec]) {
    const int t = threadIdx.x % T, group = threadIdx.x / T;
    int phase = 0;
    float w[NV][kVec];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * T + t) * kVec;
        const int n = count_of(K, at);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            sum[i][j] = make_float2(0.0f, 0.0f);
            w[i][j] = 0.0f;
        }
        if (n > 0) load8<TAIL>(gamma + at, n, w[i]);
    }
    for (int64_t m0 = first; m0 < M; m0 += step) {
        const int64_t m = m0 + group;
        const bool row = m < M;
        const size_t base = static_cast<size_t>(m) * K;
        const float mu = row ? mean[m] : 0.0f, rs = row ? rstd[m] : 0.0f;
        float xh[NV][kVec], g[NV][kVec];
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * T + t) * kVec;
            const int n = row ? count_of(K, at) : 0;
            if (n > 0) {
                load8<TAIL>(x + base + at, n, xh[i]);
                load8<TAIL>(dy + base + at, n, g[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * T + t) * kVec;
            const int n = row ? count_of(K, at) : 0;
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    xh[i][j] = !TAIL || j < n ? (xh[i][j] - mu) * rs : 0.0f;
                    if (SUMS) {
                        sum[i][j].x += g[i][j] * xh[i][j];
                        sum[i][j].y += g[i][j];
                    }
                    g[i][j] *= w[i][j];
                    s.x += g[i][j];
                    s.y += g[i][j] * xh[i][j];
                }
            }
        }
        if (dx) {
            s = row_sums<T, BLOCK, true>(s, red, phase);
            const float m1 = s.x / K, m2 = s.y / K;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int at = (i * T + t) * kVec;
                const int n = row ? count_of(K, at) : 0;
                if (n > 0) {
#pragma unroll
                    for (int j = 0; j < kVec; ++j) g[i][j] = rs * (g[i][j] - m1 - xh[i][j] * m2);
                    store8<TAIL>(dx + base + at, n, g[i]);
                }
            }
        }
    }
}

// Block b takes rows b * ROWS + r, stepping by the grid; the block joins its row
// groups' column sums in LDS, group by group, and writes partial[b][0 or 1][k].
template <typename X, typename G, int T, int NV, int BLOCK, bool TAIL>
__global__ __launch_bounds__(BLOCK) void layernorm_backward_kernel(const X* dy, const X* __restrict__ x,
                                                                   const G* __restrict__ gamma,
                                                                   const float* __restrict__ mean,
                                                                   const float* __restrict__ rstd, X* dx,
                                                                   float* __restrict__ partial, int64_t M, int K) {
    constexpr int ROWS = BLOCK / T;
    __shared__ float2 red[2 * BLOCK / 64];
    __shared__ float2 join[ROWS > 1 ? T * NV * kVec : 1];
    const int t = threadIdx.x % T, group = threadIdx.x / T;
    float2 sum[NV][kVec];  // (dgamma, dbeta) of this thread's columns
    backward_rows_of<X, G, T, NV, BLOCK, TAIL, true>(dy, x, gamma, mean, rstd, dx, M, K,
                                                     static_cast<int64_t>(blockIdx.x) * ROWS,
                                                     static_cast<int64_t>(gridDim.x) * ROWS, red, sum);
    if (!partial) return;
    if constexpr (ROWS > 1) {
        // join[] is laid out [i][j][t]: consecutive threads, consecutive pairs
        for (int r = ROWS - 1; r > 0; --r) {
            if (group == r) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) join[(i * kVec + j) * T + t] = sum[i][j];
            }
            __syncthreads();
            if (group == r - 1) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const float2 o = join[(i * kVec + j) * T + t];
                        sum[i][j].x += o.x;
                        sum[i][j].y += o.y;
                    }
            }
            __syncthreads();
        }
        if (group != 0) return;
    }
    float* out = partial + static_cast<size_t>(blockIdx.x) * 2 * K;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * T + t) * kVec;
        const int n = count_of(K, at);
        if (n > 0) {
            float a[kVec], b[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                a[j] = sum[i][j].x;
                b[j] = sum[i][j].y;
            }
            store8<TAIL>(out + at, n, a);
            store8<TAIL>(out + K + at, n, b);
        }
    }
}

// Both in one launch for small inputs, without partial rows: the first blocks take
// a strip of kStrip vectors of columns over all rows each, the rest a group of
// rows each.  dy and x are read twice, the second time from cache, so dx must be
// apart from them.
constexpr int kStrip = 2;  // 16 columns
template <typename X, typename G, int T, int NV, bool TAIL>
__global__ __launch_bounds__(256) void layernorm_backward_small(const X* dy, const X* __restrict__ x,
                                                                const G* __restrict__ gamma,
                                                                const float* __restrict__ mean,
                                                                const float* __restrict__ rstd, X* dx,
                                                                G* __restrict__ dgamma, G* __restrict__ dbeta, int M,
                                                                int K, int strips) {
    constexpr int WAVES = 4, ROWS = 256 / kStrip;
    __shared__ float2 red[2 * WAVES];
    __shared__ float2 join[WAVES][kStrip * kVec];
    if (static_cast<int>(blockIdx.x) >= strips) {
        float2 none[NV][kVec];
        const int64_t at = static_cast<int64_t>(blockIdx.x - strips) * (256 / T);
        backward_rows_of<X, G, T, NV, 256, TAIL, false>(dy, x, gamma, mean, rstd, dx, M, K, at, M, red, none);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, vec = lane % kStrip;
    const int at = (static_cast<int>(blockIdx.x) * kStrip + vec) * kVec, n = count_of(K, at);
    float2 sum[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum[j] = make_float2(0.0f, 0.0f);
    if (n > 0) {
#pragma unroll 4
        for (int m = threadIdx.x / kStrip; m < M; m += ROWS) {
            const size_t o = static_cast<size_t>(m) * K + at;
            const float mu = mean[m], rs = rstd[m];
            float a[kVec], g[kVec];
            load8<TAIL>(x + o, n, a);
            load8<TAIL>(dy + o, n, g);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                sum[j].x += g[j] * ((a[j] - mu) * rs);
                sum[j].y += g[j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
#pragma unroll
        for (int off = kStrip; off < 64; off <<= 1) {
            sum[j].x += __shfl_xor(sum[j].x, off);
            sum[j].y += __shfl_xor(sum[j].y, off);
        }
        if (lane < kStrip) join[wave][vec * kVec + j] = sum[j];
    }
    __syncthreads();
    const int k = static_cast<int>(blockIdx.x) * kStrip * kVec + threadIdx.x;
    if (threadIdx.x < kStrip * kVec && k < K) {
        float2 s = join[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            s.x += join[w][threadIdx.x].x;
            s.y += join[w][threadIdx.x].y;
        }
        if (dgamma) store1(dgamma + k, s.x);
        if (dbeta) store1(dbeta + k, s.y);
    }
}

// Rows too long for registers: dx of one row a block.
template <typename X, typename G>
__global__ __launch_bounds__(kLong) void layernorm_dx_long(const X* dy, const X* __restrict__ x,
                                                           const G* __restrict__ gamma,
                                                           const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, X* dx, int64_t M, int K) {
    __shared__ float2 red[2 * kLong / 64];
    int phase = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const size_t base = static_cast<size_t>(m) * K;
        const float mu = mean[m], rs = rstd[m];
        float2 s = make_float2(0.0f, 0.0f);
        for (int k = threadIdx.x; k < K; k += kLong) {
            const float g = load1(dy + base + k) * load1(gamma + k);
            s.x += g;
            s.y += g * ((load1(x + base + k) - mu) * rs);
        }
        s = row_sums<kLong, kLong, true>(s, red, phase);
        const float m1 = s.x / K, m2 = s.y / K;
        for (int k = threadIdx.x; k < K; k += kLong) {
            const float g = load1(dy + base + k) * load1(gamma + k);
            const float xh = (load1(x + base + k) - mu) * rs;
            store1(dx + base + k, rs * (g - m1 - xh * m2));
        }
    }
}

// ... and their partial column sums: one thread a column, rows of one group.
template <typename X>
__global__ __launch_bounds__(256) void layernorm_columns_long(const X* __restrict__ dy, const X* __restrict__ x,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd,
                                                              float* __restrict__ partial, int64_t M, int K) {
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= K) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        const size_t at = static_cast<size_t>(m) * K + k;
        const float d = load1(dy + at);
        dg += d * ((load1(x + at) - mean[m]) * rstd[m]);
        db += d;
    }
    float* out = partial + static_cast<size_t>(blockIdx.y) * 2 * K;
    out[k] = dg;
    out[K + k] = db;
}

// The partial rows joined in a fixed order: a block takes 32 columns of the
// [groups][2 K] matrix, thread (c, r) the rows r, r + 8, ...  Bound by latency: 8
// MB (K = 4096) in 4.9 us, most of it the launch and one chain of 32 loads.
template <typename G>
__global__ __launch_bounds__(256) void layernorm_join_kernel(const float* __restrict__ partial, G* __restrict__ dgamma,
                                                             G* __restrict__ dbeta, int groups, int K) {
    __shared__ float part[8][32];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int64_t wide = 2 * static_cast<int64_t>(K);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 32 + c;
    float s = 0.0f;
    if (at < wide) {
#pragma unroll 16
        for (int p = r; p < groups; p += 8) s += partial[p * wide + at];
    }
    part[r][c] = s;
    __syncthreads();
    if (r == 0 && at < wide) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][c];
        if (at < K) {
            if (dgamma) store1(dgamma + at, s);
        } else if (dbeta) {
            store1(dbeta + (at - K), s);
        }
    }
}

// ------------------------------------------------------------------ launches
constexpr int64_t kMaxBlocks = int64_t(1) << 20;  // rows beyond that loop

unsigned grid_for(int64_t rows, int64_t most) { return static_cast<unsigned>(rows < most ? rows : most); }

// Blocks of the forward where they keep gamma and beta: enough to fill the card
// and to even out, few enough that each has many rows.  16384 x 4096 (blocks of
// 256): 62.5 us with 2048, 55.9 with 4096, 66.5 with one a row; 4096 x 16384
// (blocks of 512, four vectors a thread): 70.4 with 2048, 65.4 with 1024, 61.8
// with 512.
constexpr int64_t keep_blocks(int block, int nv) { return nv == 4 ? 512 : int64_t(4096) * 256 / block; }

template <typename X, typename G, int T, int NV>
void forward_rows(const NormArgs& a, hipStream_t s) {
    constexpr int BLOCK = T < 256 ? 256 : T;
    const int64_t groups = (a.M + BLOCK / T - 1) / (BLOCK / T);
    const dim3 grid(grid_for(groups, T < 1024 ? keep_blocks(BLOCK, NV) : kMaxBlocks));
    auto k = a.K % kVec ? layernorm_forward_kernel<X, G, T, NV, BLOCK, true>
                        : layernorm_forward_kernel<X, G, T, NV, BLOCK, false>;
    hipLaunchKernelGGL(k, grid, dim3(BLOCK), 0, s, static_cast<const X*>(a.x), static_cast<const G*>(a.gamma),
                       static_cast<const G*>(a.beta), static_cast<X*>(a.y), a.mean, a.rstd, a.M, a.K, a.eps);
}

// Threads a row: one wave up to 1024 elements (no barrier; 16384 x 768: 15.9 us
// against 25.2 with 256 threads), then 256 and 512 with up to two vectors each
// (8192 x 8192: 59.5 us with 512 x 2, 78.1 with 256 x 4), then 512 x 4 (4096 x
// 16384: 61.8 us, 74.9 with 1024 x 2) and 1024 x 4.
template <typename X, typename G>
void forward(const NormArgs& a, hipStream_t s) {
    const int vecs = (a.K + kVec - 1) / kVec;
    if (vecs <= 64) return forward_rows<X, G, 64, 1>(a, s);
    if (vecs <= 128) return forward_rows<X, G, 64, 2>(a, s);
    if (vecs <= 256) return forward_rows<X, G, 256, 1>(a, s);
    if (vecs <= 512) return forward_rows<X, G, 256, 2>(a, s);
    if (vecs <= 1024) return forward_rows<X, G, 512, 2>(a, s);
    if (vecs <= 2048) return forward_rows<X, G, 512, 4>(a, s);
    if (vecs <= 4096) return forward_rows<X, G, 1024, 4>(a, s);
    hipLaunchKernelGGL((layernorm_forward_long<X, G>), dim3(grid_for(a.M, kMaxBlocks)), dim3(kLong), 0, s,
                       static_cast<const X*>(a.x), static_cast<const G*>(a.gamma), static_cast<const G*>(a.beta),
                       static_cast<X*>(a.y), a.mean, a.rstd, a.M, a.K, a.eps);
}

// Rows and elements up to which the backward pass is one launch, by the time of a
// call that the host makes: there a strip's block of four waves reads its columns,
// at about 25 bytes a ns, in the host's time for the two launches.  Where the device
// alone counts (a captured graph, a queue that runs ahead) two launches are mostly
// ahead from 1024 rows on.  A call as the host makes it, one launch against two, in us,
// bf16 / float32: 512 x 768 14.8 / 14.4 against 18.2 / 18.4, 1024 x 4096 15.6 / 18.3
// against 18.2 / 18.0, 1280 x 1283 15.1 / 14.1 against 18.1 / 18.2, 1280 x 4096 18.3 /
// 22.2 against 18.5 / 20.6, 2048 x 2048 17.3 / 23.6 against 18.2.  On the device
// alone: 512 x 4096 12.5 / 14.4 against 16.3 / 16.2, 1024 x 768 10.5 / 14.6 against
// 11.5 / 11.4, 1024 x 4096 19.2 / 21.6 against 18.3 / 19.9.
constexpr int64_t kSmallRows = 1280, kSmallElements = int64_t(4) << 20;

// How the backward pass splits the rows.
struct Split {
    int T;       // threads a row, 0: too long for registers
    int block;   // threads a block
    int groups;  // blocks, and partial rows
};

// One block a compute unit.  128 / 256 / 512, backward in us: 16384 x 4096: 132 /
// 86 / 93; 16384 x 768: 32.5 / 26 / 33.5; 4096 x 8192: 82 / 53 / 54.
constexpr int kGroups = 256;

Split split_of(int64_t M, int32_t K) {
    const int vecs = (K + kVec - 1) / kVec;
    Split p;
    p.T = vecs <= 128 ? 64 : vecs <= 512 ? 256 : vecs <= 2048 ? 1024 : 0;
    if (p.T == 0) {
        p.block = kLong;
        p.groups = static_cast<int>(M < kGroups ? M : kGroups);
        return p;
    }
    // small row counts take small blocks, so that they still spread out (512 x
    // 768: 10.8 us against 14.8; 16384 x 768 the other way: 36 against 26)
    p.block = p.T == 1024 || M >= int64_t(kGroups) * (1024 / p.T) ? 1024 : 256;
    const int64_t need = (M + p.block / p.T - 1) / (p.block / p.T);
    p.groups = static_cast<int>(need < kGroups ? need : kGroups);
    return p;
}

template <typename X, typename G, int T, int NV, int BLOCK>
void backward_rows(const NormArgs& a, int groups, float* partial, hipStream_t s) {
    auto k = a.K % kVec ? layernorm_backward_kernel<X, G, T, NV, BLOCK, true>
                        : layernorm_backward_kernel<X, G, T, NV, BLOCK, false>;
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(groups)), dim3(BLOCK), 0, s, static_cast<const X*>(a.dy),
                       static_cast<const X*>(a.x), static_cast<const G*>(a.gamma), a.mean_in, a.rstd_in,
                       static_cast<X*>(a.dx), partial, a.M, a.K);
}

template <typename X, typename G, int T, int NV>
void backward_small(const NormArgs& a, hipStream_t s) {
    const int strips = a.dgamma || a.dbeta ? (a.K + kStrip * kVec - 1) / (kStrip * kVec) : 0;
    const int64_t rows = a.dx ? (a.M + 256 / T - 1) / (256 / T) : 0;
    auto k = a.K % kVec ? layernorm_backward_small<X, G, T, NV, true> : layernorm_backward_small<X, G, T, NV, false>;
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(strips + rows)), dim3(256), 0, s, static_cast<const X*>(a.dy),
                       static_cast<const X*>(a.x), static_cast<const G*>(a.gamma), a.mean_in, a.rstd_in,
                       static_cast<X*>(a.dx), static_cast<G*>(a.dgamma), static_cast<G*>(a.dbeta),
                       static_cast<int>(a.M), a.K, strips);
}

// Whether two [M][K] arrays share memory.
bool overlap(const void* a, const void* b, size_t bytes) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + bytes && q < p + bytes;
}

template <typename X>
bool is_small(const NormArgs& a) {
    const size_t bytes = static_cast<size_t>(a.M) * a.K * sizeof(X);
    return a.M > 0 && a.M <= kSmallRows && a.M * a.K <= kSmallElements && a.K <= 4096 &&
           !(a.dx && (overlap(a.dx, a.dy, bytes) || overlap(a.dx, a.x, bytes)));
}

template <typename X, typename G>
void backward(const NormArgs& a, hipStream_t s) {
    const Split p = split_of(a.M, a.K);
    const bool sums = a.dgamma || a.dbeta;
    if (is_small<X>(a)) {
        const int vecs = (a.K + kVec - 1) / kVec;
        return vecs <= 64    ? backward_small<X, G, 64, 1>(a, s)
               : vecs <= 128 ? backward_small<X, G, 64, 2>(a, s)
               : vecs <= 256 ? backward_small<X, G, 256, 1>(a, s)
                             : backward_small<X, G, 256, 2>(a, s);
    }
    float* partial = sums ? a.partial : nullptr;
    if (a.M > 0 && p.T == 0) {
        // the column sums first: dx may be dy itself
        if (sums)
            hipLaunchKernelGGL((layernorm_columns_long<X>),
                               dim3(static_cast<unsigned>((a.K + 255) / 256), static_cast<unsigned>(p.groups)),
                               dim3(256), 0, s, static_cast<const X*>(a.dy), static_cast<const X*>(a.x), a.mean_in,
                               a.rstd_in, partial, a.M, a.K);
        if (a.dx)
            hipLaunchKernelGGL((layernorm_dx_long<X, G>), dim3(grid_for(a.M, kMaxBlocks)), dim3(kLong), 0, s,
                               static_cast<const X*>(a.dy), static_cast<const X*>(a.x),
                               static_cast<const G*>(a.gamma), a.mean_in, a.rstd_in, static_cast<X*>(a.dx), a.M, a.K);
    } else if (a.M > 0) {
        const int vecs = (a.K + kVec - 1) / kVec;
        if (p.T == 64 && vecs <= 64)
            p.block == 256 ? backward_rows<X, G, 64, 1, 256>(a, p.groups, partial, s)
                           : backward_rows<X, G, 64, 1, 1024>(a, p.groups, partial, s);
        else if (p.T == 64)
            p.block == 256 ? backward_rows<X, G, 64, 2, 256>(a, p.groups, partial, s)
                           : backward_rows<X, G, 64, 2, 1024>(a, p.groups, partial, s);
        else if (p.T == 256 && vecs <= 256)
            p.block == 256 ? backward_rows<X, G, 256, 1, 256>(a, p.groups, partial, s)
                           : backward_rows<X, G, 256, 1, 1024>(a, p.groups, partial, s);
        else if (p.T == 256)
            p.block == 256 ? backward_rows<X, G, 256, 2, 256>(a, p.groups, partial, s)
                           : backward_rows<X, G, 256, 2, 1024>(a, p.groups, partial, s);
        else if (vecs <= 1024)
            backward_rows<X, G, 1024, 1, 1024>(a, p.groups, partial, s);
        else
            backward_rows<X, G, 1024, 2, 1024>(a, p.groups, partial, s);
    }
    if (sums)
        hipLaunchKernelGGL((layernorm_join_kernel<G>), dim3(static_cast<unsigned>((2 * int64_t(a.K) + 31) / 32)),
                           dim3(256), 0, s, partial, static_cast<G*>(a.dgamma), static_cast<G*>(a.dbeta), p.groups,
                           a.K);
}

}  // namespace

size_t layernorm_backward_workspace(int64_t M, int32_t K) {
    return static_cast<size_t>(split_of(M, K).groups) * 2 * static_cast<size_t>(K) * sizeof(float);
}

ss1_status launch_layernorm_forward(const NormArgs& a) {
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    if (a.dtype == SS1_F32)
        forward<float, float>(a, s);
    else if (a.affine_dtype == SS1_F32)
        forward<uint16_t, float>(a, s);
    else
        forward<uint16_t, uint16_t>(a, s);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

ss1_status launch_layernorm_backward(const NormArgs& a) {
    hipStream_t s = static_cast<hipStream_t>(a.stream);
    if (a.dtype == SS1_F32)
        backward<float, float>(a, s);
    else if (a.affine_dtype == SS1_F32)
        backward<uint16_t, float>(a, s);
    else
        backward<uint16_t, uint16_t>(a, s);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace ss1
