// The global gradient norm over many tensors, its clip coefficient, and
// clipping in place (ss1_gradnorm, ss1_gradnorm_clip).
//
// Each work item is a run of kNormChunk elements of one tensor; a block takes a
// run of consecutive items and leaves one partial sum.  The product of two
// float32 values is exact in float64 and the sums stay there, so gradients of
// 1e-30 or 1e30 count like any other and the order of the sum does not show in
// the result.  The partial sums are added by whoever needs the norm: one block
// that writes it, or every block of the clipping pass for itself (at most
// kNormMost doubles), which saves a launch between the two passes.
//
// Bound by memory: 118M bf16 values (236 MB) are summed in 47 us (5.0 TB/s, the
// rate of a large copy; 39 us over the same ones again and again) and clipped in 73
// more, read and written (6.5 TB/s); the clipping pass finds nothing of the first
// one's reads in the last-level cache, in either direction.  Gradients that earlier
// calls have just clipped are summed in 68 us, beside the writes that are still on
// their way to memory: such a call takes 142 us.  20M bf16 values take 10.4 us and the last sum 3.8; below
// that the two launches are the time (400 tensors of 1.5M values together: 11.9
// us a call).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ss1_model_ops.h"

namespace ss1 {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;
constexpr int kPasses = static_cast<int>(kNormChunk / (kThreads * kVec));
static_assert(kNormChunk % (kThreads * kVec) == 0, "a chunk is whole passes of the block");

// Eight bf16 or float32 values as they lie in memory.
struct RawH {
    uint4 a;
};
struct RawF {
    uint4 a, b;
};

__device__ __forceinline__ void load_raw(const uint16_t* p, RawH& r) { r.a = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void load_raw(const float* p, RawF& r) {
    r.a = *reinterpret_cast<const uint4*>(p);
    r.b = *reinterpret_cast<const uint4*>(p + 4);
}
__device__ __forceinline__ void widen(const RawH& r, float (&v)[kVec]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen(const RawF& r, float (&v)[kVec]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }
__device__ __forceinline__ float widen(float f) { return f; }

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[kVec]) {
    uint4 o;
    o.x = bf16_bits(v[0]) | bf16_bits(v[1]) << 16;
    o.y = bf16_bits(v[2]) | bf16_bits(v[3]) << 16;
    o.z = bf16_bits(v[4]) | bf16_bits(v[5]) << 16;
    o.w = bf16_bits(v[6]) | bf16_bits(v[7]) << 16;
    *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(bf16_bits(v)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// A block's work items, 64 at a time: lane l of every wave holds the l-th one's
// address, elements left in its tensor and type, so that the chain of reads
// (item, entry) is paid once for 64 items and not before each one's data (the
// call over 400 small tensors: 13.6 -> 12.3 us).
struct Items {
    uint64_t at;
    int64_t left;  // 0: none
    int32_t dtype;

    __device__ __forceinline__ void load(const ss1_gradnorm_entry* entries, int count, const int32_t* map, int64_t i,
                                         int64_t end) {
        at = 0;
        left = 0;
        dtype = SS1_F32;
        if (i >= end) return;
        const int item = map[2 * i];
        const int64_t begin = static_cast<int64_t>(map[2 * i + 1]) * kNormChunk;
        if (item < 0 || item >= count || begin < 0) return;
        const ss1_gradnorm_entry e = entries[item];
        if (begin >= e.numel) return;
        at = reinterpret_cast<uint64_t>(e.grad) + static_cast<uint64_t>(begin) * (e.dtype == SS1_F32 ? 4 : 2);
        left = e.numel - begin;
        dtype = e.dtype;
    }
};
struct Item {
    uint64_t at;
    int n;  // of the chunk: at most kNormChunk
    bool f32;
};
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ Item item_at(const Items& t, int lane) {
    const uint64_t left = static_cast<uint64_t>(lane_value(static_cast<uint32_t>(t.left >> 32), lane)) << 32 |
                          lane_value(static_cast<uint32_t>(t.left), lane);
    Item r;
    r.at = static_cast<uint64_t>(lane_value(static_cast<uint32_t>(t.at >> 32), lane)) << 32 |
           lane_value(static_cast<uint32_t>(t.at), lane);
    r.n = left < static_cast<uint64_t>(kNormChunk) ? static_cast<int>(left) : static_cast<int>(kNormChunk);
    r.f32 = lane_value(static_cast<uint32_t>(t.dtype), lane) == SS1_F32;
    return r;
}

// A thread's share of a chunk as it lies in memory: kPasses vectors of bf16, or
// twice as many of float32; of a tensor's last chunk the whole vectors that are
// there (zeros for the others) and one of the elements behind them, so that such a
// chunk too is one trip to memory and not one for every 256 elements.
struct Raw {
    uint4 v[2 * kPasses];
    uint32_t tail;
    __device__ __forceinline__ void load(const Item& t) {
        const uint4* p = reinterpret_cast<const uint4*>(t.at) + threadIdx.x;
        tail = 0;
        if (t.n == kNormChunk) {
            if (t.f32) {
#pragma unroll
                for (int i = 0; i < 2 * kPasses; ++i) v[i] = p[i * kThreads];
            } else {
#pragma unroll
                for (int i = 0; i < kPasses; ++i) v[i] = p[i * kThreads];
            }
            return;
        }
        const int per = t.f32 ? 4 : 8, whole = t.n / per, rest = t.n % per;
#pragma unroll
        for (int i = 0; i < 2 * kPasses; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (static_cast<int>(threadIdx.x) + i * kThreads < whole) v[i] = p[i * kThreads];
        }
        if (static_cast<int>(threadIdx.x) < rest) {
            const int at = whole * per + threadIdx.x;
            tail = t.f32 ? reinterpret_cast<const uint32_t*>(t.at)[at]
                         : static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(t.at)[at]) << 16;
        }
    }
};

__device__ __forceinline__ double squared(uint32_t bits, double s) {
    const double d = __uint_as_float(bits);
    return fma(d, d, s);
}
__device__ __forceinline__ double squares(const Item& t, const Raw& r) {
    double s = squared(r.tail, 0.0);
    if (t.f32) {
#pragma unroll
        for (int i = 0; i < 2 * kPasses; ++i) {
            s = squared(r.v[i].x, s);
            s = squared(r.v[i].y, s);
            s = squared(r.v[i].z, s);
            s = squared(r.v[i].w, s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s = squared(w[j] << 16, s);
                s = squared(w[j] & 0xFFFF0000u, s);
            }
        }
    }
    return s;
}

// The block's sum of one double a thread, in every thread.
template <int T>
__device__ __forceinline__ double block_sum(double s, double* red) {
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    double t = red[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) t += red[w];
    return t;
}

// The items of block b of `blocks`: [first, first of the next block).
__device__ __forceinline__ int64_t first_item(int64_t chunks, int b, int blocks) {
    return chunks * b / blocks;
}

__global__ __launch_bounds__(kThreads) void gradnorm_kernel(const ss1_gradnorm_entry* __restrict__ entries, int count,
                                                            const int32_t* __restrict__ map, int64_t chunks,
                                                            double* __restrict__ partial) {
    __shared__ double red[kThreads / 64];
    const int64_t end = first_item(chunks, blockIdx.x + 1, gridDim.x);
    double s = 0.0;
    for (int64_t i0 = first_item(chunks, blockIdx.x, gridDim.x); i0 < end; i0 += 64) {
        Items items;
        items.load(entries, count, map, i0 + (threadIdx.x & 63), end);
        const int n = end - i0 < 64 ? static_cast<int>(end - i0) : 64;
        // the next item's data is on its way while one is summed
        Item cur = item_at(items, 0);
        Raw raw;
        raw.load(cur);
        for (int k = 0; k < n; ++k) {
            Item next{0, 0, true};
            Raw ahead;
            if (k + 1 < n) {
                next = item_at(items, k + 1);
                ahead.load(next);
            }
            s += squares(cur, raw);
            cur = next;
            raw = ahead;
        }
    }
    s = block_sum<kThreads>(s, red);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

struct Norm {
    float norm, coef;
};

// Norm and coefficient from the partial sums, in every thread: the same order
// in every block that asks.
template <int T>
__device__ __forceinline__ Norm finish(const double* __restrict__ partial, int parts, double max_norm, double* red) {
    constexpr int kLoads = static_cast<int>(kNormMost) / T;  // all in flight together
    double v[kLoads], s = 0.0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = threadIdx.x + i * T < parts ? partial[threadIdx.x + i * T] : 0.0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) s += v[i];
    const double norm = sqrt(block_sum<T>(s, red));
    Norm r;
    r.norm = static_cast<float>(norm);
    r.coef = norm > max_norm ? static_cast<float>(max_norm / norm) : norm != norm ? r.norm : 1.0f;
    return r;
}

constexpr int kFinishThreads = 1024;
__global__ __launch_bounds__(kFinishThreads) void gradnorm_finish_kernel(const double* __restrict__ partial, int parts,
                                                                         double max_norm, float* __restrict__ norm,
                                                                         float* __restrict__ coef) {
    __shared__ double red[kFinishThreads / 64];
    const Norm r = finish<kFinishThreads>(partial, parts, max_norm, red);
    if (threadIdx.x != 0) return;
    if (norm) *norm = r.norm;
    if (coef) *coef = r.coef;
}

template <typename T, typename R>
__device__ __forceinline__ void scale_chunk(T* p, int64_t n, float coef) {
    if (n >= kNormChunk) {
        R r[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) load_raw(p + (i * kThreads + threadIdx.x) * kVec, r[i]);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            float v[kVec];
            widen(r[i], v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] *= coef;
            store8(p + (i * kThreads + threadIdx.x) * kVec, v);
        }
        return;
    }
    for (int64_t i = threadIdx.x * kVec; i < n; i += kThreads * kVec) {
        const int m = n - i < kVec ? static_cast<int>(n - i) : kVec;
        for (int j = 0; j < m; ++j) store1(p + i + j, widen(p[i + j]) * coef);
    }
}

__global__ __launch_bounds__(kThreads) void gradclip_kernel(const ss1_gradnorm_entry* __restrict__ entries, int count,
                                                            const int32_t* __restrict__ map, int64_t chunks,
                                                            const double* __restrict__ partial, double max_norm,
                                                            float* __restrict__ norm, float* __restrict__ coef) {
    __shared__ double red[kThreads / 64];
    const Norm r = finish<kThreads>(partial, gridDim.x, max_norm, red);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (norm) *norm = r.norm;
        if (coef) *coef = r.coef;
    }
    if (r.coef == 1.0f) return;
    const int64_t end = first_item(chunks, blockIdx.x + 1, gridDim.x);
    for (int64_t i = first_item(chunks, blockIdx.x, gridDim.x); i < end; ++i) {
        const int item = map[2 * i];
        const int64_t part = map[2 * i + 1];
        if (item < 0 || item >= count || part < 0) continue;
        const ss1_gradnorm_entry e = entries[item];
        const int64_t begin = part * kNormChunk;
        if (begin >= e.numel) continue;
        if (e.dtype == SS1_F32)
            scale_chunk<float, RawF>(static_cast<float*>(e.grad) + begin, e.numel - begin, r.coef);
        else
            scale_chunk<uint16_t, RawH>(static_cast<uint16_t*>(e.grad) + begin, e.numel - begin, r.coef);
    }
}

void launch_partial(const GradNormArgs& a) {
    if (a.chunks == 0) return;
    hipLaunchKernelGGL(gradnorm_kernel, dim3(gradnorm_blocks(a.chunks)), dim3(kThreads), 0,
                       static_cast<hipStream_t>(a.stream), a.entries, a.count, a.map, a.chunks, a.partial);
}

}  // namespace

ss1_status launch_gradnorm(const GradNormArgs& a) {
    launch_partial(a);
    hipLaunchKernelGGL(gradnorm_finish_kernel, dim3(1), dim3(kFinishThreads), 0, static_cast<hipStream_t>(a.stream),
                       a.partial, gradnorm_blocks(a.chunks), a.max_norm, a.norm, a.coef);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

ss1_status launch_gradnorm_clip(const GradNormArgs& a) {
    if (a.chunks == 0) return launch_gradnorm(a);
    launch_partial(a);
    hipLaunchKernelGGL(gradclip_kernel, dim3(gradnorm_blocks(a.chunks)), dim3(kThreads), 0,
                       static_cast<hipStream_t>(a.stream), a.entries, a.count, a.map, a.chunks, a.partial, a.max_norm,
                       a.norm, a.coef);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

}  // namespace ss1
