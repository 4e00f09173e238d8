// The product of two block-scaled E4M3 matrices (ss1_matmul_fp8_blocks and the
// dense layer's forward and gradients): y[m][n] = sum over blocks t of 128 of
// 2^(ea[m][t] + eb[n][t]) * sum_{k in t} a[m][k] * b[n][k].
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over 128
// elements and takes a power-of-two scale for every row of both operands, so a
// block of the format is one instruction and its scales cost nothing but their
// loads.  The instruction sums over k, so any assignment of the 128 elements to
// lanes and registers serves as long as both operands use the same one.
//
// That instruction lines the products of a block up at the largest and keeps 18
// bits below it (measured: a relative error of 1e-5 to 5e-5 of a sum over 128).
// A bf16 y does not see it beside its own rounding (4e-3); a float32 y does, and
// is computed on the bf16 matrix cores instead, at half the rate: every code
// times its scale is a bf16 value, so v_cvt_scalef32_pk_bf16_fp8 (one vector
// instruction for two, full rate) widens the operands exactly as they leave LDS
// and the sums are float32's (8e-8).
//
// Rates: 4096 x 14336 x 4096 to bf16 231 us (2080 TFLOP/s; a library product of
// plain E4M3 of this size 194 us), 8192^3 448 us (2450), 8192 x 1280 x 5120 52
// us (57; both over the same operands again and again, over six sets in turn
// 63), the float32 gradient 5120 x 1280 x 8192 about 105 us (a library product
// of bf16: 105).  The large tiles are bound by the way from L2 into LDS beside
// the matrix cores: of 192 x 256, these are busy 42% of the time, the texture
// path 68%, no LDS conflicts; its loads alone take 170 to 217 us, its MFMAs
// alone 178.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "ss1_blocks.h"
#include "ss1_dense8_choice.h"
#include "ss1_device.h"
#include "ss1_dma.h"
#include "ss1_model_ops.h"

namespace ss1 {

namespace {

using dev::f32x4;
using dev::i32x4;
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kKS = SS1_FP8_BLOCK;  // elements (bytes) of a stage

// One wave-wide load of 4 bytes per lane: lane l writes its 4 bytes at LDS
// byte address lds + 4*l.  As dev::lds_dma16 otherwise (no register result;
// the stage barriers order it).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma4(i32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                 "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Row p of a wave's weight tile in LDS (TN = 16 * FN rows) holds column
// neuron(p) of the output: with it the lane that holds rows 4q .. 4q+3 of every
// 16-row block holds 4 * FN consecutive columns.
template <int FN>
__device__ __forceinline__ int out_column(int p) {
    const int nb = p / 16, r = p % 16;
    return (r / 4) * 4 * FN + nb * 4 + r % 4;
}

// N consecutive outputs of a row that has `left` from there on; a row of an odd
// width starts anywhere, so the vectors are not aligned.
typedef blocks::u32x4 u32x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any2 __attribute__((aligned(2)));
template <int N>
__device__ __forceinline__ void store_run(uint16_t* p, const float (&v)[N], int left) {
    if (left >= N) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = dev::pack_bf16(v[2 * i], v[2 * i + 1]);
        if constexpr (N == 8) *reinterpret_cast<blocks::u32x4_any2*>(p) = u32x4{w[0], w[1], w[2], w[3]};
        else *reinterpret_cast<u32x2_any2*>(p) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
        for (int i = 0; i < N - 1; ++i)
            if (i < left) p[i] = dev::to_bf16_bits(v[i]);
    }
}
template <int N>
__device__ __forceinline__ void store_run(float* p, const float (&v)[N], int left) {
    if (left >= N) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<blocks::u32x4_any4*>(p + i) = u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]),
                                                                  __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])};
    } else {
#pragma unroll
        for (int i = 0; i < N - 1; ++i)
            if (i < left) p[i] = v[i];
    }
}

// 32 codes of a row as four bf16 operands of v_mfma_f32_16x16x32_bf16, times
// the row's scale.
struct Wide {
    dev::bf16x8 t[4];
};
__device__ __forceinline__ Wide widen(const i32x8& v, float scale) {
    Wide o;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        uint4 w;
        const uint32_t lo = static_cast<uint32_t>(v[2 * t]), hi = static_cast<uint32_t>(v[2 * t + 1]);
        w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
        w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
        w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
        w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
        o.t[t] = __builtin_bit_cast(dev::bf16x8, w);
    }
    return o;
}

// Block: WM x WN waves on a tile of BM rows of a and BN rows of b; NSTG LDS
// buffers, filled by direct loads NSTG - 1 stages ahead.  Rows of 128 bytes,
// XOR-swizzled in 16-byte pieces.  The scales of a stage come as one word a
// row, four blocks of 128 at a time (their byte is picked by the stage).
//
// SPLIT: the reduction is cut into `splits` runs of stages, one a block each;
// y then is float32 [splits][M][N], added in order by join_splits_kernel.
struct TileArgs {
    BlocksView a, b;
    void* y;
    int M, N, K;
    int n_mt, n_nt;
    int splits;
};

template <int BM, int BN, int WM, int WN, int NSTG, bool F32, bool SPLIT>
__device__ __forceinline__ void matmul_tile(const TileArgs& p, int block) {
    const BlocksView &a = p.a, &b = p.b;
    void* __restrict__ y = p.y;
    const int M = p.M, N = p.N, K = p.K, n_mt = p.n_mt, n_nt = p.n_nt, splits = p.splits;
    constexpr int NWV = WM * WN;
    constexpr int TM = BM / WM, TN = BN / WN;
    constexpr int FM = TM / 16, FN = TN / 16;
    constexpr int AI = BM / 8 / NWV, BI = BN / 8 / NWV;
    constexpr int SA = BM * kKS, SBB = BN * kKS, SS = (BM + BN) * 4;
    constexpr int SB = SA + SBB + SS;
    constexpr int SL = (BM + BN) / 64, SI = (SL + NWV - 1) / NWV;  // loads of 64 scale words: all, of a wave
    static_assert(BM % 64 == 0 && BN % 64 == 0, "a load's scales belong to one operand");
    constexpr int DPW = AI + BI + SI;

    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    constexpr int GM = 4;
    const int part = SPLIT ? block % splits : 0;
    const int tile = dev::xcd_tile(SPLIT ? block / splits : block, n_mt * n_nt);
    const int strip = tile / (GM * n_nt);
    const int gm = min(GM, n_mt - strip * GM);
    const int rem = tile - strip * GM * n_nt;
    const int m0 = (strip * GM + rem % gm) * BM;
    const int n0 = (rem / gm) * BN;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // the block's stages: [first, last); runs start at a scale word
    const int words = (K / kKS + 3) / 4;
    const int first_stage = SPLIT ? words * part / splits * 4 : 0;
    const int nstage = (SPLIT ? min(words * (part + 1) / splits * 4, K / kKS) : K / kKS) - first_stage;

    const i32x4 ar = dev::dma_rsrc(a.codes + static_cast<size_t>(m0) * K,
                                   static_cast<uint32_t>(static_cast<size_t>(min(BM, M - m0)) * K));
    const i32x4 br = dev::dma_rsrc(b.codes + static_cast<size_t>(n0) * K,
                                   static_cast<uint32_t>(static_cast<size_t>(min(BN, N - n0)) * K));
    const int lr = lane >> 3;
    const int pc = (lane & 7) ^ dev::swz_key<kKS>(wave * 8 + lr);
    const uint32_t a_voff = static_cast<uint32_t>(lr * K + pc * 16);
    uint32_t b_voff[BI];
#pragma unroll
    for (int ii = 0; ii < BI; ++ii) {
        const int p = (wave + NWV * ii) * 8 + lr;
        const int n = (p / TN) * TN + out_column<FN>(p % TN);
        b_voff[ii] = static_cast<uint32_t>(n * K + pc * 16);
    }
    // the wave's scale words, 64 a load: rows of a, or of b (the last load is
    // made twice where the waves do not share them evenly)
    i32x4 sr[SI];
    uint32_t s_voff[SI], s_lds[SI];
#pragma unroll
    for (int ii = 0; ii < SI; ++ii) {
        const int l = min(wave + NWV * ii, SL - 1);
        const bool of_a = l < BM / 64;
        const int sp = (of_a ? l : l - BM / 64) * 64 + lane;
        const BlocksView& sv = of_a ? a : b;
        const int s0 = of_a ? m0 : n0;
        const int srow = of_a ? sp : (sp / TN) * TN + out_column<FN>(sp % TN);
        const int64_t first = s0 >> sv.shift;
        const int64_t rows = ((sv.rows + (int64_t(1) << sv.shift) - 1) >> sv.shift) - first;
        const int span = ((of_a ? BM : BN) >> sv.shift) + 1;
        sr[ii] = dev::dma_rsrc(sv.scale + first * sv.scale_cols,
                               static_cast<uint32_t>((rows < span ? rows : span) * sv.scale_cols));
        s_voff[ii] = static_cast<uint32_t>((((s0 + srow) >> sv.shift) - first) * sv.scale_cols);
        s_lds[ii] = static_cast<uint32_t>(l * 256);
    }

    const uint32_t lds0 = dev::lds_address(smem);
    auto dma = [&](int s, int buf) {
        const uint32_t base = lds0 + static_cast<uint32_t>(buf * SB);
        const uint32_t k0 = static_cast<uint32_t>((first_stage + s) * kKS);
#pragma unroll
        for (int ii = 0; ii < AI; ++ii) {
            const int row0 = (wave + NWV * ii) * 8;
            dev::lds_dma16(ar, base + row0 * kKS, a_voff + static_cast<uint32_t>(row0 * K), k0);
        }
#pragma unroll
        for (int ii = 0; ii < BI; ++ii)
            dev::lds_dma16(br, base + SA + (wave + NWV * ii) * 8 * kKS, b_voff[ii], k0);
#pragma unroll
        for (int ii = 0; ii < SI; ++ii)
            lds_dma4(sr[ii], base + SA + SBB + s_lds[ii], s_voff[ii], static_cast<uint32_t>((first_stage + s) & ~3));
    };

    const int fr = lane & 15, q = lane >> 4;
    const int key = dev::swz_key<kKS>(fr);
    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto step = [&](int s, int buf) {
        if (NSTG >= 3 && nstage - 1 - s >= NSTG - 2) dev::dma_stage_barrier<(NSTG - 2) * DPW>();
        else dev::dma_stage_barrier<0>();
        if (s + NSTG - 1 < nstage) dma(s + NSTG - 1, (buf + NSTG - 1) % NSTG);
        const uint8_t* S = smem + buf * SB;
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(S + SA + SBB);
        const int byte = 8 * (s & 3);
        auto operand = [&](const uint8_t* row) {
            const uint4 u = *reinterpret_cast<const uint4*>(row + ((q ^ key) << 4));
            const uint4 w = *reinterpret_cast<const uint4*>(row + (((q + 4) ^ key) << 4));
            return i32x8{static_cast<int>(u.x), static_cast<int>(u.y), static_cast<int>(u.z), static_cast<int>(u.w),
                         static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w)};
        };
        // The first rows of a are read first, then b's, so that the first MFMA
        // waits for two reads and not for all.  From there on the next 16 rows of
        // a are read while the MFMAs of these run; left alone, the compiler reads
        // them behind those MFMAs and waits.
        auto rows = [&](int j) { return operand(S + (wm * TM + j * 16 + fr) * kKS); };
        auto word = [&](int j) { return sc[wm * TM + j * 16 + fr]; };
        i32x8 av = rows(0), bv[FN];
        uint32_t aw = word(0), bw[FN];
#pragma unroll
        for (int i = 0; i < FN; ++i) bw[i] = sc[BM + wn * TN + i * 16 + fr];
#pragma unroll
        for (int i = 0; i < FN; ++i) bv[i] = operand(S + SA + (wn * TN + i * 16 + fr) * kKS);
        __builtin_amdgcn_sched_barrier(0);
        auto scale = [&](uint32_t w) { return __uint_as_float((w >> byte & 0xFFu) << 23); };
        Wide bx[F32 ? FN : 1];
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < FN; ++i) bx[i] = widen(bv[i], scale(bw[i]));
        } else {
#pragma unroll
            for (int i = 0; i < FN; ++i) bw[i] >>= byte;
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            i32x8 an = av;
            uint32_t nw = aw;
            if (j + 1 < FM) {
                an = rows(j + 1);
                nw = word(j + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (F32) {
                const Wide ax = widen(av, scale(aw));
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < FN; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bx[i].t[t], ax.t[t], acc[i][j], 0, 0, 0);
            } else {
                const int as = static_cast<int>(aw >> byte);
#pragma unroll
                for (int i = 0; i < FN; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        bv[i], av, acc[i][j], 0, 0, 0, static_cast<int>(bw[i]), 0, as);
            }
            __builtin_amdgcn_sched_barrier(0);
            av = an;
            aw = nw;
        }
        __builtin_amdgcn_s_setprio(0);
    };
#pragma unroll
    for (int p = 0; p < NSTG - 1; ++p)
        if (p < nstage) dma(p, p);
    for (int s1 = 0; s1 < nstage; s1 += NSTG) {
#pragma unroll
        for (int u = 0; u < NSTG; ++u)
            if (s1 + u < nstage) step(s1 + u, u);
    }

    // lane holds columns nbase + 4 i .. + 3 (i < FN) of the rows m0 + .. + fr
    const int nbase = n0 + wn * TN + q * 4 * FN;
    constexpr int RUN = FN % 2 == 0 ? 8 : 4;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int m = m0 + wm * TM + j * 16 + fr;
        if (m >= M) continue;
#pragma unroll
        for (int h = 0; h < 4 * FN / RUN; ++h) {
            const int n = nbase + RUN * h;
            if (n >= N) continue;
            float v[RUN];
#pragma unroll
            for (int i = 0; i < RUN; ++i) v[i] = acc[(RUN * h + i) / 4][j][i % 4];
            const size_t at = (static_cast<size_t>(part) * M + m) * N + n;
            if constexpr (F32 || SPLIT) store_run(static_cast<float*>(y) + at, v, N - n);
            else store_run(static_cast<uint16_t*>(y) + at, v, N - n);
        }
    }
}

// ------------------------------------------------------------- few tokens
// Up to 16 rows of a (tokens) against all of b (a weight): the weight's bytes
// are the time, so a wave reads its operands of b straight from global memory,
// 4 blocks of 128 of 16 rows at a time and one such unit ahead.  A block is 16
// rows of b; its NW waves share the reduction in contiguous runs of units and
// meet in LDS, added in order.  One token 4096 -> 14336 (59 MB) 11.7 us a call,
// 5.0 TB/s.
//
// With X the rows of a are x itself, quantised by every block for itself into
// LDS (M * K elements of L2 traffic and about 10 instructions an element and
// block, against a launch); its loads are issued before the weight's, since
// loads return in order, and the weight's are in flight meanwhile.
constexpr int kUnit = 4;  // blocks of 128 of a unit: the scales of one word

struct FewArgs {
    BlocksView a, b;
    const void* x;
    int64_t xcols;
    void* y;
    int M, N, K;
};

// smem: with X the codes and scales of x; part: the waves' sums.
template <typename X, bool F32, int NW>
__device__ __forceinline__ void few_rows_block(const FewArgs& p, int block, uint8_t* smem, f32x4 (*part)[64]) {
    constexpr bool INSIDE = !__is_same(X, void);
    constexpr int kAhead = 4;  // passes over x whose loads are issued before the weight's
    const BlocksView &a = p.a, &b = p.b;
    const X* __restrict__ x = static_cast<const X*>(p.x);
    void* __restrict__ y = p.y;
    const int64_t xcols = p.xcols;
    const int M = p.M, N = p.N, K = p.K;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, q = lane >> 4;
    const int n0 = block * 16;
    const int nkb = K / kKS;
    const int units = (nkb + kUnit - 1) / kUnit;
    const int u0 = units * wave / NW, u1 = units * (wave + 1) / NW;

    // x: 16 lanes take a block of 128 of a row
    const int pitch = K + 16;  // 16 rows' pieces on distinct banks
    uint8_t* s_scale = smem + static_cast<size_t>(M) * pitch;
    const int items = INSIDE ? M * nkb : 0;
    constexpr int G = NW * 4;
    using T = typename std::conditional<INSIDE, X, float>::type;
    blocks::Eight<T> v[INSIDE ? kAhead : 1];
    auto fetch = [&](int it, blocks::Eight<T>& r) {
        if constexpr (INSIDE) {
            const int m = it / nkb, kb = it % nkb;
            r.load(x + m * xcols, kb * kKS + (lane & 15) * 8, xcols);
        }
    };
    if constexpr (INSIDE) {
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
            const int it = p * G + (tid >> 4);
            if (it < items) fetch(it, v[p]);
        }
    }

    const __amdgpu_buffer_rsrc_t br = dev::make_rsrc(b.codes + static_cast<size_t>(n0) * K,
                                                     static_cast<uint32_t>(static_cast<size_t>(min(16, N - n0)) * K));
    const uint32_t b_voff = static_cast<uint32_t>(fr * K + q * 16);
    const int n = min(n0 + fr, N - 1);
    const uint8_t* b_scale = b.scale + (static_cast<int64_t>(n) >> b.shift) * b.scale_cols;
    const int mr = min(fr, M - 1);  // columns of tokens past M are not stored
    const uint8_t* a_row = INSIDE ? nullptr : a.codes + static_cast<size_t>(mr) * K + q * 16;
    const uint8_t* a_scale = INSIDE ? nullptr : a.scale + (static_cast<int64_t>(mr) >> a.shift) * a.scale_cols;

    struct Unit {
        uint4 w[kUnit][2];
        uint4 t[INSIDE ? 1 : kUnit][2];
        uint32_t ws, ts;
    };
    auto load = [&](int u, Unit& o) {
        o.ws = *reinterpret_cast<const uint32_t*>(b_scale + u * kUnit);
        if constexpr (!INSIDE) o.ts = *reinterpret_cast<const uint32_t*>(a_scale + u * kUnit);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            // blocks past the last one of K: past the end of the row, and not used
            const uint32_t k = static_cast<uint32_t>(min(u * kUnit + i, nkb - 1) * kKS);
            o.w[i][0] = dev::buf_load16(br, b_voff, k);
            o.w[i][1] = dev::buf_load16(br, b_voff + 64, k);
            if constexpr (!INSIDE) {
                o.t[i][0] = *reinterpret_cast<const uint4*>(a_row + k);
                o.t[i][1] = *reinterpret_cast<const uint4*>(a_row + k + 64);
            }
        }
    };
    Unit cur, next;
    if (u0 < u1) load(u0, cur);

    if constexpr (INSIDE) {
        auto put = [&](int it, const blocks::Eight<T>& r) {
            const int m = it / nkb, kb = it % nkb;
            bool special;
            const uint32_t byte = blocks::scale_byte(blocks::max16(blocks::finite_top(r, special)));
            const uint2 w = blocks::codes_of(r, blocks::scale_of(byte), special);
            *reinterpret_cast<uint2*>(smem + m * pitch + kb * kKS + (lane & 15) * 8) = w;
            if ((lane & 15) == 0) s_scale[m * nkb + kb] = static_cast<uint8_t>(byte);
        };
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
            const int it = p * G + (tid >> 4);
            if (it < items) put(it, v[p]);
        }
        for (int it = kAhead * G + (tid >> 4); it < items; it += G) {
            fetch(it, v[0]);
            put(it, v[0]);
        }
        dev::lds_barrier();
    }

    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto octet = [](const uint4& u, const uint4& w) {
        return i32x8{static_cast<int>(u.x), static_cast<int>(u.y), static_cast<int>(u.z), static_cast<int>(u.w),
                     static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w)};
    };
    for (int u = u0; u < u1; ++u) {
        if (u + 1 < u1) load(u + 1, next);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const int kb = u * kUnit + i;
            if (kb >= nkb) break;
            i32x8 tv;
            uint32_t ts;
            if constexpr (INSIDE) {
                const uint8_t* r = smem + mr * pitch + kb * kKS + q * 16;
                tv = octet(*reinterpret_cast<const uint4*>(r), *reinterpret_cast<const uint4*>(r + 64));
                ts = s_scale[mr * nkb + kb];
            } else {
                tv = octet(cur.t[i][0], cur.t[i][1]);
                ts = cur.ts >> (8 * i);
            }
            const i32x8 wv = octet(cur.w[i][0], cur.w[i][1]);
            const uint32_t ws = cur.ws >> (8 * i);
            if constexpr (F32) {
                const Wide ww = widen(wv, __uint_as_float((ws & 0xFFu) << 23));
                const Wide tw = widen(tv, __uint_as_float((ts & 0xFFu) << 23));
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww.t[t], tw.t[t], acc, 0, 0, 0);
            } else {
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, tv, acc, 0, 0, 0, static_cast<int>(ws), 0,
                                                                       static_cast<int>(ts));
            }
        }
        cur = next;
    }
    part[wave][lane] = acc;
    dev::lds_barrier();
    if (wave != 0 || fr >= M) return;
    f32x4 sum = part[0][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += part[w][lane];
    const int c = n0 + 4 * q;
    if (c >= N) return;
    const size_t at = static_cast<size_t>(fr) * N + c;
    const float out[4] = {sum[0], sum[1], sum[2], sum[3]};
    if constexpr (F32) store_run(static_cast<float*>(y) + at, out, N - c);
    else store_run(static_cast<uint16_t*>(y) + at, out, N - c);
}

template <typename X, bool F32>
__global__ __launch_bounds__(kFewThreads) void few_rows_kernel(FewArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ f32x4 part[kFewWaves][64];
    few_rows_block<X, F32, kFewWaves>(p, static_cast<int>(blockIdx.x), smem, part);
}

FewArgs few_args(const MatmulBlocksArgs& p) {
    return {p.a, p.b, p.x, p.xcols, p.y, static_cast<int>(p.M), static_cast<int>(p.N), static_cast<int>(p.K)};
}

template <typename X, bool F32>
ss1_status launch_few(const MatmulBlocksArgs& p) {
    const size_t lds = __is_same(X, void) ? 0 : static_cast<size_t>(up_to(p.M * (p.K + 16 + p.K / kKS), 16));
    hipLaunchKernelGGL((few_rows_kernel<X, F32>), dim3(static_cast<unsigned>((p.N + 15) / 16)), dim3(kFewThreads), lds,
                       static_cast<hipStream_t>(p.stream), few_args(p));
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

template <int BM, int BN, int WM, int WN, int NSTG, bool F32, bool SPLIT>
__global__ __launch_bounds__(WM * WN * 64) void matmul_blocks_kernel(TileArgs p) {
    matmul_tile<BM, BN, WM, WN, NSTG, F32, SPLIT>(p, blockIdx.x);
}

// Two small products side by side: the blocks of one, then of the other.  Each
// goes the way that it would go alone (by the weight's rows, or in 64 x 64 tiles),
// so that its sums are the same bits with the other and without (4 tokens, 500 ->
// 2048, float32: 8.5 us of kernels, 13.6 with few rows in tiles too).
struct SideArgs {
    TileArgs tile;
    int blocks;
    bool few;
};

template <bool F32>
__device__ __forceinline__ void matmul_side(const SideArgs& s, int block) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const TileArgs& t = s.tile;
    if (s.few)
        few_rows_block<void, F32, kFewWaves>({t.a, t.b, nullptr, 0, t.y, t.M, t.N, t.K}, block, nullptr,
                                             reinterpret_cast<f32x4(*)[64]>(smem));
    else matmul_tile<64, 64, 2, 2, 4, F32, false>(t, block);
}

template <bool F32P, bool F32Q>
__global__ __launch_bounds__(kFewThreads) void matmul_pair_kernel(SideArgs p, SideArgs q) {
    const int block = static_cast<int>(blockIdx.x);
    if (block < p.blocks) matmul_side<F32P>(p, block);
    else matmul_side<F32Q>(q, block - p.blocks);
}

// y = the sum over the splits, in order.
template <typename T>
__global__ __launch_bounds__(256) void join_splits_kernel(const float* __restrict__ part, T* __restrict__ y,
                                                          int64_t outputs, int splits) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (at >= outputs) return;
    const int n = outputs - at < 4 ? static_cast<int>(outputs - at) : 4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (outputs % 4 == 0) {
        for (int s = 0; s < splits; ++s) sum += *reinterpret_cast<const f32x4*>(part + s * outputs + at);
    } else {
        for (int s = 0; s < splits; ++s)
            for (int i = 0; i < n; ++i) sum[i] += part[s * outputs + at + i];
    }
    const float out[4] = {sum[0], sum[1], sum[2], sum[3]};
    store_run(y + at, out, n);
}

template <int BM, int BN>
TileArgs tile_args(const MatmulBlocksArgs& p, void* y, int splits) {
    return {p.a, p.b, y, static_cast<int>(p.M), static_cast<int>(p.N), static_cast<int>(p.K),
            static_cast<int>((p.M + BM - 1) / BM), static_cast<int>((p.N + BN - 1) / BN), splits};
}
template <typename K>
bool allow_lds(K kern, size_t lds) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(lds)) == hipSuccess;
}

template <int BM, int BN, int WM, int WN, int NSTG, bool F32, bool SPLIT = false>
ss1_status launch_tile(const MatmulBlocksArgs& p, int splits = 1) {
    constexpr size_t lds = static_cast<size_t>(NSTG) * (BM + BN) * (kKS + 4);
    const TileArgs t = tile_args<BM, BN>(p, SPLIT ? p.workspace : p.y, splits);
    auto kern = &matmul_blocks_kernel<BM, BN, WM, WN, NSTG, F32, SPLIT>;
    if (!allow_lds(kern, lds)) return SS1_ERR_HIP;
    const hipStream_t stream = static_cast<hipStream_t>(p.stream);
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(t.n_mt) * t.n_nt * splits), dim3(WM * WN * 64), lds, stream, t);
    if constexpr (SPLIT) {
        const int64_t outputs = p.M * p.N;
        using T = typename std::conditional<F32, float, uint16_t>::type;
        hipLaunchKernelGGL(join_splits_kernel<T>, dim3(static_cast<unsigned>((outputs + 1023) / 1024)), dim3(256), 0,
                           stream, static_cast<const float*>(p.workspace), static_cast<T*>(p.y), outputs, splits);
    }
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

SideArgs side_args(const MatmulBlocksArgs& p) {
    const TileArgs t = tile_args<64, 64>(p, p.y, 1);
    const bool few = few_rows(p.M, p.N, p.K);
    return {t, few ? static_cast<int>((p.N + 15) / 16) : t.n_mt * t.n_nt, few};
}

template <bool F32P, bool F32Q>
ss1_status launch_pair_t(const MatmulBlocksArgs& p, const MatmulBlocksArgs& q) {
    constexpr size_t lds = static_cast<size_t>(4) * 128 * (kKS + 4);
    const SideArgs a = side_args(p), b = side_args(q);
    auto kern = &matmul_pair_kernel<F32P, F32Q>;
    if (!allow_lds(kern, lds)) return SS1_ERR_HIP;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(a.blocks + b.blocks)), dim3(kFewThreads), lds,
                       static_cast<hipStream_t>(p.stream), a, b);
    return hipGetLastError() == hipSuccess ? SS1_OK : SS1_ERR_HIP;
}

template <bool F32>
ss1_status launch_choice(const MatmulBlocksArgs& p) {
    const Choice c = choose(p.M, p.N, p.K, F32);
    if (c.splits > 1) return launch_tile<64, 64, 2, 2, 4, F32, true>(p, c.splits);
    switch (c.tile) {
        case kTile64: return launch_tile<64, 64, 2, 2, 4, F32>(p);
        case kTile64x128: return launch_tile<64, 128, 2, 2, 3, F32>(p);
        case kTile128: return launch_tile<128, 128, 2, 2, 2, F32>(p);
        case kTile192: return launch_tile<192, 256, 2, 4, 2, F32>(p);
        default:
            if constexpr (F32) return SS1_ERR_HIP;  // not chosen
            else return launch_tile<256, 256, 2, 4, 2, false>(p);
    }
}

}  // namespace

size_t matmul_blocks_workspace(int64_t M, int64_t N, int64_t K) {
    if (M == 0 || N == 0 || few_rows(M, N, K)) return 0;
    // y's type is not known here: room for either
    const int a = choose(M, N, K, false).splits, b = choose(M, N, K, true).splits;
    const int splits = a > b ? a : b;
    return splits > 1 ? static_cast<size_t>(splits) * M * N * 4 : 0;
}

bool matmul_takes_x(int64_t M, int64_t N, int64_t K) { return few_rows_take_x(M, N, K); }

ss1_status launch_matmul_blocks(const MatmulBlocksArgs& p) {
    const bool f32 = p.dtype == SS1_F32;
    if (p.x) return f32 ? launch_few<float, true>(p) : launch_few<uint16_t, false>(p);  // y has x's dtype
    if (few_rows(p.M, p.N, p.K)) return f32 ? launch_few<void, true>(p) : launch_few<void, false>(p);
    return f32 ? launch_choice<true>(p) : launch_choice<false>(p);
}

// Both in one launch where they are small: 333 tokens, 500 -> 768, float32, take
// 17.2 us a call that way and 20.1 in two, which is the host's time either way.
ss1_status launch_matmul_pair(const MatmulBlocksArgs& p, const MatmulBlocksArgs& q) {
    const bool fp = p.dtype == SS1_F32, fq = q.dtype == SS1_F32;
    if (!pairable(p.M, p.N, p.K, fp) || !pairable(q.M, q.N, q.K, fq)) {
        const ss1_status st = launch_matmul_blocks(p);
        return st == SS1_OK ? launch_matmul_blocks(q) : st;
    }
    if (fp) return fq ? launch_pair_t<true, true>(p, q) : launch_pair_t<true, false>(p, q);
    return fq ? launch_pair_t<false, true>(p, q) : launch_pair_t<false, false>(p, q);
}

}  // namespace ss1
