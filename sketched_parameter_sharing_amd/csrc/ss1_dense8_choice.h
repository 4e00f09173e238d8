// Which way a product of block-scaled E4M3 matrices goes, by its sizes alone:
// the tile, whether the reduction is split, by the weight's rows, with x quantised
// inside, beside another product.  Host code without HIP, so that a test on the
// host can ask which sizes reach which kernel.
#pragma once

#include <stdint.h>

#include "../../include/ss1.h"

namespace ss1 {

// ----------------------------------------------------------------- few rows
// Rows of a that the kernel for few rows takes, and how much of x a block quantises:
// 16 tokens 768 -> 768 take 8.3 us a call with x quantised inside and 12 with a
// launch for it, one token 4096 -> 14336 11.7 and 26.5; 4 tokens 14336 -> 4096,
// which a block would need 57 KB for, 23 and 16.
constexpr int64_t kFewRows = 16;
constexpr int64_t kInsideRows = 4;                 // rows for which a's reads do not count
constexpr int64_t kInsideBytes = 32768;            // codes of x in a block's LDS
constexpr int64_t kInsideAll = int64_t(20) << 20;  // elements that all blocks together quantise
constexpr int kFewWaves = 4, kFewThreads = kFewWaves * 64;

// Up to 16 rows go by the weight's rows where what all blocks read of a (M * K
// bytes each) stays below 24 MB.  us of kernels that way and in tiles, bf16 y:
//   M, N, K               MB                       M, N, K               MB
//   16,  1280,  5120       6    7.7    8.7         8,  8192,  4096      16   10.5   12.1
//   16,  4096,  4096      16    6.7   10.0         8, 14336,  4096      28   16.3   15.9
//   16,  6144,  4096      24   11.0   11.1         8,  8192,  8192      32   17.9   20.0
//   16,  5120,  5120      25   12.9   13.0         8,  4096, 14336      28   16.5   18.3
//   16,  8192,  4096      32   12.2   12.4         5, 14336,  4096      18   14.7   16.0
//   16, 14336,  4096      56   19.4   15.8         5, 16384,  8192      40   29.0   35.2
// The rule is out by at most 21% there (5 rows, 40 MB), and by 18% where the weight
// has few rows and is deep (16, 1024, 8192: 10.5 and 8.9).
// From 2^28 rows of the weight on the blocks of 16 would be too many: a grid's
// threads are numbered in 32 bits.
inline bool few_rows(int64_t M, int64_t N, int64_t K) {
    const int64_t blocks = (N + 15) / 16;
    return K > 0 && M <= kFewRows && blocks * kFewThreads < int64_t(1) << 32 &&
           (M <= kInsideRows || blocks * M * K <= int64_t(24) << 20);
}

// Whether x itself (not its codes) is taken: its codes and scales fit into a block's LDS.
inline bool few_rows_take_x(int64_t M, int64_t N, int64_t K) {
    return few_rows(M, N, K) && M * (K + 16 + K / SS1_FP8_BLOCK) <= kInsideBytes &&
           (N + 15) / 16 * M * K <= kInsideAll;
}

// -------------------------------------------------------------------- tiles
// The tiles and what they take, in us: a round of blocks is stages of 128 deep
// (first number each) and a prologue and epilogue (second), with at most one
// block a compute unit, and with as many as fit.  Fitted to 27 products of 64 to
// 16384 rows, 768 to 14336 columns and 768 to 14336 deep in each type of y; the
// model below picks the fastest of them or one within 5%.  256 x 256 holds too
// many registers for a float32 y's operands.
//   M, N, K (bf16)        64x64  64x128  128x128  192x256  256x256   us a product
//   64, 14336, 4096        12.5    16.6     23.6     36.4     47.1
//   1024, 4096, 4096       30.0    25.0     27.4     39.6     50.5
//   2048, 4096, 4096       55.9    45.2     35.7     43.0     52.3
//   8192, 1280, 5120       93.3    73.1     68.2     51.5     64.0
//   4096, 4096, 4096        107    84.2     66.6     81.1     58.4
//   4096, 14336, 4096       429     338      264      231      231
//   8192, 8192, 8192        889     702      548      510      448
enum Tile { kTile64, kTile64x128, kTile128, kTile192, kTile256, kTiles };
struct RoundUs {
    double stage, ends;
};
struct TileRate {
    int bm, bn, fit;
    RoundUs alone[2], full[2];  // bf16 y, float32 y
};
constexpr TileRate kRates[kTiles] = {
    {64, 64, 2, {{0.26, 1.1}, {0.43, 1.1}}, {{0.41, 0.7}, {0.57, 1.6}}},
    {64, 128, 2, {{0.39, 1.9}, {0.69, 3.5}}, {{0.64, 0.8}, {0.93, 3.8}}},
    {128, 128, 2, {{0.62, 2.7}, {1.00, 5.3}}, {{1.10, 1.8}, {1.49, 7.1}}},
    {192, 256, 1, {{1.02, 4.7}, {1.95, 10.1}}, {{1.33, 4.4}, {2.08, 13.8}}},
    {256, 256, 1, {{1.38, 5.7}, {0, 0}}, {{1.66, 5.2}, {0, 0}}}};
constexpr int64_t kCUs = 256;
constexpr double kLaunchUs = 3.0;       // of the launch that joins splits
constexpr double kJoinBytesUs = 4.0e6;  // bytes a us of partial sums, written and read

struct Choice {
    Tile tile;
    int splits;
};

inline double tile_us(const TileRate& r, int64_t blocks, int64_t stages, bool f32) {
    const int64_t per = (blocks + kCUs - 1) / kCUs;
    const RoundUs& u = per <= 1 ? r.alone[f32] : r.full[f32];
    return static_cast<double>((per + r.fit - 1) / r.fit) * (static_cast<double>(stages) * u.stage + u.ends);
}

inline Choice choose(int64_t M, int64_t N, int64_t K, bool f32) {
    const int64_t stages = K / SS1_FP8_BLOCK;
    Choice best{kTile64, 1};
    double us = 1e30;
    for (int t = 0; t < (f32 ? kTile256 : kTiles); ++t) {
        const TileRate& r = kRates[t];
        const int64_t tiles = ((M + r.bm - 1) / r.bm) * ((N + r.bn - 1) / r.bn);
        const double u = tile_us(r, tiles, stages, f32);
        if (u < us) {
            us = u;
            best = {static_cast<Tile>(t), 1};
        }
        if (t != kTile64) continue;
        // long reductions of few tiles: runs of at least four stages, a block each
        for (int splits = 2; splits <= 8 && splits * 4 <= stages; splits *= 2) {
            const double run = static_cast<double>(splits) * M * N * 8.0 / kJoinBytesUs;
            const double v = tile_us(r, tiles * splits, (stages + splits - 1) / splits, f32) + kLaunchUs + run;
            if (v < us) {
                us = v;
                best = {kTile64, splits};
            }
        }
    }
    return best;
}

// Whether a product goes by the weight's rows, or by 64 x 64 tiles in one round
// with no splits.
inline bool pairable(int64_t M, int64_t N, int64_t K, bool f32) {
    const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
    if (K == 0 || tiles > kCUs) return false;
    if (few_rows(M, N, K)) return true;
    const Choice c = choose(M, N, K, f32);
    return c.tile == kTile64 && c.splits == 1;
}

}  // namespace ss1
