// Internal declarations of the operators at a model's ends and of its dense
// layers (embedding, gradient norm, block-scaled E4M3 matrices): the checked
// arguments that the ABI layer hands to the kernel launchers.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/ss1.h"

namespace ss1 {

// ------------------------------------------------------------ gradient norm
// Elements of one work item, and blocks (partial sums) of a call: an item each
// for up to kNormMost of them, else kNormBlocks blocks (all on the card at once)
// with a run of consecutive items each.  Measured against items of 8192 over at
// most 2048 blocks: 20M bf16 12.8 us for 17.0, 5M float32 9.5 for 13.0, 118M
// bf16 46.9 for 50.8 (tensors' last items read as vectors came later).
constexpr int64_t kNormChunk = 4096;
constexpr int64_t kNormMost = 2048, kNormBlocks = 1024;
inline int gradnorm_blocks(int64_t chunks) {
    return static_cast<int>(chunks <= kNormMost ? chunks : kNormBlocks);
}

struct GradNormArgs {
    const ss1_gradnorm_entry* entries;
    const int32_t* map;
    int64_t chunks;
    int32_t count;
    double max_norm;
    float* norm;  // may be null
    float* coef;  // may be null
    double* partial;
    void* stream;
};

inline size_t gradnorm_workspace(int64_t chunks) {
    return static_cast<size_t>(gradnorm_blocks(chunks)) * sizeof(double);
}
ss1_status launch_gradnorm(const GradNormArgs& a);
ss1_status launch_gradnorm_clip(const GradNormArgs& a);

// ---------------------------------------------------------------- embedding
struct EmbeddingArgs {
    const void* ids;
    int32_t id_bytes;
    int32_t accumulate;
    int64_t M;
    int64_t V;
    int32_t K;
    int32_t table_dtype;  // of E, dE
    int32_t row_dtype;    // of y, dy
    float scale;
    const void* E;
    void* y;
    const void* dy;
    void* dE;
    void* workspace;
    void* stream;
};

ss1_status launch_embedding_forward(const EmbeddingArgs& a);
size_t embedding_backward_workspace(int64_t M, int64_t V, int32_t K);
ss1_status launch_embedding_backward(const EmbeddingArgs& a);

// --------------------------------------------- block-scaled E4M3 matrices
inline int64_t up_to(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
// Bytes of a row of codes, and of a row of scales.
inline int64_t block_code_cols(int64_t cols) { return up_to(cols, SS1_FP8_BLOCK); }
inline int64_t block_scale_cols(int64_t cols) { return up_to(block_code_cols(cols) / SS1_FP8_BLOCK, 4); }

struct BlocksView {
    uint8_t* codes;  // null: not wanted
    uint8_t* scale;
    int64_t rows;
    int64_t code_cols;   // bytes of a row of codes
    int64_t scale_cols;  // bytes of a row of scales
    int32_t shift;       // rows of one scale: 1 << shift (0 or 7)
};

struct QuantizeBlocksArgs {
    const void* x;
    int64_t R, C;
    int32_t dtype;
    BlocksView q, qt;
    void* stream;
};

ss1_status launch_quantize_blocks(const QuantizeBlocksArgs& a);

struct MatmulBlocksArgs {
    BlocksView a, b;
    int64_t M, N;
    int64_t K;  // code_cols of both: a multiple of 128
    void* y;
    int32_t dtype;
    void* workspace;
    void* stream;
    // instead of a's codes: x [M][xcols] of y's dtype, quantised by the kernel itself
    const void* x = nullptr;
    int64_t xcols = 0;
};

// Partial sums of a product, 0 where one block finishes its outputs.
size_t matmul_blocks_workspace(int64_t M, int64_t N, int64_t K);
// Whether a product over x itself (not its codes) is offered at this size.
bool matmul_takes_x(int64_t M, int64_t N, int64_t K);
ss1_status launch_matmul_blocks(const MatmulBlocksArgs& a);
// Two products that do not depend on each other; they may share a workspace.
ss1_status launch_matmul_pair(const MatmulBlocksArgs& p, const MatmulBlocksArgs& q);

}  // namespace ss1
