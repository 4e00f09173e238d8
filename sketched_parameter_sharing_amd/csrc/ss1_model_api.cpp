// The C ABI of the operators at a model's ends and of its dense layers:
// argument checks, then the launches.  Every check of a call runs on the host
// before any HIP call, so a call that fails a check has enqueued nothing.
#include <math.h>
#include <stdint.h>

#include "ss1_model_ops.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_dtype(int32_t t) { return t == SS1_F32 || t == SS1_BF16; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
// a grid's threads are numbered in 32 bits: rows of a table over 64 rows a block
constexpr int64_t kMaxTable = int64_t(1) << 29;
constexpr int64_t kMaxWidth = int64_t(1) << 16;
// tokens of an embedding's gradient: places rounded up to whole tiles stay under 2^31
constexpr int64_t kMaxGradTokens = int64_t(1) << 30;
// tiles of 128 x 128 of a matrix that is quantised, and of a product
constexpr int64_t kMaxQuantTiles = int64_t(1) << 24;
constexpr int64_t kMaxTiles = int64_t(1) << 22;
// 256 rows of codes stay within 2^31 bytes
constexpr int64_t kMaxReduction = int64_t(1) << 23;

#define SS1_TRY(expr)                      \
    do {                                   \
        const ss1_status st_ = (expr);     \
        if (st_ != SS1_OK) return st_;     \
    } while (0)

// A [rows][cols] matrix of float32 or bf16, its product of sizes under 2^40;
// the data pointer only when `data`.
ss1_status check_matrix(const ss1_tensor* t, bool data) {
    if (!t) return SS1_ERR_NULL;
    if (t->reserved != 0) return SS1_ERR_SHAPE;
    if (!valid_dtype(t->dtype)) return SS1_ERR_DTYPE;
    if (t->rows < 0 || t->rows > kMaxRows || t->cols < 0 || t->cols > kMaxRows) return SS1_ERR_SHAPE;
    if (t->rows > 0 && t->cols > (int64_t(1) << 40) / t->rows) return SS1_ERR_SHAPE;
    if (!data) return SS1_OK;
    if (t->rows > 0 && t->cols > 0 && !t->data) return SS1_ERR_NULL;
    return aligned(t->data, 16) ? SS1_OK : SS1_ERR_ALIGN;
}

// Fewer than `most` tiles of 128 x 128.
ss1_status check_tiles(int64_t rows, int64_t cols, int64_t most) {
    const int64_t r = (rows + 127) / 128, c = (cols + 127) / 128;
    return r > 0 && c > (most - 1) / r ? SS1_ERR_SHAPE : SS1_OK;
}

ss1_status check_sizes(const ss1_tensor* t, int64_t rows, int64_t cols) {
    return t->rows == rows && t->cols == cols ? SS1_OK : SS1_ERR_SHAPE;
}

ss1_status check_workspace(const void* workspace, size_t have, size_t need) {
    if (need == 0) return SS1_OK;
    if (!workspace) return SS1_ERR_NULL;
    if (!aligned(workspace, 16)) return SS1_ERR_ALIGN;
    return have < need ? SS1_ERR_SHAPE : SS1_OK;
}

}  // namespace

// ------------------------------------------------------------- gradient norm
extern "C" ss1_status ss1_gradnorm_plan(const ss1_gradnorm_entry* entries, int32_t count, int64_t* chunks,
                                        int32_t* map) {
    if (!chunks || (count > 0 && !entries)) return SS1_ERR_NULL;
    if (count < 0 || count >= (1 << 23)) return SS1_ERR_SHAPE;
    int64_t n = 0;
    for (int32_t i = 0; i < count; ++i) {
        const ss1_gradnorm_entry& e = entries[i];
        if (e.reserved != 0) return SS1_ERR_SHAPE;
        if (!valid_dtype(e.dtype)) return SS1_ERR_DTYPE;
        if (e.numel < 0 || e.numel >= (int64_t(1) << 39)) return SS1_ERR_SHAPE;
        if (e.numel == 0) continue;
        if (!e.grad) return SS1_ERR_NULL;
        if (!aligned(e.grad, 16)) return SS1_ERR_ALIGN;
        const int64_t c = (e.numel + ss1::kNormChunk - 1) / ss1::kNormChunk;
        if (n + c > kMaxRows) return SS1_ERR_SHAPE;
        if (map)
            for (int64_t j = 0; j < c; ++j) {
                map[2 * (n + j)] = i;
                map[2 * (n + j) + 1] = static_cast<int32_t>(j);
            }
        n += c;
    }
    *chunks = n;
    return SS1_OK;
}

extern "C" ss1_status ss1_gradnorm_query(int64_t chunks, size_t* bytes) {
    if (!bytes) return SS1_ERR_NULL;
    if (chunks < 0 || chunks > kMaxRows) return SS1_ERR_SHAPE;
    *bytes = ss1::gradnorm_workspace(chunks);
    return SS1_OK;
}

namespace {

ss1_status gradnorm(const ss1_gradnorm_entry* entries, int32_t count, const int32_t* map, int64_t chunks,
                    double max_norm, float* norm, float* coef, void* workspace, size_t workspace_bytes, void* stream,
                    bool clip) {
    if (count < 0 || chunks < 0 || chunks > kMaxRows || !(max_norm >= 0.0)) return SS1_ERR_SHAPE;
    if (!aligned(norm, 4) || !aligned(coef, 4)) return SS1_ERR_ALIGN;
    if (chunks > 0) {
        if (!entries || !map) return SS1_ERR_NULL;
        if (!aligned(entries, 8) || !aligned(map, 4)) return SS1_ERR_ALIGN;
        SS1_TRY(check_workspace(workspace, workspace_bytes, ss1::gradnorm_workspace(chunks)));
    }
    if (!norm && !coef && (!clip || chunks == 0)) return SS1_OK;
    const ss1::GradNormArgs a{entries, map,  chunks, count, max_norm, norm, coef, static_cast<double*>(workspace), stream};
    return clip ? ss1::launch_gradnorm_clip(a) : ss1::launch_gradnorm(a);
}

}  // namespace

extern "C" ss1_status ss1_gradnorm(const ss1_gradnorm_entry* entries, int32_t count, const int32_t* map,
                                   int64_t chunks, double max_norm, float* norm, float* coef, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    return gradnorm(entries, count, map, chunks, max_norm, norm, coef, workspace, workspace_bytes, stream, false);
}

extern "C" ss1_status ss1_gradnorm_clip(const ss1_gradnorm_entry* entries, int32_t count, const int32_t* map,
                                        int64_t chunks, double max_norm, float* norm, float* coef, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    return gradnorm(entries, count, map, chunks, max_norm, norm, coef, workspace, workspace_bytes, stream, true);
}

// ----------------------------------------------------------------- embedding
namespace {

ss1_status check_tokens(const ss1_tokens* t, bool data) {
    if (!t) return SS1_ERR_NULL;
    if (t->reserved != 0 || t->count < 0 || t->count > kMaxRows) return SS1_ERR_SHAPE;
    if (t->bytes != 4 && t->bytes != 8) return SS1_ERR_DTYPE;
    if (!data || t->count == 0) return SS1_OK;
    if (!t->id) return SS1_ERR_NULL;
    return aligned(t->id, static_cast<uintptr_t>(t->bytes)) ? SS1_OK : SS1_ERR_ALIGN;
}

ss1_status check_table(const ss1_tensor* E, bool data) {
    SS1_TRY(check_matrix(E, data));
    return E->rows >= kMaxTable || E->cols < 1 || E->cols > kMaxWidth ? SS1_ERR_SHAPE : SS1_OK;
}

ss1::EmbeddingArgs embedding_args(const ss1_tokens* tokens, const ss1_tensor* table, const ss1_tensor* rows,
                                  float scale, void* stream) {
    ss1::EmbeddingArgs a{};
    a.ids = tokens->id;
    a.id_bytes = tokens->bytes;
    a.M = tokens->count;
    a.V = table->rows;
    a.K = static_cast<int32_t>(table->cols);
    a.table_dtype = table->dtype;
    a.row_dtype = rows->dtype;
    a.scale = scale;
    a.stream = stream;
    return a;
}

}  // namespace

extern "C" ss1_status ss1_embedding_forward(const ss1_tokens* tokens, const ss1_tensor* E, float scale, ss1_tensor* y,
                                            void* stream) {
    if (!tokens || !E || !y) return SS1_ERR_NULL;
    SS1_TRY(check_tokens(tokens, true));
    SS1_TRY(check_table(E, true));
    SS1_TRY(check_matrix(y, true));
    SS1_TRY(check_sizes(y, tokens->count, E->cols));
    if (!isfinite(scale)) return SS1_ERR_SHAPE;
    if (tokens->count == 0) return SS1_OK;
    ss1::EmbeddingArgs a = embedding_args(tokens, E, y, scale, stream);
    a.E = E->data;
    a.y = y->data;
    return ss1::launch_embedding_forward(a);
}

extern "C" ss1_status ss1_embedding_backward_query(const ss1_tokens* tokens, const ss1_tensor* dE, size_t* bytes) {
    if (!bytes) return SS1_ERR_NULL;
    SS1_TRY(check_tokens(tokens, false));
    SS1_TRY(check_table(dE, false));
    if (tokens->count >= kMaxGradTokens) return SS1_ERR_SHAPE;
    if (tokens->count > 0 && dE->cols > (int64_t(1) << 40) / tokens->count) return SS1_ERR_SHAPE;
    *bytes = ss1::embedding_backward_workspace(tokens->count, dE->rows, static_cast<int32_t>(dE->cols));
    return SS1_OK;
}

extern "C" ss1_status ss1_embedding_backward(const ss1_tensor* dy, const ss1_tokens* tokens, float scale,
                                             int32_t accumulate, ss1_tensor* dE, void* workspace,
                                             size_t workspace_bytes, void* stream) {
    if (!dy || !tokens || !dE) return SS1_ERR_NULL;
    SS1_TRY(check_tokens(tokens, true));
    SS1_TRY(check_table(dE, true));
    SS1_TRY(check_matrix(dy, true));
    SS1_TRY(check_sizes(dy, tokens->count, dE->cols));
    if (tokens->count >= kMaxGradTokens) return SS1_ERR_SHAPE;
    if (!isfinite(scale) || (accumulate != 0 && accumulate != 1)) return SS1_ERR_SHAPE;
    SS1_TRY(check_workspace(workspace, workspace_bytes,
                            ss1::embedding_backward_workspace(tokens->count, dE->rows,
                                                              static_cast<int32_t>(dE->cols))));
    if (dE->rows == 0 || (tokens->count == 0 && accumulate)) return SS1_OK;
    ss1::EmbeddingArgs a = embedding_args(tokens, dE, dy, scale, stream);
    a.accumulate = accumulate;
    a.dy = dy->data;
    a.dE = dE->data;
    a.workspace = workspace;
    return ss1::launch_embedding_backward(a);
}

// ---------------------------------------------- block-scaled E4M3 matrices
namespace {

ss1_status check_blocks(const ss1_fp8_blocks* b, bool data) {
    if (!b) return SS1_ERR_NULL;
    if (b->reserved != 0 || (b->block != 1 && b->block != SS1_FP8_BLOCK)) return SS1_ERR_SHAPE;
    if (b->rows < 0 || b->rows > kMaxRows || b->cols < 0 || b->cols > kMaxRows) return SS1_ERR_SHAPE;
    if (b->rows > 0 && b->cols > (int64_t(1) << 40) / b->rows) return SS1_ERR_SHAPE;
    if (!data) return SS1_OK;
    if (b->rows > 0 && b->cols > 0 && (!b->codes || !b->scale)) return SS1_ERR_NULL;
    return aligned(b->codes, 16) && aligned(b->scale, 4) ? SS1_OK : SS1_ERR_ALIGN;
}

ss1_status check_blocks_sizes(const ss1_fp8_blocks* b, int64_t rows, int64_t cols) {
    return b->rows == rows && b->cols == cols ? SS1_OK : SS1_ERR_SHAPE;
}

// A side of a product: its reduction is short enough for 32-bit offsets over a
// tile's rows.
ss1_status check_operand(const ss1_fp8_blocks* b, bool data) {
    SS1_TRY(check_blocks(b, data));
    return b->cols < kMaxReduction ? SS1_OK : SS1_ERR_SHAPE;
}

ss1::BlocksView view_of(const ss1_fp8_blocks* b) {
    return {static_cast<uint8_t*>(b->codes),      b->scale, b->rows, ss1::block_code_cols(b->cols),
            ss1::block_scale_cols(b->cols), b->block == 1 ? 0 : 7};
}

// Codes and scales of a [rows][cols] matrix with a scale for 128 elements of a
// row, at `at` in a workspace; the place behind them.
size_t blocks_bytes(int64_t rows, int64_t cols) {
    return static_cast<size_t>(ss1::up_to(rows * ss1::block_code_cols(cols), 16) +
                               ss1::up_to(rows * ss1::block_scale_cols(cols), 16));
}
ss1::BlocksView blocks_in(void* workspace, size_t at, int64_t rows, int64_t cols) {
    uint8_t* p = static_cast<uint8_t*>(workspace) + at;
    const int64_t cp = ss1::block_code_cols(cols);
    return {p, p + ss1::up_to(rows * cp, 16), rows, cp, ss1::block_scale_cols(cols), 0};
}

ss1::MatmulBlocksArgs product(const ss1::BlocksView& a, const ss1::BlocksView& b, const ss1_tensor* y, void* workspace,
                              void* stream) {
    ss1::MatmulBlocksArgs p{};
    p.a = a;
    p.b = b;
    p.M = y->rows;
    p.N = y->cols;
    p.K = b.code_cols;
    p.y = y->data;
    p.dtype = y->dtype;
    p.workspace = workspace;
    p.stream = stream;
    return p;
}

size_t product_bytes(int64_t M, int64_t N, int64_t cols) {
    return ss1::matmul_blocks_workspace(M, N, ss1::block_code_cols(cols));
}

}  // namespace

extern "C" ss1_status ss1_quantize_fp8_blocks(const ss1_tensor* x, ss1_fp8_blocks* q, ss1_fp8_blocks* qt,
                                              void* stream) {
    if (!x) return SS1_ERR_NULL;
    SS1_TRY(check_matrix(x, true));
    SS1_TRY(check_tiles(x->rows, x->cols, kMaxQuantTiles));
    if (q) {
        SS1_TRY(check_blocks(q, true));
        SS1_TRY(check_blocks_sizes(q, x->rows, x->cols));
    }
    if (qt) {
        SS1_TRY(check_blocks(qt, true));
        SS1_TRY(check_blocks_sizes(qt, x->cols, x->rows));
    }
    if ((!q && !qt) || x->rows == 0 || x->cols == 0) return SS1_OK;
    ss1::QuantizeBlocksArgs a{};
    a.x = x->data;
    a.R = x->rows;
    a.C = x->cols;
    a.dtype = x->dtype;
    if (q) a.q = view_of(q);
    if (qt) a.qt = view_of(qt);
    a.stream = stream;
    return ss1::launch_quantize_blocks(a);
}

extern "C" ss1_status ss1_matmul_fp8_blocks_query(const ss1_fp8_blocks* a, const ss1_fp8_blocks* b, size_t* bytes) {
    if (!bytes) return SS1_ERR_NULL;
    SS1_TRY(check_operand(a, false));
    SS1_TRY(check_operand(b, false));
    if (a->cols != b->cols) return SS1_ERR_SHAPE;
    SS1_TRY(check_tiles(a->rows, b->rows, kMaxTiles));
    *bytes = product_bytes(a->rows, b->rows, a->cols);
    return SS1_OK;
}

extern "C" ss1_status ss1_matmul_fp8_blocks(const ss1_fp8_blocks* a, const ss1_fp8_blocks* b, ss1_tensor* y,
                                            void* workspace, size_t workspace_bytes, void* stream) {
    if (!a || !b || !y) return SS1_ERR_NULL;
    SS1_TRY(check_operand(a, true));
    SS1_TRY(check_operand(b, true));
    if (a->cols != b->cols) return SS1_ERR_SHAPE;
    SS1_TRY(check_tiles(a->rows, b->rows, kMaxTiles));
    SS1_TRY(check_matrix(y, true));
    SS1_TRY(check_sizes(y, a->rows, b->rows));
    SS1_TRY(check_workspace(workspace, workspace_bytes, product_bytes(a->rows, b->rows, a->cols)));
    if (y->rows == 0 || y->cols == 0) return SS1_OK;
    return ss1::launch_matmul_blocks(product(view_of(a), view_of(b), y, workspace, stream));
}

// -------------------------------------------------------------- dense layers
namespace {

// Workspace of a dense layer's calls: the codes made in the call, then the
// partial sums of its products (which follow each other and share them).
size_t dense_forward_bytes(int64_t M, int64_t N, int64_t K) {
    const size_t codes = ss1::matmul_takes_x(M, N, ss1::block_code_cols(K)) ? 0 : blocks_bytes(M, K);
    return codes + product_bytes(M, N, K);
}
size_t dense_backward_bytes(int64_t M, int64_t N, int64_t K, bool dx, bool dW) {
    const size_t px = dx ? product_bytes(M, K, N) : 0, pw = dW ? product_bytes(N, K, M) : 0;
    return (dx ? blocks_bytes(M, N) : 0) + (dW ? blocks_bytes(N, M) : 0) + (px > pw ? px : pw);
}

ss1_status check_dense_forward(const ss1_tensor* x, const ss1_fp8_blocks* w, bool data) {
    SS1_TRY(check_matrix(x, data));
    SS1_TRY(check_operand(w, data));
    if (x->cols != w->cols) return SS1_ERR_SHAPE;
    SS1_TRY(check_tiles(x->rows, x->cols, kMaxQuantTiles));
    return check_tiles(x->rows, w->rows, kMaxTiles);
}

// xt is [K][M] (block 1), wt is [K][N], dy is [M][N].
ss1_status check_dense_backward(const ss1_tensor* dy, const ss1_fp8_blocks* xt, const ss1_fp8_blocks* wt, bool data) {
    SS1_TRY(check_matrix(dy, data));
    const int64_t M = dy->rows, N = dy->cols;
    SS1_TRY(check_tiles(M, N, kMaxQuantTiles));
    if (wt) {
        SS1_TRY(check_operand(wt, data));
        if (wt->cols != N) return SS1_ERR_SHAPE;
        SS1_TRY(check_tiles(M, wt->rows, kMaxTiles));
    }
    if (xt) {
        SS1_TRY(check_operand(xt, data));
        if (xt->cols != M) return SS1_ERR_SHAPE;
        SS1_TRY(check_tiles(N, xt->rows, kMaxTiles));
    }
    return wt && xt && wt->rows != xt->rows ? SS1_ERR_SHAPE : SS1_OK;
}

}  // namespace

extern "C" ss1_status ss1_dense_forward_fp8_query(const ss1_tensor* x, const ss1_fp8_blocks* w, size_t* bytes) {
    if (!x || !w || !bytes) return SS1_ERR_NULL;
    SS1_TRY(check_dense_forward(x, w, false));
    *bytes = dense_forward_bytes(x->rows, w->rows, x->cols);
    return SS1_OK;
}

extern "C" ss1_status ss1_dense_forward_fp8(const ss1_tensor* x, const ss1_fp8_blocks* w, ss1_tensor* y,
                                            ss1_fp8_blocks* xt, void* workspace, size_t workspace_bytes,
                                            void* stream) {
    if (!x || !w || !y) return SS1_ERR_NULL;
    SS1_TRY(check_dense_forward(x, w, true));
    const int64_t M = x->rows, K = x->cols, N = w->rows;
    SS1_TRY(check_matrix(y, true));
    if (y->dtype != x->dtype) return SS1_ERR_DTYPE;
    SS1_TRY(check_sizes(y, M, N));
    if (xt) {
        SS1_TRY(check_blocks(xt, true));
        SS1_TRY(check_blocks_sizes(xt, K, M));
        if (xt->block != 1) return SS1_ERR_SHAPE;
    }
    SS1_TRY(check_workspace(workspace, workspace_bytes, dense_forward_bytes(M, N, K)));
    if (M == 0) return SS1_OK;
    const bool inside = ss1::matmul_takes_x(M, N, ss1::block_code_cols(K));
    ss1::QuantizeBlocksArgs q{};
    q.x = x->data;
    q.R = M;
    q.C = K;
    q.dtype = x->dtype;
    q.stream = stream;
    size_t at = 0;
    if (!inside && N > 0) {
        q.q = blocks_in(workspace, 0, M, K);
        at = blocks_bytes(M, K);
    }
    if (xt) q.qt = view_of(xt);
    if (K > 0 && (q.q.codes || q.qt.codes)) SS1_TRY(ss1::launch_quantize_blocks(q));
    if (N == 0) return SS1_OK;
    ss1::MatmulBlocksArgs p = product(q.q, view_of(w), y, static_cast<uint8_t*>(workspace) + at, stream);
    if (inside) {
        p.x = x->data;
        p.xcols = K;
    }
    return ss1::launch_matmul_blocks(p);
}

extern "C" ss1_status ss1_dense_backward_fp8_query(const ss1_tensor* dy, const ss1_fp8_blocks* xt,
                                                   const ss1_fp8_blocks* wt, size_t* bytes) {
    if (!dy || !bytes) return SS1_ERR_NULL;
    SS1_TRY(check_dense_backward(dy, xt, wt, false));
    *bytes = dense_backward_bytes(dy->rows, dy->cols, wt ? wt->rows : xt ? xt->rows : 0, wt != nullptr, xt != nullptr);
    return SS1_OK;
}

extern "C" ss1_status ss1_dense_backward_fp8(const ss1_tensor* dy, const ss1_fp8_blocks* xt, const ss1_fp8_blocks* wt,
                                             ss1_tensor* dx, ss1_tensor* dW, void* workspace, size_t workspace_bytes,
                                             void* stream) {
    if (!dy || (dx && !wt) || (dW && !xt)) return SS1_ERR_NULL;
    SS1_TRY(check_dense_backward(dy, dW ? xt : nullptr, dx ? wt : nullptr, true));
    const int64_t M = dy->rows, N = dy->cols, K = dx ? wt->rows : dW ? xt->rows : 0;
    if (dx) {
        SS1_TRY(check_matrix(dx, true));
        if (dx->dtype != dy->dtype) return SS1_ERR_DTYPE;
        SS1_TRY(check_sizes(dx, M, K));
    }
    if (dW) {
        SS1_TRY(check_matrix(dW, true));
        SS1_TRY(check_sizes(dW, N, K));
        if (xt->block != 1) return SS1_ERR_SHAPE;
    }
    const size_t need = dense_backward_bytes(M, N, K, dx != nullptr, dW != nullptr);
    SS1_TRY(check_workspace(workspace, workspace_bytes, need));
    // an empty side leaves the other's sum over it: zeros, by the products below
    const bool do_dx = dx && M > 0 && K > 0, do_dW = dW && N > 0 && K > 0;
    if (!do_dx && !do_dW) return SS1_OK;
    ss1::QuantizeBlocksArgs q{};
    q.x = dy->data;
    q.R = M;
    q.C = N;
    q.dtype = dy->dtype;
    q.stream = stream;
    size_t at = 0;
    if (do_dx) {
        q.q = blocks_in(workspace, at, M, N);
        at += blocks_bytes(M, N);
    }
    if (do_dW) {
        q.qt = blocks_in(workspace, at, N, M);
        at += blocks_bytes(N, M);
    }
    if (M > 0 && N > 0) SS1_TRY(ss1::launch_quantize_blocks(q));
    void* rest = static_cast<uint8_t*>(workspace) + at;
    if (!do_dW) return ss1::launch_matmul_blocks(product(q.q, view_of(wt), dx, rest, stream));
    if (!do_dx) return ss1::launch_matmul_blocks(product(q.qt, view_of(xt), dW, rest, stream));
    return ss1::launch_matmul_pair(product(q.q, view_of(wt), dx, rest, stream),
                                   product(q.qt, view_of(xt), dW, rest, stream));
}
