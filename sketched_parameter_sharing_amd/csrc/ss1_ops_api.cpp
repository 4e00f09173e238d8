// The C ABI of the operators around an SS1 layer: argument checks, then the
// launch.  Every check runs on the host before any HIP call, so a call that
// fails a check has enqueued nothing.
#include <math.h>
#include <stdint.h>

#include "ss1_ops.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_dtype(int32_t t) { return t == SS1_F32 || t == SS1_BF16; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxCols = int64_t(1) << 24;
// 128 rows of an adapter or 64 of x stay within 2^31 bytes
constexpr int64_t kMaxAdapterCols = int64_t(1) << 22;
// segments plus M / 16 tiles of tokens, and adapters plus the parts of the outer
// products, are numbered in 32 bits
constexpr int32_t kMaxCount = int32_t(1) << 30;

// x of a layer norm: sizes and dtype.
ss1_status check_norm_x(const ss1_tensor* x) {
    if (!x) return SS1_ERR_NULL;
    if (x->reserved != 0) return SS1_ERR_SHAPE;
    if (!valid_dtype(x->dtype)) return SS1_ERR_DTYPE;
    if (x->rows < 0 || x->rows > kMaxRows || x->cols < 1 || x->cols >= kMaxCols) return SS1_ERR_SHAPE;
    if (x->rows > 0 && x->cols > (int64_t(1) << 40) / x->rows) return SS1_ERR_SHAPE;
    return SS1_OK;
}

// A [rows][cols] tensor of the given dtype with 16-byte aligned data.
ss1_status check_like(const ss1_tensor* t, int64_t rows, int64_t cols, int32_t dtype) {
    if (t->reserved != 0) return SS1_ERR_SHAPE;
    if (!valid_dtype(t->dtype) || t->dtype != dtype) return SS1_ERR_DTYPE;
    if (t->rows != rows || t->cols != cols) return SS1_ERR_SHAPE;
    if (rows > 0 && cols > 0 && !t->data) return SS1_ERR_NULL;
    if (!aligned(t->data, 16)) return SS1_ERR_ALIGN;
    return SS1_OK;
}

ss1_status check_gamma(const ss1_tensor* g, int64_t K, int32_t xdtype) {
    if (!g) return SS1_ERR_NULL;
    if (g->dtype != SS1_F32 && g->dtype != xdtype) return SS1_ERR_DTYPE;
    return check_like(g, 1, K, g->dtype);
}

#define SS1_TRY(expr)                      \
    do {                                   \
        const ss1_status st_ = (expr);     \
        if (st_ != SS1_OK) return st_;     \
    } while (0)

}  // namespace

// ---------------------------------------------------------------- layer norm
extern "C" ss1_status ss1_layernorm_forward(const ss1_tensor* x, const ss1_tensor* gamma, const ss1_tensor* beta,
                                            float eps, ss1_tensor* y, float* mean, float* rstd, void* stream) {
    if (!x || !gamma || !y) return SS1_ERR_NULL;
    SS1_TRY(check_norm_x(x));
    SS1_TRY(check_like(x, x->rows, x->cols, x->dtype));
    SS1_TRY(check_gamma(gamma, x->cols, x->dtype));
    if (beta) SS1_TRY(check_like(beta, 1, x->cols, gamma->dtype));
    SS1_TRY(check_like(y, x->rows, x->cols, x->dtype));
    if (!(eps >= 0.0f) || !isfinite(eps)) return SS1_ERR_SHAPE;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return SS1_ERR_ALIGN;
    if (x->rows == 0) return SS1_OK;
    ss1::NormArgs a{};
    a.x = x->data;
    a.gamma = gamma->data;
    a.beta = beta ? beta->data : nullptr;
    a.y = y->data;
    a.mean = mean;
    a.rstd = rstd;
    a.M = x->rows;
    a.K = static_cast<int32_t>(x->cols);
    a.dtype = x->dtype;
    a.affine_dtype = gamma->dtype;
    a.eps = eps;
    a.stream = stream;
    return ss1::launch_layernorm_forward(a);
}

extern "C" ss1_status ss1_layernorm_backward_query(const ss1_tensor* x, size_t* bytes) {
    if (!x || !bytes) return SS1_ERR_NULL;
    SS1_TRY(check_norm_x(x));
    *bytes = ss1::layernorm_backward_workspace(x->rows, static_cast<int32_t>(x->cols));
    return SS1_OK;
}

extern "C" ss1_status ss1_layernorm_backward(const ss1_tensor* dy, const ss1_tensor* x, const ss1_tensor* gamma,
                                             const float* mean, const float* rstd, ss1_tensor* dx,
                                             ss1_tensor* dgamma, ss1_tensor* dbeta, void* workspace,
                                             size_t workspace_bytes, void* stream) {
    if (!dy || !x || !gamma) return SS1_ERR_NULL;
    SS1_TRY(check_norm_x(x));
    const int64_t M = x->rows, K = x->cols;
    SS1_TRY(check_like(x, M, K, x->dtype));
    SS1_TRY(check_like(dy, M, K, x->dtype));
    SS1_TRY(check_gamma(gamma, K, x->dtype));
    if (dx) SS1_TRY(check_like(dx, M, K, x->dtype));
    if (dgamma) SS1_TRY(check_like(dgamma, 1, K, gamma->dtype));
    if (dbeta) SS1_TRY(check_like(dbeta, 1, K, gamma->dtype));
    if (M > 0 && (!mean || !rstd)) return SS1_ERR_NULL;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return SS1_ERR_ALIGN;
    if (!dx && !dgamma && !dbeta) return SS1_OK;
    const size_t need = dgamma || dbeta ? ss1::layernorm_backward_workspace(M, static_cast<int32_t>(K)) : 0;
    if (need > 0) {
        if (!workspace) return SS1_ERR_NULL;
        if (!aligned(workspace, 16)) return SS1_ERR_ALIGN;
        if (workspace_bytes < need) return SS1_ERR_SHAPE;
    }
    if (M == 0 && !dgamma && !dbeta) return SS1_OK;
    ss1::NormArgs a{};
    a.x = x->data;
    a.gamma = gamma->data;
    a.dy = dy->data;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.dx = dx ? dx->data : nullptr;
    a.dgamma = dgamma ? dgamma->data : nullptr;
    a.dbeta = dbeta ? dbeta->data : nullptr;
    a.partial = static_cast<float*>(workspace);
    a.M = M;
    a.K = static_cast<int32_t>(K);
    a.dtype = x->dtype;
    a.affine_dtype = gamma->dtype;
    a.stream = stream;
    return ss1::launch_layernorm_backward(a);
}

// ------------------------------------------------------------------ adapters
namespace {

// The adapters' factors and sizes; data pointers only when `data`.
ss1_status check_adapters(const ss1_adapters* ad, bool data) {
    if (!ad) return SS1_ERR_NULL;
    const ss1_tensor &A = ad->A, &B = ad->B;
    if (A.reserved != 0 || B.reserved != 0) return SS1_ERR_SHAPE;
    if (!valid_dtype(A.dtype) || B.dtype != A.dtype) return SS1_ERR_DTYPE;
    if (A.rows < 0 || A.rows > kMaxRows || B.rows != A.rows) return SS1_ERR_SHAPE;
    const int64_t unit = A.dtype == SS1_BF16 ? 8 : 4;
    for (const int64_t n : {A.cols, B.cols})
        if (n < unit || n >= kMaxAdapterCols || n % unit) return SS1_ERR_SHAPE;
    if (ad->count < 0 || ad->count >= kMaxCount || ad->max_rank < 0 || ad->max_rank > SS1_MAX_RANK) return SS1_ERR_SHAPE;
    if (!data) return SS1_OK;
    if (A.rows > 0 && (!A.data || !B.data)) return SS1_ERR_NULL;
    if (!ad->row || (ad->count > 0 && !ad->scale)) return SS1_ERR_NULL;
    if (!aligned(A.data, 16) || !aligned(B.data, 16) || !aligned(ad->row, 4) || !aligned(ad->scale, 4))
        return SS1_ERR_ALIGN;
    return SS1_OK;
}

ss1_status check_segments(const ss1_segments* s) {
    if (!s) return SS1_ERR_NULL;
    if (s->reserved != 0 || s->count < 0 || s->count >= kMaxCount) return SS1_ERR_SHAPE;
    if (s->count > 0 && (!s->offset || !s->adapter)) return SS1_ERR_NULL;
    if (!aligned(s->offset, 4) || !aligned(s->adapter, 4)) return SS1_ERR_ALIGN;
    return SS1_OK;
}

ss1_status check_tokens(int64_t M, const ss1_adapters* ad) {
    if (M < 0 || M > kMaxRows) return SS1_ERR_SHAPE;
    const int64_t wide = ad->A.cols > ad->B.cols ? ad->A.cols : ad->B.cols;
    if (M > 0 && wide > (int64_t(1) << 40) / M) return SS1_ERR_SHAPE;
    return SS1_OK;
}

ss1_status check_workspace(const void* workspace, size_t have, size_t need) {
    if (need == 0) return SS1_OK;
    if (!workspace) return SS1_ERR_NULL;
    if (!aligned(workspace, 16)) return SS1_ERR_ALIGN;
    return have < need ? SS1_ERR_SHAPE : SS1_OK;
}

void fill_adapter(const ss1_adapters* ad, const ss1_segments* s, int64_t M, void* workspace, void* stream,
                  ss1::AdapterArgs* a) {
    a->ad = {ad->row,   ad->scale, s->offset, s->adapter, ad->count, s->count, static_cast<int32_t>(ad->A.rows),
             ad->max_rank, static_cast<int32_t>(M)};
    // no rows, no adapters or no ranks: every token goes without
    if (ad->A.rows == 0 || ad->max_rank == 0) a->ad.E = 0;
    a->A = ad->A.data;
    a->B = ad->B.data;
    a->K = static_cast<int32_t>(ad->A.cols);
    a->N = static_cast<int32_t>(ad->B.cols);
    a->dtype = ad->A.dtype;
    a->workspace = workspace;
    a->stream = stream;
}

size_t forward_bytes(int64_t M, const ss1_adapters* ad) {
    // as fill_adapter: no rows or no ranks count as no adapters
    const int32_t E = ad->A.rows == 0 || ad->max_rank == 0 ? 0 : ad->count;
    return ss1::adapter_forward_workspace(M, static_cast<int32_t>(ad->A.cols), static_cast<int32_t>(ad->B.cols), E,
                                          static_cast<int32_t>(ad->A.rows), ad->max_rank, ad->A.dtype);
}

size_t backward_bytes(int64_t M, const ss1_adapters* ad) {
    // as fill_adapter: no rows or no ranks count as no adapters
    const int32_t E = ad->A.rows == 0 || ad->max_rank == 0 ? 0 : ad->count;
    return ss1::adapter_backward_workspace(M, static_cast<int32_t>(ad->A.cols), static_cast<int32_t>(ad->B.cols), E,
                                          static_cast<int32_t>(ad->A.rows), ad->max_rank, ad->A.dtype);
}

}  // namespace

extern "C" ss1_status ss1_adapter_forward_query(int64_t M, const ss1_adapters* adapters, size_t* bytes) {
    if (!bytes) return SS1_ERR_NULL;
    SS1_TRY(check_adapters(adapters, false));
    SS1_TRY(check_tokens(M, adapters));
    *bytes = forward_bytes(M, adapters);
    return SS1_OK;
}

extern "C" ss1_status ss1_adapter_backward_query(int64_t M, const ss1_adapters* adapters, size_t* bytes) {
    if (!bytes) return SS1_ERR_NULL;
    SS1_TRY(check_adapters(adapters, false));
    SS1_TRY(check_tokens(M, adapters));
    *bytes = backward_bytes(M, adapters);
    return SS1_OK;
}

extern "C" ss1_status ss1_adapter_forward(const ss1_tensor* x, const ss1_adapters* adapters,
                                          const ss1_segments* segments, const ss1_tensor* base, ss1_tensor* y,
                                          ss1_tensor* v, void* workspace, size_t workspace_bytes, void* stream) {
    if (!x || !adapters || !segments || !y) return SS1_ERR_NULL;
    SS1_TRY(check_adapters(adapters, true));
    SS1_TRY(check_segments(segments));
    const int64_t M = x->rows;
    SS1_TRY(check_tokens(M, adapters));
    const int32_t dt = adapters->A.dtype;
    SS1_TRY(check_like(x, M, adapters->A.cols, dt));
    SS1_TRY(check_like(y, M, adapters->B.cols, dt));
    if (base) SS1_TRY(check_like(base, M, adapters->B.cols, dt));
    if (v) SS1_TRY(check_like(v, M, adapters->max_rank, SS1_F32));
    SS1_TRY(check_workspace(workspace, workspace_bytes, forward_bytes(M, adapters)));
    if (M == 0) return SS1_OK;
    ss1::AdapterArgs a{};
    fill_adapter(adapters, segments, M, workspace, stream, &a);
    a.x = x->data;
    a.base = base ? base->data : nullptr;
    a.y = y->data;
    a.v = v && adapters->max_rank > 0 ? static_cast<float*>(v->data) : nullptr;
    return ss1::launch_adapter_forward(a);
}

extern "C" ss1_status ss1_adapter_backward(const ss1_tensor* dy, const ss1_tensor* x, const ss1_tensor* v,
                                           const ss1_adapters* adapters, const ss1_segments* segments,
                                           const ss1_tensor* dx_base, ss1_tensor* dx, ss1_tensor* dA,
                                           ss1_tensor* dB, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dy || !x || !adapters || !segments || (dB && !v)) return SS1_ERR_NULL;
    SS1_TRY(check_adapters(adapters, true));
    SS1_TRY(check_segments(segments));
    const int64_t M = x->rows, K = adapters->A.cols, N = adapters->B.cols, R = adapters->A.rows;
    SS1_TRY(check_tokens(M, adapters));
    const int32_t dt = adapters->A.dtype;
    SS1_TRY(check_like(x, M, K, dt));
    SS1_TRY(check_like(dy, M, N, dt));
    if (v) SS1_TRY(check_like(v, M, adapters->max_rank, SS1_F32));
    if (dx_base) SS1_TRY(check_like(dx_base, M, K, dt));
    if (dx) SS1_TRY(check_like(dx, M, K, dt));
    if (dA) SS1_TRY(check_like(dA, R, K, dt));
    if (dB) SS1_TRY(check_like(dB, R, N, dt));
    SS1_TRY(check_workspace(workspace, workspace_bytes, backward_bytes(M, adapters)));
    if (!dx && !dA && !dB) return SS1_OK;
    if (M == 0 && R == 0) return SS1_OK;
    ss1::AdapterArgs a{};
    fill_adapter(adapters, segments, M, workspace, stream, &a);
    a.x = x->data;
    a.dy = dy->data;
    a.v = v ? static_cast<float*>(v->data) : nullptr;
    a.base = dx_base ? dx_base->data : nullptr;
    a.dx = dx && M > 0 ? dx->data : nullptr;
    a.dA = dA && R > 0 ? dA->data : nullptr;
    a.dB = dB && R > 0 ? dB->data : nullptr;
    return ss1::launch_adapter_backward(a);
}

// --------------------------------------------------------------------- AdamW
extern "C" ss1_status ss1_adamw_plan(const ss1_adamw_entry* entries, int32_t count, int64_t* chunks, int32_t* map) {
    if (!chunks || (count > 0 && !entries)) return SS1_ERR_NULL;
    if (count < 0 || count >= (1 << 23)) return SS1_ERR_SHAPE;
    int64_t n = 0;
    for (int32_t i = 0; i < count; ++i) {
        const ss1_adamw_entry& e = entries[i];
        if (!valid_dtype(e.param_dtype) || !valid_dtype(e.grad_dtype) ||
            (e.state_dtype != SS1_F32 && e.state_dtype != SS1_FP8_E4M3))
            return SS1_ERR_DTYPE;
        if (e.numel < 0 || e.numel >= (int64_t(1) << 39)) return SS1_ERR_SHAPE;
        if (!(e.weight_decay >= 0.0f) || !isfinite(e.weight_decay)) return SS1_ERR_SHAPE;
        if (e.master && e.param_dtype != SS1_BF16) return SS1_ERR_SHAPE;
        if (e.numel == 0) continue;
        if (!e.param || !e.grad || !e.m || !e.v) return SS1_ERR_NULL;
        if (e.state_dtype == SS1_FP8_E4M3 && (!e.m_scale || !e.v_scale)) return SS1_ERR_NULL;
        for (const void* p : {static_cast<const void*>(e.param), e.grad, static_cast<const void*>(e.m),
                              static_cast<const void*>(e.v), static_cast<const void*>(e.master)})
            if (!aligned(p, 16)) return SS1_ERR_ALIGN;
        if (!aligned(e.m_scale, 4) || !aligned(e.v_scale, 4)) return SS1_ERR_ALIGN;
        const int64_t c = (e.numel + ss1::kAdamWChunk - 1) / ss1::kAdamWChunk;
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

extern "C" ss1_status ss1_adamw_step(const ss1_adamw_entry* entries, int32_t count, const int32_t* map,
                                     int64_t chunks, const ss1_adamw_hyper* hyper, void* stream) {
    if (!hyper) return SS1_ERR_NULL;
    if (count < 0 || chunks < 0 || chunks > kMaxRows || hyper->step < 1) return SS1_ERR_SHAPE;
    const double b1 = hyper->beta1, b2 = hyper->beta2;
    if (!(b1 >= 0.0 && b1 < 1.0) || !(b2 >= 0.0 && b2 < 1.0)) return SS1_ERR_SHAPE;
    for (const double d : {hyper->lr, hyper->eps, hyper->grad_scale})
        if (!(d >= 0.0) || !isfinite(d)) return SS1_ERR_SHAPE;
    if (chunks == 0) return SS1_OK;
    if (!entries || !map) return SS1_ERR_NULL;
    if (!aligned(entries, 8) || !aligned(map, 4) || !aligned(hyper->grad_scale_dev, 4)) return SS1_ERR_ALIGN;
    ss1::AdamWCoef c;
    c.beta1 = static_cast<float>(b1);
    c.one_minus_beta1 = static_cast<float>(1.0 - b1);
    c.beta2 = static_cast<float>(b2);
    c.one_minus_beta2 = static_cast<float>(1.0 - b2);
    const double t = static_cast<double>(hyper->step);
    c.step_size = static_cast<float>(hyper->lr / (1.0 - pow(b1, t)));
    c.inv_sqrt_c2 = static_cast<float>(1.0 / sqrt(1.0 - pow(b2, t)));
    c.eps = static_cast<float>(hyper->eps);
    c.grad_scale = static_cast<float>(hyper->grad_scale);
    c.grad_scale_dev = hyper->grad_scale_dev;
    c.lr = hyper->lr;
    c.seed = hyper->seed;
    return ss1::launch_adamw(entries, count, map, chunks, c, stream);
}
