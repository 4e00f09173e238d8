// Internal declarations of the operators around an SS1 layer (layer norm,
// low-rank adapters, AdamW): the checked arguments that the ABI layer hands
// to the kernel launchers.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/ss1.h"

namespace ss1 {

struct NormArgs {
    const void* x;
    const void* gamma;
    const void* beta;  // forward; may be null
    const void* dy;    // backward
    const float* mean_in;
    const float* rstd_in;
    float* mean;       // forward; may be null
    float* rstd;
    void* y;           // forward
    void* dx;          // backward; may be null
    void* dgamma;
    void* dbeta;
    float* partial;    // backward workspace
    int64_t M;
    int32_t K;
    int32_t dtype;         // of x, y, dy, dx
    int32_t affine_dtype;  // of gamma, beta, dgamma, dbeta
    float eps;
    void* stream;
};

size_t layernorm_backward_workspace(int64_t M, int32_t K);
ss1_status launch_layernorm_forward(const NormArgs& a);
ss1_status launch_layernorm_backward(const NormArgs& a);

// The adapters and segments as the kernels read them.
struct AdapterView {
    const int32_t* row;
    const float* scale;
    const int32_t* seg;
    const int32_t* seg_adapter;
    int32_t E;         // adapters
    int32_t S;         // segments
    int32_t R;         // rows of A and B
    int32_t max_rank;
    int32_t M;         // tokens
};

struct AdapterArgs {
    AdapterView ad;
    const void* A;
    const void* B;
    int32_t K, N;
    int32_t dtype;
    const void* x;
    const void* base;  // forward: base; backward: dx_base; may be null
    void* y;           // forward
    float* v;          // forward: written, may be null; backward: read
    const void* dy;    // backward
    void* dx;
    void* dA;
    void* dB;
    void* workspace;
    void* stream;
};

size_t adapter_forward_workspace(int64_t M, int32_t K, int32_t N, int32_t E, int32_t R, int32_t max_rank,
                                 int32_t dtype);
size_t adapter_backward_workspace(int64_t M, int32_t K, int32_t N, int32_t E, int32_t R, int32_t max_rank,
                                  int32_t dtype);
ss1_status launch_adapter_forward(const AdapterArgs& a);
ss1_status launch_adapter_backward(const AdapterArgs& a);

// Elements of one work item of the AdamW step (a multiple of SS1_ADAMW_BLOCK).
constexpr int64_t kAdamWChunk = 2048;

// The step's coefficients, rounded once from the caller's doubles.
struct AdamWCoef {
    float beta1, one_minus_beta1, beta2, one_minus_beta2;
    float step_size;     // lr / (1 - beta1^step)
    float inv_sqrt_c2;   // 1 / sqrt(1 - beta2^step)
    float eps;
    float grad_scale;
    const float* grad_scale_dev;
    double lr;
    uint64_t seed;
};

ss1_status launch_adamw(const ss1_adamw_entry* entries, int32_t count, const int32_t* map, int64_t chunks,
                        const AdamWCoef& coef, void* stream);

}  // namespace ss1
