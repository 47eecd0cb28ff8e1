// Launchers of the operators of include/mps_train.h (kernels_act8.hip,
// kernels_wgrad.hip, kernels_policy.hip).  Arguments are checked by the
// callers in train_api.cpp; rows >= 1 and cols >= 1 here.
#pragma once

#include <hip/hip_runtime_api.h>

#include <stddef.h>
#include <stdint.h>

namespace mps {

// A row-major matrix of bf16 or fp32 elements; `stride` in elements.
struct Matrix {
    const void* data;
    int64_t stride;
};
struct MatrixOut {
    void* data;
    int64_t stride;
};

// An 8-bit activation's bytes.
struct Codes {
    const uint8_t* codes;
    const uint8_t* scales;
};
struct CodesOut {
    uint8_t* codes;
    uint8_t* scales;
};

hipError_t launch_act8_save(Matrix x, bool bf16, int64_t rows, int64_t cols, CodesOut out,
                            hipStream_t stream);
hipError_t launch_act8_load(Codes in, int64_t rows, int64_t cols, MatrixOut x, bool bf16,
                            hipStream_t stream);

hipError_t launch_act8_rmsnorm(Matrix x, bool bf16, int64_t rows, int64_t cols, const float* weight,
                               float eps, MatrixOut y, float* rstd, CodesOut kept,
                               hipStream_t stream);

size_t rmsnorm_backward_scratch(int64_t rows, int64_t cols);
hipError_t launch_act8_rmsnorm_backward(Matrix dy, bool bf16, Codes kept, const float* rstd,
                                        int64_t rows, int64_t cols, const float* weight,
                                        Matrix residual, MatrixOut dx, float* dweight,
                                        bool accumulate, CodesOut out, void* scratch,
                                        hipStream_t stream);

hipError_t launch_act8_swiglu(Matrix gate, Matrix up, bool bf16, int64_t rows, int64_t cols,
                              MatrixOut out, CodesOut kept_gate, CodesOut kept_up,
                              hipStream_t stream);
hipError_t launch_act8_swiglu_backward(Matrix dout, bool bf16, Codes gate, Codes up, int64_t rows,
                                       int64_t cols, MatrixOut dgate, MatrixOut dup, CodesOut out,
                                       hipStream_t stream);

size_t weight_grad_scratch(int64_t tokens, int64_t out_features, int64_t in_features);
// tokens may be 0 (dw is then zeroed, or left as it is with accumulate).
hipError_t launch_act8_weight_grad(Matrix dy, bool dy_bf16, Codes x, int64_t tokens,
                                   int64_t out_features, int64_t in_features, void* dw,
                                   bool dw_bf16, bool accumulate, void* scratch,
                                   hipStream_t stream);

struct PolicyArgs {
    Matrix logits;
    int64_t rows, vocab;
    const int64_t* labels;
    const float* old_logp;  // NULL: log-probabilities only
    const float* ref_logp;  // or NULL
    const float* advantage;
    const float* weight;
    double clip_low, clip_high, kl_coef;
    float* loss;            // NULL: log-probabilities only
    MatrixOut dlogits;      // data NULL: no gradient
    float* token_logp;      // or NULL
    float* token_kl;        // or NULL
};
size_t policy_scratch(int64_t rows, int64_t vocab);
// rows may be 0 (the loss is then written as 0).
hipError_t launch_policy_loss(const PolicyArgs& a, bool bf16, void* scratch, hipStream_t stream);

// Writes n fp32 zeros (a fill kernel, so that it may be captured).
hipError_t launch_zero(float* x, int64_t n, hipStream_t stream);

}  // namespace mps
