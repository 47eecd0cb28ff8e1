// C ABI of the operators before the optimizer step (include/mps_train.h):
// argument checks and launches.  Nothing is kept between calls.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "../../include/mps_train.h"
#include "errors.h"
#include "train_kernels.h"

namespace {

using mps::fail;
using mps::ok;

constexpr int64_t kMostRows = (1ll << 31) - 1;
constexpr int64_t kMostCols = 1ll << 27;
constexpr int64_t kMostStride = (1ll << 31) - 1;
constexpr int64_t kMostTiles = 1ll << 21;  // of 128 x 128 values of a weight gradient
constexpr size_t kWorkspaceAlign = 256;

int elem_bytes(mps_dtype t) { return t == MPS_DTYPE_BF16 ? 2 : 4; }

int check_dtype(mps_dtype t, const char* name)
{
    if (t == MPS_DTYPE_F32 || t == MPS_DTYPE_BF16) return MPS_OK;
    return fail(MPS_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", name, static_cast<int>(t));
}

int check_shape(int64_t rows, int64_t cols, const char* rows_name, const char* cols_name)
{
    if (rows < 0 || rows > kMostRows) {
        return fail(MPS_ERR_INVALID_ARGUMENT, "%s = %lld: 0 to 2^31 - 1", rows_name, static_cast<long long>(rows));
    }
    if (cols < 1 || cols > kMostCols) {
        return fail(MPS_ERR_INVALID_ARGUMENT, "%s = %lld: 1 to 2^27", cols_name, static_cast<long long>(cols));
    }
    return MPS_OK;
}

// The memory of one argument: `rows` stretches of `row_bytes`, `stride_bytes`
// apart (a vector is one row).
struct Area {
    const char* name;
    uintptr_t at;
    uint64_t rows, row_bytes, stride_bytes;
    bool written;
};

uint64_t extent(const Area& a) { return a.rows == 0 || a.row_bytes == 0 ? 0 : (a.rows - 1) * a.stride_bytes + a.row_bytes; }

// Two areas with elements in common.  Matrices of one stride that lie in
// different columns of the same rows (halves of one matrix) have none.
bool overlap(const Area& a, const Area& b)
{
    const uint64_t ea = extent(a), eb = extent(b);
    if (ea == 0 || eb == 0 || a.at + ea <= b.at || b.at + eb <= a.at) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride_bytes == b.stride_bytes) {
        const Area& low = a.at <= b.at ? a : b;
        const Area& high = a.at <= b.at ? b : a;
        const uint64_t off = (high.at - low.at) % low.stride_bytes;
        return !(off >= low.row_bytes && off + high.row_bytes <= low.stride_bytes);
    }
    return true;
}

class Checks {
public:
    // A matrix argument; NULL is an error where it has elements.
    Checks& matrix(const char* name, const void* p, mps_dtype t, int64_t rows, int64_t cols, int64_t stride, bool written)
    {
        if (rc_) return *this;
        if (stride < cols || stride > kMostStride) {
            rc_ = fail(MPS_ERR_INVALID_ARGUMENT, "%s: stride %lld, with rows of %lld", name, static_cast<long long>(stride),
                       static_cast<long long>(cols));
            return *this;
        }
        return area(name, p, elem_bytes(t), rows, static_cast<uint64_t>(cols) * elem_bytes(t),
                    static_cast<uint64_t>(stride) * elem_bytes(t), written);
    }

    Checks& vector(const char* name, const void* p, int elem, int64_t n, bool written)
    {
        return area(name, p, elem, 1, static_cast<uint64_t>(n) * elem, static_cast<uint64_t>(n) * elem, written);
    }

    Checks& kept(const char* name, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool written)
    {
        const int64_t row = MPS_ACT8_ROW(cols);
        area(name, codes, 16, 1, static_cast<uint64_t>(rows * row), static_cast<uint64_t>(rows * row), written);
        return area(name, scales, 1, 1, static_cast<uint64_t>(rows * (row / MPS_Q8_BLOCK)),
                    static_cast<uint64_t>(rows * (row / MPS_Q8_BLOCK)), written);
    }

    Checks& workspace(void* p, size_t bytes, size_t need)
    {
        if (rc_ || need == 0) return *this;
        if (!p) rc_ = fail(MPS_ERR_WORKSPACE, "workspace is NULL");
        else if (reinterpret_cast<uintptr_t>(p) % kWorkspaceAlign) rc_ = fail(MPS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
        else if (bytes < need) rc_ = fail(MPS_ERR_WORKSPACE, "workspace too small: %zu bytes, %zu needed", bytes, need);
        else areas_[n_++] = {"workspace", reinterpret_cast<uintptr_t>(p), 1, need, need, true};
        return *this;
    }

    // Argument `a` may be the same memory as argument `b`, element by element.
    Checks& may_be_same(const char* a, const char* b)
    {
        same_[n_same_][0] = a;
        same_[n_same_++][1] = b;
        return *this;
    }

    int done()
    {
        if (rc_) return rc_;
        for (int i = 0; i < n_; ++i) {
            for (int j = 0; j < i; ++j) {
                const Area &a = areas_[i], &b = areas_[j];
                if (!(a.written || b.written) || !overlap(a, b) || allowed(a, b)) continue;
                return fail(MPS_ERR_INVALID_ARGUMENT, "%s and %s overlap", b.name, a.name);
            }
        }
        return MPS_OK;
    }

private:
    Checks& area(const char* name, const void* p, int align, int64_t rows, uint64_t row_bytes, uint64_t stride_bytes, bool written)
    {
        if (rc_ || rows == 0 || row_bytes == 0) return *this;
        if (!p) rc_ = fail(MPS_ERR_INVALID_ARGUMENT, "%s is NULL", name);
        else if (reinterpret_cast<uintptr_t>(p) % align) rc_ = fail(MPS_ERR_INVALID_ARGUMENT, "%s is not %d-byte aligned", name, align);
        else areas_[n_++] = {name, reinterpret_cast<uintptr_t>(p), static_cast<uint64_t>(rows), row_bytes, stride_bytes, written};
        return *this;
    }

    bool allowed(const Area& a, const Area& b) const
    {
        if (a.at != b.at || a.row_bytes != b.row_bytes || (a.rows > 1 && a.stride_bytes != b.stride_bytes)) return false;
        for (int i = 0; i < n_same_; ++i) {
            if ((a.name == same_[i][0] && b.name == same_[i][1]) || (b.name == same_[i][0] && a.name == same_[i][1])) return true;
        }
        return false;
    }

    int rc_ = MPS_OK;
    Area areas_[16];
    int n_ = 0;
    const char* same_[4][2];
    int n_same_ = 0;
};

int launched(hipError_t e, const char* what)
{
    if (e != hipSuccess) return fail(MPS_ERR_DEVICE, "%s launch: %s", what, hipGetErrorString(e));
    return ok();
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int weight_grad_shape(int64_t tokens, int64_t out_features, int64_t in_features)
{
    int rc = check_shape(tokens, out_features, "tokens", "out_features");
    if (!rc) rc = check_shape(tokens, in_features, "tokens", "in_features");
    if (rc) return rc;
    if (((out_features + 127) / 128) * ((in_features + 127) / 128) > kMostTiles) {
        return fail(MPS_ERR_INVALID_ARGUMENT, "a weight gradient of more than 2^21 tiles of 128 x 128");
    }
    return MPS_OK;
}

}  // namespace

extern "C" {

int act8_save(const void* d_x, mps_dtype x_dtype, int64_t x_stride, int64_t rows, int64_t cols, uint8_t* d_codes,
              uint8_t* d_scales, void* stream)
{
    int rc = check_dtype(x_dtype, "x_dtype");
    if (!rc) rc = check_shape(rows, cols, "rows", "cols");
    if (rc) return rc;
    rc = Checks().matrix("x", d_x, x_dtype, rows, cols, x_stride, false).kept("codes", d_codes, d_scales, rows, cols, true).done();
    if (rc || rows == 0) return rc ? rc : ok();
    return launched(mps::launch_act8_save({d_x, x_stride}, x_dtype == MPS_DTYPE_BF16, rows, cols, {d_codes, d_scales},
                                          as_stream(stream)), "act8_save");
}

int act8_load(const uint8_t* d_codes, const uint8_t* d_scales, int64_t rows, int64_t cols, void* d_x, mps_dtype x_dtype,
              int64_t x_stride, void* stream)
{
    int rc = check_dtype(x_dtype, "x_dtype");
    if (!rc) rc = check_shape(rows, cols, "rows", "cols");
    if (rc) return rc;
    rc = Checks().kept("codes", d_codes, d_scales, rows, cols, false).matrix("x", d_x, x_dtype, rows, cols, x_stride, true).done();
    if (rc || rows == 0) return rc ? rc : ok();
    return launched(mps::launch_act8_load({d_codes, d_scales}, rows, cols, {d_x, x_stride}, x_dtype == MPS_DTYPE_BF16,
                                          as_stream(stream)), "act8_load");
}

int act8_rmsnorm(const void* d_x, mps_dtype x_dtype, int64_t x_stride, int64_t rows, int64_t cols, const float* d_weight,
                 double eps, void* d_y, int64_t y_stride, float* d_rstd, uint8_t* d_codes, uint8_t* d_scales, void* stream)
{
    int rc = check_dtype(x_dtype, "x_dtype");
    if (!rc) rc = check_shape(rows, cols, "rows", "cols");
    if (rc) return rc;
    const float eps32 = static_cast<float>(eps);
    if (!std::isfinite(eps) || !std::isfinite(eps32) || !(eps32 > 0.0f)) {
        return fail(MPS_ERR_INVALID_ARGUMENT, "eps must be finite and > 0 in fp32");
    }
    rc = Checks()
             .matrix("x", d_x, x_dtype, rows, cols, x_stride, false)
             .vector("weight", d_weight, 4, cols, false)
             .matrix("y", d_y, x_dtype, rows, cols, y_stride, true)
             .vector("rstd", d_rstd, 4, rows, true)
             .kept("codes", d_codes, d_scales, rows, cols, true)
             .done();
    if (rc || rows == 0) return rc ? rc : ok();
    return launched(mps::launch_act8_rmsnorm({d_x, x_stride}, x_dtype == MPS_DTYPE_BF16, rows, cols, d_weight, eps32,
                                             {d_y, y_stride}, d_rstd, {d_codes, d_scales}, as_stream(stream)), "act8_rmsnorm");
}

size_t act8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols)
{
    if (check_shape(rows, cols, "rows", "cols")) return 0;
    ok();
    return rows == 0 ? 0 : mps::rmsnorm_backward_scratch(rows, cols);
}

int act8_rmsnorm_backward(const void* d_dy, mps_dtype dy_dtype, int64_t dy_stride, const uint8_t* d_codes,
                          const uint8_t* d_scales, const float* d_rstd, int64_t rows, int64_t cols, const float* d_weight,
                          const void* d_residual, int64_t residual_stride, void* d_dx, int64_t dx_stride, float* d_dweight,
                          int accumulate, uint8_t* d_out_codes, uint8_t* d_out_scales, void* d_workspace,
                          size_t workspace_bytes, void* stream)
{
    int rc = check_dtype(dy_dtype, "dy_dtype");
    if (!rc) rc = check_shape(rows, cols, "rows", "cols");
    if (rc) return rc;
    if (!d_out_codes != !d_out_scales && rows > 0) {
        return fail(MPS_ERR_INVALID_ARGUMENT, "out_codes and out_scales: both or neither");
    }
    Checks c;
    c.matrix("dy", d_dy, dy_dtype, rows, cols, dy_stride, false)
        .kept("codes", d_codes, d_scales, rows, cols, false)
        .vector("rstd", d_rstd, 4, rows, false)
        .vector("weight", d_weight, 4, cols, false)
        .matrix("dx", d_dx, dy_dtype, rows, cols, dx_stride, true)
        .vector("dweight", d_dweight, 4, cols, true)
        .may_be_same("dx", "dy")
        .may_be_same("dx", "residual");
    if (d_residual) c.matrix("residual", d_residual, dy_dtype, rows, cols, residual_stride, false);
    if (d_out_codes) c.kept("out_codes", d_out_codes, d_out_scales, rows, cols, true);
    rc = c.workspace(d_workspace, workspace_bytes, rows == 0 ? 0 : mps::rmsnorm_backward_scratch(rows, cols)).done();
    if (rc) return rc;
    if (rows == 0) {
        if (accumulate) return ok();
        return launched(mps::launch_zero(d_dweight, cols, as_stream(stream)), "act8_rmsnorm_backward");
    }
    return launched(mps::launch_act8_rmsnorm_backward({d_dy, dy_stride}, dy_dtype == MPS_DTYPE_BF16, {d_codes, d_scales},
                                                      d_rstd, rows, cols, d_weight, {d_residual, residual_stride},
                                                      {d_dx, dx_stride}, d_dweight, accumulate != 0,
                                                      {d_out_codes, d_out_scales}, d_workspace, as_stream(stream)),
                    "act8_rmsnorm_backward");
}

int act8_swiglu(const void* d_gate, int64_t gate_stride, const void* d_up, int64_t up_stride, mps_dtype dtype, int64_t rows,
                int64_t cols, void* d_out, int64_t out_stride, uint8_t* d_gate_codes, uint8_t* d_gate_scales,
                uint8_t* d_up_codes, uint8_t* d_up_scales, void* stream)
{
    int rc = check_dtype(dtype, "dtype");
    if (!rc) rc = check_shape(rows, cols, "rows", "cols");
    if (rc) return rc;
    rc = Checks()
             .matrix("gate", d_gate, dtype, rows, cols, gate_stride, false)
             .matrix("up", d_up, dtype, rows, cols, up_stride, false)
             .matrix("out", d_out, dtype, rows, cols, out_stride, true)
             .kept("gate_codes", d_gate_codes, d_gate_scales, rows, cols, true)
             .kept("up_codes", d_up_codes, d_up_scales, rows, cols, true)
             .done();
    if (rc || rows == 0) return rc ? rc : ok();
    return launched(mps::launch_act8_swiglu({d_gate, gate_stride}, {d_up, up_stride}, dtype == MPS_DTYPE_BF16, rows, cols,
                                            {d_out, out_stride}, {d_gate_codes, d_gate_scales}, {d_up_codes, d_up_scales},
                                            as_stream(stream)), "act8_swiglu");
}

int act8_swiglu_backward(const void* d_dout, mps_dtype dtype, int64_t dout_stride, const uint8_t* d_gate_codes,
                         const uint8_t* d_gate_scales, const uint8_t* d_up_codes, const uint8_t* d_up_scales, int64_t rows,
                         int64_t cols, void* d_dgate, int64_t dgate_stride, void* d_dup, int64_t dup_stride,
                         uint8_t* d_out_codes, uint8_t* d_out_scales, void* stream)
{
    int rc = check_dtype(dtype, "dtype");
    if (!rc) rc = check_shape(rows, cols, "rows", "cols");
    if (rc) return rc;
    if (!d_out_codes != !d_out_scales && rows > 0) {
        return fail(MPS_ERR_INVALID_ARGUMENT, "out_codes and out_scales: both or neither");
    }
    Checks c;
    c.matrix("dout", d_dout, dtype, rows, cols, dout_stride, false)
        .kept("gate_codes", d_gate_codes, d_gate_scales, rows, cols, false)
        .kept("up_codes", d_up_codes, d_up_scales, rows, cols, false)
        .matrix("dgate", d_dgate, dtype, rows, cols, dgate_stride, true)
        .matrix("dup", d_dup, dtype, rows, cols, dup_stride, true)
        .may_be_same("dgate", "dout")
        .may_be_same("dup", "dout");
    if (d_out_codes) c.kept("out_codes", d_out_codes, d_out_scales, rows, cols, true);
    rc = c.done();
    if (rc || rows == 0) return rc ? rc : ok();
    return launched(mps::launch_act8_swiglu_backward({d_dout, dout_stride}, dtype == MPS_DTYPE_BF16,
                                                     {d_gate_codes, d_gate_scales}, {d_up_codes, d_up_scales}, rows, cols,
                                                     {d_dgate, dgate_stride}, {d_dup, dup_stride},
                                                     {d_out_codes, d_out_scales}, as_stream(stream)), "act8_swiglu_backward");
}

size_t act8_weight_grad_workspace_bytes(int64_t tokens, int64_t out_features, int64_t in_features)
{
    if (weight_grad_shape(tokens, out_features, in_features)) return 0;
    ok();
    return mps::weight_grad_scratch(tokens, out_features, in_features);
}

int act8_weight_grad(const void* d_dy, mps_dtype dy_dtype, int64_t dy_stride, const uint8_t* d_codes,
                     const uint8_t* d_scales, int64_t tokens, int64_t out_features, int64_t in_features, void* d_dw,
                     mps_dtype dw_dtype, int accumulate, void* d_workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_dtype(dy_dtype, "dy_dtype");
    if (!rc) rc = check_dtype(dw_dtype, "dw_dtype");
    if (!rc) rc = weight_grad_shape(tokens, out_features, in_features);
    if (rc) return rc;
    rc = Checks()
             .matrix("dy", d_dy, dy_dtype, tokens, out_features, dy_stride, false)
             .kept("codes", d_codes, d_scales, tokens, in_features, false)
             .vector("dw", d_dw, elem_bytes(dw_dtype), out_features * in_features, true)
             .workspace(d_workspace, workspace_bytes, mps::weight_grad_scratch(tokens, out_features, in_features))
             .done();
    if (rc) return rc;
    if (tokens == 0 && accumulate) return ok();
    return launched(mps::launch_act8_weight_grad({d_dy, dy_stride}, dy_dtype == MPS_DTYPE_BF16, {d_codes, d_scales}, tokens,
                                                 out_features, in_features, d_dw, dw_dtype == MPS_DTYPE_BF16,
                                                 accumulate != 0, d_workspace, as_stream(stream)), "act8_weight_grad");
}

size_t policy_loss_workspace_bytes(int64_t rows, int64_t vocab)
{
    if (check_shape(rows, vocab, "rows", "vocab")) return 0;
    ok();
    return rows == 0 ? 0 : mps::policy_scratch(rows, vocab);
}

int policy_loss(const void* d_logits, mps_dtype logits_dtype, int64_t logits_stride, int64_t rows, int64_t vocab,
                const int64_t* d_labels, const float* d_old_logp, const float* d_ref_logp, const float* d_advantage,
                const float* d_weight, double clip_low, double clip_high, double kl_coef, float* d_loss, void* d_dlogits,
                int64_t dlogits_stride, float* d_token_logp, float* d_token_kl, void* d_workspace, size_t workspace_bytes,
                void* stream)
{
    int rc = check_dtype(logits_dtype, "logits_dtype");
    if (!rc) rc = check_shape(rows, vocab, "rows", "vocab");
    if (rc) return rc;
    if (!(clip_low >= 0.0 && clip_low < 1.0)) return fail(MPS_ERR_INVALID_ARGUMENT, "clip_low must be in [0, 1)");
    if (!(clip_high >= 0.0) || !std::isfinite(clip_high)) return fail(MPS_ERR_INVALID_ARGUMENT, "clip_high must be finite and >= 0");
    if (!(kl_coef >= 0.0) || !std::isfinite(kl_coef)) return fail(MPS_ERR_INVALID_ARGUMENT, "kl_coef must be finite and >= 0");
    if (!d_ref_logp && kl_coef != 0.0 && rows > 0) return fail(MPS_ERR_INVALID_ARGUMENT, "kl_coef without ref_logp");
    Checks c;
    c.matrix("logits", d_logits, logits_dtype, rows, vocab, logits_stride, false)
        .vector("labels", d_labels, 8, rows, false)
        .vector("old_logp", d_old_logp, 4, rows, false)
        .vector("advantage", d_advantage, 4, rows, false)
        .vector("weight", d_weight, 4, rows, false)
        .vector("loss", d_loss, 4, 1, true)
        .may_be_same("dlogits", "logits");
    if (d_ref_logp) c.vector("ref_logp", d_ref_logp, 4, rows, false);
    if (d_dlogits) c.matrix("dlogits", d_dlogits, logits_dtype, rows, vocab, dlogits_stride, true);
    if (d_token_logp) c.vector("token_logp", d_token_logp, 4, rows, true);
    if (d_token_kl) c.vector("token_kl", d_token_kl, 4, rows, true);
    rc = c.workspace(d_workspace, workspace_bytes, rows == 0 ? 0 : mps::policy_scratch(rows, vocab)).done();
    if (rc) return rc;
    const mps::PolicyArgs a{{d_logits, logits_stride}, rows, vocab, d_labels, d_old_logp, d_ref_logp, d_advantage, d_weight,
                            clip_low, clip_high, kl_coef, d_loss, {d_dlogits, dlogits_stride}, d_token_logp, d_token_kl};
    return launched(mps::launch_policy_loss(a, logits_dtype == MPS_DTYPE_BF16, d_workspace, as_stream(stream)), "policy_loss");
}

int token_logprobs(const void* d_logits, mps_dtype logits_dtype, int64_t logits_stride, int64_t rows, int64_t vocab,
                   const int64_t* d_labels, float* d_token_logp, void* d_workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_dtype(logits_dtype, "logits_dtype");
    if (!rc) rc = check_shape(rows, vocab, "rows", "vocab");
    if (rc) return rc;
    rc = Checks()
             .matrix("logits", d_logits, logits_dtype, rows, vocab, logits_stride, false)
             .vector("labels", d_labels, 8, rows, false)
             .vector("token_logp", d_token_logp, 4, rows, true)
             .workspace(d_workspace, workspace_bytes, rows == 0 ? 0 : mps::policy_scratch(rows, vocab))
             .done();
    if (rc || rows == 0) return rc ? rc : ok();
    const mps::PolicyArgs a{{d_logits, logits_stride}, rows, vocab, d_labels, nullptr, nullptr, nullptr, nullptr, 0.0, 0.0, 0.0,
                            nullptr, {nullptr, 0}, d_token_logp, nullptr};
    return launched(mps::launch_policy_loss(a, logits_dtype == MPS_DTYPE_BF16, d_workspace, as_stream(stream)), "token_logprobs");
}

}  // extern "C"
