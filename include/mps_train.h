/*
 * mps_train.h — C ABI of the operators that stand before the optimizer step
 * on one GPU (AMD Instinct MI355X, gfx950): activations kept in 8 bits for
 * the backward pass, the weight gradients made from them, and the clipped
 * policy loss whose gradient starts that pass.  In the same library as
 * mps_adamw.h, whose error codes, dtypes and 8-bit runs it uses:
 *
 *   forward     act8_save / act8_rmsnorm / act8_swiglu keep what the backward
 *               pass needs in one byte per element instead of two or four
 *   loss        policy_loss writes the gradient of the logits in the pass
 *               that computes the loss (token_logprobs gives the old and
 *               reference log-probabilities it takes)
 *   backward    act8_swiglu_backward and act8_rmsnorm_backward read the kept
 *               bytes, and can make their forward outputs again as 8-bit
 *               activations; act8_weight_grad multiplies those by the output
 *               gradients, into the fp32 or bf16 buffers of the step's list
 *   step        grad_norm_sq / adamw_clipped_step of mps_adamw.h
 *
 * An 8-bit activation x[rows, cols] is
 *   codes  [rows, P]       one OCP FP8 E4M3 code per element, with
 *                          P = MPS_ACT8_ROW(cols), cols rounded up to whole
 *                          runs of MPS_Q8_BLOCK = 32;
 *   scales [rows, P / 32]  one scale byte b per run.
 * An element's value is code * 2^(b - 127); the scale of a run and the
 * rounding of its elements follow the rule of the first moment's state in
 * mps_adamw.h (smallest exponent >= -127 under which the largest magnitude
 * fits 448; nearest code, ties to even; a run with a NaN or an infinity has
 * b = 255 and codes 0xFF and reads back as NaN).  Runs start at each row's
 * first element.  The elements behind `cols` count as zeros: the writing
 * calls store them, the reading calls rely on them for nothing but that
 * their bytes exist.
 *
 * Conventions shared by every entry point, beyond those of mps_adamw.h
 * (device pointers, stream, return codes, adamw_last_error; no call waits on
 * the host, allocates, or copies from it, so every call may be captured in a
 * graph at once):
 *   - Matrices are row-major: `stride` is the distance of two rows in
 *     elements, at least the row's length; the elements of a row are
 *     contiguous.  Any element-aligned start and any stride are accepted.
 *     `codes` must be 16-byte aligned; scales, codes and weight gradients
 *     have no stride of their own (rows follow each other).
 *   - rows == 0 is a call with nothing to do, except that gradients summed
 *     over the rows are then zeros (or stay, with accumulate) and a loss is 0.
 *   - An output may not overlap an input or another output, except where an
 *     entry point says so; such calls are refused.
 *   - A workspace holds nothing from one call to the next: any 256-byte
 *     aligned memory of the stated size will do, without release.  Calls that
 *     may run at the same time need workspaces of their own (as do captured
 *     graphs that may be replayed at the same time).
 *   - Results do not depend on the order in which the device runs blocks:
 *     the same call on the same data gives the same bits.
 *   - Sizes: 0 <= rows (tokens) < 2^31, 1 <= cols (features, vocab) <= 2^27,
 *     strides below 2^31; a matrix may have more than 2^32 elements.
 */
#ifndef MPS_TRAIN_H
#define MPS_TRAIN_H

#include "mps_adamw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Codes in a row of an 8-bit activation of `cols` columns. */
#define MPS_ACT8_ROW(cols) (((int64_t)(cols) + MPS_Q8_BLOCK - 1) / MPS_Q8_BLOCK * MPS_Q8_BLOCK)

/*
 * act8_save — keep x[rows, cols] in 8 bits.
 * act8_load — the values that 8-bit activations stand for, rounded once to
 * the type of x (exact for fp32; for bf16 only values below its normal range
 * round).
 *   x_dtype : MPS_DTYPE_F32 or MPS_DTYPE_BF16.
 */
int act8_save(const void* d_x, mps_dtype x_dtype, int64_t x_stride, int64_t rows, int64_t cols,
              uint8_t* d_codes, uint8_t* d_scales, void* stream);
int act8_load(const uint8_t* d_codes, const uint8_t* d_scales, int64_t rows, int64_t cols,
              void* d_x, mps_dtype x_dtype, int64_t x_stride, void* stream);

/*
 * act8_rmsnorm — per row of x, with r = 1 / sqrt(mean(x^2) + eps):
 *     y = (x * r) * weight
 * and what the backward pass needs: r (fp32, one per row) and x in 8 bits.
 * y comes from x itself; sums and products in fp32, y rounded once.
 *   x_dtype : the type of x and y.
 *   d_weight: fp32 [cols].       eps: finite, > 0.
 */
int act8_rmsnorm(const void* d_x, mps_dtype x_dtype, int64_t x_stride, int64_t rows, int64_t cols,
                 const float* d_weight, double eps, void* d_y, int64_t y_stride, float* d_rstd,
                 uint8_t* d_codes, uint8_t* d_scales, void* stream);

/*
 * act8_rmsnorm_backward — from the gradient dy of y, with xh = x * r of the
 * kept x and r and g = dy * weight:
 *     dx      = r * (g - xh * mean(g * xh))  [+ residual]
 *     dweight = [dweight +] sum over the rows of dy * xh
 * and, where d_out_codes is not NULL, xh * weight in 8 bits: the norm's
 * output again, for act8_weight_grad of the projections behind it.
 *   dy_dtype   : the type of dy, dx and the residual's gradient.
 *   d_residual : the gradient that reaches x by the residual connection,
 *                [rows, cols], or NULL; dx may be the same memory (same
 *                pointer and stride), or that of dy.
 *   d_dweight  : fp32 [cols]; accumulate non-zero adds to what it holds.
 */
size_t act8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols);
int act8_rmsnorm_backward(const void* d_dy, mps_dtype dy_dtype, int64_t dy_stride,
                          const uint8_t* d_codes, const uint8_t* d_scales, const float* d_rstd,
                          int64_t rows, int64_t cols, const float* d_weight,
                          const void* d_residual, int64_t residual_stride, void* d_dx,
                          int64_t dx_stride, float* d_dweight, int accumulate,
                          uint8_t* d_out_codes, uint8_t* d_out_scales, void* d_workspace,
                          size_t workspace_bytes, void* stream);

/*
 * act8_swiglu — out = gate * sigmoid(gate) * up, keeping gate and up in 8
 * bits.  gate and up may be the two halves of one matrix (the same stride).
 * Products in fp32, out rounded once; a sigmoid below fp32's normal range,
 * 2^-126 (a gate below -87.3), counts as 0, also in the backward pass.
 *   dtype : the type of gate, up and out.
 */
int act8_swiglu(const void* d_gate, int64_t gate_stride, const void* d_up, int64_t up_stride,
                mps_dtype dtype, int64_t rows, int64_t cols, void* d_out, int64_t out_stride,
                uint8_t* d_gate_codes, uint8_t* d_gate_scales, uint8_t* d_up_codes,
                uint8_t* d_up_scales, void* stream);

/*
 * act8_swiglu_backward — from the gradient dout of out, with g and u the kept
 * gate and up and s = sigmoid(g):
 *     dgate = dout * u * s * (1 + g * (1 - s)),   dup = dout * g * s
 * and, where d_out_codes is not NULL, g * s * u in 8 bits: the forward output
 * again, for act8_weight_grad of the projection behind it.
 *   dtype : the type of dout, dgate and dup; dgate or dup may be the same
 *           memory as dout (same pointer and stride).
 */
int act8_swiglu_backward(const void* d_dout, mps_dtype dtype, int64_t dout_stride,
                         const uint8_t* d_gate_codes, const uint8_t* d_gate_scales,
                         const uint8_t* d_up_codes, const uint8_t* d_up_scales, int64_t rows,
                         int64_t cols, void* d_dgate, int64_t dgate_stride, void* d_dup,
                         int64_t dup_stride, uint8_t* d_out_codes, uint8_t* d_out_scales,
                         void* stream);

/*
 * act8_weight_grad — the weight gradient of y = x W^T, from the gradient
 * dy[tokens, out_features] of y and the kept x[tokens, in_features]:
 *     dw[n, k] = [dw[n, k] +] sum over t of dy[t, n] * x[t, k]
 * The products of an E4M3 code, its power of two and a bf16 gradient are
 * formed exactly and summed in fp32 by the matrix cores (bf16 operands; the
 * one rounding on the way in is that of kept values below 2^-126, which bf16
 * holds with fewer bits).  fp32 gradients enter as three bf16 parts each,
 * which hold all their 24 bits down to 2^-133.  dw is rounded once, after the sum with what
 * it held.
 *   dy_dtype   : MPS_DTYPE_F32 or MPS_DTYPE_BF16.
 *   d_dw       : fp32 or bf16 (dw_dtype) [out_features, in_features], e.g.
 *                the gradient buffer of an mps_tensor; any element-aligned
 *                start.  accumulate non-zero adds to what it holds (micro-
 *                batches; fold 1/K into the step's grad_scale).
 */
size_t act8_weight_grad_workspace_bytes(int64_t tokens, int64_t out_features, int64_t in_features);
int act8_weight_grad(const void* d_dy, mps_dtype dy_dtype, int64_t dy_stride,
                     const uint8_t* d_codes, const uint8_t* d_scales, int64_t tokens,
                     int64_t out_features, int64_t in_features, void* d_dw, mps_dtype dw_dtype,
                     int accumulate, void* d_workspace, size_t workspace_bytes, void* stream);

/*
 * policy_loss — the clipped policy loss of answer tokens with a KL term, and
 * its gradient with respect to the logits, in one call.  Per row t, with
 * l = x[label] - logsumexp(x), ratio = exp(l - old), d = ref - l:
 *     kl     = exp(d) - d - 1                            (0 without ref)
 *     loss_t = weight * (kl_coef * kl - min(ratio * A, clip(ratio) * A))
 *     clip(ratio) = min(max(ratio, 1 - clip_low), 1 + clip_high)
 *     *d_loss = sum over t of loss_t
 *     dlogits = (d loss_t / d l) * (onehot(label) - softmax(x))
 * where the min gives both sides at a tie, the gradient of the unclipped one.
 * An advantage of 0 contributes nothing to either, whatever the ratio, and a
 * kl_coef of 0 nothing, whatever the KL term: with ref_logp given, token_kl is
 * then written and loss and gradient are those of the call without it.
 * Row statistics in fp32 with fp64 sums, one value per row in fp64; outputs
 * rounded once.
 *
 * A row is left out (loss, l, kl and gradient 0; its logits are not read)
 * when its label is outside [0, vocab) or its weight is 0, and so is a row
 * whose logits are all -inf.  Single logits of -inf are tokens the
 * vocabulary does not offer (a label among them has l = -inf: a ratio of 0
 * and an infinite KL term); a NaN or +inf logit makes its row NaN (in the loss
 * where its advantage or the KL term counts).
 *
 *   d_logits, logits_dtype, logits_stride : [rows, vocab].
 *   d_labels     : int64 [rows].
 *   d_old_logp, d_advantage, d_weight : fp32 [rows]; the weight holds the
 *                  mask and the mean's divisor (1 / answer tokens).
 *   d_ref_logp   : fp32 [rows], or NULL for no KL term (kl_coef must be 0).
 *   clip_low in [0, 1), clip_high >= 0, kl_coef >= 0; finite.
 *   d_loss       : fp32, written.
 *   d_dlogits    : [rows, vocab] of logits_dtype, or NULL for the loss alone;
 *                  may be d_logits itself with the same stride.
 *   d_token_logp, d_token_kl : fp32 [rows], or NULL.
 */
size_t policy_loss_workspace_bytes(int64_t rows, int64_t vocab);
int policy_loss(const void* d_logits, mps_dtype logits_dtype, int64_t logits_stride, int64_t rows,
                int64_t vocab, const int64_t* d_labels, const float* d_old_logp,
                const float* d_ref_logp, const float* d_advantage, const float* d_weight,
                double clip_low, double clip_high, double kl_coef, float* d_loss, void* d_dlogits,
                int64_t dlogits_stride, float* d_token_logp, float* d_token_kl, void* d_workspace,
                size_t workspace_bytes, void* stream);

/*
 * token_logprobs — l = x[label] - logsumexp(x) of every row, fp32: the old
 * and reference log-probabilities that policy_loss takes, by the same
 * arithmetic.  0 for a row whose label is outside [0, vocab) or whose logits
 * are all -inf.  The workspace is policy_loss's.
 */
int token_logprobs(const void* d_logits, mps_dtype logits_dtype, int64_t logits_stride,
                   int64_t rows, int64_t vocab, const int64_t* d_labels, float* d_token_logp,
                   void* d_workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MPS_TRAIN_H */
