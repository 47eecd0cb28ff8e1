/*
 * mps_model.h — C ABI of the operators at the two ends of a model in training
 * on one GPU (AMD Instinct MI355X, gfx950): the embedding lookup and its
 * gradient, dropout whose mask is never stored, and a linear head under a
 * cross entropy that holds no more than a piece of its logits.  In the same
 * library as mps_adamw.h and mps_train.h, whose error codes, dtypes and conventions
 * (device pointers, streams, strides, overlaps, workspaces, rows == 0, results
 * that do not depend on the order of blocks, no call that waits, allocates or
 * copies) hold here as well:
 *
 *   forward     embedding; dropout on a sublayer's output
 *   loss        linear_cross_entropy: loss and both gradients of the head
 *               (linear_token_logprobs gives the old and reference
 *               log-probabilities that policy_loss of mps_train.h takes)
 *   backward    dropout on the gradient (the same call), embedding_backward
 *               into the gradient buffer of the step's list; with one table
 *               for both ends, accumulated onto the head's gradient
 *   step        grad_norm_sq / adamw_clipped_step of mps_adamw.h, whose step
 *               counter dropout reads
 */
#ifndef MPS_MODEL_H
#define MPS_MODEL_H

#include "mps_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * embedding — out[t, :] = scale * table[ids[t], :], rounded once; zeros where
 * ids[t] is outside [0, vocab).
 *   d_ids : int64 [tokens].
 *   dtype : the type of table and out, MPS_DTYPE_F32 or MPS_DTYPE_BF16.
 *   scale : finite in fp32.
 */
int embedding(const int64_t* d_ids, int64_t tokens, const void* d_table, mps_dtype dtype,
              int64_t table_stride, int64_t vocab, int64_t features, double scale, void* d_out,
              int64_t out_stride, void* stream);

/*
 * embedding_backward — the table's gradient, from the gradient dout of out:
 *     dtable[v, :] = [dtable[v, :] +] scale * sum over the t with ids[t] = v of dout[t, :]
 * Sums in fp32, over a row's tokens in ascending order (in fixed pieces, where
 * there are many); rounded once, after the sum with what dtable held.  Tokens
 * whose id is outside [0, vocab) have no part in it.
 *   dout_dtype : MPS_DTYPE_F32 or MPS_DTYPE_BF16.
 *   d_dtable   : fp32 or bf16 (dtable_dtype) [vocab, features], e.g. the
 *                gradient buffer of an mps_tensor; any element-aligned start.
 *                accumulate non-zero adds to what it holds and touches the
 *                rows that have tokens; zero writes every row.
 */
size_t embedding_backward_workspace_bytes(int64_t tokens, int64_t vocab, int64_t features);
int embedding_backward(const void* d_dout, mps_dtype dout_dtype, int64_t dout_stride,
                       const int64_t* d_ids, int64_t tokens, int64_t vocab, int64_t features,
                       double scale, void* d_dtable, mps_dtype dtable_dtype, int accumulate,
                       void* d_workspace, size_t workspace_bytes, void* stream);

/*
 * dropout — out = [residual +] (dropped ? 0 : x / (1 - q)), and, called with
 * the same p, seed, site and step on the gradient of out, without a residual,
 * its own backward pass.  Which elements are dropped is computed again in
 * every call and stored nowhere:
 *     a row's elements go in units of eight; unit u of row r takes the four
 *     words of Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011) with the key
 *     (seed's low word, seed's high word) and the counter
 *     (low and high word of r * ceil(cols / 8) + u, site, step);
 *     element i of the unit has the low (i even) or high (i odd) 16 bits of
 *     word i / 2, and is dropped where they are below q * 65536, with q the
 *     multiple of 2^-16 nearest to p (ties to even).
 * What an element draws depends on its place, the row's length and these
 * numbers alone, not on strides, types or the device.  A dropped element's
 * value reaches nothing (a NaN there gives 0).
 *   dtype   : the type of x, residual and out.
 *   p       : in [0, 1].  With q = 1 everything is dropped.
 *   site    : tells the dropouts of a step apart (layer, micro-batch).
 *   d_step  : int32 device counter, e.g. that of the optimizer step, so that
 *             a replayed graph draws anew every step; NULL counts as 0.
 *   d_residual : [rows, cols], or NULL.
 *   d_out   : may be the same memory as x or residual (same pointer and stride).
 */
int dropout(const void* d_x, mps_dtype dtype, int64_t x_stride, int64_t rows, int64_t cols,
            double p, uint64_t seed, uint32_t site, const int32_t* d_step, const void* d_residual,
            int64_t residual_stride, void* d_out, int64_t out_stride, void* stream);

/*
 * linear_cross_entropy — the cross entropy of a linear head, and its
 * gradients, in one call that holds no more than a piece of the logits.  With x[t, v] the product of
 * row t of hidden and row v of weight, and l_t = x[t, labels[t]] -
 * logsumexp(x[t, :]):
 *     *d_loss = - sum over t of token_weight[t] * l_t
 *     g[t, v] = token_weight[t] * (softmax(x[t, :])[v] - (v == labels[t]))
 *     dhidden = g weight,   dweight = [dweight +] g^T hidden
 * The logits are made in pieces of the vocabulary; where gradients are asked
 * for, all but the last piece's are made twice.  Products of bf16 operands are
 * exact and summed in fp32; fp32 operands enter as three bf16 parts each,
 * whose sum they are, and the six products of parts that can reach 2^-16 of
 * the largest are summed (what is left out is below 2^-22 of |x| |w|).  Row
 * statistics in fp32 with fp64 sums, one value per row in fp64.
 * With bf16 operands g is rounded to bf16, also where dweight is fp32 (which is
 * 1.5e-5 to 2e-4 of its norm off by it, rows that are no token's label 1.6e-3),
 * but at the labels, where it is largest, to 16 bits; with fp32 operands it
 * keeps its 24.  The last piece's bf16 g comes of exponentials that are kept to 3.4e-4
 * of themselves (zeros below 2^-64 of the largest of 128 neighbouring
 * entries; g of the other pieces reaches down to 2^-126).  Sums in fp32;
 * gradients are rounded once, after the sum with what dweight held.
 *
 * A row is left out (l 0, no part in the loss or dweight, zeros in dhidden;
 * nothing of its hidden state is read) when its label is outside [0, vocab) or
 * its weight is 0; rows that are left out cost next to nothing.  A value that
 * is not finite makes the rows and gradients that it reaches NaN; but with bf16
 * operands, whose products are made as they are, an entry with a logit of minus
 * infinity has the probability 0 and leaves l of its row finite.
 *
 *   dtype          : of hidden, weight and dhidden.
 *   d_hidden       : [tokens, features].      d_weight : [vocab, features].
 *   d_labels       : int64 [tokens].          d_token_weight : fp32 [tokens];
 *                    the mask and the mean's divisor.
 *   d_loss         : fp32, written.
 *   d_dhidden      : [tokens, features], or NULL.
 *   d_dweight      : fp32 or bf16 (dweight_dtype) [vocab, features], e.g. the
 *                    gradient buffer of an mps_tensor; any element-aligned
 *                    start; or NULL.  accumulate non-zero adds to what it holds.
 *   d_token_logp   : fp32 [tokens], l, or NULL.
 *   tokens <= 2^24, features <= 2^20.
 * The workspace: without gradients the packed hidden states (2 bytes a value,
 * fp32: 6), up to 128 MB of statistics (128 bytes a token where that is more),
 * and up to 512 MB for a piece of a weight that cannot be read as it lies; with
 * gradients also an fp32 dhidden (several, where it has few tiles), and for a
 * piece's g and what is packed of its weight half of what the logits would take
 * in the operands' type, but up to 512 MB where that is more and 2 GB where that
 * is less (2048 entries at least).  A bf16 weight can be read as it lies where
 * features are a multiple of 64, rows start at 16 bytes and the stride is at
 * most 2^21; up to 64 tokens any weight can, and without gradients where tokens
 * times vocab, each rounded up to 256, is at most 2^22.
 */
size_t linear_cross_entropy_workspace_bytes(int64_t tokens, int64_t vocab, int64_t features,
                                            mps_dtype dtype, int gradients);
int linear_cross_entropy(const void* d_hidden, mps_dtype dtype, int64_t hidden_stride,
                         int64_t tokens, int64_t features, const void* d_weight,
                         int64_t weight_stride, int64_t vocab, const int64_t* d_labels,
                         const float* d_token_weight, float* d_loss, void* d_dhidden,
                         int64_t dhidden_stride, void* d_dweight, mps_dtype dweight_dtype,
                         int accumulate, float* d_token_logp, void* d_workspace,
                         size_t workspace_bytes, void* stream);

/*
 * linear_token_logprobs — l of every row, fp32, by the same arithmetic; 0 for a
 * row whose label is outside [0, vocab).  The workspace is
 * linear_cross_entropy's without gradients.
 */
int linear_token_logprobs(const void* d_hidden, mps_dtype dtype, int64_t hidden_stride,
                          int64_t tokens, int64_t features, const void* d_weight,
                          int64_t weight_stride, int64_t vocab, const int64_t* d_labels,
                          float* d_token_logp, void* d_workspace, size_t workspace_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MPS_MODEL_H */
