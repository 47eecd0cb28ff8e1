// gfx950 kernels of the clipped policy loss, its gradient with respect to the
// logits, and the log-probabilities of the labels.
//
// Every row is reduced to its largest logit and the sum of e^(x - max); one value per row (ratio, clip, KL term, the slope d loss / d l)
// is computed in fp64, and the gradient is slope * (onehot - softmax).
#include <hip/hip_runtime.h>

#include "rows.h"
#include "train_kernels.h"

namespace mps {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// 2^((x - top) log2(e)), the form that also holds at the type's lowest values
// (where x log2(e) itself is no fp32 number).
__device__ __forceinline__ float exp_below(float x, float top) { return __builtin_amdgcn_exp2f((x - top) * kLog2e); }

// A share of a row: its largest logit and the sum of e^(x - top).  An empty
// share, or one of -inf logits only, is {-inf, 0}; a NaN or +inf logit makes
// the sum NaN.
struct Share {
    float top;
    double sum;
};

__device__ __forceinline__ Share join(const Share& a, const Share& b)
{
    const float top = fmaxf(a.top, b.top);
    const float base = top == -INFINITY ? 0.0f : top;
    return {top, a.sum * static_cast<double>(exp_below(a.top, base)) + b.sum * static_cast<double>(exp_below(b.top, base))};
}

// One value a row: what the row gives to the loss, and the two factors of
// its gradient, dlogits = slope * onehot + factor * e^(x - top).
struct RowResult {
    double loss;
    float logp, kl, slope, factor, top;
};

// `share` is the whole row's; `label_logit` its label's.  A row that is left
// out never comes here.
__device__ __forceinline__ RowResult row_result(const PolicyArgs& a, int64_t row, const Share& share, float label_logit)
{
    RowResult r = {};
    if (share.top == -INFINITY && share.sum == 0.0) return r;  // nothing to choose from: left out
    r.top = share.top;
    const double logp = static_cast<double>(label_logit) - static_cast<double>(share.top) - log(share.sum);
    r.logp = static_cast<float>(logp);
    if (!a.loss) return r;
    const double w = a.weight[row], adv = a.advantage[row];
    double gain = 0.0, slope = 0.0;
    if (adv != 0.0) {
        const double ratio = exp(logp - static_cast<double>(a.old_logp[row]));
        const double low = 1.0 - a.clip_low, high = 1.0 + a.clip_high;
        const double held = ratio < low ? low : (ratio > high ? high : ratio);  // a NaN stays one
        const double plain = ratio * adv, clipped = held * adv;
        const bool flat = plain > clipped;
        gain = flat ? clipped : plain;
        slope = flat ? 0.0 : -plain;
    }
    if (a.ref_logp) {
        const double d = static_cast<double>(a.ref_logp[row]) - logp;
        const double q = exp(d);
        const double kl = q == INFINITY ? q : q - d - 1.0;  // the label has no probability left
        r.kl = static_cast<float>(kl);
        gain -= a.kl_coef * kl;
        slope += a.kl_coef * (1.0 - q);
    }
    r.loss = -w * gain;
    slope *= w;
    r.slope = static_cast<float>(slope);
    r.factor = static_cast<float>(-slope / share.sum);
    return r;
}

// Whether a row takes part at all.
__device__ __forceinline__ bool row_live(const PolicyArgs& a, int64_t row)
{
    const int64_t label = a.labels[row];
    return label >= 0 && label < a.vocab && !(a.weight && a.weight[row] == 0.0f);
}

// The block's shares joined in a fixed order; every thread gets the result.
__device__ __forceinline__ Share block_join(Share s, Share* lds)
{
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const Share o = {__shfl_xor(s.top, off, kWave), __shfl_xor(s.sum, off, kWave)};
        s = (threadIdx.x & off) ? join(o, s) : join(s, o);
    }
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = s;
    __syncthreads();
    Share r = lds[0];
    for (int w = 1; w < static_cast<int>(blockDim.x) / kWave; ++w) r = join(r, lds[w]);
    return r;
}

// Units of eight logits of one share of a row: [first, last).
struct Span {
    int64_t first, last;
};
__device__ __forceinline__ Span span_of(int64_t vocab, int shares, int share)
{
    const int64_t units = (vocab + kUnit - 1) / kUnit;
    const int64_t per = (units + shares - 1) / shares;
    const int64_t first = per * share;
    return {first, first + per < units ? first + per : units};
}

// Shares of every row: block (row, share).
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void policy_shares_kernel(PolicyArgs a, int shares, Share* out)
{
    __shared__ Share lds[kWavesPerBlock];
    const Span span = span_of(a.vocab, shares, blockIdx.y);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (!row_live(a, row)) continue;
        Share s = {-INFINITY, 0.0};
        for (int64_t u = span.first + threadIdx.x; u < span.last; u += kBlock) {
            float x[kUnit], top = -INFINITY, sum = 0.0f;
            const int64_t c = u * kUnit, n = a.vocab - c;
            widen<kBf16>(load8<kBf16>(a.logits.data, row * a.logits.stride + c, n), x);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
                x[i] = i < n ? x[i] : -INFINITY;
                top = fmaxf(top, x[i]);
            }
            top = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < kUnit; ++i) sum += exp_below(x[i], top);
            s = join(s, {sum == 0.0f ? -INFINITY : top, static_cast<double>(sum)});
        }
        s = block_join(s, lds);
        if (threadIdx.x == 0) out[row * shares + blockIdx.y] = s;
    }
}

// Joins the shares of a row, and writes this block's part of the gradient;
// the first share's block writes the row's own results.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void policy_rows_kernel(PolicyArgs a, int shares, const Share* in, double* row_loss)
{
    const Span span = span_of(a.vocab, shares, blockIdx.y);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        RowResult r = {};
        int64_t label = -1;
        if (row_live(a, row)) {
            label = a.labels[row];
            float x;
            if (kBf16) x = bf16_lo(static_cast<const uint16_t*>(a.logits.data)[row * a.logits.stride + label]);
            else x = static_cast<const float*>(a.logits.data)[row * a.logits.stride + label];
            Share s = in[row * shares];
            for (int i = 1; i < shares; ++i) s = join(s, in[row * shares + i]);
            r = row_result(a, row, s, x);
        }
        if (blockIdx.y == 0 && threadIdx.x == 0) {
            if (a.token_logp) a.token_logp[row] = r.logp;
            if (a.token_kl) a.token_kl[row] = r.kl;
            if (row_loss) row_loss[row] = r.loss;
        }
        if (!a.dlogits.data) continue;
        const bool flat = r.slope == 0.0f && r.factor == 0.0f;  // zeros, whatever the logits
        for (int64_t u = span.first + threadIdx.x; u < span.last; u += kBlock) {
            float x[kUnit] = {};
            const int64_t c = u * kUnit, n = a.vocab - c;
            if (!flat) {
                widen<kBf16>(load8<kBf16>(a.logits.data, row * a.logits.stride + c, n), x);
#pragma unroll
                for (int i = 0; i < kUnit; ++i) {
                    x[i] = r.factor * exp_below(x[i], r.top);
                    if (c + i == label) x[i] += r.slope;
                }
            }
            store8<kBf16>(x, a.dlogits.data, row * a.dlogits.stride + c, n);
        }
    }
}

// *loss = the n values' sum, in a fixed order.
__global__ __launch_bounds__(kBlock) void policy_total_kernel(const double* values, int64_t n, float* loss)
{
    __shared__ double lds[kWavesPerBlock];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kBlock) s += values[i];
    s = block_sum(s, lds);
    if (threadIdx.x == 0) *loss = static_cast<float>(s);
}

constexpr int kMostRowBlocks = 1 << 20;

// Blocks that share a row: enough for two blocks per CU, of at least 16
// units per thread each.
int shares_of(int64_t rows, int64_t vocab)
{
    const int64_t most = (vocab + kUnit * kBlock * 4 - 1) / (kUnit * kBlock * 4);
    int64_t s = 1024 / (rows > 0 ? rows : 1);
    if (s > most) s = most;
    return static_cast<int>(s < 1 ? 1 : s);
}

}  // namespace

size_t policy_scratch(int64_t rows, int64_t vocab)
{
    return static_cast<size_t>(rows) * (shares_of(rows, vocab) * sizeof(Share) + sizeof(double));
}

hipError_t launch_policy_loss(const PolicyArgs& a, bool bf16, void* scratch, hipStream_t stream)
{
    const int shares = shares_of(a.rows, a.vocab);
    Share* parts = static_cast<Share*>(scratch);
    double* row_loss = a.loss ? reinterpret_cast<double*>(parts + a.rows * shares) : nullptr;
    if (a.rows > 0) {
        const dim3 grid(static_cast<uint32_t>(a.rows < kMostRowBlocks ? a.rows : kMostRowBlocks), shares);
        if (bf16) {
            policy_shares_kernel<true><<<grid, kBlock, 0, stream>>>(a, shares, parts);
            policy_rows_kernel<true><<<grid, kBlock, 0, stream>>>(a, shares, parts, row_loss);
        } else {
            policy_shares_kernel<false><<<grid, kBlock, 0, stream>>>(a, shares, parts);
            policy_rows_kernel<false><<<grid, kBlock, 0, stream>>>(a, shares, parts, row_loss);
        }
    }
    if (a.loss) policy_total_kernel<<<1, kBlock, 0, stream>>>(row_loss, a.rows, a.loss);
    return hipGetLastError();
}

}  // namespace mps
