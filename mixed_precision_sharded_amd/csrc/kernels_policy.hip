// gfx950 kernels of the clipped policy loss, its gradient with respect to the
// logits, and the log-probabilities of the labels.
//
// Every row is reduced to its largest logit and the sum of e^(x - max), one
// pass with a running maximum; one value per row (ratio, clip, KL term, the
// slope d loss / d l) is computed in fp64, and the gradient is slope * (onehot
// - softmax).  The logits are read and the gradient written once, 4 bytes a
// logit in bf16, so many rows are bound by memory: 8192 x 128256 bf16 791 us
// (5.3 TB/s), 4000 x 32003 fp32 216 us (4.7 TB/s).  Few rows are bound by two
// launches that wait for one another: 24 x 128256 bf16 13 us.
#include <hip/hip_runtime.h>

#include "rows.h"
#include "train_kernels.h"

namespace mps {
namespace {

// Cache policy of the gradient's stores (2: nontemporal).  The rows in work
// stay in the cache and the gradient passes it by: with the default 8192 x
// 128256 bf16 took 2 % longer, 1000 x 50257 58 us and not 41.  The logits' loads keep the default
// (nontemporal, 5-40 % slower: the second reading then misses).
constexpr int kGradientPolicy = 2;
constexpr int kLogitsPolicy = 0;
constexpr double kLog2eWide = 1.44269504088896340736;
constexpr float kLog2e = static_cast<float>(kLog2eWide);
constexpr float kLog2eLow = static_cast<float>(kLog2eWide - static_cast<double>(kLog2e));

// e^(x - top) as 2^((x - top) log2(e)), the form that also holds at the type's
// lowest values (where x log2(e) itself is no fp32 number).  log2(e) is in two
// parts: what the first one lacks, 1.3e-8 of every exponent, has one sign in
// all of a row's terms (kl of 1000 x 32003 fp32 was off by 1.5e-7 with one
// part, is by 4.8e-8, and takes 0.3 to 1.2 % longer).  The rounding of the
// exponent has no sign and stays.
__device__ __forceinline__ float exp_below(float x, float top)
{
    const float d = x - top;
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, kLog2e, d * kLog2eLow));
}

// The same for a gradient that is rounded to bf16: by the first part alone.
template <bool kBf16>
__device__ __forceinline__ float exp_for_store(float x, float top)
{
    return kBf16 ? __builtin_amdgcn_exp2f((x - top) * kLog2e) : exp_below(x, top);
}

// A share of a row: its largest logit and the sum of e^(x - top).  An empty
// share, or one of -inf logits only, is {-inf, 0}; a NaN or +inf logit makes
// the sum NaN.
struct Share {
    float top;
    double sum;
};

// The share of a wavefront, from its lanes' tops and sums; every lane gets it.
__device__ __forceinline__ Share wave_share(float top, float sum)
{
    float most = top;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, kWave));
    const float base = most == -INFINITY ? 0.0f : most;
    return {most, wave_sum(static_cast<double>(sum * exp_below(top, base)))};
}

// The sum of a share under a larger top: in fp64, since few factors decide a
// row's sum here (in fp32 their errors, 1e-7 each, showed in the loss).
__device__ __forceinline__ double rescaled(const Share& s, float top)
{
    const float base = top == -INFINITY ? 0.0f : top;
    return s.sum * exp2((static_cast<double>(s.top) - static_cast<double>(base)) * kLog2eWide);
}

// Joins the shares of each group of kLanes lanes (a power of two), in a fixed
// order; every lane of the group gets the result.
template <int kLanes>
__device__ __forceinline__ Share lanes_join(const Share& s)
{
    float top = s.top;
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
    double sum = rescaled(s, top);
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor(sum, off, kWave);
    return {top, sum};
}

// What one row gives to the loss, and the two factors of its gradient,
// dlogits = slope * onehot + factor * e^(x - top).
struct RowResult {
    double loss;
    float logp, kl, slope, factor, top, label_logit;
};

// The fp64 part of a row, for the lanes that own one.  Not inlined: its
// registers would count for the streaming loops, which want many wavefronts.
__device__ __attribute__((noinline)) RowResult row_values(float top, double sum, float label_logit, bool loss_too, bool with_ref,
                                                          float old_logp, float ref_logp, float advantage, float weight,
                                                          double low, double high, double kl_coef)
{
    RowResult r = {};
    if (top == -INFINITY && sum == 0.0) return r;  // nothing to choose from: left out
    r.top = top;
    r.label_logit = label_logit;
    const double logp = (static_cast<double>(label_logit) - static_cast<double>(top)) - log(sum);
    r.logp = static_cast<float>(logp);
    if (!loss_too) return r;
    const double w = weight, adv = advantage;
    double gain = 0.0, slope = 0.0;
    if (adv != 0.0) {
        const double ratio = exp(logp - static_cast<double>(old_logp));
        const double held = ratio < low ? low : (ratio > high ? high : ratio);  // a NaN stays one
        const double plain = ratio * adv, clipped = held * adv;
        const bool flat = plain > clipped;
        gain = flat ? clipped : plain;
        slope = flat ? 0.0 : -plain;
    }
    if (with_ref) {
        const double d = static_cast<double>(ref_logp) - logp;
        const double q = exp(d);
        const double kl = q == INFINITY ? q : q - d - 1.0;  // the label has no probability left
        r.kl = static_cast<float>(kl);
        if (kl_coef != 0.0) {  // else the term is only watched: no 0 * inf of it in the loss
            gain -= kl_coef * kl;
            slope += kl_coef * (1.0 - q);
        }
    }
    r.loss = -w * gain;
    slope *= w;
    r.slope = static_cast<float>(slope);
    r.factor = static_cast<float>(-slope / sum);
    return r;
}

__device__ __forceinline__ float logit_at(const PolicyArgs& a, bool bf16, int64_t i)
{
    if (bf16) return bf16_lo(static_cast<const uint16_t*>(a.logits.data)[i]);
    return static_cast<const float*>(a.logits.data)[i];
}

__device__ __forceinline__ void store_logit(const PolicyArgs& a, bool bf16, int64_t i, float v)
{
    if (bf16) static_cast<uint16_t*>(a.dlogits.data)[i] = bf16_one(v);
    else static_cast<float*>(a.dlogits.data)[i] = v;
}

// The logit of a live row's label.
__device__ __forceinline__ float label_logit_of(const PolicyArgs& a, bool bf16, int64_t row)
{
    return logit_at(a, bf16, row * a.logits.stride + a.labels[row]);
}

// Whether a row takes part at all.
__device__ __forceinline__ bool row_live(const PolicyArgs& a, int64_t row)
{
    const int64_t label = a.labels[row];
    return label >= 0 && label < a.vocab && !(a.weight && a.weight[row] == 0.0f);
}

// The result of a live row whose share and label's logit these are, and its
// own outputs; one lane per row.
__device__ __forceinline__ RowResult finish_row(const PolicyArgs& a, int64_t row, bool live, const Share& s, float label_logit)
{
    RowResult r = {};
    if (live) {
        const bool loss_too = a.loss != nullptr, with_ref = a.ref_logp != nullptr;
        r = row_values(s.top, s.sum, label_logit, loss_too, with_ref,
                       loss_too ? a.old_logp[row] : 0.0f, with_ref ? a.ref_logp[row] : 0.0f, loss_too ? a.advantage[row] : 0.0f,
                       loss_too ? a.weight[row] : 0.0f, 1.0 - a.clip_low, 1.0 + a.clip_high, a.kl_coef);
    }
    if (a.token_logp) a.token_logp[row] = r.logp;
    if (a.token_kl) a.token_kl[row] = r.kl;
    return r;
}

constexpr int kDeep = 4;  // units of eight logits that a thread has under way

// A thread's running largest logit, and the sum under it.
struct Running {
    float top = -INFINITY, sum = 0.0f;

    template <bool kBf16>
    __device__ __forceinline__ void take(const Raw8<kBf16>& raw)
    {
        float x[kUnit];
        widen<kBf16>(raw, x);
        const float most = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        const float now = fmaxf(top, most), under = now == -INFINITY ? 0.0f : now;
        const float before = sum * exp_below(top, under);
        top = now;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) x[i] = exp_below(x[i], under);
        sum = before + (((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])));
    }

    __device__ __forceinline__ void take(float x)
    {
        const float now = fmaxf(top, x), under = now == -INFINITY ? 0.0f : now;
        sum = sum * exp_below(top, under) + exp_below(x, under);
        top = now;
    }
};

// The whole units of (a stretch of) a row, through a buffer resource: a 32-bit
// offset per access, where a pointer would take two registers.  A unit behind the last one reads as zeros and is
// not stored.  An fp32 unit is two accesses of 16 bytes a lane.  Where a wavefront has 64 whole units before it, unit u
// means the 16 bytes u % 64 of their first half and of their second one, so that each access of the wavefront is one
// stretch and not every other 16 bytes of it (4000 x 32003 250 us without, 205 with).
template <bool kBf16>
struct Units {
    static constexpr uint32_t kBytes = kUnit * (kBf16 ? 2 : 4);
    __amdgpu_buffer_rsrc_t r;
    uint32_t count;

    __device__ __forceinline__ Units(const void* data, int64_t at, uint32_t units)
        : r(rsrc(uniform_ptr(static_cast<const char*>(data) + at * (kBf16 ? 2 : 4)), units * kBytes)), count(units)
    {
    }

    // Whether unit u is one of 64 whole ones in two halves.
    __device__ __forceinline__ bool halves(uint32_t unit) const { return !kBf16 && (unit | (kWave - 1)) < count; }

    // Offsets of a unit's first and second 16 bytes.
    struct Places {
        uint32_t first, second;
    };
    __device__ __forceinline__ Places places(uint32_t unit) const
    {
        const uint32_t lane = unit % kWave;
        if (halves(unit)) return {unit * kBytes - lane * 16, unit * kBytes - lane * 16 + kWave * 16};
        return {unit * kBytes, unit * kBytes + 16};
    }

    // The thread, of kTeam, that has element `at` of the stretch (units u, u + kTeam, .. of thread u), or that takes it
    // behind the last whole unit.
    template <int kTeam>
    __device__ __forceinline__ uint32_t owner(uint32_t at) const
    {
        const uint32_t unit = at / kUnit;
        if (unit >= count) return at % kUnit;
        if (!halves(unit)) return unit % kTeam;
        return (unit / kWave * kWave + at / 4 % kWave) % kTeam;
    }

    // Every offset is in the vector operand.  A scalar offset does not take
    // part in the resource's bounds check; and 16-byte stores with a scalar
    // offset in a register were seen to send data that the next instructions
    // had already overwritten (the compiler leaves the one wait state out that
    // it puts behind a store without one).
    __device__ __forceinline__ Raw8<kBf16> load(uint32_t unit) const
    {
        Raw8<kBf16> v;
        const Places p = places(unit);
        v.v[0] = __builtin_amdgcn_raw_buffer_load_b128(r, p.first, 0, kLogitsPolicy);
        if (!kBf16) v.v[kBf16 ? 0 : 1] = __builtin_amdgcn_raw_buffer_load_b128(r, p.second, 0, kLogitsPolicy);
        return v;
    }

    __device__ __forceinline__ void store(const float (&x)[kUnit], uint32_t unit) const
    {
        if (kBf16) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = bf16_pack2(x[2 * i], x[2 * i + 1]);
            __builtin_amdgcn_raw_buffer_store_b128(w, r, unit * kBytes, 0, kGradientPolicy);
        } else {
            const Places p = places(unit);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 w = {__float_as_uint(x[4 * h]), __float_as_uint(x[4 * h + 1]), __float_as_uint(x[4 * h + 2]),
                                 __float_as_uint(x[4 * h + 3])};
                __builtin_amdgcn_raw_buffer_store_b128(w, r, h == 0 ? p.first : p.second, 0, kGradientPolicy);
            }
        }
    }

    // Stores factor * e^(x - top) of a unit.
    __device__ __forceinline__ void give(const Raw8<kBf16>& raw, float factor, float top, uint32_t unit) const
    {
        float x[kUnit];
        widen<kBf16>(raw, x);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) x[i] = factor * exp_for_store<kBf16>(x[i], top);
        store(x, unit);
    }
};

// Forgets, for the compiler, what is known of these registers.  Without it
// the widened values of one pass over a kept row are held for the next, twice
// the row's size in registers that are not there.
template <bool kBf16>
__device__ __forceinline__ void forget(Raw8<kBf16>& r)
{
#pragma unroll
    for (int i = 0; i < (kBf16 ? 1 : 2); ++i) asm volatile("" : "+v"(r.v[i]));
}

// Reads thread t's part (of kTeam threads) of the logits [first, last) of a
// row, both in whole units except that `last` may be the row's end; the share
// of its whole wavefront.
template <bool kBf16, int kTeam>
__device__ __forceinline__ Share read_share(const PolicyArgs& a, int64_t row, int64_t first, int64_t last, int t)
{
    const uint32_t count = static_cast<uint32_t>(last - first), full = count / kUnit;
    const Units<kBf16> in(a.logits.data, row * a.logits.stride + first, full);
    Running run;
    uint32_t u = t;
    for (; u + (kDeep - 1) * kTeam < full; u += kDeep * kTeam) {
        Raw8<kBf16> raw[kDeep];
#pragma unroll
        for (int v = 0; v < kDeep; ++v) raw[v] = in.load(u + v * kTeam);
#pragma unroll
        for (int v = 0; v < kDeep; ++v) run.take(raw[v]);
    }
    for (; u < full; u += kTeam) run.take(in.load(u));
    if (t < static_cast<int>(count % kUnit)) run.take(logit_at(a, kBf16, row * a.logits.stride + first + full * kUnit + t));
    return wave_share(run.top, run.sum);
}

// The gradient of the logits [first, last) of a row, by thread t of kTeam;
// the thread that has stored the label's element stores it once more with the
// slope added.
template <bool kBf16, int kTeam>
__device__ __forceinline__ void write_gradient(const PolicyArgs& a, int64_t row, int64_t first, int64_t last, int t,
                                               const RowResult& r, int64_t label)
{
    const int64_t to = row * a.dlogits.stride + first;
    const uint32_t count = static_cast<uint32_t>(last - first), full = count / kUnit;
    const Units<kBf16> out(a.dlogits.data, to, full);
    const float top = r.top, factor = r.factor;
    uint32_t u = t;
    if (r.slope == 0.0f && factor == 0.0f) {  // zeros, whatever the logits
        const float x[kUnit] = {};
        for (; u < full; u += kTeam) out.store(x, u);
        if (t < static_cast<int>(count % kUnit)) store_logit(a, kBf16, to + full * kUnit + t, 0.0f);
        return;
    }
    const Units<kBf16> in(a.logits.data, row * a.logits.stride + first, full);
    for (; u + (kDeep - 1) * kTeam < full; u += kDeep * kTeam) {
        Raw8<kBf16> raw[kDeep];
#pragma unroll
        for (int v = 0; v < kDeep; ++v) raw[v] = in.load(u + v * kTeam);
#pragma unroll
        for (int v = 0; v < kDeep; ++v) out.give(raw[v], factor, top, u + v * kTeam);
    }
    for (; u < full; u += kTeam) out.give(in.load(u), factor, top, u);
    if (t < static_cast<int>(count % kUnit)) {
        const int64_t c = full * kUnit + t;
        store_logit(a, kBf16, to + c, factor * exp_below(logit_at(a, kBf16, row * a.logits.stride + first + c), top));
    }
    if (label < first || label >= last) return;
    const uint32_t at = static_cast<uint32_t>(label - first);
    if (out.template owner<kTeam>(at) == static_cast<uint32_t>(t)) store_logit(a, kBf16, to + at, factor * exp_below(r.label_logit, top) + r.slope);
}

// ------------------------------------------------------ a row per block ---

// The wavefronts' shares of a block, joined and finished by the first one;
// the result is in `result` behind the barrier.  Called by every thread.
template <bool kBf16, int kThreads>
__device__ __forceinline__ void finish_block(const PolicyArgs& a, int64_t row, bool live, Share mine, Share* shares,
                                             RowResult* result, double& total)
{
    constexpr int kWaves = kThreads / kWave;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    if (live && lane == 0) shares[wave] = mine;
    __syncthreads();
    if (wave == 0) {
        const Share s = lanes_join<kWaves>(shares[lane % kWaves]);
        if (lane == 0) {
            *result = finish_row(a, row, live, s, live ? label_logit_of(a, kBf16, row) : 0.0f);
            total += result->loss;
        }
    }
    __syncthreads();
}

// Block b takes rows b, b + grid, ..; the sum of their losses goes to
// losses[b].  The rows are read twice.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void policy_block_kernel(PolicyArgs a, double* losses)
{
    __shared__ Share shares[kWavesPerBlock];
    __shared__ RowResult result;
    double total = 0.0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const bool live = row_live(a, row);
        Share s = {-INFINITY, 0.0};
        if (live) s = read_share<kBf16, kBlock>(a, row, 0, a.vocab, threadIdx.x);
        finish_block<kBf16, kBlock>(a, row, live, s, shares, &result, total);
        if (a.dlogits.data) write_gradient<kBf16, kBlock>(a, row, 0, a.vocab, threadIdx.x, result, a.labels[row]);
    }
    if (threadIdx.x == 0 && losses) losses[blockIdx.x] = total;
}

// The same for long rows, which are kept between the passes: unit t + j *
// kThreads of thread t in registers for j < kRegs, in LDS (each thread's own
// place, so that no barrier is needed) for the next kLds, and only what lies
// behind is read again.  A register that has given its gradient asks for the
// next row's unit at once, so half of the next row is on its way while this
// one is written.  Rows of at least kThreads * kRegs units of eight.  (Of 1024
// threads each has 128 registers, and spills 12 of them in bf16, 23 in fp32.)
template <bool kBf16, int kThreads, int kRegs, int kLds>
__global__ __launch_bounds__(kThreads) void policy_kept_kernel(PolicyArgs a, double* losses)
{
    constexpr int kWords = kBf16 ? 1 : 2, kHalf = kLds / 2;
    __shared__ u32x4 kept[kLds * kWords * kThreads];
    __shared__ Share shares[kThreads / kWave];
    __shared__ RowResult result;
    const uint32_t t = threadIdx.x, full = static_cast<uint32_t>(a.vocab / kUnit), rest = static_cast<uint32_t>(a.vocab % kUnit);
    double total = 0.0;
    Raw8<kBf16> reg[kRegs];
    auto load_regs = [&](const Units<kBf16>& in) {
#pragma unroll
        for (int j = 0; j < kRegs; ++j) reg[j] = in.load(t + j * kThreads);
    };
    int64_t row = blockIdx.x;
    bool live = row < a.rows && row_live(a, row);
    if (live) load_regs(Units<kBf16>(a.logits.data, row * a.logits.stride, full));
    while (row < a.rows) {
        const Units<kBf16> in(a.logits.data, row * a.logits.stride, full);
        Share s = {-INFINITY, 0.0};
        if (live) {
            Running run;
            Raw8<kBf16> raw[kHalf];
#pragma unroll
            for (int j = 0; j < kHalf; ++j) raw[j] = in.load(t + (kRegs + j) * kThreads);
#pragma unroll
            for (int j = 0; j < kRegs; ++j) run.take(reg[j]);  // whole: the row has as many units
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < kHalf; ++j) {
                    const int at = h * kHalf + j;
                    for (int w = 0; w < kWords; ++w) kept[(at * kWords + w) * kThreads + t] = raw[j].v[w];
                    if (t + (kRegs + at) * kThreads < full) run.take(raw[j]);
                    if (h == 0) raw[j] = in.load(t + (kRegs + kHalf + j) * kThreads);
                }
            }
            for (uint32_t u = t + (kRegs + kLds) * kThreads; u < full; u += kThreads) run.take(in.load(u));
            if (t < rest) run.take(logit_at(a, kBf16, row * a.logits.stride + full * kUnit + t));
            s = wave_share(run.top, run.sum);
        }
        finish_block<kBf16, kThreads>(a, row, live, s, shares, &result, total);
        const int64_t next = row + gridDim.x;
        const bool next_live = next < a.rows && row_live(a, next);
        const Units<kBf16> coming(a.logits.data, next * a.logits.stride, full);
        const float top = result.top, factor = result.factor, slope = result.slope;
        if (!a.dlogits.data || (slope == 0.0f && factor == 0.0f)) {  // no gradient, or zeros whatever the logits
            if (next_live) load_regs(coming);
            if (a.dlogits.data) write_gradient<kBf16, kThreads>(a, row, 0, a.vocab, t, result, -1);
        } else {
            const int64_t to = row * a.dlogits.stride;
            const Units<kBf16> out(a.dlogits.data, to, full);
#pragma unroll
            for (int j = 0; j < kRegs; ++j) {
                forget(reg[j]);
                out.give(reg[j], factor, top, t + j * kThreads);
                if (next_live) reg[j] = coming.load(t + j * kThreads);
            }
#pragma unroll
            for (int j = 0; j < kLds; ++j) {
                Raw8<kBf16> raw;
                for (int w = 0; w < kWords; ++w) raw.v[w] = kept[(j * kWords + w) * kThreads + t];
                out.give(raw, factor, top, t + (kRegs + j) * kThreads);
            }
            for (uint32_t u = t + (kRegs + kLds) * kThreads; u < full; u += kThreads) out.give(in.load(u), factor, top, u);
            if (t < rest) {
                const int64_t c = full * kUnit + t;
                store_logit(a, kBf16, to + c, factor * exp_below(logit_at(a, kBf16, row * a.logits.stride + c), top));
            }
            const uint32_t label = static_cast<uint32_t>(a.labels[row]);
            if (out.template owner<kThreads>(label) == t) store_logit(a, kBf16, to + label, factor * exp_below(result.label_logit, top) + slope);
        }
        row = next;
        live = next_live;
    }
    if (threadIdx.x == 0 && losses) losses[blockIdx.x] = total;
}

// -------------------------------------------------- a row per wavefront ---

// For short rows: a block takes kGroup rows at a time, a wavefront one of
// them after the other, and the rows' fp64 parts run side by side on kGroup
// lanes.
constexpr int kGroup = 16;

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void policy_wave_kernel(PolicyArgs a, double* losses)
{
    __shared__ Share shares[kGroup];
    __shared__ RowResult results[kGroup];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    double total = 0.0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kGroup; first < a.rows; first += static_cast<int64_t>(gridDim.x) * kGroup) {
        const int n = static_cast<int>(min(static_cast<int64_t>(kGroup), a.rows - first));
        for (int i = wave; i < n; i += kWavesPerBlock) {
            if (!row_live(a, first + i)) continue;
            const Share s = read_share<kBf16, kWave>(a, first + i, 0, a.vocab, lane);
            if (lane == 0) shares[i] = s;
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n) {
            const int64_t row = first + threadIdx.x;
            const bool live = row_live(a, row);
            results[threadIdx.x] = finish_row(a, row, live, shares[threadIdx.x], live ? label_logit_of(a, kBf16, row) : 0.0f);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 0; i < n; ++i) total += results[i].loss;
        }
        if (!a.dlogits.data) continue;
        for (int i = wave; i < n; i += kWavesPerBlock) {
            write_gradient<kBf16, kWave>(a, first + i, 0, a.vocab, lane, results[i], a.labels[first + i]);
        }
    }
    if (threadIdx.x == 0 && losses) losses[blockIdx.x] = total;
}

// -------------------------------------------------- several blocks a row ---

// Logits of one share of a row.
struct Span {
    int64_t first, last;
};
__device__ __forceinline__ Span span_of(int64_t vocab, int shares, int share)
{
    const int64_t units = (vocab + kUnit - 1) / kUnit;
    const int64_t per = (units + shares - 1) / shares * kUnit;
    return {min(per * share, vocab), min(per * (share + 1), vocab)};
}

// Shares of every row: block (row, share).  The label's logit is kept as well:
// the next kernel's blocks may write the gradient over the logits while others
// of the same row have yet to compute its result.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void policy_shares_kernel(PolicyArgs a, int shares, Share* out, float* label_logits)
{
    __shared__ Share lds[kWavesPerBlock];
    const Span span = span_of(a.vocab, shares, blockIdx.y);
    const int64_t row = blockIdx.x;
    if (!row_live(a, row)) return;
    if (blockIdx.y == 0 && threadIdx.x == 0) label_logits[row] = label_logit_of(a, kBf16, row);
    Share s = read_share<kBf16, kBlock>(a, row, span.first, span.last, threadIdx.x);
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = s;
    __syncthreads();
    if (threadIdx.x < kWave) {
        s = lanes_join<kWavesPerBlock>(lds[threadIdx.x % kWavesPerBlock]);
        if (threadIdx.x == 0) out[row * shares + blockIdx.y] = s;
    }
}

// Joins the (at most 64) shares of a row, and writes this block's part of the
// gradient; the first share's block writes the row's own results, and the
// second wavefront of the very first block computes every row's loss once
// more, a row (of at most 64) per lane, for their sum.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void policy_rows_kernel(PolicyArgs a, int shares, const Share* in, const float* label_logits)
{
    __shared__ RowResult result;
    const Span span = span_of(a.vocab, shares, blockIdx.y);
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    if (wave == 0) {
        const bool live = row_live(a, row);
        const Share s = lanes_join<kWave>(live && lane < shares ? in[row * shares + lane] : Share{-INFINITY, 0.0});
        if (lane == 0) {
            PolicyArgs mine = a;
            if (blockIdx.y != 0) mine.token_logp = mine.token_kl = nullptr;
            result = finish_row(mine, row, live, s, live ? label_logits[row] : 0.0f);
        }
    } else if (wave == 1 && a.loss && blockIdx.x == 0 && blockIdx.y == 0) {
        double loss = 0.0;
        if (lane < a.rows && row_live(a, lane)) {
            Share s = {-INFINITY, 0.0};
            for (int i = 0; i < shares; ++i) s.top = fmaxf(s.top, in[lane * shares + i].top);
            for (int i = 0; i < shares; ++i) s.sum += rescaled(in[lane * shares + i], s.top);
            PolicyArgs mine = a;
            mine.token_logp = mine.token_kl = nullptr;
            loss = finish_row(mine, lane, true, s, label_logits[lane]).loss;
        }
        loss = wave_sum(loss);
        if (lane == 0) *a.loss = static_cast<float>(loss);
    }
    __syncthreads();
    if (a.dlogits.data) write_gradient<kBf16, kBlock>(a, row, span.first, span.last, threadIdx.x, result, a.labels[row]);
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

// Which kernel takes a call, by rows and vocabulary (measured with the others
// forced on the same calls, us, over more than 1 GB of inputs in turn; bf16
// where nothing else is said):
//   - up to kWaveVocab logits a row is a wavefront's: 8000 x 5000 52 against 69
//     with a block each, 8000 x 2000 32 against 44, 30000 x 1000 49 against
//     127.  The rule does not look at the rows, and loses where they do not
//     fill the chip, sixteen to a block: 16 x 8000 38 against 12, 1000 x 8000
//     45 against 15, 1000 x 2000 23 against 13 (fp32 4000 x 5000 52 against 47);
//   - above, a block's of 256 threads that reads it twice, up to kBlockVocab
//     logits: 2000 x 9000 24 against 47 by wavefronts and 26 when the 256 keep
//     it, 8000 x 9000 77, 87 and 80.  Keeping is ahead from about 10000 on:
//     8000 x 12000 98 against 90, 2000 x 16000 42 against 35;
//   - above that, kept by a block of 512 or 1024: 1000 x 32003 35 against 43
//     read twice, 4000 x 32003 123 against 149, 8192 x 128256 791 against 1079,
//     fp32 2000 x 65000 227 against 263, 1000 x 32003 59 against 66; but 2000 x
//     20000 46 and 46, fp32 85 against 78;
//   - up to kFewRows rows of more than kShareVocab logits, blocks share a row:
//     24 x 128256 14.9 against 20.9 kept, 64 x 200000 19.0 against 33.4, 24 x
//     50257 12.0 against 15.0, fp32 64 x 128256 22.7 against 29.7; 24 x 32000
//     12 either way.  kFewRows is a wavefront's lanes (policy_rows_kernel sums
//     the loss a row per lane) and not where the two sides meet: 64 x 128256
//     takes 16.4, 65 rows, kept, 22.4.
constexpr int64_t kWaveVocab = 8192;
constexpr int64_t kBlockVocab = 16384;
constexpr int64_t kFewRows = 64;
constexpr int64_t kShareVocab = 32768;
// Logits of a share, at most (unless lanes or blocks run out): the kDeep units
// that each thread of a block has under way at once.  24 x 128256 bf16 13.4 us
// with shares just above it, 14.3 with 4096.
constexpr int kShareLogits = kDeep * kUnit * kBlock;
constexpr int kMostBlocks = 2048;
static_assert(kFewRows <= kWave, "a row per lane");

// Blocks that share a row: two blocks per CU in all, and at most a lane's
// worth.  1: a row per block or per wavefront.
int shares_of(int64_t rows, int64_t vocab)
{
    if (rows <= 0 || rows > kFewRows || vocab <= kShareVocab) return 1;
    int64_t s = (vocab + kShareLogits - 1) / kShareLogits;
    if (s > 512 / rows) s = 512 / rows;
    return static_cast<int>(s > kWave ? kWave : s);
}

}  // namespace

size_t policy_scratch(int64_t rows, int64_t vocab)
{
    const int shares = shares_of(rows, vocab);
    if (shares > 1) return static_cast<size_t>(rows) * (shares * sizeof(Share) + sizeof(float));
    return static_cast<size_t>(rows < kMostBlocks ? rows : kMostBlocks) * sizeof(double);
}

hipError_t launch_policy_loss(const PolicyArgs& a, bool bf16, void* scratch, hipStream_t stream)
{
    const int shares = shares_of(a.rows, a.vocab);
    if (shares > 1) {
        Share* parts = static_cast<Share*>(scratch);
        float* label_logits = reinterpret_cast<float*>(parts + a.rows * shares);
        const dim3 grid(static_cast<uint32_t>(a.rows), shares);
        if (bf16) {
            policy_shares_kernel<true><<<grid, kBlock, 0, stream>>>(a, shares, parts, label_logits);
            policy_rows_kernel<true><<<grid, kBlock, 0, stream>>>(a, shares, parts, label_logits);
        } else {
            policy_shares_kernel<false><<<grid, kBlock, 0, stream>>>(a, shares, parts, label_logits);
            policy_rows_kernel<false><<<grid, kBlock, 0, stream>>>(a, shares, parts, label_logits);
        }
        return hipGetLastError();
    }
    double* losses = a.loss ? static_cast<double*>(scratch) : nullptr;  // a sum per block
    int64_t n = 0;                                                      // their count
    auto blocks = [&](int64_t jobs, int most) { return static_cast<int>(n = jobs < most ? jobs : most); };
    if (a.rows > 0 && a.vocab <= kWaveVocab) {
        const int grid = blocks((a.rows + kGroup - 1) / kGroup, kMostBlocks);
        if (bf16) policy_wave_kernel<true><<<grid, kBlock, 0, stream>>>(a, losses);
        else policy_wave_kernel<false><<<grid, kBlock, 0, stream>>>(a, losses);
    } else if (a.rows > 0) {
        if (a.vocab <= kBlockVocab) {
            const int grid = blocks(a.rows, kMostBlocks);
            if (bf16) policy_block_kernel<true><<<grid, kBlock, 0, stream>>>(a, losses);
            else policy_block_kernel<false><<<grid, kBlock, 0, stream>>>(a, losses);
        } else if (bf16) {
            if (a.vocab < 1024 * 8 * 8) policy_kept_kernel<true, 512, 4, 4><<<blocks(a.rows, 256 * 2), 512, 0, stream>>>(a, losses);
            else policy_kept_kernel<true, 1024, 8, 8><<<blocks(a.rows, 256), 1024, 0, stream>>>(a, losses);
        } else {
            if (a.vocab < 1024 * 4 * 8) policy_kept_kernel<false, 512, 4, 4><<<blocks(a.rows, 256 * 2), 512, 0, stream>>>(a, losses);
            else policy_kept_kernel<false, 1024, 4, 4><<<blocks(a.rows, 256), 1024, 0, stream>>>(a, losses);
        }
    }
    if (a.loss) policy_total_kernel<<<1, kBlock, 0, stream>>>(losses, n, a.loss);
    return hipGetLastError();
}

}  // namespace mps
