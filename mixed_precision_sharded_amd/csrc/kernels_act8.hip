// gfx950 kernels of the 8-bit activations: keeping a matrix and reading it
// back, RMSNorm and SwiGLU forward (which keep their inputs) and backward
// (which read them).
//
// A lane takes eight consecutive elements of a row (16 bytes of bf16), so
// four lanes hold a run of 32: the run's largest magnitude is two exchanges
// within a quad away, the codes of a lane are one 8-byte store, and every
// access of a wavefront is contiguous.  Rows are padded to whole runs, so a
// run never spans two rows and rows of codes stay aligned whatever the
// matrix's own width and stride.
#include <hip/hip_runtime.h>

#include "rows.h"
#include "train_kernels.h"

namespace mps {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = 1.92596299112661746887e-8f;  // log2(e) - kLog2e
constexpr float kLn2 = 0.69314718055994530942f;

// ------------------------------------------------------- keep, read back ---
//
// Bound by memory: 16384 x 8192 bf16 is kept in 68 us and read back in 63 (407
// MB each, 5.9 and 6.5 TB/s).

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_save_kernel(Matrix x, int64_t rows, int64_t cols,
                                                           uint32_t per_row, CodesOut out)
{
    RowWalk w(per_row);
    for (; w.row < rows; w.next()) {
        float v[kUnit];
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        widen<kBf16>(load8<kBf16>(x.data, w.row * x.stride + c, cols - c), v);
        store_codes<false>(v, out.codes, out.scales, w.unit());
    }
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_load_kernel(Codes in, int64_t rows, int64_t cols,
                                                           uint32_t per_row, MatrixOut x)
{
    RowWalk w(per_row);
    for (; w.row < rows; w.next()) {
        float v[kUnit];
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        load_codes(in.codes, in.scales, w.unit(), v);
        store_unit<kBf16>(v, x.data, w.row * x.stride + c, cols - c);
    }
}

// ---------------------------------------------------------------- SwiGLU ---
//
// Forward: o = g s u with s = 1 / (1 + e^-g), keeping g and u.  Backward, from
// what was kept: dg = d u s (1 + g (1 - s)), du = d g s, and o once more, in 8
// bits, for the next weight gradient.  Both are bound by memory: 8192 x 14336
// bf16 forward 159 us (5.95 TB/s), backward 175 us (6.1 TB/s); the kernel of
// 333 x 5001 fp32 takes 5.3 us, its launch 8.5.

// 1 / (1 + e^-g).  The exponent -g log2(e) is rounded to n, and what the
// rounding lost is put back to first order, so the error stays near the two
// instructions' own (1 ulp each).  From |n| = 128 on, where 2^n is 0 or
// infinite and the correction would be inf * 0, it is left out.  The reciprocal
// gives 0 for results below fp32's normal range, 2^-126: g below -87.3.
__device__ __forceinline__ float sigmoid(float g)
{
    const float n = -g * kLog2e;
    const float lost = __builtin_fmaf(-g, kLog2e, -n) - g * kLog2eLow;
    const float p = __builtin_amdgcn_exp2f(n);
    const float t = fabsf(n) < 128.0f ? __builtin_fmaf(p * kLn2, lost, p) : p;
    return __builtin_amdgcn_rcpf(1.0f + t);
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_swiglu_kernel(Matrix gate, Matrix up, int64_t rows,
                                                             int64_t cols, uint32_t per_row,
                                                             MatrixOut out, CodesOut kept_gate,
                                                             CodesOut kept_up)
{
    RowWalk w(per_row);
    for (; w.row < rows; w.next()) {
        float g[kUnit], u[kUnit], o[kUnit];
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        const Raw8<kBf16> rg = load8<kBf16>(gate.data, w.row * gate.stride + c, cols - c);
        const Raw8<kBf16> ru = load8<kBf16>(up.data, w.row * up.stride + c, cols - c);
        widen<kBf16>(rg, g);
        widen<kBf16>(ru, u);
        store_codes<true>(g, kept_gate.codes, kept_gate.scales, w.unit());
        store_codes<true>(u, kept_up.codes, kept_up.scales, w.unit());
#pragma unroll
        for (int i = 0; i < kUnit; ++i) o[i] = g[i] * sigmoid(g[i]) * u[i];
        store_unit<kBf16>(o, out.data, w.row * out.stride + c, cols - c);
    }
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_swiglu_backward_kernel(
    Matrix dout, Codes gate, Codes up, int64_t rows, int64_t cols, uint32_t per_row,
    MatrixOut dgate, MatrixOut dup, CodesOut out)
{
    RowWalk w(per_row);
    for (; w.row < rows; w.next()) {
        float d[kUnit], g[kUnit], u[kUnit], dg[kUnit], du[kUnit], o[kUnit];
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        widen<kBf16>(load8<kBf16>(dout.data, w.row * dout.stride + c, cols - c), d);
        load_codes(gate.codes, gate.scales, w.unit(), g);
        load_codes(up.codes, up.scales, w.unit(), u);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const float s = sigmoid(g[i]);
            const float gs = g[i] * s;
            o[i] = gs * u[i];
            dg[i] = d[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
            du[i] = d[i] * gs;
        }
        store_unit<kBf16>(dg, dgate.data, w.row * dgate.stride + c, cols - c);
        store_unit<kBf16>(du, dup.data, w.row * dup.stride + c, cols - c);
        if (out.codes) {
            // Behind the row's end the kept bytes may hold anything.
#pragma unroll
            for (int i = 0; i < kUnit; ++i) o[i] = i < cols - c ? o[i] : 0.0f;
            store_codes<true>(o, out.codes, out.scales, w.unit());
        }
    }
}

// --------------------------------------------------------------- RMSNorm ---
//
// Forward: y = x r w with r = 1 / sqrt(mean(x^2) + eps), keeping x and r.
// Backward, with xh = x r from the kept x: dx = r (w dy - xh mean(w dy xh))
// [+ residual], dw = sum over the rows of dy xh.  Both are bound by memory:
// 8192 x 4096 bf16 forward 26.9 us (6.3 TB/s); 4096 x 8192 backward, with a
// residual and xh w in 8 bits, 49 us (5.5 TB/s; 45 and the join's 4).
//
// A team of kThreads lanes holds a whole row, kUnits units of eight per lane,
// so x (or dy) is read once, the weights once per team instead of once per
// row, and dweight's sums stay in registers over all of a team's rows.  The
// next row's loads go out before the present row's sum is waited for (except
// with two units a lane, whose registers they would not fit: the fp32 backward
// with a residual spills 26 of its 128 as it is).
template <int kThreads>
struct Team {
    static constexpr int kBlockThreads = kThreads < kBlock ? kBlock : kThreads;
    static constexpr int kTeams = kBlockThreads / kThreads;    // in a block
    static constexpr int kWaves = kThreads / kWave;            // of a team
    static_assert(kTeams == 1 || kWaves == 1, "only teams of one wavefront share a block");

    // The team's sum, the same bits in every lane.  `lds` is used in turn by
    // even and odd calls, so that one barrier separates a call's writes from
    // its reads, and its reads from the writes of the call after next.
    static __device__ __forceinline__ float sum(float x, float (&lds)[2][kWaves], int odd)
    {
        x = wave_sumf(x);
        if (kWaves == 1) return x;
        if (threadIdx.x % kWave == 0) lds[odd][threadIdx.x / kWave] = x;
        __syncthreads();
        float r = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) r += lds[odd][w];
        return r;
    }
};

template <bool kBf16, int kThreads, int kUnits>
__global__ __launch_bounds__(Team<kThreads>::kBlockThreads) void act8_rmsnorm_kernel(Matrix x, int64_t rows, int64_t cols,
                                                                                     uint32_t per_row, const float* weight,
                                                                                     float eps, MatrixOut y, float* rstd,
                                                                                     CodesOut kept)
{
    using T = Team<kThreads>;
    __shared__ float lds[2][T::kWaves];
    const uint32_t t = threadIdx.x % kThreads;
    const int64_t step = static_cast<int64_t>(gridDim.x) * T::kTeams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * T::kTeams + threadIdx.x / kThreads;
    float w[kUnits][kUnit];
    Raw8<kBf16> raw[kUnits];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int64_t c = static_cast<int64_t>(t + j * kThreads) * kUnit;
            raw[j] = load8<kBf16>(x.data, row * x.stride + c, cols - c);
        }
    };
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const int64_t c = static_cast<int64_t>(t + j * kThreads) * kUnit;
        widen<false>(load8<false>(weight, c, cols - c), w[j]);
    }
    if (row < rows) load(row);
    for (int odd = 0; row < rows; row += step, odd ^= 1) {
        float v[kUnits][kUnit], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            widen<kBf16>(raw[j], v[j]);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) sum = __builtin_fmaf(v[j][i], v[j][i], sum);
        }
        if (row + step < rows) load(row + step);
        const float mean = T::sum(sum, lds, odd) / static_cast<float>(cols);
        const float r = 1.0f / __builtin_sqrtf(mean + eps);
        if (t == 0) rstd[row] = r;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const uint32_t u = t + j * kThreads;
            if (u >= per_row) continue;
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            store_codes<true>(v[j], kept.codes, kept.scales, row * per_row + u);
            float o[kUnit];
#pragma unroll
            for (int i = 0; i < kUnit; ++i) o[i] = v[j][i] * r * w[j][i];
            store_unit<kBf16>(o, y.data, row * y.stride + c, cols - c);
        }
    }
}

// xh = x * r of a kept unit, zeros behind the row's end.
__device__ __forceinline__ void kept_xhat(u32x2 codes, uint32_t byte, int64_t n, float r, float (&xh)[kUnit])
{
    decode8(codes, byte, xh);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) xh[i] = i < n ? xh[i] * r : 0.0f;
}

// dx of one unit; `o` is free to use afterwards.
template <bool kBf16>
__device__ __forceinline__ void norm_dx(const float (&d)[kUnit], const float (&xh)[kUnit], const float (&w)[kUnit], float r,
                                        float mean, const Raw8<kBf16>* residual, MatrixOut dx, int64_t row, int64_t c,
                                        int64_t cols)
{
    float o[kUnit], res[kUnit] = {};
    if (residual) widen<kBf16>(*residual, res);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
        o[i] = r * (d[i] * w[i] - xh[i] * mean);
        if (residual) o[i] += res[i];
    }
    store_unit<kBf16>(o, dx.data, row * dx.stride + c, cols - c);
}

// Block b leaves its rows' share of dweight in row b of `partials`.
template <bool kBf16, bool kResidual, int kThreads, int kUnits>
__global__ __launch_bounds__(Team<kThreads>::kBlockThreads) void act8_rmsnorm_backward_kernel(
    Matrix dy, Codes kept, const float* rstd, int64_t rows, int64_t cols, uint32_t per_row, const float* weight,
    Matrix residual, MatrixOut dx, CodesOut out, float* partials)
{
    using T = Team<kThreads>;
    __shared__ float lds[2][T::kWaves];
    __shared__ float joined[T::kTeams > 1 ? T::kTeams : 1][T::kTeams > 1 ? kThreads * kUnits * kUnit : 1];
    const uint32_t t = threadIdx.x % kThreads;
    const int64_t step = static_cast<int64_t>(gridDim.x) * T::kTeams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * T::kTeams + threadIdx.x / kThreads;
    float w[kUnits][kUnit], acc[kUnits][kUnit] = {};
    Raw8<kBf16> raw[kUnits], res[kUnits];
    u32x2 codes[kUnits];
    uint32_t byte[kUnits];
    float r_next = 0.0f;
    auto load = [&](int64_t row) {
        r_next = rstd[row];
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const uint32_t u = t + j * kThreads;
            const int64_t c = static_cast<int64_t>(u) * kUnit, unit = row * per_row + min(u, per_row - 1);
            raw[j] = load8<kBf16, true>(dy.data, row * dy.stride + c, cols - c);
            if (kResidual) res[j] = load8<kBf16, true>(residual.data, row * residual.stride + c, cols - c);
            codes[j] = reinterpret_cast<const u32x2*>(kept.codes)[unit];
            byte[j] = kept.scales[unit / 4];
        }
    };
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const int64_t c = static_cast<int64_t>(t + j * kThreads) * kUnit;
        widen<false>(load8<false>(weight, c, cols - c), w[j]);
    }
    constexpr bool kAhead = kUnits == 1;
    if (kAhead && row < rows) load(row);
    for (int odd = 0; row < rows; row += step, odd ^= 1) {
        if (!kAhead) load(row);
        const float r = r_next;
        float d[kUnits][kUnit], xh[kUnits][kUnit], sum = 0.0f;
        Raw8<kBf16> mine[kUnits];
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int64_t c = static_cast<int64_t>(t + j * kThreads) * kUnit;
            widen<kBf16>(raw[j], d[j]);
            kept_xhat(codes[j], byte[j], cols - c, r, xh[j]);
            if (kResidual) mine[j] = res[j];
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
                sum = __builtin_fmaf(d[j][i] * w[j][i], xh[j][i], sum);
                acc[j][i] = __builtin_fmaf(d[j][i], xh[j][i], acc[j][i]);
            }
        }
        if (kAhead && row + step < rows) load(row + step);
        const float mean = T::sum(sum, lds, odd) / static_cast<float>(cols);
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const uint32_t u = t + j * kThreads;
            if (u >= per_row) continue;
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            norm_dx<kBf16>(d[j], xh[j], w[j], r, mean, kResidual ? &mine[j] : nullptr, dx, row, c, cols);
            if (out.codes) {
                float o[kUnit];
#pragma unroll
                for (int i = 0; i < kUnit; ++i) o[i] = xh[j][i] * w[j][i];
                store_codes<true>(o, out.codes, out.scales, row * per_row + u);
            }
        }
    }
    // Teams of one wavefront: joined in LDS, in team order.
    if (T::kTeams > 1) {
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
#pragma unroll
            for (int i = 0; i < kUnit; ++i) joined[threadIdx.x / kThreads][(t + j * kThreads) * kUnit + i] = acc[j][i];
        }
        __syncthreads();
        if (threadIdx.x >= kThreads) return;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
                for (int k = 1; k < T::kTeams; ++k) acc[j][i] += joined[k][(t + j * kThreads) * kUnit + i];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const uint32_t u = t + j * kThreads;
        if (u < per_row) store8<false>(acc[j], partials, (static_cast<int64_t>(blockIdx.x) * per_row + u) * kUnit, kUnit);
    }
}

// ------------------------------------------- rows longer than a block's ---

// Sum over the block in a fixed order, the same bits in every thread.
__device__ __forceinline__ float block_sumf(float x, float* lds)
{
    x = wave_sumf(x);
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = x;
    __syncthreads();
    float r = 0.0f;
    for (int w = 0; w < kWavesPerBlock; ++w) r += lds[w];
    return r;
}

// A block takes a row at a time and reads it twice.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_rmsnorm_long_kernel(Matrix x, int64_t rows, int64_t cols, uint32_t per_row,
                                                                   const float* weight, float eps, MatrixOut y, float* rstd,
                                                                   CodesOut kept)
{
    __shared__ float lds[kWavesPerBlock];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        float sum = 0.0f, v[kUnit], wt[kUnit], o[kUnit];
        for (uint32_t u = threadIdx.x; u < per_row; u += kBlock) {
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            widen<kBf16>(load8<kBf16>(x.data, row * x.stride + c, cols - c), v);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) sum = __builtin_fmaf(v[i], v[i], sum);
        }
        const float mean = block_sumf(sum, lds) / static_cast<float>(cols);
        const float r = 1.0f / __builtin_sqrtf(mean + eps);
        if (threadIdx.x == 0) rstd[row] = r;
        for (uint32_t u = threadIdx.x; u < per_row; u += kBlock) {
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            widen<kBf16>(load8<kBf16>(x.data, row * x.stride + c, cols - c), v);
            widen<false>(load8<false>(weight, c, cols - c), wt);
            store_codes<true>(v, kept.codes, kept.scales, row * per_row + u);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) o[i] = v[i] * r * wt[i];
            store8<kBf16>(o, y.data, row * y.stride + c, cols - c);
        }
    }
}

__device__ __forceinline__ void load_xhat(Codes kept, int64_t unit, int64_t n, float r, float (&xh)[kUnit])
{
    kept_xhat(reinterpret_cast<const u32x2*>(kept.codes)[unit], kept.scales[unit / 4], n, r, xh);
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_rmsnorm_backward_long_kernel(
    Matrix dy, Codes kept, const float* rstd, int64_t rows, int64_t cols, uint32_t per_row,
    const float* weight, Matrix residual, MatrixOut dx, CodesOut out)
{
    __shared__ float lds[kWavesPerBlock];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float r = rstd[row];
        float sum = 0.0f, d[kUnit], xh[kUnit], wt[kUnit];
        for (uint32_t u = threadIdx.x; u < per_row; u += kBlock) {
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            widen<kBf16>(load8<kBf16>(dy.data, row * dy.stride + c, cols - c), d);
            widen<false>(load8<false>(weight, c, cols - c), wt);
            load_xhat(kept, row * per_row + u, cols - c, r, xh);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) sum = __builtin_fmaf(d[i] * wt[i], xh[i], sum);
        }
        const float mean = block_sumf(sum, lds) / static_cast<float>(cols);
        for (uint32_t u = threadIdx.x; u < per_row; u += kBlock) {
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            widen<kBf16>(load8<kBf16>(dy.data, row * dy.stride + c, cols - c), d);
            widen<false>(load8<false>(weight, c, cols - c), wt);
            load_xhat(kept, row * per_row + u, cols - c, r, xh);
            Raw8<kBf16> res;
            if (residual.data) res = load8<kBf16>(residual.data, row * residual.stride + c, cols - c);
            norm_dx<kBf16>(d, xh, wt, r, mean, residual.data ? &res : nullptr, dx, row, c, cols);
            if (out.codes) {
                float o[kUnit];
#pragma unroll
                for (int i = 0; i < kUnit; ++i) o[i] = xh[i] * wt[i];
                store_codes<true>(o, out.codes, out.scales, row * per_row + u);
            }
        }
    }
}

// Partial sums of dweight: block (x, y) takes 256 units of columns and the
// rows y, y + gridDim.y, ...
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_rmsnorm_dweight_kernel(Matrix dy, Codes kept,
                                                                      const float* rstd, int64_t rows,
                                                                      int64_t cols, uint32_t per_row,
                                                                      float* partials)
{
    const uint32_t u = blockIdx.x * kBlock + threadIdx.x;
    if (u >= per_row) return;
    const int64_t c = static_cast<int64_t>(u) * kUnit;
    float acc[kUnit] = {}, d[kUnit], xh[kUnit];
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        widen<kBf16>(load8<kBf16>(dy.data, row * dy.stride + c, cols - c), d);
        load_xhat(kept, row * per_row + u, cols - c, rstd[row], xh);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) acc[i] = __builtin_fmaf(d[i], xh[i], acc[i]);
    }
    store8<false>(acc, partials, static_cast<int64_t>(blockIdx.y) * per_row * kUnit + c, kUnit);
}

// dweight = [dweight +] the n partial rows (`stride` floats apart): sixteen
// wavefronts take every sixteenth row each, then their sums in order.
constexpr int kParts = 16;
__global__ __launch_bounds__(kWave * kParts) void sum_partials_kernel(const float* partials, int n, int64_t stride, int64_t cols,
                                                                      float* dweight, bool accumulate)
{
    __shared__ float lds[kParts][kWave];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + threadIdx.x % kWave;
    const int part = threadIdx.x / kWave;
    float sum = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int i = part; i < n; i += kParts) sum += partials[i * stride + c];
    }
    lds[part][threadIdx.x % kWave] = sum;
    __syncthreads();
    if (part == 0 && c < cols) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) all += lds[i][threadIdx.x];
        dweight[c] = accumulate ? dweight[c] + all : all;
    }
}

__global__ __launch_bounds__(kBlock) void zero_kernel(float* x, int64_t n)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * kBlock;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n; i += step) x[i] = 0.0f;
}

uint32_t units_per_row(int64_t cols) { return static_cast<uint32_t>((cols + kRun - 1) / kRun * (kRun / kUnit)); }

// Blocks for `n` threads' worth of work, at most `most`.
int blocks_for(int64_t n, int most)
{
    const int64_t b = (n + kBlock - 1) / kBlock;
    return static_cast<int>(b < most ? b : most);
}

// Blocks of the element-wise kernels: one unit a thread (the walk goes on only
// behind 2^30 units).  Threads that come back for more stream slower: SwiGLU
// backward 8192 x 14336 takes 175 us with one unit a thread, 187 with blocks
// capped at 16384, 205 at 2048, 202 at 1024 (forward 159, 167, 183, 182; keep
// and read 16384 x 8192 135, 132, 143, 145).
constexpr int kStreamBlocks = 1 << 22;
constexpr int kRowBlocks = 2048;  // a row per block: eight blocks of 256 per CU
constexpr int kDweightSplits = 64;   // partial rows of dweight, long rows

// Calls f<threads, units> with the team that holds a row of `cols`, and the
// most blocks of it; false for rows longer than 16384.  Measured for the
// backward pass of 4096 x 8192 bf16: 1024 lanes in 256 blocks 49.2 us, in 512
// blocks 52.7, 512 lanes of two units in 256 / 512 blocks 61.9 / 65.4; 8192 x
// 4096: 512 lanes in 512 blocks 49.8, in 1024 blocks 56.1, 256 lanes of two
// units in 512 / 1024 blocks 56.7 / 63.0 (more blocks, more partial rows).
// Forward 8192 x 4096: 26.9, 30.3, 27.8, 27.3 in the same order.  These widths
// fill their teams; just above a class's edge lanes idle, and short rows wait for
// one another: backward 15000 x 576 30 us for bytes worth 12, 4000 x 2176 21.5
// for 12, 1000 x 8320 22 for 11, and by blocks that read a row twice 400 x 20000
// 43 for 11 (forward 19, 13, 11 and 16 for 7 each).
template <class F>
bool with_team(int64_t cols, F&& f)
{
    if (cols <= 512) f.template operator()<64, 1>(1024);
    else if (cols <= 2048) f.template operator()<256, 1>(1024);
    else if (cols <= 4096) f.template operator()<512, 1>(512);
    else if (cols <= 8192) f.template operator()<1024, 1>(256);
    else if (cols <= 16384) f.template operator()<1024, 2>(256);
    else return false;
    return true;
}

struct CountBlocks {
    int64_t rows;
    int grid = 0;
    template <int kThreads, int kUnits>
    void operator()(int most)
    {
        const int64_t blocks = (rows + Team<kThreads>::kTeams - 1) / Team<kThreads>::kTeams;
        grid = static_cast<int>(blocks < most ? blocks : most);
    }
};

// Blocks of the team kernels, which are also dweight's partial rows.
int team_blocks(int64_t rows, int64_t cols)
{
    CountBlocks c{rows};
    if (with_team(cols, c)) return c.grid;
    return static_cast<int>(rows < kDweightSplits ? rows : kDweightSplits);
}

struct NormForward {
    Matrix x;
    bool bf16;
    int64_t rows, cols;
    const float* weight;
    float eps;
    MatrixOut y;
    float* rstd;
    CodesOut kept;
    hipStream_t stream;
    template <int kThreads, int kUnits>
    void operator()(int)
    {
        constexpr int kBlockThreads = Team<kThreads>::kBlockThreads;
        const int grid = team_blocks(rows, cols);
        const uint32_t per_row = units_per_row(cols);
        if (bf16) act8_rmsnorm_kernel<true, kThreads, kUnits><<<grid, kBlockThreads, 0, stream>>>(x, rows, cols, per_row, weight, eps, y, rstd, kept);
        else act8_rmsnorm_kernel<false, kThreads, kUnits><<<grid, kBlockThreads, 0, stream>>>(x, rows, cols, per_row, weight, eps, y, rstd, kept);
    }
};

struct NormBackward {
    Matrix dy;
    bool bf16;
    Codes kept;
    const float* rstd;
    int64_t rows, cols;
    const float* weight;
    Matrix residual;
    MatrixOut dx;
    CodesOut out;
    float* partials;
    hipStream_t stream;
    template <int kThreads, int kUnits>
    void operator()(int)
    {
        const int grid = team_blocks(rows, cols);
        auto run = [&](auto kernel) {
            kernel<<<grid, Team<kThreads>::kBlockThreads, 0, stream>>>(dy, kept, rstd, rows, cols, units_per_row(cols), weight,
                                                                       residual, dx, out, partials);
        };
        if (bf16) {
            if (residual.data) run(act8_rmsnorm_backward_kernel<true, true, kThreads, kUnits>);
            else run(act8_rmsnorm_backward_kernel<true, false, kThreads, kUnits>);
        } else {
            if (residual.data) run(act8_rmsnorm_backward_kernel<false, true, kThreads, kUnits>);
            else run(act8_rmsnorm_backward_kernel<false, false, kThreads, kUnits>);
        }
    }
};

}  // namespace

// --------------------------------------------------------------- launchers ---

hipError_t launch_act8_save(Matrix x, bool bf16, int64_t rows, int64_t cols, CodesOut out, hipStream_t stream)
{
    const uint32_t per_row = units_per_row(cols);
    const int grid = blocks_for(rows * per_row, kStreamBlocks);
    if (bf16) act8_save_kernel<true><<<grid, kBlock, 0, stream>>>(x, rows, cols, per_row, out);
    else act8_save_kernel<false><<<grid, kBlock, 0, stream>>>(x, rows, cols, per_row, out);
    return hipGetLastError();
}

hipError_t launch_act8_load(Codes in, int64_t rows, int64_t cols, MatrixOut x, bool bf16, hipStream_t stream)
{
    const uint32_t per_row = units_per_row(cols);
    const int grid = blocks_for(rows * per_row, kStreamBlocks);
    if (bf16) act8_load_kernel<true><<<grid, kBlock, 0, stream>>>(in, rows, cols, per_row, x);
    else act8_load_kernel<false><<<grid, kBlock, 0, stream>>>(in, rows, cols, per_row, x);
    return hipGetLastError();
}

hipError_t launch_act8_rmsnorm(Matrix x, bool bf16, int64_t rows, int64_t cols, const float* weight, float eps,
                               MatrixOut y, float* rstd, CodesOut kept, hipStream_t stream)
{
    NormForward f{x, bf16, rows, cols, weight, eps, y, rstd, kept, stream};
    if (!with_team(cols, f)) {
        const uint32_t per_row = units_per_row(cols);
        const int grid = static_cast<int>(rows < kRowBlocks ? rows : kRowBlocks);
        if (bf16) act8_rmsnorm_long_kernel<true><<<grid, kBlock, 0, stream>>>(x, rows, cols, per_row, weight, eps, y, rstd, kept);
        else act8_rmsnorm_long_kernel<false><<<grid, kBlock, 0, stream>>>(x, rows, cols, per_row, weight, eps, y, rstd, kept);
    }
    return hipGetLastError();
}

size_t rmsnorm_backward_scratch(int64_t rows, int64_t cols)
{
    return static_cast<size_t>(team_blocks(rows, cols)) * units_per_row(cols) * kUnit * sizeof(float);
}

hipError_t launch_act8_rmsnorm_backward(Matrix dy, bool bf16, Codes kept, const float* rstd, int64_t rows,
                                        int64_t cols, const float* weight, Matrix residual, MatrixOut dx,
                                        float* dweight, bool accumulate, CodesOut out, void* scratch,
                                        hipStream_t stream)
{
    const uint32_t per_row = units_per_row(cols);
    float* partials = static_cast<float*>(scratch);
    const int splits = team_blocks(rows, cols);
    NormBackward f{dy, bf16, kept, rstd, rows, cols, weight, residual, dx, out, partials, stream};
    if (!with_team(cols, f)) {
        const int grid = static_cast<int>(rows < kRowBlocks ? rows : kRowBlocks);
        const dim3 tiles((per_row + kBlock - 1) / kBlock, splits);
        // dweight's sums first: dx may be written over dy.
        if (bf16) {
            act8_rmsnorm_dweight_kernel<true><<<tiles, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, partials);
            act8_rmsnorm_backward_long_kernel<true><<<grid, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, weight,
                                                                                 residual, dx, out);
        } else {
            act8_rmsnorm_dweight_kernel<false><<<tiles, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, partials);
            act8_rmsnorm_backward_long_kernel<false><<<grid, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, weight,
                                                                                  residual, dx, out);
        }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sum_partials_kernel<<<static_cast<int>((cols + kWave - 1) / kWave), kWave * kParts, 0, stream>>>(
        partials, splits, static_cast<int64_t>(per_row) * kUnit, cols, dweight, accumulate);
    return hipGetLastError();
}

hipError_t launch_act8_swiglu(Matrix gate, Matrix up, bool bf16, int64_t rows, int64_t cols, MatrixOut out,
                              CodesOut kept_gate, CodesOut kept_up, hipStream_t stream)
{
    const uint32_t per_row = units_per_row(cols);
    const int grid = blocks_for(rows * per_row, kStreamBlocks);
    if (bf16) act8_swiglu_kernel<true><<<grid, kBlock, 0, stream>>>(gate, up, rows, cols, per_row, out, kept_gate, kept_up);
    else act8_swiglu_kernel<false><<<grid, kBlock, 0, stream>>>(gate, up, rows, cols, per_row, out, kept_gate, kept_up);
    return hipGetLastError();
}

hipError_t launch_act8_swiglu_backward(Matrix dout, bool bf16, Codes gate, Codes up, int64_t rows, int64_t cols,
                                       MatrixOut dgate, MatrixOut dup, CodesOut out, hipStream_t stream)
{
    const uint32_t per_row = units_per_row(cols);
    const int grid = blocks_for(rows * per_row, kStreamBlocks);
    if (bf16) act8_swiglu_backward_kernel<true><<<grid, kBlock, 0, stream>>>(dout, gate, up, rows, cols, per_row, dgate, dup, out);
    else act8_swiglu_backward_kernel<false><<<grid, kBlock, 0, stream>>>(dout, gate, up, rows, cols, per_row, dgate, dup, out);
    return hipGetLastError();
}

hipError_t launch_zero(float* x, int64_t n, hipStream_t stream)
{
    zero_kernel<<<blocks_for(n, kStreamBlocks), kBlock, 0, stream>>>(x, n);
    return hipGetLastError();
}

}  // namespace mps
