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

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_save_kernel(Matrix x, int64_t rows, int64_t cols,
                                                           uint32_t per_row, CodesOut out)
{
    RowWalk w(static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x,
              static_cast<int64_t>(gridDim.x) * kBlock, per_row);
    for (; w.row < rows; w.next()) {
        float v[kUnit];
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        widen<kBf16>(load8<kBf16>(x.data, w.row * x.stride + c, cols - c), v);
        store_codes(v, out.codes, out.scales, w.unit());
    }
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_load_kernel(Codes in, int64_t rows, int64_t cols,
                                                           uint32_t per_row, MatrixOut x)
{
    RowWalk w(static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x,
              static_cast<int64_t>(gridDim.x) * kBlock, per_row);
    for (; w.row < rows; w.next()) {
        float v[kUnit];
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        load_codes(in.codes, in.scales, w.unit(), v);
        store8<kBf16>(v, x.data, w.row * x.stride + c, cols - c);
    }
}

// ---------------------------------------------------------------- SwiGLU ---

// 1 / (1 + e^-g).  The exponent -g log2(e) is rounded to n, and what the
// rounding lost is put back to first order, so the error stays near the two
// instructions' own (1 ulp each) for every g; far out, where 2^n is 0 or
// infinite and the correction would be inf * 0, it is left out.
__device__ __forceinline__ float sigmoid(float g)
{
    const float n = -g * kLog2e;
    const float lost = __builtin_fmaf(-g, kLog2e, -n) - g * kLog2eLow;
    const float p = __builtin_amdgcn_exp2f(n);
    const float t = fabsf(g) > 80.0f ? p : __builtin_fmaf(p * kLn2, lost, p);
    return __builtin_amdgcn_rcpf(1.0f + t);
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_swiglu_kernel(Matrix gate, Matrix up, int64_t rows,
                                                             int64_t cols, uint32_t per_row,
                                                             MatrixOut out, CodesOut kept_gate,
                                                             CodesOut kept_up)
{
    RowWalk w(static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x,
              static_cast<int64_t>(gridDim.x) * kBlock, per_row);
    for (; w.row < rows; w.next()) {
        float g[kUnit], u[kUnit], o[kUnit];
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        const Raw8<kBf16> rg = load8<kBf16>(gate.data, w.row * gate.stride + c, cols - c);
        const Raw8<kBf16> ru = load8<kBf16>(up.data, w.row * up.stride + c, cols - c);
        widen<kBf16>(rg, g);
        widen<kBf16>(ru, u);
        store_codes(g, kept_gate.codes, kept_gate.scales, w.unit());
        store_codes(u, kept_up.codes, kept_up.scales, w.unit());
#pragma unroll
        for (int i = 0; i < kUnit; ++i) o[i] = g[i] * sigmoid(g[i]) * u[i];
        store8<kBf16>(o, out.data, w.row * out.stride + c, cols - c);
    }
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_swiglu_backward_kernel(
    Matrix dout, Codes gate, Codes up, int64_t rows, int64_t cols, uint32_t per_row,
    MatrixOut dgate, MatrixOut dup, CodesOut out)
{
    RowWalk w(static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x,
              static_cast<int64_t>(gridDim.x) * kBlock, per_row);
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
        store8<kBf16>(dg, dgate.data, w.row * dgate.stride + c, cols - c);
        store8<kBf16>(du, dup.data, w.row * dup.stride + c, cols - c);
        if (out.codes) {
            // Behind the row's end the kept bytes may hold anything.
#pragma unroll
            for (int i = 0; i < kUnit; ++i) o[i] = i < cols - c ? o[i] : 0.0f;
            store_codes(o, out.codes, out.scales, w.unit());
        }
    }
}

// --------------------------------------------------------------- RMSNorm ---

// Sum over the block in a fixed order, the same bits in every thread.
__device__ __forceinline__ float block_sumf(float x, float* lds)
{
    x = wave_sumf(x);
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = x;
    __syncthreads();
    float r = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x) / kWave; ++w) r += lds[w];
    return r;
}

// A block takes a row at a time and reads it twice.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_rmsnorm_kernel(Matrix x, int64_t rows, int64_t cols,
                                                              uint32_t per_row, const float* weight,
                                                              float eps, MatrixOut y, float* rstd,
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
            store_codes(v, kept.codes, kept.scales, row * per_row + u);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) o[i] = v[i] * r * wt[i];
            store8<kBf16>(o, y.data, row * y.stride + c, cols - c);
        }
    }
}

// The kept row's unit u: xh = x * r, zeros behind the row's end.
__device__ __forceinline__ void kept_xhat(Codes kept, int64_t unit, int64_t n, float r, float (&xh)[kUnit])
{
    load_codes(kept.codes, kept.scales, unit, xh);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) xh[i] = i < n ? xh[i] * r : 0.0f;
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void act8_rmsnorm_backward_kernel(
    Matrix dy, Codes kept, const float* rstd, int64_t rows, int64_t cols, uint32_t per_row,
    const float* weight, Matrix residual, MatrixOut dx, CodesOut out)
{
    __shared__ float lds[kWavesPerBlock];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float r = rstd[row];
        float sum = 0.0f, d[kUnit], xh[kUnit], wt[kUnit], o[kUnit], res[kUnit];
        for (uint32_t u = threadIdx.x; u < per_row; u += kBlock) {
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            widen<kBf16>(load8<kBf16>(dy.data, row * dy.stride + c, cols - c), d);
            widen<false>(load8<false>(weight, c, cols - c), wt);
            kept_xhat(kept, row * per_row + u, cols - c, r, xh);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) sum = __builtin_fmaf(d[i] * wt[i], xh[i], sum);
        }
        const float mean = block_sumf(sum, lds) / static_cast<float>(cols);
        for (uint32_t u = threadIdx.x; u < per_row; u += kBlock) {
            const int64_t c = static_cast<int64_t>(u) * kUnit;
            widen<kBf16>(load8<kBf16>(dy.data, row * dy.stride + c, cols - c), d);
            widen<false>(load8<false>(weight, c, cols - c), wt);
            kept_xhat(kept, row * per_row + u, cols - c, r, xh);
            if (residual.data) widen<kBf16>(load8<kBf16>(residual.data, row * residual.stride + c, cols - c), res);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
                o[i] = r * (d[i] * wt[i] - xh[i] * mean);
                if (residual.data) o[i] += res[i];
            }
            store8<kBf16>(o, dx.data, row * dx.stride + c, cols - c);
            if (out.codes) {
#pragma unroll
                for (int i = 0; i < kUnit; ++i) o[i] = xh[i] * wt[i];
                store_codes(o, out.codes, out.scales, row * per_row + u);
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
        kept_xhat(kept, row * per_row + u, cols - c, rstd[row], xh);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) acc[i] = __builtin_fmaf(d[i], xh[i], acc[i]);
    }
    store8<false>(acc, partials, static_cast<int64_t>(blockIdx.y) * per_row * kUnit + c, kUnit);
}

// dweight = [dweight +] the n partial rows (`stride` floats apart), in order.
__global__ __launch_bounds__(kBlock) void sum_partials_kernel(const float* partials, int n, int64_t stride,
                                                              int64_t cols, float* dweight, bool accumulate)
{
    __shared__ float lds[kWavesPerBlock][kWave];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + threadIdx.x % kWave;
    const int part = threadIdx.x / kWave;
    float sum = 0.0f;
    if (c < cols) {
        for (int i = part; i < n; i += kWavesPerBlock) sum += partials[i * stride + c];
    }
    lds[part][threadIdx.x % kWave] = sum;
    __syncthreads();
    if (part == 0 && c < cols) {
        float total = accumulate ? dweight[c] : 0.0f;
        float all = 0.0f;
        for (int i = 0; i < kWavesPerBlock; ++i) all += lds[i][threadIdx.x];
        dweight[c] = total + all;
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

constexpr int kStreamBlocks = 2048;  // element-wise kernels: eight blocks of 256 per CU
constexpr int kDweightSplits = 64;   // partial rows of dweight

int dweight_splits(int64_t rows) { return static_cast<int>(rows < kDweightSplits ? rows : kDweightSplits); }

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
    const uint32_t per_row = units_per_row(cols);
    const int grid = static_cast<int>(rows < kStreamBlocks ? rows : kStreamBlocks);
    if (bf16) act8_rmsnorm_kernel<true><<<grid, kBlock, 0, stream>>>(x, rows, cols, per_row, weight, eps, y, rstd, kept);
    else act8_rmsnorm_kernel<false><<<grid, kBlock, 0, stream>>>(x, rows, cols, per_row, weight, eps, y, rstd, kept);
    return hipGetLastError();
}

size_t rmsnorm_backward_scratch(int64_t rows, int64_t cols)
{
    return static_cast<size_t>(dweight_splits(rows)) * units_per_row(cols) * kUnit * sizeof(float);
}

hipError_t launch_act8_rmsnorm_backward(Matrix dy, bool bf16, Codes kept, const float* rstd, int64_t rows,
                                        int64_t cols, const float* weight, Matrix residual, MatrixOut dx,
                                        float* dweight, bool accumulate, CodesOut out, void* scratch,
                                        hipStream_t stream)
{
    const uint32_t per_row = units_per_row(cols);
    float* partials = static_cast<float*>(scratch);
    const int splits = dweight_splits(rows);
    const int grid = static_cast<int>(rows < kStreamBlocks ? rows : kStreamBlocks);
    const dim3 tiles((per_row + kBlock - 1) / kBlock, splits);
    // dweight's sums first: dx may be written over dy.
    if (bf16) {
        act8_rmsnorm_dweight_kernel<true><<<tiles, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, partials);
        act8_rmsnorm_backward_kernel<true><<<grid, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, weight,
                                                                        residual, dx, out);
    } else {
        act8_rmsnorm_dweight_kernel<false><<<tiles, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, partials);
        act8_rmsnorm_backward_kernel<false><<<grid, kBlock, 0, stream>>>(dy, kept, rstd, rows, cols, per_row, weight,
                                                                         residual, dx, out);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sum_partials_kernel<<<static_cast<int>((cols + kWave - 1) / kWave), kBlock, 0, stream>>>(
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
