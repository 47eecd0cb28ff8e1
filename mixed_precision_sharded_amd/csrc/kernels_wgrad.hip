// gfx950 kernel of the weight gradient from 8-bit activations:
//     dw[n, k] = sum over t of dy[t, n] * x[t, k]
// on the matrix cores.  An E4M3 code has four significant bits and its scale
// is a power of two, so a kept value is a bf16 value exactly and its product
// with a bf16 gradient has at most 12 significant bits: bf16 operands with
// fp32 sums lose nothing on the way in.  fp32 gradients are split into three
// bf16 parts of eight bits each, whose sum they are.
//
// Both operands lie with the summed index t as their slow one, while a lane
// of the matrix instruction wants eight t of one column.  Tiles are staged in
// LDS as they lie (rows of t) and read with the transposing LDS load, which
// hands each lane four t of one column.
#include <hip/hip_runtime.h>

#include "rows.h"
#include "train_kernels.h"

namespace mps {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileT = 32;   // t per stage: two matrix instructions deep
constexpr int kTile = 128;   // rows (n) and columns (k) of a block's tile
constexpr int kFrag = 32;    // rows and columns of one matrix instruction

// Byte offset in a staged tile [kTileT][kTile] of bf16 of the 16-byte chunk
// `chunk` of row t.  A transposing load reads 32 bytes from each of four
// consecutive rows per 16 lanes; the exclusive-or sends the four rows to
// different banks.
__device__ __forceinline__ uint32_t chunk_at(int t, int chunk)
{
    return static_cast<uint32_t>(t * kTile * 2 + ((chunk ^ ((t & 3) << 2)) << 4));
}

// Four t (t0 .. t0 + 3) of column `col` for each lane of a group of 16, whose
// lanes hold 16 consecutive columns from col0 on.
__device__ __forceinline__ bf16x4 read_transposed(const char* tile, int t0, int col0, int lane16)
{
    const int t = t0 + lane16 / 4;
    const int col = col0 + lane16 % 4 * 4;
    const char* p = tile + chunk_at(t, col / 8) + (col % 8) * 2;
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                          (__attribute__((address_space(3))) s16x4*)p));
}

// The operand of one matrix instruction: columns col0 .. col0 + 31 (lane %
// 32), t0 + 8 * (lane / 32) .. + 7.
__device__ __forceinline__ bf16x8 read_operand(const char* tile, int t0, int col0, int lane)
{
    const int t = t0 + lane / 32 * 8, c = col0 + lane % 32 / 16 * 16;
    const bf16x4 lo = read_transposed(tile, t, c, lane % 16);
    const bf16x4 hi = read_transposed(tile, t + 4, c, lane % 16);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// An fp32 value as three bf16 parts: the leading eight bits, the next eight,
// the rest (cut off, not rounded, so each remainder is exact and no part
// overflows).  A value that is not finite is its own first part.
__device__ __forceinline__ void split3(float x, uint32_t (&part)[3])
{
    const uint32_t bits = __float_as_uint(x);
    if ((bits & 0x7f800000u) == 0x7f800000u) {
        part[0] = (bits >> 16) | ((bits & 0x7fffffu) ? 0x40u : 0u);
        part[1] = part[2] = 0;
        return;
    }
    part[0] = bits >> 16;
    const float rest = x - __uint_as_float(bits & 0xffff0000u);
    part[1] = __float_as_uint(rest) >> 16;
    const float last = rest - __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
    part[2] = __float_as_uint(last) >> 16;
}

// dw (or partial) value at (n, k).
template <bool kDwBf16>
__device__ __forceinline__ void store_dw(void* dw, int64_t i, float v, bool accumulate)
{
    if (kDwBf16) {
        uint16_t* p = static_cast<uint16_t*>(dw) + i;
        *p = bf16_one(accumulate ? bf16_lo(*p) + v : v);
    } else {
        float* p = static_cast<float*>(dw) + i;
        *p = accumulate ? *p + v : v;
    }
}

// One tile of dw over the t of [t_first, t_last): block (tile, split).
template <bool kDyBf16, bool kDwBf16>
__global__ __launch_bounds__(kBlock) void weight_grad_kernel(Matrix dy, Codes x, int64_t tokens, int64_t n_all,
                                                             int64_t k_all, int64_t per_split, uint32_t tiles_k,
                                                             void* dw, bool accumulate, float* partials)
{
    constexpr int kParts = kDyBf16 ? 1 : 3;
    __shared__ __attribute__((aligned(16))) char tile_a[kParts][kTileT * kTile * 2];
    __shared__ __attribute__((aligned(16))) char tile_b[kTileT * kTile * 2];
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / tiles_k) * kTile;
    const int64_t k0 = static_cast<int64_t>(blockIdx.x % tiles_k) * kTile;
    const int64_t padded = (k_all + kRun - 1) / kRun * kRun;
    const int64_t t_first = blockIdx.y * per_split;
    const int64_t t_last = min(t_first + per_split, tokens);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int wn = wave / 2 * 64, wk = wave % 2 * 64;
    f32x16 acc[2][2] = {};

    for (int64_t t0 = t_first; t0 < t_last; t0 += kTileT) {
        __syncthreads();
        // 512 chunks of eight columns of each operand, two per thread.
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int unit = threadIdx.x + j * kBlock;
            const int t = unit / 16, chunk = unit % 16;
            const bool live = t0 + t < t_last;
            const int64_t n = n0 + chunk * 8;
            const int64_t have = live ? n_all - n : 0;
            const Raw8<kDyBf16> raw = load8<kDyBf16>(dy.data, (t0 + t) * dy.stride + n, have);
            if (kDyBf16) {
                *reinterpret_cast<u32x4*>(tile_a[0] + chunk_at(t, chunk)) = raw.v[0];
            } else {
                float v[kUnit];
                uint32_t part[kUnit][3];
                widen<kDyBf16>(raw, v);
#pragma unroll
                for (int i = 0; i < kUnit; ++i) split3(v[i], part[i]);
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    u32x4 w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = part[2 * i][p] | part[2 * i + 1][p] << 16;
                    *reinterpret_cast<u32x4*>(tile_a[p] + chunk_at(t, chunk)) = w;
                }
            }
            const int64_t k = k0 + chunk * 8;
            u32x2 codes{0, 0};
            uint32_t byte = 0;
            if (live && k < padded) {
                const int64_t u = ((t0 + t) * padded + k) / kUnit;
                codes = reinterpret_cast<const u32x2*>(x.codes)[u];
                byte = x.scales[u / 4];
            }
            const float scale = __uint_as_float(byte << 23);
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], scale, false));
                w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], scale, true));
            }
            *reinterpret_cast<u32x4*>(tile_b + chunk_at(t, chunk)) = w;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kTileT; t += 16) {
            bf16x8 b[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) b[j] = read_operand(tile_b, t, wk + j * kFrag, lane);
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 a = read_operand(tile_a[p], t, wn + i * kFrag, lane);
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[j], acc[i][j], 0, 0, 0);
                }
            }
        }
    }
    // Lane l of a result holds column l % 32 and the rows 8 (r / 4) + 4 (l / 32) + r % 4.
    float* mine = partials ? partials + static_cast<int64_t>(blockIdx.y) * n_all * k_all : nullptr;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t k = k0 + wk + j * kFrag + lane % 32;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t n = n0 + wn + i * kFrag + r / 4 * 8 + lane / 32 * 4 + r % 4;
                if (n < n_all && k < k_all) {
                    if (mine) mine[n * k_all + k] = acc[i][j][r];
                    else store_dw<kDwBf16>(dw, n * k_all + k, acc[i][j][r], accumulate);
                }
            }
        }
    }
}

// dw = [dw +] the splits' partial sums, in split order.
template <bool kDwBf16>
__global__ __launch_bounds__(kBlock) void weight_grad_join_kernel(const float* partials, int splits, int64_t count,
                                                                  void* dw, bool accumulate)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * kBlock;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < count; i += step) {
        float sum = 0.0f;
        for (int s = 0; s < splits; ++s) sum += partials[s * count + i];
        store_dw<kDwBf16>(dw, i, sum, accumulate);
    }
}

struct Shape {
    int64_t tiles_n, tiles_k, per_split;
    int splits;
};

// Enough blocks for the chip's 256 CUs, each with at least 16 stages.
Shape shape_of(int64_t tokens, int64_t n, int64_t k)
{
    Shape s;
    s.tiles_n = (n + kTile - 1) / kTile;
    s.tiles_k = (k + kTile - 1) / kTile;
    const int64_t tiles = s.tiles_n * s.tiles_k;
    const int64_t stages = (tokens + kTileT - 1) / kTileT;
    int64_t splits = 512 / tiles;
    if (splits > stages / 16) splits = stages / 16;
    if (splits < 1) splits = 1;
    const int64_t per = (stages + splits - 1) / splits;
    s.per_split = per * kTileT;
    s.splits = static_cast<int>(per > 0 ? (stages + per - 1) / per : 1);
    return s;
}

}  // namespace

size_t weight_grad_scratch(int64_t tokens, int64_t out_features, int64_t in_features)
{
    const Shape s = shape_of(tokens, out_features, in_features);
    return s.splits > 1 ? static_cast<size_t>(s.splits) * out_features * in_features * sizeof(float) : 0;
}

hipError_t launch_act8_weight_grad(Matrix dy, bool dy_bf16, Codes x, int64_t tokens, int64_t out_features,
                                   int64_t in_features, void* dw, bool dw_bf16, bool accumulate, void* scratch,
                                   hipStream_t stream)
{
    const Shape s = shape_of(tokens, out_features, in_features);
    float* partials = s.splits > 1 ? static_cast<float*>(scratch) : nullptr;
    const dim3 grid(static_cast<uint32_t>(s.tiles_n * s.tiles_k), s.splits);
    const uint32_t tk = static_cast<uint32_t>(s.tiles_k);
    auto run = [&](auto kernel) {
        kernel<<<grid, kBlock, 0, stream>>>(dy, x, tokens, out_features, in_features, s.per_split, tk, dw, accumulate,
                                            partials);
    };
    if (dy_bf16) {
        if (dw_bf16) run(weight_grad_kernel<true, true>);
        else run(weight_grad_kernel<true, false>);
    } else {
        if (dw_bf16) run(weight_grad_kernel<false, true>);
        else run(weight_grad_kernel<false, false>);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !partials) return e;
    const int64_t count = out_features * in_features;
    const int64_t blocks = (count + kBlock - 1) / kBlock;
    const int join_grid = static_cast<int>(blocks < 2048 ? blocks : 2048);
    if (dw_bf16) weight_grad_join_kernel<true><<<join_grid, kBlock, 0, stream>>>(partials, s.splits, count, dw, accumulate);
    else weight_grad_join_kernel<false><<<join_grid, kBlock, 0, stream>>>(partials, s.splits, count, dw, accumulate);
    return hipGetLastError();
}

}  // namespace mps
