// gfx950 kernel of the weight gradient from 8-bit activations:
//     dw[n, k] = sum over t of dy[t, n] * x[t, k]
// on the matrix cores.  An E4M3 code has four significant bits and its scale
// is a power of two, so a kept value of 2^-126 or more is a bf16 value exactly
// (a smaller one rounds to the bits that bf16 has left there) and its product
// with a bf16 gradient has at most 12 significant bits: bf16 operands with
// fp32 sums lose nothing else on the way in.  fp32 gradients are split into
// three bf16 parts of eight bits each, whose sum they are down to 2^-133, where
// bf16 ends.
//
// Both operands lie with the summed index t as their slow one, while a lane
// of the matrix instruction wants eight t of one column.  Tiles are staged in
// LDS as they lie (rows of t) and read with the transposing LDS load, which
// hands each lane four t of one column.
//
// Large products are bound by the matrix instructions (8192 x 4096 x 4096 bf16
// 208 us, 1320 TF/s, their pipes busy 75 % of the cycles; fp32 594 us, three
// products at 1390 TF/s; a chip under this load lowers its clock), small ones
// by the stages' waits and the launch (fp32 777 x 1000 x 2051 25.6 us).  Adding
// to what dw holds is a load, a sum and a store per value behind the product:
// 8192 x 4096 x 4096 305 us into fp32, 267 into bf16.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "mfma.h"
#include "rows.h"
#include "train_kernels.h"

namespace mps {
namespace {

constexpr int kStageBf16 = 64, kStageF32 = 32;  // t per stage of the tiles of 128 and 64

// Eight fp32 values as three bf16 parts each: the leading eight bits, the next
// eight, the rest (cut off, not rounded, so each remainder is exact and no
// part overflows; bits below 2^-133 are lost).  A value that is not finite is its own first part: the
// remainder of an infinity is a NaN, and is set to zero, as a NaN's is, whose
// quiet bit keeps it one in the upper half.
__device__ __forceinline__ void split3(const Raw8<false>& raw, u32x4 (&part)[3])
{
    constexpr uint32_t kUpper = 0x07060302;  // the upper halves of two words
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[3][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float x = __builtin_canonicalizef(__uint_as_float(raw.v[i / 2][i % 2 * 2 + h]));
            w[0][h] = __float_as_uint(x);
            const float rest = x - __uint_as_float(w[0][h] & 0xffff0000u);
            w[1][h] = rest == rest ? __float_as_uint(rest) : 0u;
            const float last = __uint_as_float(w[1][h]) - __uint_as_float(w[1][h] & 0xffff0000u);
            w[2][h] = __float_as_uint(last);
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) part[p][i] = __builtin_amdgcn_perm(w[p][1], w[p][0], kUpper);
    }
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

// Block b of `tiles` takes this tile: the device hands consecutive blocks to
// its eight XCDs in turn, so each XCD (and its L2) gets a stretch of
// neighbouring tiles, which share rows of dy.
struct Tile {
    int64_t n, k;
};
__device__ __forceinline__ Tile tile_of(uint32_t b, uint32_t tiles, uint32_t tiles_k)
{
    const uint32_t each = tiles / 8, more = tiles % 8, xcd = b % 8;
    const uint32_t t = xcd * each + min(xcd, more) + b / 8;
    return {static_cast<int64_t>(t / tiles_k), static_cast<int64_t>(t % tiles_k)};
}

// Where a block's tile goes: dw itself, or its split's partial sums.
struct Target {
    void* dw;
    float* partials;  // or NULL
    bool accumulate;
    int64_t n_all, k_all;
};

// Stores a wavefront's kI x kJ results, whose first element is (n0, k0): lane
// l of a result holds column l % 32 and the rows 8 (r / 4) + 4 (l / 32) + r % 4.
template <bool kEdge, bool kBf16, bool kAccumulate, int kI, int kJ>
__device__ __forceinline__ void store_results(const f32x16 (&acc)[kI][kJ], void* out, int64_t n0, int64_t k0, int64_t n_all,
                                              int64_t k_all)
{
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int i = 0; i < kI; ++i) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int64_t n = n0 + i * kFrag + r / 4 * 8 + lane / 32 * 4 + r % 4;
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int64_t k = k0 + j * kFrag + lane % 32;
                if (!kEdge || (n < n_all && k < k_all)) store_dw<kBf16>(out, n * k_all + k, acc[i][j][r], kAccumulate);
            }
        }
    }
}

template <bool kDwBf16, int kI, int kJ>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[kI][kJ], const Target& to, int64_t n0, int64_t k0)
{
    const bool edge = n0 + kI * kFrag > to.n_all || k0 + kJ * kFrag > to.k_all;
    if (to.partials) {
        float* mine = to.partials + static_cast<int64_t>(blockIdx.y) * to.n_all * to.k_all;
        if (edge) store_results<true, false, false>(acc, mine, n0, k0, to.n_all, to.k_all);
        else store_results<false, false, false>(acc, mine, n0, k0, to.n_all, to.k_all);
    } else if (to.accumulate) {
        if (edge) store_results<true, kDwBf16, true>(acc, to.dw, n0, k0, to.n_all, to.k_all);
        else store_results<false, kDwBf16, true>(acc, to.dw, n0, k0, to.n_all, to.k_all);
    } else {
        if (edge) store_results<true, kDwBf16, false>(acc, to.dw, n0, k0, to.n_all, to.k_all);
        else store_results<false, kDwBf16, false>(acc, to.dw, n0, k0, to.n_all, to.k_all);
    }
}

// One tile of dw over the t of [t_first, t_last): block (tile, split).
template <bool kDyBf16, bool kDwBf16, int kTile>
__global__ __launch_bounds__(kBlock, 2) void weight_grad_kernel(Matrix dy, Codes x, int64_t tokens, int64_t n_all,
                                                                int64_t k_all, int64_t per_split, uint32_t tiles_k,
                                                                Target to)
{
    constexpr int kParts = kDyBf16 ? 1 : 3, kTileT = kDyBf16 ? kStageBf16 : kStageF32;
    constexpr int kBytes = kTileT * kTile * 2;
    __shared__ __attribute__((aligned(16))) char lds[2][kParts + 1][kBytes];  // parts of dy, then x
    const Tile tile = tile_of(blockIdx.x, gridDim.x, tiles_k);
    const int64_t n0 = tile.n * kTile, k0 = tile.k * kTile;
    const int64_t padded = (k_all + kRun - 1) / kRun * kRun;
    const int64_t t_first = blockIdx.y * per_split;
    const int64_t t_last = min(t_first + per_split, tokens);
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    constexpr int kI = kTile / 64;  // a wavefront's results: kI x kI of 32 x 32
    const int wn = wave / 2 * (kTile / 2), wk = wave % 2 * (kTile / 2);
    f32x16 acc[kI][kI] = {};

    // Chunks of eight columns: a thread has the same one of every kStep-th row.
    constexpr int kChunks = kTile / 8, kStep = kBlock / kChunks, kOwn = kTileT / kStep;
    const int t_own = tid / kChunks, chunk = tid % kChunks;
    const int64_t n = n0 + chunk * 8, k = k0 + chunk * 8;
    Raw8<kDyBf16> raw[kOwn];
    u32x2 codes[kOwn];
    uint32_t byte[kOwn];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int64_t t = t0 + t_own + j * kStep;
            raw[j] = load8<kDyBf16>(dy.data, t * dy.stride + n, t < t_last ? n_all - n : 0);
        }
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int64_t t = t0 + t_own + j * kStep;
            codes[j] = u32x2{0, 0};
            byte[j] = 0;
            if (t < t_last && k < padded) {
                const int64_t u = (t * padded + k) / kUnit;
                codes[j] = reinterpret_cast<const u32x2*>(x.codes)[u];
                byte[j] = x.scales[u / 4];
            }
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const uint32_t at = chunk_at<kTile>(t_own + j * kStep, chunk);
            u32x4 part[3];
            if constexpr (kDyBf16) part[0] = raw[j].v[0];
            else split3(raw[j], part);
#pragma unroll
            for (int p = 0; p < kParts; ++p) *reinterpret_cast<u32x4*>(lds[buf][p] + at) = part[p];
        }
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const float scale = __uint_as_float(byte[j] << 23);
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[j][i], scale, false));
                w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[j][i], scale, true));
            }
            *reinterpret_cast<u32x4*>(lds[buf][kParts] + chunk_at<kTile>(t_own + j * kStep, chunk)) = w;
        }
    };

    load(t_first);
    put(0);
    load(t_first + kTileT);
    __syncthreads();
    int buf = 0;
    for (int64_t t0 = t_first; t0 < t_last; t0 += kTileT, buf ^= 1) {
#pragma unroll
        for (int t = 0; t < kTileT; t += 16) {
            bf16x8 b[kI];
#pragma unroll
            for (int j = 0; j < kI; ++j) b[j] = read_operand<kTile>(lds[buf][kParts], t, wk + j * kFrag, lane);
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    const bf16x8 a = read_operand<kTile>(lds[buf][p], t, wn + i * kFrag, lane);
#pragma unroll
                    for (int j = 0; j < kI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[j], acc[i][j], 0, 0, 0);
                }
            }
        }
        put(buf ^ 1);  // read last before the barrier that began this stage
        load(t0 + 2 * kTileT);
        __syncthreads();
    }
    store_tile<kDwBf16>(acc, to, n0 + wn, k0 + wk);
}

// ------------------------------------------------------------- wide tiles ---
//
// 256 x 256 of dw per block, four wavefronts of 128 x 128 each (256 of a
// SIMD's 512 registers per lane hold the sums), stages of 64 t, two of them
// in LDS.  Per stage and wavefront: 64 matrix instructions of 32 cycles; per
// CU 128 KB read from LDS and 64 KB written, 1536 of those 2048 cycles, so
// the tile cannot be smaller, and the LDS accesses have to run beside the
// matrix instructions.  A stage is therefore unrolled into four steps of 16
// t, and a step's code reads the operands of the next one, moves a share of
// the next stage from registers to LDS and asks memory for a share of the one
// after that, all between its own 16 matrix instructions.  The block meets
// once per stage, before the last step: by then every operand of the stage is
// in registers and the next stage is in LDS.  fp32 gradients have stages of 32
// t, whose three parts of dy and x take the same room: six steps, 96 matrix
// instructions for the same bytes, with the splitting beside them.
//
// Rows behind the last token come as zeros of both operands (the buffer
// resources end with the split's tokens); columns behind the matrix's own
// read what lies there and are not stored.  Where dy's rows are not whole
// 16-byte chunks (kAligned false: an odd width, stride or start) the last
// chunk of a row reaches into the next row, which is harmless except in the
// very last one: that token is left out of the stages and added to the sums
// at the end, and the rows behind it are cleared in registers (8192 x 4095 x
// 4096 bf16 240 us, fp32 630; this form spills 178 registers, the aligned one at
// most 6).

constexpr int kWideTile = 256;
constexpr int kWideRow = kWideTile * 2;  // bytes of a staged row
constexpr int kWideBf16 = 64, kWideF32 = 32;  // t per stage

__device__ __forceinline__ uint32_t wide_chunk_at(int t, int chunk)
{
    return static_cast<uint32_t>(t * kWideRow + ((chunk ^ ((t & 3) << 2)) << 4));
}

// A thread's share of a stage on its way from memory.
template <bool kDyBf16>
struct WideStage {
    static constexpr int kT = kDyBf16 ? kWideBf16 : kWideF32;
    static constexpr int kRows = kT / 8;            // units of eight of dy, eight rows apart
    static constexpr int kUnits = kT / 16;          // units of sixteen codes, sixteen rows apart
    u32x4 dy[8];                                    // kRows units, of one or two chunks
    u32x4 codes[kUnits];
    uint32_t scale[kUnits];
};

template <bool kDyBf16, bool kAligned, bool kDwBf16>
__global__ __launch_bounds__(kBlock, 1) void weight_grad_wide_kernel(Matrix dy, Codes x, int64_t tokens, int64_t n_all,
                                                                     int64_t k_all, int64_t per_split, uint32_t tiles_k,
                                                                     Target to)
{
    using Stage = WideStage<kDyBf16>;
    constexpr int kT = Stage::kT, kE = kDyBf16 ? 2 : 4, kParts = kDyBf16 ? 1 : 3;
    constexpr int kOperand = kT * kWideRow;            // bytes of a staged operand
    constexpr int kX = 2 * kParts * kOperand;          // dy's parts: two stages, then x: two stages
    __shared__ __attribute__((aligned(16))) char lds[kX + 2 * kOperand];
    const Tile tile = tile_of(blockIdx.x, gridDim.x, tiles_k);
    const int64_t n0 = tile.n * kWideTile;
    const int64_t k0 = tile.k * kWideTile;
    const int64_t padded = (k_all + kRun - 1) / kRun * kRun;
    const int64_t t_first = blockIdx.y * per_split;
    const int64_t t_last = min(t_first + per_split, kAligned ? tokens : tokens - 1);
    const int stages = static_cast<int>((t_last - t_first + kT - 1) / kT);
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int wn = wave / 2 * 128, wk = wave % 2 * 128;

    // Where this thread's share of a stage lies, in bytes from the stage's first row.
    const uint32_t dy_row = static_cast<uint32_t>(dy.stride) * kE, x_row = static_cast<uint32_t>(padded);
    const uint32_t dy_off = (tid / 32) * dy_row + (tid % 32) * 8u * kE;  // + 8 rows per unit
    const uint32_t x_off = (tid / 16) * x_row + (tid % 16) * 16u;       // + 16 rows per unit
    const uint32_t s_off = (tid / 16) * (x_row / 32) + (tid % 16) / 2;
    const char* dy_base = static_cast<const char*>(dy.data) + n0 * kE;
    const uint8_t* x_base = x.codes + k0;
    const uint8_t* s_base = x.scales + k0 / kRun;

    // The operands' bytes behind a stage's first row, `row` for each of its tokens and `less` fewer in the last one; the
    // stage behind the split's tokens, and those that follow, reach nothing.
    const int t_count = static_cast<int>(max(t_last - t_first, static_cast<int64_t>(0)));
    const int whole = t_count / kT, rest = t_count % kT;
    const uint32_t dy_less = static_cast<uint32_t>((dy.stride - n_all + n0) * kE), x_less = static_cast<uint32_t>(k0);
    auto reach = [&](int s, uint32_t row, uint32_t less) {
        const uint32_t last = rest ? rest * row - less : 0u;
        return s < whole ? kT * row - less : (s == whole ? last : 0u);
    };
    const char* dy_stage = dy_base + t_first * dy_row;
    const uint8_t* x_stage = x_base + t_first * x_row;
    const uint8_t* s_stage = s_base + t_first * (x_row / 32);
    auto load_dy = [&](Stage& w, int s, const char* at, int first, int count) __attribute__((always_inline)) {
        uint32_t bytes = 0;
        if (kAligned) {
            bytes = reach(s, dy_row, dy_less);
        } else {  // to the end of the matrix, which the last stages reach
            const int64_t left = (tokens - t_first - static_cast<int64_t>(s) * kT) * dy_row - dy_less;
            const uint32_t most = left < 0 ? 0u : static_cast<uint32_t>(min(left, static_cast<int64_t>(2 * kT) * dy_row));
            // Said to be uniform: each load would be a loop over the lanes' resources otherwise.
            bytes = __builtin_amdgcn_readfirstlane(most);
        }
        const __amdgpu_buffer_rsrc_t r = rsrc(at, bytes);
#pragma unroll
        for (int j = first; j < first + count; ++j) {
#pragma unroll
            for (int h = 0; h < kE / 2; ++h) w.dy[j * (kE / 2) + h] = load_u32x4<0>(r, dy_off + j * 8 * dy_row + h * 16);
        }
    };
    auto load_x = [&](Stage& w, int s, const uint8_t* at, const uint8_t* scales_at, int first, int count) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t r = rsrc(at, reach(s, x_row, x_less));
        const __amdgpu_buffer_rsrc_t rs = rsrc(scales_at, reach(s, x_row / 32, x_less / 32));
#pragma unroll
        for (int j = first; j < first + count; ++j) {
            w.codes[j] = load_u32x4<0>(r, x_off + j * 16 * x_row);
            w.scale[j] = __builtin_amdgcn_raw_buffer_load_b8(rs, s_off + j * 16 * (x_row / 32), 0, 0);
        }
    };
    const uint32_t dy_at = wide_chunk_at(tid / 32, tid % 32);              // + 8 rows: the same t & 3
    // A unit fills two chunks.  Eight lanes write at a time; the last four of them take their second chunk first, so
    // that the eight are spread over all banks (with every lane's first chunk first, each write took twice as long).
    const bool swap = tid & 4;
    const uint32_t x_at = kX + wide_chunk_at(tid / 16, tid % 16 * 2) + (swap ? 16 : 0);  // + 16 rows
    const uint32_t x_at2 = x_at ^ 16;
    auto put_dy = [&](const Stage& w, int s, int buf, int first, int count) __attribute__((always_inline)) {
#pragma unroll
        for (int j = first; j < first + count; ++j) {
            Raw8<kDyBf16> raw;
#pragma unroll
            for (int h = 0; h < kE / 2; ++h) {
                raw.v[h] = w.dy[j * (kE / 2) + h];
                if (!kAligned) {
                    const uint32_t keep = s * kT + tid / 32 + j * 8 < t_count ? ~0u : 0u;
                    raw.v[h] = raw.v[h] & u32x4{keep, keep, keep, keep};
                }
            }
            u32x4 part[3];
            if constexpr (kDyBf16) part[0] = raw.v[0];
            else split3(raw, part);
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                *reinterpret_cast<u32x4*>(lds + (buf * kParts + p) * kOperand + dy_at + j * 8 * kWideRow) = part[p];
            }
        }
    };
    auto put_x = [&](const Stage& w, int buf, int first, int count) __attribute__((always_inline)) {
#pragma unroll
        for (int j = first; j < first + count; ++j) {
            const float scale = __uint_as_float(w.scale[j] << 23);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x2 c = swap == (h == 0) ? u32x2{w.codes[j][2], w.codes[j][3]} : u32x2{w.codes[j][0], w.codes[j][1]};
                u32x4 v;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], scale, false));
                    v[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], scale, true));
                }
                *reinterpret_cast<u32x4*>(lds + buf * kOperand + (h == 0 ? x_at : x_at2) + j * 16 * kWideRow) = v;
            }
        }
    };
    // Operand addresses: column block i of 32 sits at chunk 4 i, whose exclusive-or with the row is the lane's own.
    uint32_t a_at[4], b_at[4];
    {
        const int l16 = lane % 16, t = lane / 32 * 8 + l16 / 4;
        const int low = lane % 32 / 16 * 2 + l16 % 4 / 2;  // chunk within the 32 columns
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t at = t * kWideRow + (((i ^ (t & 3)) * 4 + low) << 4) + l16 % 2 * 8;
            a_at[i] = at + wn * 2;
            b_at[i] = at + wk * 2 + kX;
        }
    }
    auto read4 = [&](bf16x8 (&v)[4], const uint32_t (&at)[4], int offset) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char* p = lds + at[i] + offset;
            const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                             (__attribute__((address_space(3))) s16x4*)p));
            const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                             (__attribute__((address_space(3))) s16x4*)(p + 4 * kWideRow)));
            v[i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };

    f32x16 acc[4][4] = {};
    bf16x8 a[2][4], b[2][4];
    Stage w;
    auto read_a = [&](int h, int buf, int step, int part) __attribute__((always_inline)) {
        read4(a[h], a_at, (buf * kParts + part) * kOperand + step * 16 * kWideRow);
    };
    auto read_b = [&](int h, int buf, int step) __attribute__((always_inline)) { read4(b[h], b_at, buf * kOperand + step * 16 * kWideRow); };
    auto multiply = [&](int ha, int hb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[ha][i], b[hb][j], acc[i][j], 0, 0, 0);
        }
    };
    const int64_t dy_step = static_cast<int64_t>(kT) * dy_row, x_step = static_cast<int64_t>(kT) * x_row;
    auto advance = [&]() __attribute__((always_inline)) { dy_stage += dy_step, x_stage += x_step, s_stage += x_step / 32; };
    load_dy(w, 0, dy_stage, 0, Stage::kRows);
    load_x(w, 0, x_stage, s_stage, 0, Stage::kUnits);
    put_dy(w, 0, 0, 0, Stage::kRows);
    put_x(w, 0, 0, Stage::kUnits);
    // From here on the pointers are, for bf16, at the stage behind the one in work, whose last two units of x are still to
    // come, and for fp32 at the one after that.
    advance();
    load_dy(w, 1, dy_stage, 0, Stage::kRows);
    load_x(w, 1, x_stage, s_stage, 0, 2);
    if (!kDyBf16) advance();
    __syncthreads();
    read_a(0, 0, 0, 0);
    read_b(0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    auto stage_bf16 = [&](int s, int buf) __attribute__((always_inline)) {
        read_a(1, buf, 1, 0);
        read_b(1, buf, 1);
        load_x(w, s + 1, x_stage, s_stage, 2, 2);
        multiply(0, 0);
        put_dy(w, s + 1, buf ^ 1, 0, 4);
        put_x(w, buf ^ 1, 0, 1);
        advance();
        order_step<16, 6, 4>();
        read_a(0, buf, 2, 0);
        read_b(0, buf, 2);
        load_dy(w, s + 2, dy_stage, 0, 4);
        load_x(w, s + 2, x_stage, s_stage, 0, 1);
        multiply(1, 1);
        put_dy(w, s + 1, buf ^ 1, 4, 4);
        put_x(w, buf ^ 1, 1, 1);
        order_step<16, 6, 6>();
        read_a(1, buf, 3, 0);
        read_b(1, buf, 3);
        load_dy(w, s + 2, dy_stage, 4, 4);
        load_x(w, s + 2, x_stage, s_stage, 1, 1);
        multiply(0, 0);
        put_x(w, buf ^ 1, 2, 2);
        order_step<16, 4, 6>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        read_a(0, buf ^ 1, 0, 0);
        read_b(0, buf ^ 1, 0);
        multiply(1, 1);
        order_step<16, 0, 0>();
    };
    // fp32: six steps, each part of dy for each of the two sixteens of t; what a step puts away, the next one asks for.
    auto stage_f32 = [&](int s, int buf) __attribute__((always_inline)) {
        read_a(1, buf, 0, 1);
        multiply(0, 0);
        put_dy(w, s + 1, buf ^ 1, 0, 1);
        order_step<8, 3, 0>();
        read_a(0, buf, 0, 2);
        load_dy(w, s + 2, dy_stage, 0, 1);
        multiply(1, 0);
        put_dy(w, s + 1, buf ^ 1, 1, 1);
        order_step<8, 3, 2>();
        read_a(1, buf, 1, 0);
        read_b(1, buf, 1);
        load_dy(w, s + 2, dy_stage, 1, 1);
        multiply(0, 0);
        put_x(w, buf ^ 1, 0, 2);
        order_step<16, 4, 2>();
        read_a(0, buf, 1, 1);
        load_x(w, s + 2, x_stage, s_stage, 0, 2);
        multiply(1, 1);
        put_dy(w, s + 1, buf ^ 1, 2, 1);
        order_step<8, 3, 4>();
        read_a(1, buf, 1, 2);
        load_dy(w, s + 2, dy_stage, 2, 1);
        multiply(0, 1);
        put_dy(w, s + 1, buf ^ 1, 3, 1);
        order_step<8, 3, 2>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        read_a(0, buf ^ 1, 0, 0);
        read_b(0, buf ^ 1, 0);
        load_dy(w, s + 2, dy_stage, 3, 1);
        multiply(1, 1);
        advance();
        order_step<16, 0, 2>();
    };
    auto stage = [&](int s, int buf) __attribute__((always_inline)) {
        if constexpr (kDyBf16) stage_bf16(s, buf);
        else stage_f32(s, buf);
    };
    // Two stages a round, so that the buffers' addresses are constants of the code (4 % faster).
    int s = 0;
    for (; s + 1 < stages; s += 2) {
        stage(s, 0);
        stage(s + 1, 1);
    }
    if (s < stages) stage(s, 0);
    if (!kAligned && t_first + per_split >= tokens) {
        const int64_t t = tokens - 1;
        float xv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t k = min(k0 + wk + j * kFrag + lane % 32, padded - 1);
            xv[j] = decode1<true>(x.codes[t * padded + k], scale_value(x.scales[t * (padded / kRun) + k / kRun]));
        }
        auto last = [&](int64_t n) {
            if (kDyBf16) return bf16_lo(static_cast<const uint16_t*>(dy.data)[t * dy.stride + n]);
            return static_cast<const float*>(dy.data)[t * dy.stride + n];
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float d = last(min(n0 + wn + i * kFrag + r / 4 * 8 + lane / 32 * 4 + r % 4, n_all - 1));
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j][r] = __builtin_fmaf(d, xv[j], acc[i][j][r]);
            }
        }
    }
    store_tile<kDwBf16>(acc, to, n0 + wn, k0 + wk);
}

// dw = [dw +] the splits' partial sums, in split order; four values a thread
// (partial sums are 16-byte aligned where count % 4 == 0, else one by one).
template <bool kDwBf16, int kWidth>
__global__ __launch_bounds__(kBlock) void weight_grad_join_kernel(const float* partials, int splits, int64_t count,
                                                                  void* dw, bool accumulate)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * kBlock * kWidth;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * kWidth; i < count; i += step) {
        float sum[kWidth] = {};
#pragma unroll 8
        for (int s = 0; s < splits; ++s) {
            const float* p = partials + s * count + i;
            if (kWidth == 4) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
                for (int j = 0; j < kWidth; ++j) sum[j] += v[j];
            } else {
                sum[0] += *p;
            }
        }
#pragma unroll
        for (int j = 0; j < kWidth; ++j) store_dw<kDwBf16>(dw, i + j, sum[j], accumulate);
    }
}

// A tile's edge, its stage, and two measured times of a stage of it (us): on a
// CU of its own, and per block where several share a CU.
struct TileKind {
    int edge, stage_t;
    double alone_us, shared_us;
};
constexpr TileKind kWide[2] = {{kWideTile, kWideF32, 2.3, 2.3}, {kWideTile, kWideBf16, 1.6, 1.6}};  // one block fills a CU
constexpr TileKind kMid[2] = {{128, kStageF32, 1.14, 0.84}, {128, kStageBf16, 1.0, 0.70}};  // [bf16]
constexpr TileKind kSmall[2] = {{64, kStageF32, 0.60, 0.30}, {64, kStageBf16, 0.54, 0.29}};

struct Plan {
    int edge = 0;  // of the tile
    int64_t tiles_n, tiles_k, per_split;
    int splits;
};

// Partial sums, at most: a workspace of 256 MB.  fp32 16384 x 14336 x 4096
// takes 4.81 ms for it and 4.43 split in two, with 470 MB.
constexpr double kMostPartials = 1 << 26;

// The tile and the count of splits of the tokens under which the work should
// take least: the busiest CU's stages, and with splits the partial sums' way
// to memory and back (4 TB/s) and their join.  With each choice forced (us):
// 8192 x 4096 x 4096 bf16 207 wide, 358 at 128, 585 at 64; 2048 x 4096 x 1024
// 40, 36, 40; 1000 x 1000 x 1000 19.7, 16.3 and 10.8; fp32 777 x 1000 x 2051 31
// at 128 and 25.6 at 64, 2048 x 4096 x 4096 157 wide and 223 at 128, 8192 x
// 4096 x 4096 594, 868 and 1222.
Plan plan_of(int64_t tokens, int64_t n, int64_t k, bool bf16, bool wide)
{
    Plan best;
    double least = 0.0;
    const double values = static_cast<double>(n) * static_cast<double>(k);
    for (const TileKind& kind : {kSmall[bf16], kMid[bf16], kWide[bf16]}) {
        if (kind.edge == kWideTile && !wide) continue;
        const int64_t tiles_n = (n + kind.edge - 1) / kind.edge, tiles_k = (k + kind.edge - 1) / kind.edge;
        const int64_t stages = (tokens + kind.stage_t - 1) / kind.stage_t;
        for (int64_t c = 1; c <= 32 && (c == 1 || (2 * c <= stages && static_cast<double>(c) * values <= kMostPartials)); ++c) {
            const int64_t each = (stages + c - 1) / c;
            const double on_cu = static_cast<double>((tiles_n * tiles_k * c + 255) / 256) * kind.shared_us;
            const double cost = static_cast<double>(each) * (on_cu > kind.alone_us ? on_cu : kind.alone_us) +
                                (c > 1 ? 3.0 + (2.0 * static_cast<double>(c) + 1.0) * values * 4.0 / 4.0e6 : 0.0);
            if (best.edge == 0 || cost < least) {
                least = cost;
                best.edge = kind.edge;
                best.tiles_n = tiles_n;
                best.tiles_k = tiles_k;
                best.per_split = each * kind.stage_t;
                best.splits = static_cast<int>(each > 0 ? (stages + each - 1) / each : 1);
            }
        }
    }
    return best;
}

// Whether dy's rows are whole 16-byte chunks.
bool chunk_rows(const Matrix& dy, bool bf16, int64_t n)
{
    const int64_t chunk = bf16 ? 8 : 4;
    return n % chunk == 0 && dy.stride % chunk == 0 && reinterpret_cast<uintptr_t>(dy.data) % 16 == 0;
}

// The wide tile takes rows that keep two stages' offsets below 2^32 bytes.
bool wide_fits(int64_t dy_stride, bool dy_bf16, int64_t n, int64_t k)
{
    return dy_stride < 1 << (dy_bf16 ? 23 : 22) && n >= 64 && k >= 64 && k <= 1 << 25;
}

size_t scratch_of(const Plan& s, int64_t n, int64_t k)
{
    return s.splits > 1 ? static_cast<size_t>(s.splits) * n * k * sizeof(float) : 0;
}

}  // namespace

// Whichever plan the gradient's type and stride will give.
size_t weight_grad_scratch(int64_t tokens, int64_t out_features, int64_t in_features)
{
    size_t most = 0;
    for (const bool bf16 : {false, true}) {
        for (const bool wide : {false, true}) {
            if (wide && !wide_fits(out_features, bf16, out_features, in_features)) continue;
            const size_t need = scratch_of(plan_of(tokens, out_features, in_features, bf16, wide), out_features, in_features);
            if (need > most) most = need;
        }
    }
    return most;
}

hipError_t launch_act8_weight_grad(Matrix dy, bool dy_bf16, Codes x, int64_t tokens, int64_t out_features,
                                   int64_t in_features, void* dw, bool dw_bf16, bool accumulate, void* scratch,
                                   hipStream_t stream)
{
    const Plan s = plan_of(tokens, out_features, in_features, dy_bf16, wide_fits(dy.stride, dy_bf16, out_features, in_features));
    float* partials = s.splits > 1 ? static_cast<float*>(scratch) : nullptr;
    const dim3 grid(static_cast<uint32_t>(s.tiles_n * s.tiles_k), s.splits);
    const uint32_t tk = static_cast<uint32_t>(s.tiles_k);
    auto run = [&](auto kernel) {
        kernel<<<grid, kBlock, 0, stream>>>(dy, x, tokens, out_features, in_features, s.per_split, tk,
                                            Target{dw, partials, accumulate, out_features, in_features});
    };
    if (s.edge == kWideTile) {
        auto wide = [&](auto bf16, auto aligned) {
            if (dw_bf16) run(weight_grad_wide_kernel<bf16.value, aligned.value, true>);
            else run(weight_grad_wide_kernel<bf16.value, aligned.value, false>);
        };
        const std::true_type yes;
        const std::false_type no;
        if (chunk_rows(dy, dy_bf16, out_features)) dy_bf16 ? wide(yes, yes) : wide(no, yes);
        else dy_bf16 ? wide(yes, no) : wide(no, no);
    } else if (s.edge == 128) {
        if (dy_bf16) {
            if (dw_bf16) run(weight_grad_kernel<true, true, 128>);
            else run(weight_grad_kernel<true, false, 128>);
        } else {
            if (dw_bf16) run(weight_grad_kernel<false, true, 128>);
            else run(weight_grad_kernel<false, false, 128>);
        }
    } else {
        if (dy_bf16) {
            if (dw_bf16) run(weight_grad_kernel<true, true, 64>);
            else run(weight_grad_kernel<true, false, 64>);
        } else {
            if (dw_bf16) run(weight_grad_kernel<false, true, 64>);
            else run(weight_grad_kernel<false, false, 64>);
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !partials) return e;
    const int64_t count = out_features * in_features;
    const int width = count % 4 == 0 ? 4 : 1;
    const int64_t blocks = (count + kBlock * width - 1) / (kBlock * width);
    const int join_grid = static_cast<int>(blocks < 1 << 20 ? blocks : 1 << 20);
    auto join = [&](auto kernel) { kernel<<<join_grid, kBlock, 0, stream>>>(partials, s.splits, count, dw, accumulate); };
    if (width == 4) {
        if (dw_bf16) join(weight_grad_join_kernel<true, 4>);
        else join(weight_grad_join_kernel<false, 4>);
    } else {
        if (dw_bf16) join(weight_grad_join_kernel<true, 1>);
        else join(weight_grad_join_kernel<false, 1>);
    }
    return hipGetLastError();
}

}  // namespace mps
