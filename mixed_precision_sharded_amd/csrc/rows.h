// Device helpers of the row-matrix operators (8-bit activations, weight
// gradients, the policy loss): eight consecutive elements of a row at a time,
// their 8-bit form, and reductions in fp32.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "device.h"
#include "fp8.h"

namespace mps {
namespace {

constexpr int kRun = 32;   // elements that share a scale byte (MPS_Q8_BLOCK)
constexpr int kUnit = 8;   // elements a lane takes at a time: four lanes hold a run

// Vectors at any element's address: a global access of 16 bytes needs no
// alignment on this chip, so rows of any start and stride take one path.
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight elements as they lie in memory.
template <bool kBf16>
struct Raw8 {
    u32x4 v[kBf16 ? 1 : 2];
};

// kStream: past the cache, for matrices that a kernel reads once (the norm's
// backward 4096 x 8192 53.2 -> 48.5 us; forward kernels, whose inputs another
// kernel has just written, lose up to 17 % by it at sizes that fit the cache).
template <bool kBf16, bool kStream = false>
__device__ __forceinline__ Raw8<kBf16> load_full(const void* base, int64_t at)
{
    Raw8<kBf16> r;
    if (kBf16) {
        const auto* p = reinterpret_cast<const u32x4_at2*>(static_cast<const uint16_t*>(base) + at);
        r.v[0] = kStream ? __builtin_nontemporal_load(p) : *p;
    } else {
        const auto* p = reinterpret_cast<const u32x4_at4*>(static_cast<const float*>(base) + at);
        r.v[0] = kStream ? __builtin_nontemporal_load(p) : p[0];
        r.v[kBf16 ? 0 : 1] = kStream ? __builtin_nontemporal_load(p + 1) : p[1];
    }
    return r;
}

// Elements at .. at + 7, of which the first n exist (zeros behind them).
template <bool kBf16, bool kStream = false>
__device__ __forceinline__ Raw8<kBf16> load8(const void* base, int64_t at, int64_t n)
{
    if (n >= kUnit) return load_full<kBf16, kStream>(base, at);
    Raw8<kBf16> r{};
    for (int i = 0; i < kUnit - 1; ++i) {
        if (i >= n) break;
        if (kBf16) {
            const uint32_t h = static_cast<const uint16_t*>(base)[at + i];
            const uint32_t word = (i & 1) ? h << 16 : h;
            if (i / 2 == 0) r.v[0][0] |= word;
            else if (i / 2 == 1) r.v[0][1] |= word;
            else if (i / 2 == 2) r.v[0][2] |= word;
            else r.v[0][3] |= word;
        } else {
            const uint32_t word = static_cast<const uint32_t*>(base)[at + i];
            constexpr int kHi = kBf16 ? 0 : 1;
            if (i == 0) r.v[0][0] = word;
            else if (i == 1) r.v[0][1] = word;
            else if (i == 2) r.v[0][2] = word;
            else if (i == 3) r.v[0][3] = word;
            else if (i == 4) r.v[kHi][0] = word;
            else if (i == 5) r.v[kHi][1] = word;
            else r.v[kHi][2] = word;
        }
    }
    return r;
}

template <bool kBf16>
__device__ __forceinline__ void widen(const Raw8<kBf16>& r, float (&x)[kUnit])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            x[2 * i] = bf16_lo(r.v[0][i]);
            x[2 * i + 1] = bf16_hi(r.v[0][i]);
        } else {
            x[i] = __uint_as_float(r.v[0][i]);
            x[4 + i] = __uint_as_float(r.v[kBf16 ? 0 : 1][i]);
        }
    }
}

// Round (bf16: to nearest, ties to even) and store the first n of eight.
// Whole vectors go out nontemporally: nothing of what these operators write is
// read again by the same kernel, and the lines they would push out of L2 are
// (RMSNorm 8192 x 4096 31.1 -> 26.7 us, SwiGLU backward 8192 x 14336 185 ->
// 175 us, 1024 x 14336 forward 21.2 -> 19.0 us).
template <bool kBf16>
__device__ __forceinline__ void store8(const float (&x)[kUnit], void* base, int64_t at, int64_t n)
{
    if (n >= kUnit) {
        if (kBf16) {
            u32x4_at2 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = bf16_pack2(x[2 * i], x[2 * i + 1]);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4_at2*>(static_cast<uint16_t*>(base) + at));
        } else {
            auto* p = reinterpret_cast<u32x4_at4*>(static_cast<float*>(base) + at);
            const u32x4_at4 lo = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
            const u32x4_at4 hi = {__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])};
            __builtin_nontemporal_store(lo, p);
            __builtin_nontemporal_store(hi, p + 1);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kUnit - 1; ++i) {
        if (i >= n) break;
        if (kBf16) static_cast<uint16_t*>(base)[at + i] = bf16_one(x[i]);
        else static_cast<float*>(base)[at + i] = x[i];
    }
}

// ------------------------------------------------------- the 8-bit form ---

// Largest over the four lanes of a quad (the lanes that hold one run).
__device__ __forceinline__ uint32_t quad_max(uint32_t x)
{
    constexpr int kQuadSwap1 = 0xb1;  // quad_perm [1,0,3,2]
    constexpr int kQuadSwap2 = 0x4e;  // quad_perm [2,3,0,1]
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), kQuadSwap1, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), kQuadSwap2, 0xf, 0xf, false)));
    return x;
}

// store8 of a unit of a row, by the quads of lanes that hold its runs (they
// come here together).  An fp32 unit is two stores of 16 bytes; of a whole run
// the lanes first exchange, so that each of its two stores is 64 bytes in one
// piece and not every other 16 of 128 (fp32 8192 x 8192 kept and read back 158
// -> 133 us, RMSNorm 119 -> 105, SwiGLU backward 4096 x 8192 96.8 -> 91.2; not
// so RMSNorm of rows of 20000, 41.9 -> 43.4, which takes store8).
template <bool kBf16>
__device__ __forceinline__ void store_unit(const float (&x)[kUnit], void* base, int64_t at, int64_t n)
{
    const int q = threadIdx.x % 4;
    if (kBf16 || n + q * kUnit < kRun) return store8<kBf16>(x, base, at, n);
    constexpr int kLower = 0x50, kUpper = 0xfa;  // quad_perm [0,0,1,1] and [2,2,3,3]
    u32x4_at4 first, second;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int lo = __float_as_int(x[i]), hi = __float_as_int(x[4 + i]);
        const int a = __builtin_amdgcn_update_dpp(0, lo, kLower, 0xf, 0xf, false);
        const int b = __builtin_amdgcn_update_dpp(0, hi, kLower, 0xf, 0xf, false);
        const int c = __builtin_amdgcn_update_dpp(0, lo, kUpper, 0xf, 0xf, false);
        const int d = __builtin_amdgcn_update_dpp(0, hi, kUpper, 0xf, 0xf, false);
        first[i] = static_cast<uint32_t>(q & 1 ? b : a);
        second[i] = static_cast<uint32_t>(q & 1 ? d : c);
    }
    auto* p = reinterpret_cast<u32x4_at4*>(static_cast<float*>(base) + at - q * (kUnit / 2));
    __builtin_nontemporal_store(first, p);
    __builtin_nontemporal_store(second, p + 4);
}

// Encode this lane's eight elements, the quad's lanes holding one run, and
// store them as unit `unit` of the matrix (eight codes; the quad's first
// lane writes the scale byte).  The four lanes come here together.
// kStream: codes past the cache, for kernels that write other matrices too
// (with the stores above, SwiGLU backward 8192 x 14336 175 -> 174, forward 163
// -> 158 us; a matrix that is kept and read back at once is 4 % faster without).
template <bool kStream>
__device__ __forceinline__ void store_codes(const float (&x)[kUnit], uint8_t* codes, uint8_t* scales,
                                            int64_t unit)
{
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) most = max(most, abs_bits(x[i]));
    const uint32_t byte = scale_byte<kE4M3TopExp>(quad_max(most));
    const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
    const u32x2 word = {encode4<true>(lo, byte), encode4<true>(hi, byte)};
    if (kStream) __builtin_nontemporal_store(word, reinterpret_cast<u32x2*>(codes) + unit);
    else reinterpret_cast<u32x2*>(codes)[unit] = word;
    if (unit % 4 == 0) scales[unit / 4] = static_cast<uint8_t>(byte);
}

// Eight codes to the values they stand for: the conversion takes 2^(b - 127)
// as an fp32 scale whose exponent field is b, 0 and 255 (NaN) included.
__device__ __forceinline__ void decode8(u32x2 c, uint32_t byte, float (&x)[kUnit])
{
    const float scale = __uint_as_float(byte << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[i], scale, false);
        const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[i], scale, true);
        x[4 * i] = lo[0];
        x[4 * i + 1] = lo[1];
        x[4 * i + 2] = hi[0];
        x[4 * i + 3] = hi[1];
    }
}

__device__ __forceinline__ void load_codes(const uint8_t* codes, const uint8_t* scales, int64_t unit,
                                           float (&x)[kUnit])
{
    decode8(reinterpret_cast<const u32x2*>(codes)[unit], scales[unit / 4], x);
}

// ---------------------------------------------------- the walk over rows ---

// The units of a matrix, `per_row` to a row, in order from this thread's first
// on, a grid of kBlock threads apart (below 2^31): one division at the start,
// none behind it.
struct RowWalk {
    int64_t row;
    uint32_t col, d_row, d_col, per_row;

    __device__ __forceinline__ explicit RowWalk(uint32_t units_per_row) : per_row(units_per_row)
    {
        const uint32_t first = blockIdx.x * kBlock + threadIdx.x, step = gridDim.x * kBlock;
        const uint32_t r = first / units_per_row;
        row = r;
        col = first - r * units_per_row;
        d_row = step / units_per_row;
        d_col = step - d_row * units_per_row;
    }

    __device__ __forceinline__ void next()
    {
        row += d_row;
        col += d_col;
        if (col >= per_row) {
            col -= per_row;
            ++row;
        }
    }

    __device__ __forceinline__ int64_t unit() const { return row * per_row + col; }
};

// ------------------------------------------------------ reductions (fp32) ---

template <int kCtrl>
__device__ __forceinline__ float dpp_movef(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kCtrl, 0xf, 0xf, false));
}

// Sum over the wavefront, the same bits in every lane; all lanes active.
__device__ __forceinline__ float wave_sumf(float x)
{
    x += dpp_movef<0xb1>(x);
    x += dpp_movef<0x4e>(x);
    x += dpp_movef<0x141>(x);
    x += dpp_movef<0x140>(x);
    x += __shfl_xor(x, 16, kWave);
    x += __shfl_xor(x, 32, kWave);
    return x;
}

}  // namespace
}  // namespace mps
