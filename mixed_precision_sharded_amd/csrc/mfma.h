// Device helpers of the products on the matrix cores (kernels_wgrad.hip,
// kernels_head.hip): operands staged in LDS as rows of the summed index, and
// the order of a step's instructions.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace mps {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFrag = 32;    // rows and columns of one matrix instruction

// Byte offset in a staged tile [t][kCols] of bf16 of the 16-byte chunk
// `chunk` of row t.  A transposing load reads 32 bytes from each of four
// consecutive rows per 16 lanes; the exclusive-or sends the four rows to
// different banks (rows of 64 columns lie two to the banks' 256 bytes).
template <int kCols>
__device__ __forceinline__ uint32_t chunk_at(int t, int chunk)
{
    const int mixed = kCols == 64 ? chunk ^ ((t & 2) << 1) : chunk ^ ((t & 3) << 2);
    return static_cast<uint32_t>(t * kCols * 2 + (mixed << 4));
}

// Four consecutive t of one column for each lane of a group of 16, whose lanes
// hold 16 consecutive columns.  p: the lane's own four columns of row lane / 4.
__device__ __forceinline__ bf16x4 load_transposed(const char* p)
{
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// The same in a staged tile: t0 .. t0 + 3, columns from col0 on.
template <int kCols>
__device__ __forceinline__ bf16x4 read_transposed(const char* tile, int t0, int col0, int lane16)
{
    const int t = t0 + lane16 / 4;
    const int col = col0 + lane16 % 4 * 4;
    return load_transposed(tile + chunk_at<kCols>(t, col / 8) + (col % 8) * 2);
}

// The operand of one matrix instruction: columns col0 .. col0 + 31 (lane %
// 32), t0 + 8 * (lane / 32) .. + 7.
template <int kCols>
__device__ __forceinline__ bf16x8 read_operand(const char* tile, int t0, int col0, int lane)
{
    const int t = t0 + lane / 32 * 8, c = col0 + lane % 32 / 16 * 16;
    const bf16x4 lo = read_transposed<kCols>(tile, t, c, lane % 16);
    const bf16x4 hi = read_transposed<kCols>(tile, t + 4, c, lane % 16);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The order of a step's sixteen matrix instructions: its LDS reads behind the
// first eight (where there are 12, one and two in turn) and a write behind each
// of the next, with a load from memory behind each of the first.  Asked for
// one by one, the compiler gathers them before or behind the matrix
// instructions, which then wait: a weight gradient of 8192 x 4096 x 4096 takes
// 267 instead of 220 us; one read behind each of the sixteen, with the writes
// last, took 238.
template <int kReads, int kWrites, int kLoads>
__device__ __forceinline__ void order_step()
{
    constexpr int kMfma = 0x008, kVmemRead = 0x020, kLdsRead = 0x100, kLdsWrite = 0x200;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        if (i < 8) {
            if constexpr (kReads == 16) __builtin_amdgcn_sched_group_barrier(kLdsRead, 2, 0);
            else if constexpr (kReads == 12) {
                if (i % 2) __builtin_amdgcn_sched_group_barrier(kLdsRead, 2, 0);
                else __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
            }
            else __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
        } else if (i - 8 < kWrites) {
            __builtin_amdgcn_sched_group_barrier(kLdsWrite, 1, 0);
        }
        if (i < kLoads) __builtin_amdgcn_sched_group_barrier(kVmemRead, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace
}  // namespace mps
