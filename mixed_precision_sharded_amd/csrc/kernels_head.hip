// gfx950 kernels of a linear head under a cross entropy whose logits
//     x[t, v] = sum over k of h[t, k] w[v, k]
// are never kept: loss = sum over t of c_t (lse_t - x[t, label_t]) and, with
// g[t, v] = c_t (e^(x[t, v] - lse_t) - onehot),
//     dh[t, k] = sum over v of g[t, v] w[v, k],   dw[v, k] = sum over t of g[t, v] h[t, k].
//
// The rows that take part are packed first, in the order of their labels, so
// that the others cost nothing and what lies in them reaches nothing.  A first
// product leaves, for every row and stretch of 128 logits, the largest and the
// sum of the exponentials under it; joined, they give lse.  Then piece by piece
// of the vocabulary the same product is made again, its tiles turned into g in
// a workspace, and g goes into the two gradients' products.  The last piece of
// the first pass leaves its exponentials in that workspace, so that its logits
// are made once (8192 x 128256 x 4096, where that is half of them: 22.1 ms; 25.3
// with none).
// What a bf16 g loses at the label, where it is largest, is added again: to
// dh with the label's row of w, to dw as a few more stages of the product of
// the tile that holds the label (rows of neighbouring labels lie together).
// With it the gradients of 24 x 128256 x 4096 are 0.0017 of their norm off,
// the rounding of the result alone; without it 0.0026.
// All products of more than 64 tokens (the logits: of more than 64 tiles) are one
// kernel over tiles of 256 x 256 on the matrix cores: bf16 operands, fp32 sums.
// fp32 operands are split into three bf16 parts each, and six products of parts
// are summed.
//
// Large products are bound by the power that the matrix cores may draw: 8192 x
// 128256 x 4096 runs them at 1300 TF/s, about 70 % of the cycles at 1.65 GHz, where
// the library's best kernel for the logits has 83 % of them at 1.4 GHz and the
// same time; other orders of a stage's instructions, or its loads a stage
// earlier, change nothing.  Few tokens are bound by the readings of w and the
// writing of dw: 24 x 128256 x 4096 591 us for 3.15 GB.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "mfma.h"
#include "model_kernels.h"
#include "parts.h"
#include "rows.h"

namespace mps {
namespace {

constexpr int kTile = 256;       // of m and of n
constexpr int kStage = 64;       // of k
constexpr int kOperand = kTile * kStage * 2;  // bytes of a staged operand
constexpr int kB = 2 * kOperand;              // A: two stages, then B: two stages
constexpr int kGroup = 8;        // tiles of n in a patch of neighbouring ones

constexpr double kLog2eWide = 1.44269504088896340736;
constexpr float kLog2e = static_cast<float>(kLog2eWide);
constexpr float kLog2eLow = static_cast<float>(kLog2eWide - static_cast<double>(kLog2e));

// e^(x - top) and its logarithm to base 2, log2(e) in two parts (the error of
// one has the same sign in all of a row's terms).
__device__ __forceinline__ float log2_below(float x, float top)
{
    const float d = x - top;
    return __builtin_fmaf(d, kLog2e, d * kLog2eLow);
}
__device__ __forceinline__ float exp_below(float x, float top) { return __builtin_amdgcn_exp2f(log2_below(x, top)); }

// ------------------------------------------------------------ the product ---

// What the products are for: statistics and g have m = vocabulary, n = tokens;
// dh has m = tokens, n = features; dw has m = vocabulary, n = features.
// kKept leaves the logits beside their statistics, kExp their exponentials.
enum class Kind { kStats, kKept, kExp, kGrad, kHidden, kWeight };

// D[m, n] = sum over k of A[m, k] B[n, k].  An operand is `parts` matrices,
// `plane` bytes apart, whose rows are `stride` bytes apart: rows of m (or n)
// along k, or, where k is the slow index, rows of k along m (or n).
struct Side {
    const char* data;
    int64_t plane;
    uint32_t stride;
};
struct Product {
    Side a, b;
    int64_t m, n, k;     // the one that counts tokens is their most
    const int32_t* live; // how many tokens there are
    int32_t parts;       // 1 or 3
    int32_t splits;      // of k
};

struct Target {
    // kStats
    float2* stats;           // [stretch of the vocabulary][row]
    float* label_logit;
    // kGrad
    const float* top;
    const float* factor;
    const float* slope;
    // and kWeight
    const int32_t* labels;   // of the packed rows
    int64_t first;           // vocabulary entry of m = 0
    int64_t rows;            // packed rows, padded: the statistics' row length
    // kWeight
    const int32_t* tile_rows;  // the first row whose label is in a tile of the vocabulary or behind it
    const float* lost;       // what a bf16 g at the row's label lacks
    // kGrad, kHidden, kWeight; kStats: where the logits are kept (fp32), or NULL
    void* out;
    int64_t out_stride, out_plane;  // elements
    bool accumulate, bf16;
};

// The three bf16 parts of eight fp32 values: each the nearest to what is left,
// and together all of their 24 bits.  The first is held to the largest finite
// bf16 number; an infinity or a NaN shows in the second.
__device__ __forceinline__ void split(const float (&x)[kUnit], u32x4 (&part)[3])
{
    constexpr float kMost = 0x1.fep127f;
#pragma unroll
    for (int i = 0; i < kUnit; i += 2) {
        float left[2] = {x[i], x[i + 1]};
        part[0][i / 2] = bf16_pack2(__builtin_amdgcn_fmed3f(left[0], -kMost, kMost), __builtin_amdgcn_fmed3f(left[1], -kMost, kMost));
#pragma unroll
        for (int p = 1; p < 3; ++p) {
            left[0] -= bf16_lo(part[p - 1][i / 2]);
            left[1] -= bf16_hi(part[p - 1][i / 2]);
            part[p][i / 2] = bf16_pack2(left[0], left[1]);
        }
    }
}

// One operand's staged tile.  Rows along k ("fast"): 256 rows of 64 k, 128
// bytes each; sixteen lanes read one 16-byte chunk from each of sixteen rows,
// and the exclusive-or with half the row spreads them over all banks.  Rows
// of k ("slow"): 64 rows of 256 columns, read with the transposing load, four
// consecutive rows of 32 bytes at a time, sent to different banks.
template <bool kSlow>
struct Staged {
    static constexpr int kReads = kSlow ? 8 : 4;   // LDS reads of a step
    uint32_t offset, row_step, put_at, read_at[4];
    const char* at;

    __device__ __forceinline__ void init(const Side& s, int64_t first, int tid, int wave_first, int lds_at)
    {
        const int lane = tid % kWave;
        if (kSlow) {
            const int t = tid / 32, chunk = tid % 32;
            offset = t * s.stride + chunk * 16;
            row_step = 8 * s.stride;
            put_at = lds_at + t * 512 + ((chunk ^ ((t & 3) << 2)) << 4);
            const int l16 = lane % 16, rt = lane / 32 * 8 + l16 / 4;
            const int low = lane % 32 / 16 * 2 + l16 % 4 / 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                read_at[i] = lds_at + rt * 512 + (((i ^ (rt & 3)) * 4 + low) << 4) + l16 % 2 * 8 + wave_first * 2;
            }
            at = s.data + first * 2;
        } else {
            const int row = tid / 8, chunk = tid % 8;
            offset = row * s.stride + chunk * 16;
            row_step = 32 * s.stride;
            put_at = lds_at + row * 128 + ((chunk ^ ((row >> 1) & 7)) << 4);
            const int rr = wave_first + lane % 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) read_at[i] = lds_at + rr * 128 + (((i * 2 + lane / 32) ^ ((rr >> 1) & 7)) << 4);
            at = s.data + first * s.stride;
        }
    }

    template <int kFirst, int kCount>
    __device__ __forceinline__ void load(u32x4 (&v)[8], const char* stage, uint32_t bytes) const
    {
        const __amdgpu_buffer_rsrc_t r = rsrc(stage, bytes);
#pragma unroll
        for (int j = kFirst; j < kFirst + kCount; ++j) v[j] = load_u32x4<0>(r, offset + j * row_step);
    }

    template <int kFirst, int kCount>
    __device__ __forceinline__ void put(const u32x4 (&v)[8], char* lds, int buf) const
    {
#pragma unroll
        for (int j = kFirst; j < kFirst + kCount; ++j) *reinterpret_cast<u32x4*>(lds + put_at + buf * kOperand + j * 4096) = v[j];
    }

    // The four operands of 32 rows, 16 k from 16 * step on.
    __device__ __forceinline__ void read(bf16x8 (&v)[4], const char* lds, int buf, int step) const
    {
        if (kSlow) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char* p = lds + read_at[i] + buf * kOperand + step * 16 * 512;
                const bf16x4 lo = load_transposed(p), hi = load_transposed(p + 4 * 512);
                v[i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = *reinterpret_cast<const bf16x8*>(lds + read_at[step] + buf * kOperand + i * kFrag * 128);
            }
        }
    }
};

template <Kind kKind, int kParts>
__device__ void finish_tile(const f32x16 (&acc)[4][4], char* lds, const Product& p, const Target& to, int64_t m0, int64_t n0,
                            int64_t live, int64_t m_tile, uint32_t split);

// One tile of one split, by one thread block.
template <Kind kKind, int kParts>
__device__ __forceinline__ void product(Product p, const Target& to, char* lds, uint32_t block)
{
    constexpr bool kASlow = kKind == Kind::kWeight;
    constexpr bool kBSlow = kKind == Kind::kWeight || kKind == Kind::kHidden;
    const int64_t live = __builtin_amdgcn_readfirstlane(*p.live);
    if (kKind != Kind::kHidden && kKind != Kind::kWeight) p.n = live;
    if (kKind == Kind::kHidden) p.m = live;
    if (kKind == Kind::kWeight) p.k = live;

    // The tile: the device hands consecutive blocks to its eight XCDs in
    // turn, and each XCD (and its L2) gets a stretch of tiles of which 32
    // neighbours form a patch of kGroup tiles of n by four of m (8192 x 128256
    // x 4096 22.0 ms with groups of 8, 22.2 with 4, 22.4 with 6, 22.5 with 16);
    // the tiles of one split lie together, since they share all they read.
    const uint32_t tiles_m = static_cast<uint32_t>((p.m + kTile - 1) / kTile), tiles_n = static_cast<uint32_t>((p.n + kTile - 1) / kTile);
    const uint32_t tiles = tiles_m * tiles_n, in_all = kKind == Kind::kHidden ? tiles * p.splits : tiles;
    const uint32_t each = in_all / 8, more = in_all % 8, xcd = block % 8;
    if (block / 8 >= each + (xcd < more ? 1 : 0)) return;
    const uint32_t of_all = xcd * each + min(xcd, more) + block / 8;
    const uint32_t split = kKind == Kind::kHidden ? __builtin_amdgcn_readfirstlane(of_all / tiles) : 0, t = of_all - split * tiles;
    const uint32_t group = t / (kGroup * tiles_m), in_group = t - group * kGroup * tiles_m;
    const uint32_t width = min(static_cast<uint32_t>(kGroup), tiles_n - group * kGroup);
    const int64_t m_tile = in_group / width;
    const int64_t m0 = m_tile * kTile;
    const int64_t n0 = static_cast<int64_t>(group * kGroup + in_group % width) * kTile;

    const int tid = threadIdx.x, wave = tid / kWave;
    Staged<kASlow> a;
    Staged<kBSlow> b;
    a.init(p.a, m0, tid, wave / 2 * 128, 0);
    b.init(p.b, n0, tid, wave % 2 * 128, kB);

    // This block's stages: those of its split, for every pair of parts.
    const int all = static_cast<int>((p.k + kStage - 1) / kStage);
    const int per = kKind == Kind::kHidden ? (all + p.splits - 1) / p.splits : all;
    const int s_first = min(static_cast<int>(split) * per, all), per_pair = min(per, all - s_first);
    constexpr int pair_first = kParts == 1 ? kPairs - 1 : 0;
    const int stages = (kPairs - pair_first) * per_pair;
    const int64_t a_step = kASlow ? static_cast<int64_t>(kStage) * p.a.stride : kStage * 2;
    const int64_t b_step = kBSlow ? static_cast<int64_t>(kStage) * p.b.stride : kStage * 2;
    const char* a_first = a.at + s_first * a_step;
    const char* b_first = b.at + s_first * b_step;
    const int64_t k_left = p.k - static_cast<int64_t>(s_first) * kStage;
    // Bytes that a stage reaches from its first one on.  What lies behind reads as zeros: rows of m and n that are not
    // stored, and rows of k that are none.
    const uint32_t a_fast = static_cast<uint32_t>(min(p.m - m0, static_cast<int64_t>(kTile)) - 1) * p.a.stride + kStage * 2;
    const uint32_t b_fast = static_cast<uint32_t>(min(p.n - n0, static_cast<int64_t>(kTile)) - 1) * p.b.stride + kStage * 2;
    // Columns in whole chunks (rows of k are padded to them): a word that ends behind the last byte would read as zero.
    const uint32_t a_cols = (static_cast<uint32_t>(min(p.m - m0, static_cast<int64_t>(kTile))) + 7) / 8 * 16;
    const uint32_t b_cols = (static_cast<uint32_t>(min(p.n - n0, static_cast<int64_t>(kTile))) + 7) / 8 * 16;
    auto slow_bytes = [&](int kk, uint32_t stride, uint32_t cols) {
        const int64_t rows = min(k_left - static_cast<int64_t>(kk) * kStage, static_cast<int64_t>(kStage));
        return static_cast<uint32_t>(rows - 1) * stride + cols;
    };

    // The stage that is being asked for.
    const char* a_at = a_first + part_a(pair_first) * p.a.plane;
    const char* b_at = b_first + part_b(pair_first) * p.b.plane;
    uint32_t a_bytes = 0, b_bytes = 0;
    int kk = 0, pair = pair_first;
    auto reach = [&]() __attribute__((always_inline)) {
        const bool there = pair < kPairs && per_pair > 0;
        a_bytes = there ? (kASlow ? slow_bytes(kk, p.a.stride, a_cols) : a_fast) : 0;
        b_bytes = there ? (kBSlow ? slow_bytes(kk, p.b.stride, b_cols) : b_fast) : 0;
        a_bytes = __builtin_amdgcn_readfirstlane(a_bytes);
        b_bytes = __builtin_amdgcn_readfirstlane(b_bytes);
    };
    auto advance = [&]() __attribute__((always_inline)) {
        a_at += a_step;
        b_at += b_step;
        if (++kk >= per_pair) {
            kk = 0;
            ++pair;
            a_at = a_first + part_a(pair) * p.a.plane;
            b_at = b_first + part_b(pair) * p.b.plane;
        }
        reach();
    };

    f32x16 acc[4][4] = {};
    bf16x8 av[2][4], bv[2][4];
    u32x4 ra[8], rb[8];
    auto multiply = [&](int h) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av[h][i], bv[h][j], acc[i][j], 0, 0, 0);
        }
    };
    if constexpr (kKind == Kind::kWeight && kParts == 1) {
        // What g lost at the labels among this tile's entries: one value a row of k.
        const int tile = static_cast<int>((to.first + m0) / kTile);
        const int k_begin = __builtin_amdgcn_readfirstlane(to.tile_rows[tile]);
        const int k_end = __builtin_amdgcn_readfirstlane(to.tile_rows[tile + 1]);
        for (int k0 = k_begin / kStage * kStage; k0 < k_end; k0 += kStage) {
            b.template load<0, 8>(rb, b.at + k0 / kStage * b_step, slow_bytes(k0 / kStage, p.b.stride, b_cols));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = k0 + tid / 32 + j * 8;
                const bool some = row >= k_begin && row < k_end;
                const int at = some ? static_cast<int>(to.labels[row] - to.first - m0) : -1;
                const uint32_t bits = some ? bf16_one(to.lost[row]) : 0;
                const uint32_t word = at % 2 ? bits << 16 : bits;
#pragma unroll
                for (int i = 0; i < 4; ++i) ra[j][i] = at / 2 == tid % 32 * 4 + i && some ? word : 0;
            }
            a.template put<0, 8>(ra, lds, 0);
            b.template put<0, 8>(rb, lds, 0);
            __syncthreads();
#pragma unroll 1
            for (int step = 0; step < 4; ++step) {
                a.read(av[0], lds, 0, step);
                b.read(bv[0], lds, 0, step);
                multiply(0);
            }
            __syncthreads();
        }
    }
    reach();
    a.template load<0, 8>(ra, a_at, a_bytes);
    b.template load<0, 8>(rb, b_at, b_bytes);
    a.template put<0, 8>(ra, lds, 0);
    b.template put<0, 8>(rb, lds, 0);
    advance();
    a.template load<0, 8>(ra, a_at, a_bytes);
    b.template load<0, 8>(rb, b_at, b_bytes);
    advance();
    __syncthreads();
    a.read(av[0], lds, 0, 0);
    b.read(bv[0], lds, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    // A stage: four steps of 16 matrix instructions of 32 cycles, 2500 cycles in all.  A step reads the operands of the next
    // one; the first three put the next stage, which is in registers, into LDS, and ask for the one after it into the
    // registers that they freed.
    constexpr int kReads = Staged<kASlow>::kReads + Staged<kBSlow>::kReads;
    auto stage = [&](int buf) __attribute__((always_inline)) {
        a.read(av[1], lds, buf, 1);
        b.read(bv[1], lds, buf, 1);
        multiply(0);
        a.template put<0, 6>(ra, lds, buf ^ 1);
        order_step<kReads, 6, 0>();
        a.read(av[0], lds, buf, 2);
        b.read(bv[0], lds, buf, 2);
        a.template load<0, 6>(ra, a_at, a_bytes);
        multiply(1);
        a.template put<6, 2>(ra, lds, buf ^ 1);
        b.template put<0, 4>(rb, lds, buf ^ 1);
        order_step<kReads, 6, 6>();
        a.read(av[1], lds, buf, 3);
        b.read(bv[1], lds, buf, 3);
        a.template load<6, 2>(ra, a_at, a_bytes);
        b.template load<0, 4>(rb, b_at, b_bytes);
        multiply(0);
        b.template put<4, 4>(rb, lds, buf ^ 1);
        order_step<kReads, 4, 6>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        a.read(av[0], lds, buf ^ 1, 0);
        b.read(bv[0], lds, buf ^ 1, 0);
        b.template load<4, 4>(rb, b_at, b_bytes);
        multiply(1);
        advance();
        order_step<kReads, 0, 4>();
    };
    // Two stages a round, so that the buffers' addresses are constants of the code.
    int s = 0;
    for (; s + 1 < stages; s += 2) {
        stage(0);
        stage(1);
    }
    if (s < stages) stage(0);
    finish_tile<kKind, kParts>(acc, lds, p, to, m0, n0, live, m_tile, split);
}

template <Kind kKind, int kParts>
__global__ __launch_bounds__(kBlock, 1) void product_kernel(Product p, Target to)
{
    __shared__ __attribute__((aligned(16))) char lds[4 * kOperand];
    product<kKind, kParts>(p, to, lds, blockIdx.x);
}

// The loss: the rows' in a fixed order, by one block.
__device__ __forceinline__ void sum_loss(const double* rows, const int32_t* live, float* loss, double* lds)
{
    const int64_t n = live ? *live : 0;
    double sum = 0.0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < n; i += kBlock) sum += rows[i];
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) *loss = static_cast<float>(sum);
}

// Both gradients in one launch: dh's few long tiles (`hidden_blocks`), then dw's many short ones, which fill the device to
// the end; a last block has the loss, where it is asked for.
template <int kParts>
__global__ __launch_bounds__(kBlock, 1) void gradients_kernel(Product dh, Target dh_to, uint32_t hidden_blocks, Product dw, Target dw_to,
                                                              const double* row_loss, float* loss)
{
    __shared__ __attribute__((aligned(16))) char lds[4 * kOperand];
    if (loss && blockIdx.x + 1 == gridDim.x) {
        sum_loss(row_loss, dh.live, loss, reinterpret_cast<double*>(lds));
    } else if (blockIdx.x < hidden_blocks) {
        product<Kind::kHidden, kParts>(dh, dh_to, lds, blockIdx.x);
    } else {
        product<Kind::kWeight, kParts>(dw, dw_to, lds, blockIdx.x - hidden_blocks);
    }
}

// Lane l of a result holds column n = l % 32 and the rows m = 8 (r / 4) + 4 (l / 32) + r % 4.
__device__ __forceinline__ int row_of(int r, int lane) { return r / 4 * 8 + lane / 32 * 4 + r % 4; }

// Sixteen values that lie in a row of results; the values of the others stay where they are (all of them read at once
// do not fit beside the sums).
struct Sixteen {
    float x[16];
    __device__ __forceinline__ Sixteen(const f32x16& v)
    {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = v[r];
    }
};

// For each token of the tile: the largest of this wavefront's 128 logits, the
// sum of e^(x - largest), and its label's logit where it is among them.
// kLogits: also leaves the logits, rows of tokens, for a later pass; rows that are none are stored outside the buffer, which
// drops them without a branch.  kExp: puts e^(x - largest) in 16 bits into LDS as tile_row_at says: minus its logarithm to
// base 2 in steps of 1 / kLogSteps.  So every one of them down to 2^-64 of the largest is kept to 2^-11 ln 2 = 3.4e-4 of
// itself (fp16 keeps the large ones to 4.9e-4, and of what is beside a label with nearly all of its row it loses bits below
// 2^-14 and everything below 2^-25); smaller ones, the largest code, are zeros.
enum class Keep { kNone, kLogits, kExp };

// Where four entries from `entry` on, of a tile's row t, lie in LDS: rows of 256 entries of 16 bits, whose 16-byte chunks
// are spread by the row's number.
__device__ __forceinline__ uint32_t tile_row_at(int t, int entry) { return t * 512 + ((entry / 8 ^ (t & 31)) << 4) + entry % 8 * 2; }

// And from there to memory, 512 bytes of a row at a time.
__device__ __forceinline__ void store_tile_rows(const char* lds, const Target& to, int64_t m0, int64_t n0)
{
    const int tid = threadIdx.x;
    char* out = static_cast<char*>(to.out) + (n0 * to.out_stride + m0) * 2;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
        const int t = tid / 32 + j * 8, chunk = tid % 32;
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + t * 512 + ((chunk ^ (t & 31)) << 4));
        *reinterpret_cast<u32x4*>(out + static_cast<int64_t>(t) * to.out_stride * 2 + chunk * 16) = v;
    }
}

constexpr float kLogSteps = 1024.0f;
constexpr uint32_t kLogMost = 65535;  // of what the logarithms are held to

// Two logarithms, at most 0, as codes: to the nearest step, both ends held (a NaN gives 0, but then its row's sum is one).
__device__ __forceinline__ uint32_t log_pack2(float a, float b)
{
    constexpr float kUnits = -kLogSteps / static_cast<float>(kLogMost);
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_u16(a * kUnits, b * kUnits));
}

// The power of two that a code stands for, under 2^top.
__device__ __forceinline__ float log_value(uint32_t code, float top)
{
    return code == kLogMost ? 0.0f : __builtin_amdgcn_exp2f(__builtin_fmaf(static_cast<float>(code), -1.0f / kLogSteps, top));
}

template <bool kEdge, Keep kKeep, int kI, int kJ>
__device__ __forceinline__ void stats_of(const f32x16 (&acc)[kI][kJ], const Target& to, int there, int64_t mw, int64_t row0, int64_t live,
                                         float2* stats, char* lds = nullptr)
{
    const int lane = threadIdx.x % kWave;
    const uint32_t row_bytes = kKeep == Keep::kLogits ? static_cast<uint32_t>(to.out_stride) * 4 : 0;
    const __amdgpu_buffer_rsrc_t logits = rsrc(uniform_ptr(static_cast<float*>(to.out) + row0 * to.out_stride + mw), 128 * row_bytes);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int64_t row = row0 + j * kFrag + lane % 32;
        const uint32_t offset = row < live ? (j * kFrag + lane % 32) * row_bytes + lane / 32 * 16 : 0x80000000u;
        const int64_t label = row < live ? to.labels[row] - to.first - mw : -1;
        const bool here = label >= 0 && label < there;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const Sixteen v(acc[i][j]);
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, !kEdge || i * kFrag + row_of(r, lane) < there ? v.x[r] : -INFINITY);
        }
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        const float under = top == -INFINITY ? 0.0f : top;
        float part[4] = {};
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const Sixteen v(acc[i][j]);
            float log[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                log[r] = log2_below(!kEdge || i * kFrag + row_of(r, lane) < there ? v.x[r] : -INFINITY, under);
                part[r % 4] += __builtin_amdgcn_exp2f(log[r]);
            }
            if (kKeep == Keep::kExp) {
                const int wave = threadIdx.x / kWave, t = wave % 2 * 128 + j * kFrag + lane % 32;
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const u32x2 w = {log_pack2(log[r], log[r + 1]), log_pack2(log[r + 2], log[r + 3])};
                    *reinterpret_cast<u32x2*>(lds + tile_row_at(t, wave / 2 * 128 + i * kFrag + row_of(r, lane))) = w;
                }
            }
            if (kKeep == Keep::kLogits) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4 w = {v.x[4 * q], v.x[4 * q + 1], v.x[4 * q + 2], v.x[4 * q + 3]};
                    asm volatile("" : "+v"(w));  // in registers of its own, not where the sums are: those would be spilled
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), logits, offset + i * kFrag * 4 + q * 32, 0, 0);
                }
            }
            if (__any(here && label / kFrag == i)) {
                float x = 0.0f;
                bool mine = false;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const bool hit = here && label == i * kFrag + row_of(r, lane);
                    x = hit ? v.x[r] : x;
                    mine = mine || hit;
                }
                if (mine) to.label_logit[row] = x;
            }
        }
        float sum = (part[0] + part[1]) + (part[2] + part[3]);
        sum += __shfl_xor(sum, 32, kWave);
        if (lane < 32 && row < live) stats[row] = float2{top, sum};
    }
}

// g at a logit.  For bf16 with the first part of log2(e) alone: 1.3e-8 of the value for each that the logit lies below the
// largest, 1.2e-6 at the most, where bf16 keeps 3.9e-3.
template <int kParts>
__device__ __forceinline__ float grad_at(float x, float top, float factor)
{
    return factor * (kParts == 1 ? __builtin_amdgcn_exp2f((x - top) * kLog2e) : exp_below(x, top));
}

// g of the tile, through LDS (rows of 256 entries, whose 16-byte chunks are
// spread by the row's number) to rows of 512 bytes in memory.  Entries and
// rows that are none are zeros.
template <bool kEdge>
__device__ __forceinline__ void grad_tile(const f32x16 (&acc)[4][4], char* lds, const Target& to, int there, int64_t m0, int64_t n0,
                                          int64_t live)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int wm = wave / 2 * 128, wn = wave % 2 * 128;
    __syncthreads();  // the stages have been read
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int t = wn + j * kFrag + lane % 32;
        const int64_t row = n0 + t;
        const bool some = row < live;
        const float top = some ? to.top[row] : 0.0f, factor = some ? to.factor[row] : 0.0f, slope = some ? to.slope[row] : 0.0f;
        const int64_t label = some ? to.labels[row] - to.first - m0 - wm : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Sixteen v(acc[i][j]);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                v.x[r] = grad_at<1>(v.x[r], top, factor);
                if (kEdge) v.x[r] = some && i * kFrag + row_of(r, lane) < there ? v.x[r] : 0.0f;
            }
            if (__any(label >= 0 && label < there && label / kFrag == i)) {
#pragma unroll
                for (int r = 0; r < 16; ++r) v.x[r] -= label == i * kFrag + row_of(r, lane) && label < there ? slope : 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const u32x2 w = {bf16_pack2(v.x[r], v.x[r + 1]), bf16_pack2(v.x[r + 2], v.x[r + 3])};
                *reinterpret_cast<u32x2*>(lds + tile_row_at(t, wm + i * kFrag + row_of(r, lane))) = w;
            }
        }
    }
    __syncthreads();
    store_tile_rows(lds, to, m0, n0);
}

// Rows of values, added to what is there where `kAccumulate`: 32 of those are asked for at once (one by one, each waits for
// the one before).
template <bool kBf16, bool kAccumulate, bool kEdge>
__device__ __forceinline__ void values_of(const f32x16 (&acc)[4][4], const Product& p, const Target& to, int64_t m0, int64_t n0,
                                          uint32_t split)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    uint16_t* const out16 = static_cast<uint16_t*>(to.out) + split * to.out_plane;
    float* const out32 = static_cast<float*>(to.out) + split * to.out_plane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m_first = m0 + wave / 2 * 128 + i * kFrag, n_first = n0 + wave % 2 * 128 + lane % 32;
#pragma unroll
        for (int half = 0; half < 16; half += 8) {
            float old[8][4];
            if (kAccumulate) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int64_t m = m_first + row_of(half + r, lane), row = (kEdge ? min(m, p.m - 1) : m) * to.out_stride;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t n = n_first + j * kFrag, at = row + (kEdge ? min(n, p.n - 1) : n);
                        old[r][j] = kBf16 ? bf16_lo(out16[at]) : out32[at];
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int64_t m = m_first + row_of(half + r, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t n = n_first + j * kFrag, at = m * to.out_stride + n;
                    if (kEdge && !(m < p.m && n < p.n)) continue;
                    const float v = kAccumulate ? old[r][j] + acc[i][j][half + r] : acc[i][j][half + r];
                    if (kBf16) out16[at] = bf16_one(v);
                    else out32[at] = v;
                }
            }
        }
    }
}

template <bool kBf16>
__device__ __forceinline__ void finish_values(const f32x16 (&acc)[4][4], const Product& p, const Target& to, int64_t m0, int64_t n0,
                                              uint32_t split)
{
    const bool edge = m0 + kTile > p.m || n0 + kTile > p.n;
    if (to.accumulate) {
        if (edge) values_of<kBf16, true, true>(acc, p, to, m0, n0, split);
        else values_of<kBf16, true, false>(acc, p, to, m0, n0, split);
    } else {
        if (edge) values_of<kBf16, false, true>(acc, p, to, m0, n0, split);
        else values_of<kBf16, false, false>(acc, p, to, m0, n0, split);
    }
}

template <Kind kKind, int kParts>
__device__ __forceinline__ void finish_tile(const f32x16 (&acc)[4][4], char* lds, const Product& p, const Target& to, int64_t m0,
                                            int64_t n0, int64_t live, int64_t m_tile, uint32_t split)
{
    const int wave = threadIdx.x / kWave;
    const int64_t mw = m0 + wave / 2 * 128;
    const int there = static_cast<int>(min(p.m - mw, static_cast<int64_t>(128)));  // of a wavefront's 128 entries; may be <= 0
    if constexpr (kKind == Kind::kStats || kKind == Kind::kKept || kKind == Kind::kExp) {
        float2* stats = to.stats + (m_tile * 2 + wave / 2) * to.rows;
        const int64_t row0 = n0 + wave % 2 * 128;
        constexpr Keep kKeep = kKind == Kind::kKept ? Keep::kLogits : (kKind == Kind::kExp ? Keep::kExp : Keep::kNone);
        if (kKeep == Keep::kExp) __syncthreads();  // the stages have been read
        if (there < 128) stats_of<true, kKeep>(acc, to, there, mw, row0, live, stats, lds);
        else stats_of<false, kKeep>(acc, to, there, mw, row0, live, stats, lds);
        if (kKeep == Keep::kExp) {
            __syncthreads();
            store_tile_rows(lds, to, m0, n0);
        }
    } else if constexpr (kKind == Kind::kGrad) {
        if (m0 + kTile > p.m || n0 + kTile > live) grad_tile<true>(acc, lds, to, there, m0, n0, live);
        else grad_tile<false>(acc, lds, to, there, m0, n0, live);
    } else if (kKind == Kind::kHidden || !to.bf16) {
        finish_values<false>(acc, p, to, m0, n0, split);
    } else {
        finish_values<true>(acc, p, to, m0, n0, split);
    }
}

// ------------------------------------------------------------ few tokens ---

// Up to here the products have kernels of their own: 24 x 128256 x 4096 591 us, 1066 by the tiles of 256 x 256; with 100
// tokens the statistics took 250 us by kernels for 128 and take 210-230 by those tiles.
constexpr int kFewTokens = 64;

// The tile of 64 entries of a block of few_stats_kernel: the last blocks have the entries that dh's splits begin with, which
// are still in the last-level cache then (24 x 128256 x 4096 614 -> 596 us).
__device__ __forceinline__ uint32_t few_tile(const Product& p)
{
    const uint32_t tiles = static_cast<uint32_t>((p.m + 63) / 64), per = (tiles + p.splits - 1) / p.splits;
    return blockIdx.x % p.splits * per + (per - 1 - blockIdx.x / p.splits);
}

// The target of the packed rows from `row` on.
__device__ __forceinline__ Target from_row(Target to, int64_t row)
{
    to.stats += row;
    to.label_logit += row;
    to.labels += row;
    if (to.out) to.out = static_cast<float*>(to.out) + row * to.out_stride;
    return to;
}

// The end of few_stats_kernel: wavefronts wm and wm + 1 have 32 entries' logits, each from half of every stage's k.
template <int kJ>
__device__ __forceinline__ void finish_few(f32x16 (&acc)[1][kJ], char* lds, int64_t m, int64_t m0, const Target& to, int64_t live)
{
    const int tid = threadIdx.x, lane = tid % kWave, wm = tid / kWave / 2, wk = tid / kWave % 2;
    f32x4* half = reinterpret_cast<f32x4*>(lds) + wm * kJ * 4 * kWave;
    if (wk == 1) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                half[(j * 4 + q) * kWave + lane] = f32x4{acc[0][j][4 * q], acc[0][j][4 * q + 1], acc[0][j][4 * q + 2], acc[0][j][4 * q + 3]};
            }
        }
    }
    __syncthreads();
    float2* const joined = reinterpret_cast<float2*>(lds + 2 * kJ * 4 * kWave * 16);
    if (wk == 0) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 v = half[(j * 4 + q) * kWave + lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][j][4 * q + i] += v[i];
            }
        }
        const int64_t mw = m0 + wm * 32;
        const int there = static_cast<int>(min(m - mw, static_cast<int64_t>(32)));  // may be <= 0
        float2* mine = joined + wm * kJ * 32;
        if (to.out) {
            if (there < 32) stats_of<true, Keep::kLogits>(acc, to, there, mw, 0, live, mine);
            else stats_of<false, Keep::kLogits>(acc, to, there, mw, 0, live, mine);
        } else {
            if (there < 32) stats_of<true, Keep::kNone>(acc, to, there, mw, 0, live, mine);
            else stats_of<false, Keep::kNone>(acc, to, there, mw, 0, live, mine);
        }
    }
    __syncthreads();
    if (tid < kJ * 32 && tid < live) {
        const float2 v = joined[tid], w = joined[kJ * 32 + tid];
        const float top = fmaxf(v.x, w.x), under = top == -INFINITY ? 0.0f : top;
        to.stats[m0 / 64 * to.rows + tid] = float2{top, v.y * exp_below(v.x, under) + w.y * exp_below(w.x, under)};
    }
}

// kStats and kKept for 32 * kJ tokens (blockIdx.y: which): 64 entries of the
// vocabulary a block, in stages of 128 k (256 bytes of a row of w at a time), two of them in
// LDS and one on its way in registers; two wavefronts have 32 entries each and
// half of a stage's k.  Bound by the one reading of w, of which several blocks a
// CU have 16 KB each under way; the 256-wide tile would spend up to eight times
// the matrix instructions.
// kAny: w is read as it lies, whatever its rows' start and length (log-probabilities of 24 x 128256 x 4001 607 -> 228 us,
// the loss 1552 -> 919, against packing it first; buffer loads of whole stages are a little faster where they can be, 4096
// features 201 us and not 211).
template <int kJ, bool kAny>
__global__ __launch_bounds__(kBlock, 2) void few_stats_kernel(Product p, Matrix w, int64_t cols, Target to)
{
    constexpr int kA = 64 * 256, kBuf = kA + kJ * 32 * 256;
    __shared__ __attribute__((aligned(16))) char lds[2 * kBuf];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int64_t m0 = static_cast<int64_t>(few_tile(p)) * 64, row0 = blockIdx.y * (32 * kJ), live = __builtin_amdgcn_readfirstlane(*p.live) - row0;
    if (live <= 0 || m0 >= p.m) return;
    to = from_row(to, row0);
    const int stages = static_cast<int>((p.k + 127) / 128);

    const int row = tid / 16, chunk = tid % 16;
    const uint32_t a_off = row * p.a.stride + chunk * 16, b_off = row * p.b.stride + chunk * 16;
    const uint32_t put_at = row * 256 + ((chunk ^ row) << 4);  // + 16 rows: 4096
    const uint32_t a_bytes = static_cast<uint32_t>(min(p.m - m0, static_cast<int64_t>(64)) - 1) * p.a.stride + 256;
    const uint32_t b_bytes = (32 * kJ - 1) * p.b.stride + 256;
    // Where the last stage has 64 k, its upper half is asked for outside the buffer.
    const int half_stage = p.k % 128 ? stages - 1 : -1;
    const char *a_at = p.a.data + m0 * p.a.stride, *b_at = p.b.data + row0 * p.b.stride;
    int kk = 0;
    u32x4 ra[4], rb[2 * kJ];
    auto load = [&]() __attribute__((always_inline)) {  // nothing behind the last stage
        const uint32_t less = kk == half_stage ? 128 : 0, out = less && chunk >= 8 ? 0x80000000u : 0;
        const __amdgpu_buffer_rsrc_t br = rsrc(uniform_ptr(b_at), kk < stages ? b_bytes - less : 0);
        if constexpr (kAny) {
            const int64_t k = static_cast<int64_t>(kk) * 128 + chunk * kUnit;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + row + j * 16;
                ra[j] = load8<true>(w.data, m * w.stride + k, m < p.m ? cols - k : 0).v[0];
            }
        } else {
            const __amdgpu_buffer_rsrc_t ar = rsrc(uniform_ptr(a_at), kk < stages ? a_bytes - less : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) ra[j] = load_u32x4<0>(ar, a_off + j * 16 * p.a.stride + out);
        }
#pragma unroll
        for (int j = 0; j < 2 * kJ; ++j) rb[j] = load_u32x4<0>(br, b_off + j * 16 * p.b.stride + out);
        a_at += 256;
        b_at += 256;
        ++kk;
    };
    auto put = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4*>(lds + buf * kBuf + put_at + j * 4096) = ra[j];
#pragma unroll
        for (int j = 0; j < 2 * kJ; ++j) *reinterpret_cast<u32x4*>(lds + buf * kBuf + kA + put_at + j * 4096) = rb[j];
    };
    const int wm = wave / 2, wk = wave % 2;
    f32x16 sums[4][kJ] = {};  // a step's each: shorter sums are more exact (40 x 32000 x 4096: log-probabilities 1.1e-7 off, not 3.3e-7)
    load();
    put(0);
    load();
    __syncthreads();
    for (int s = 0; s < stages; ++s) {
        const char* buf = lds + (s & 1) * kBuf;
#pragma unroll
        for (int step = 0; step < 4; ++step) {
            const uint32_t at = lane % 32 * 256 + (((wk * 8 + step * 2 + lane / 32) ^ (lane % 16)) << 4);
            const bf16x8 a = *reinterpret_cast<const bf16x8*>(buf + wm * 8192 + at);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const bf16x8 b = *reinterpret_cast<const bf16x8*>(buf + kA + j * 8192 + at);
                sums[step][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, sums[step][j], 0, 0, 0);
            }
        }
        put((s + 1) & 1);  // read last before the barrier that began this stage
        load();
        __syncthreads();
    }
    f32x16 acc[1][kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) acc[0][j] = (sums[0][j] + sums[1][j]) + (sums[2][j] + sums[3][j]);
    finish_few<kJ>(acc, lds, p.m, m0, to, live);
}

// The same for fp32: stages of 64 k of w, split into their parts on their way into LDS, so that w is read once and as it lies
// (packed first and read part by part, 2 x 181889 x 1971 took 1480 us).
template <int kJ>
__global__ __launch_bounds__(kBlock, 2) void few_stats_f32_kernel(Product p, Matrix w, int64_t cols, Target to)
{
    constexpr int kA = 64 * 128, kB32 = 32 * kJ * 128;  // of one part
    __shared__ __attribute__((aligned(16))) char lds[3 * (kA + kB32)];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int64_t m0 = static_cast<int64_t>(few_tile(p)) * 64, row0 = blockIdx.y * (32 * kJ), live = __builtin_amdgcn_readfirstlane(*p.live) - row0;
    if (live <= 0 || m0 >= p.m) return;
    to = from_row(to, row0);
    Raw8<false> ra[2];
    u32x4 rb[3][kJ];
    auto load = [&](int64_t k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t m = m0 + tid / 8 + i * 32, k = k0 + tid % 8 * kUnit;
            ra[i] = load8<false>(w.data, m * w.stride + k, m < p.m ? cols - k : 0);
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const char* at = p.b.data + part * p.b.plane + (row0 + tid / 8 + j * 32) * p.b.stride + k0 * 2 + tid % 8 * 16;
                rb[part][j] = k0 < p.k ? *reinterpret_cast<const u32x4*>(at) : u32x4{0, 0, 0, 0};
            }
        }
    };
    const uint32_t put_at = tid / 8 * 128 + ((tid % 8 ^ (tid / 16 & 7)) << 4);  // + 32 rows: 4096
    const int wm = wave / 2, wk = wave % 2;
    f32x16 acc[1][kJ] = {};
    load(0);
    for (int64_t k0 = 0; k0 < p.k; k0 += kStage) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x[kUnit];
            widen<false>(ra[i], x);
            u32x4 part[3];
            split(x, part);
#pragma unroll
            for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x4*>(lds + q * kA + put_at + i * 4096) = part[q];
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) *reinterpret_cast<u32x4*>(lds + 3 * kA + part * kB32 + put_at + j * 4096) = rb[part][j];
        }
        __syncthreads();
        load(k0 + kStage);
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            const uint32_t at = lane % 32 * 128 + (((wk * 4 + step * 2 + lane / 32) ^ (lane % 32 >> 1 & 7)) << 4);
            bf16x8 a[3], b[3][kJ];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                a[q] = *reinterpret_cast<const bf16x8*>(lds + q * kA + wm * 4096 + at);
#pragma unroll
                for (int j = 0; j < kJ; ++j) b[q][j] = *reinterpret_cast<const bf16x8*>(lds + 3 * kA + q * kB32 + j * 4096 + at);
            }
#pragma unroll
            for (int pair = 0; pair < kPairs; ++pair) {
#pragma unroll
                for (int j = 0; j < kJ; ++j) acc[0][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[part_a(pair)], b[part_b(pair)][j], acc[0][j], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    finish_few<kJ>(acc, lds, p.m, m0, to, live);
}

// kWeight for at most kT tokens: one or two steps of the matrix instruction a
// tile, so that the tile's way to memory is all there is.  A block has 256
// features (fp32: 128), whose operands stay in registers, and takes one tile of
// 64 entries after the other, the next one's g on its way; rows of 512 bytes go
// out through LDS.  Several blocks a CU.
template <int kParts, int kT, bool kBf16, bool kAccumulate>
__global__ __launch_bounds__(kBlock, kT == 32 && !kAccumulate ? (kParts == 1 ? (kBf16 ? 4 : 2) : 3) : 2) void few_weight_kernel(Product p, Target to, uint32_t per_block)
{
    constexpr int kCols = kParts == 1 ? 256 : 128, kJ = kCols / 128, kSteps = kT / 16;
    constexpr int kG = kT * 128, kH = kT * kCols * 2, kUnits = kT * 8 / kBlock;  // 16-byte units of g a thread
    constexpr int kElem = kBf16 ? 2 : 4, kOut = 64 * kCols * kElem;
    constexpr int kGs = kParts == 1 ? 2 : 3;  // g's parts, or g and what it lost
    constexpr int kFirst = kParts == 1 ? kPairs - 1 : 0;
    __shared__ __attribute__((aligned(16))) char lds[kGs * kG + (kParts * kH > kOut ? kParts * kH : kOut)];
    char* const rest = lds + kGs * kG;  // the hidden states, then the results
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int live = __builtin_amdgcn_readfirstlane(*p.live);
    const uint32_t across = static_cast<uint32_t>((p.n + kCols - 1) / kCols);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x % across) * kCols;
    const int64_t m_first = static_cast<int64_t>(blockIdx.x / across) * per_block * 64;
    const int64_t m_last = min(m_first + static_cast<int64_t>(per_block) * 64, p.m);

    // Rows behind the last one are zeros; columns behind the last one are padding of the workspace, or zeros.
    const u32x4 none = {0, 0, 0, 0};
    u32x4 g[kParts][kUnits];
    int64_t label[kUnits];  // of the unit's first entry
    uint32_t lost[kUnits];
    const int64_t of_lane = lane < live ? to.labels[lane] - to.first : -1;
    auto load = [&](int64_t m0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int t = tid / 8 + i * 32, chunk = tid % 8;
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                const char* from = p.a.data + part * p.a.plane + t * static_cast<int64_t>(p.a.stride) + m0 * 2 + chunk * 16;
                g[part][i] = t < live && m0 < m_last ? *reinterpret_cast<const u32x4*>(from) : none;
            }
        }
    };
    load(m_first);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int t = tid / 8 + i * 32;
        label[i] = kParts == 1 && t < live ? to.labels[t] - to.first - tid % 8 * 8 : -1;
        lost[i] = kParts == 1 && t < live ? bf16_one(to.lost[t]) : 0;
    }
    for (int u = tid; u < kT * (kCols / 8); u += kBlock) {
        const int t = u / (kCols / 8), chunk = u % (kCols / 8);
        const int64_t c = n0 + chunk * 8;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            const char* from = p.b.data + part * p.b.plane + t * static_cast<int64_t>(p.b.stride) + c * 2;
            *reinterpret_cast<u32x4*>(rest + part * kH + chunk_at<kCols>(t, chunk)) = t < live && c < p.n ? *reinterpret_cast<const u32x4*>(from) : none;
        }
    }
    __syncthreads();
    bf16x8 b[kParts][kSteps][kJ];
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) b[part][step][j] = read_operand<kCols>(rest + part * kH, step * 16, wave * (kCols / 4) + j * kFrag, lane);
        }
    }
#pragma unroll 1
    for (int64_t m0 = m_first; m0 < m_last; m0 += 64) {
        const bool lost_too = kParts == 1 && __any(of_lane >= m0 && of_lane < m0 + 64);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const uint32_t at = chunk_at<64>(tid / 8 + i * 32, tid % 8);
#pragma unroll
            for (int part = 0; part < kParts; ++part) *reinterpret_cast<u32x4*>(lds + part * kG + at) = g[part][i];
            if (lost_too) {
                const int64_t l = label[i] - m0;
                const bool here = label[i] >= 0 && l >= 0 && l < 8;
                const uint32_t word = l % 2 ? lost[i] << 16 : lost[i];
                u32x4 v = none;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = here && l / 2 == k ? word : 0;
                *reinterpret_cast<u32x4*>(lds + kG + at) = v;
            }
        }
        __syncthreads();  // also: the results of the tile before have been read
        load(m0 + 64);
        f32x16 acc[2][kJ] = {};
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
#pragma unroll
            for (int pair = kFirst; pair < kPairs; ++pair) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 a = read_operand<64>(lds + part_a(pair) * kG, step * 16, i * kFrag, lane);
#pragma unroll
                    for (int j = 0; j < kJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[part_b(pair)][step][j], acc[i][j], 0, 0, 0);
                }
            }
            if (lost_too) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 a = read_operand<64>(lds + kG, step * 16, i * kFrag, lane);
#pragma unroll
                    for (int j = 0; j < kJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[0][step][j], acc[i][j], 0, 0, 0);
                }
            }
        }
        const int col = wave * (kCols / 4) + lane % 32;
        if constexpr (kAccumulate) {  // 32 rows at a time, in fp32, to what is there, rounded after the sum
            constexpr int kRowUnits = kCols / kUnit, kMine = 32 * kRowUnits / kBlock;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                Raw8<kBf16> old[kMine];
                int64_t at[kMine], there[kMine];
#pragma unroll
                for (int k = 0; k < kMine; ++k) {
                    const int u = k * kBlock + tid, c = u % kRowUnits * kUnit;
                    const int64_t m = m0 + i * kFrag + u / kRowUnits;
                    at[k] = m * to.out_stride + n0 + c;
                    there[k] = m < p.m ? p.n - n0 - c : 0;
                    old[k] = load8<kBf16>(to.out, at[k], there[k]);
                }
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) reinterpret_cast<float*>(rest)[row_of(r, lane) * kCols + col + j * kFrag] = acc[i][j][r];
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kMine; ++k) {
                    const f32x4* v = reinterpret_cast<const f32x4*>(rest + (k * kBlock + tid) * kUnit * 4);
                    const f32x4 lo = v[0], hi = v[1];
                    float x[kUnit];
                    widen<kBf16>(old[k], x);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x[q] += lo[q];
                        x[4 + q] += hi[q];
                    }
                    store8<kBf16>(x, to.out, at[k], there[k]);
                }
                __syncthreads();
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int at = (i * kFrag + row_of(r, lane)) * kCols + col + j * kFrag;
                    if (kBf16) reinterpret_cast<uint16_t*>(rest)[at] = bf16_one(acc[i][j][r]);
                    else reinterpret_cast<float*>(rest)[at] = acc[i][j][r];
                }
            }
        }
        __syncthreads();
        // A thread has the same 16 bytes of every kDown-th row.
        constexpr int kEach = 16 / kElem, kRowUnits = kCols / kEach, kDown = kBlock / kRowUnits;
        const int row = tid / kRowUnits, c = tid % kRowUnits * kEach;
        const int left = static_cast<int>(min(p.n - n0 - c, static_cast<int64_t>(kEach)));
        const int rows = static_cast<int>(min(p.m - m0, static_cast<int64_t>(64)));
        char* out = static_cast<char*>(to.out) + ((m0 + row) * to.out_stride + n0 + c) * kElem;
        const int64_t step = to.out_stride * kDown * kElem;
        const char* from = rest + tid * 16;
        if (left == kEach) {
#pragma unroll
            for (int i = 0; i < 64 / kDown; ++i) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(from + i * kBlock * 16);
                if (row + i * kDown < rows) __builtin_nontemporal_store(u32x4_at2{v[0], v[1], v[2], v[3]}, reinterpret_cast<u32x4_at2*>(out));
                out += step;
            }
        } else if (left > 0) {
#pragma unroll 1
            for (int i = 0; i < 64 / kDown && row + i * kDown < rows; ++i) {
#pragma unroll 1
                for (int k = 0; k < left; ++k) {
                    if (kBf16) reinterpret_cast<uint16_t*>(out)[k] = reinterpret_cast<const uint16_t*>(from + i * kBlock * 16)[k];
                    else reinterpret_cast<float*>(out)[k] = reinterpret_cast<const float*>(from + i * kBlock * 16)[k];
                }
                out += step;
            }
        }
    }
}

// A unit of the weight's as its bf16 parts.
template <int kParts>
__device__ __forceinline__ void parts_of(const Raw8<kParts == 1>& raw, u32x4 (&part)[kParts])
{
    if constexpr (kParts == 1) {
        part[0] = raw.v[0];
    } else {
        float x[kUnit];
        widen<false>(raw, x);
        split(x, part);
    }
}

// kHidden for at most 32 * kJ tokens and any weight: 128 features a block, stages of 64 entries of the vocabulary, whose rows
// of w are split into their parts on their way into LDS.  A block has a share of the entries.
template <int kParts, int kJ>
__global__ __launch_bounds__(kBlock, 2) void few_hidden_any_kernel(Product p, Matrix w, int64_t cols, Target to)
{
    constexpr int kA = 32 * kJ * 128, kW = 64 * 256;  // of one part
    constexpr int kFirst = kParts == 1 ? kPairs - 1 : 0;
    __shared__ __attribute__((aligned(16))) char lds[kParts * (kA + kW)];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int live = __builtin_amdgcn_readfirstlane(*p.live);
    if (live == 0) return;
    const uint32_t across = static_cast<uint32_t>((cols + 127) / 128);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x % across) * 128;
    const int split_of = static_cast<int>(blockIdx.x / across);
    const int64_t all = (p.k + kStage - 1) / kStage, per = (all + p.splits - 1) / p.splits;
    const int64_t v_first = min(split_of * per, all) * kStage, v_last = min(v_first + per * kStage, p.k);
    Raw8<kParts == 1> rw[4];
    u32x4 ra[kParts][kJ];
    auto load = [&](int64_t v0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t v = v0 + tid / 16 + i * 16, c = n0 + tid % 16 * kUnit;
            rw[i] = load8<kParts == 1>(w.data, v * w.stride + c, v < v_last ? cols - c : 0);
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int t = tid / 8 + j * 32;
                const char* at = p.a.data + part * p.a.plane + t * static_cast<int64_t>(p.a.stride) + v0 * 2 + tid % 8 * 16;
                ra[part][j] = t < live && v0 < v_last ? *reinterpret_cast<const u32x4*>(at) : u32x4{0, 0, 0, 0};
            }
        }
    };
    const uint32_t put_at = tid / 8 * 128 + ((tid % 8 ^ (tid / 16 & 7)) << 4);  // + 32 rows: 4096
    f32x16 acc[kJ] = {};
    load(v_first);
    for (int64_t v0 = v_first; v0 < v_last; v0 += kStage) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 part[kParts];
            parts_of<kParts>(rw[i], part);
#pragma unroll
            for (int q = 0; q < kParts; ++q) *reinterpret_cast<u32x4*>(lds + kParts * kA + q * kW + chunk_at<128>(tid / 16 + i * 16, tid % 16)) = part[q];
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) *reinterpret_cast<u32x4*>(lds + part * kA + put_at + j * 4096) = ra[part][j];
        }
        __syncthreads();
        load(v0 + kStage);
#pragma unroll
        for (int step = 0; step < 4; ++step) {
            const uint32_t at = lane % 32 * 128 + (((step * 2 + lane / 32) ^ (lane % 32 >> 1 & 7)) << 4);
            bf16x8 a[kParts][kJ], b[kParts];
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                b[q] = read_operand<128>(lds + kParts * kA + q * kW, step * 16, wave * 32, lane);
#pragma unroll
                for (int j = 0; j < kJ; ++j) a[q][j] = *reinterpret_cast<const bf16x8*>(lds + q * kA + j * 4096 + at);
            }
#pragma unroll
            for (int pair = kFirst; pair < kPairs; ++pair) {
#pragma unroll
                for (int j = 0; j < kJ; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[part_a(pair)][j], b[part_b(pair)], acc[j], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    const int64_t n = n0 + wave * 32 + lane % 32;
    if (n >= cols) return;
    float* out = static_cast<float*>(to.out) + split_of * to.out_plane + n;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        float old[16] = {};
        if (to.accumulate) {
#pragma unroll
            for (int r = 0; r < 16; ++r) old[r] = out[min(j * kFrag + row_of(r, lane), live - 1) * to.out_stride];
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int t = j * kFrag + row_of(r, lane);
            if (t < live) out[t * to.out_stride] = old[r] + acc[j][r];
        }
    }
}

// ------------------------------------------------------- rows, packed ---

// Per row of the tokens that take part, in the order of their labels.
struct RowSpace {
    int32_t* live;         // how many
    int32_t* slot;         // token -> packed row, or -1
    int32_t* token;        // packed row -> token
    int32_t* label;        // of the packed row
    int32_t* tile_rows;    // the first row whose label is in a tile of the vocabulary or behind it
    float* label_logit;
    float* top;            // largest logit so far
    double* sum;           // of e^(x - top), so far
    float* factor;         // c / sum
    float* slope;          // c
    float* lost;           // what a bf16 g at the label lacks
    double* loss;
};

// A unit of a row as bf16 parts, padded with zeros to whole stages.
template <bool kBf16>
__device__ __forceinline__ void pack_unit(const Matrix& x, int64_t from, bool there, int64_t cols, const RowWalk& w, char* out, int64_t plane)
{
    const int64_t c = static_cast<int64_t>(w.col) * kUnit;
    const Raw8<kBf16> raw = load8<kBf16>(x.data, from * x.stride + c, there ? cols - c : 0);
    u32x4* to = reinterpret_cast<u32x4*>(out + w.unit() * 16);
    if constexpr (kBf16) {
        *to = raw.v[0];
    } else {
        float v[kUnit];
        widen<kBf16>(raw, v);
        u32x4 part[3];
        split(v, part);
#pragma unroll
        for (int p = 0; p < 3; ++p) to[p * (plane / 16)] = part[p];
    }
}

// A piece of the weight.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void pack_kernel(Matrix x, int64_t rows, int64_t cols, uint32_t per_row, char* out, int64_t plane)
{
    for (RowWalk w(per_row); w.row < rows; w.next()) pack_unit<kBf16>(x, w.row, true, cols, w, out, plane);
}

// The rows that take part, from the sorted tokens, and their hidden states; zeros behind the last one up to a whole tile.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void rows_kernel(SortedTokens sorted, int64_t tokens, uint32_t vocab, uint32_t tiles, RowSpace s,
                                                      float* token_logp, Matrix x, int64_t rows, int64_t cols, uint32_t per_row, char* out,
                                                      int64_t plane)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * kBlock;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < tokens; i += step) {
        const uint32_t key = sorted.keys[i], t = sorted.tokens[i];
        const bool in = key < vocab;
        s.slot[t] = in ? static_cast<int32_t>(i) : -1;
        if (in) {
            s.token[i] = static_cast<int32_t>(t);
            s.label[i] = static_cast<int32_t>(key);
            s.top[i] = -INFINITY;
            s.sum[i] = 0.0;
            if (i + 1 == tokens || sorted.keys[i + 1] >= vocab) *s.live = static_cast<int32_t>(i + 1);
        } else {
            if (i == 0) *s.live = 0;
            if (token_logp) token_logp[t] = 0.0f;
        }
    }
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i <= tiles; i += step) {
        const uint32_t first = i < tiles ? static_cast<uint32_t>(i) * kTile : vocab;
        int64_t low = 0, high = tokens;
        while (low < high) {
            const int64_t mid = (low + high) / 2;
            if (sorted.keys[mid] < first) low = mid + 1;
            else high = mid;
        }
        s.tile_rows[i] = static_cast<int32_t>(low);
    }
    for (RowWalk w(per_row); w.row < rows; w.next()) {
        if (sorted.keys[w.row / kTile * kTile] >= vocab) break;  // a tile of none, as are those behind it
        const bool there = w.row < tokens && sorted.keys[w.row] < vocab;
        pack_unit<kBf16>(x, there ? sorted.tokens[w.row] : 0, there, cols, w, out, plane);
    }
}

// ------------------------------------------------------ rows' statistics ---

constexpr int kJoinThreads = 1024;

struct Share {
    float top;
    double sum;
};

// One factor is 1.
__device__ __forceinline__ Share join(const Share& a, const Share& b)
{
    const double d = static_cast<double>(b.top) - static_cast<double>(a.top);
    if (!(d > 0.0)) return {a.top, b.top == -INFINITY ? a.sum + b.sum : a.sum + b.sum * exp2(d * kLog2eWide)};
    return {b.top, a.top == -INFINITY ? a.sum + b.sum : a.sum * exp2(-d * kLog2eWide) + b.sum};
}

// Joins `count` stretches of kJoinRows rows a block to what the rows have, in a fixed order; after the last piece of the
// vocabulary also what follows from them.
template <int kJoinRows>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const float2* stats, int64_t count, int64_t padded, RowSpace s, bool last,
                                                            const float* token_weight, float* token_logp)
{
    constexpr int kRuns = kJoinThreads / kJoinRows;
    __shared__ float tops[kRuns][kJoinRows];
    __shared__ double sums[kRuns][kJoinRows];
    const int at = threadIdx.x % kJoinRows, run = threadIdx.x / kJoinRows;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinRows + at, live = *s.live;
    if (static_cast<int64_t>(blockIdx.x) * kJoinRows >= live) return;
    Share mine = {-INFINITY, 0.0};
    if (row < live) {
        const int64_t each = (count + kRuns - 1) / kRuns, end = min((run + 1) * each, count);
#pragma unroll 8
        for (int64_t i = run * each; i < end; ++i) {  // fp32 factors, each of a share of the sum
            const float2 v = stats[i * padded + row];
            const float top = fmaxf(mine.top, v.x), under = top == -INFINITY ? 0.0f : top;
            mine = {top, mine.sum * static_cast<double>(exp_below(mine.top, under)) + static_cast<double>(v.y * exp_below(v.x, under))};
        }
    }
    // The largest first, so that a run's sum has one factor.
    tops[run][at] = mine.top;
    for (int half = kRuns / 2; half > 0; half /= 2) {
        __syncthreads();
        if (run < half) tops[run][at] = fmaxf(tops[run][at], tops[run + half][at]);
    }
    __syncthreads();
    const float most = tops[0][at];
    if (mine.top != most) mine.sum *= exp2((static_cast<double>(mine.top) - static_cast<double>(most)) * kLog2eWide);
    sums[run][at] = mine.sum;
    for (int half = kRuns / 2; half > 0; half /= 2) {
        __syncthreads();
        if (run < half) sums[run][at] += sums[run + half][at];
    }
    if (run != 0 || row >= live) return;
    const Share all = join({s.top[row], s.sum[row]}, {most, sums[0][at]});
    s.top[row] = all.top;
    s.sum[row] = all.sum;
    if (!last) return;
    const double logp = (static_cast<double>(s.label_logit[row]) - static_cast<double>(all.top)) - log(all.sum);
    const int32_t t = s.token[row];
    if (token_logp) token_logp[t] = static_cast<float>(logp);
    if (!token_weight) return;
    const double c = token_weight[t];
    const float slope = static_cast<float>(c), factor = static_cast<float>(c / all.sum);
    s.loss[row] = -c * logp;
    s.slope[row] = slope;
    s.factor[row] = factor;
    const float g = grad_at<1>(s.label_logit[row], all.top, factor) - slope;  // as the tile of g computes it
    s.lost[row] = g - bf16_lo(bf16_one(g));
}

// g from kept logits, its rows of the tokens that there are: entries behind the last one are zeros.  And the loss, where it
// is asked for.
template <int kParts>
__global__ __launch_bounds__(kBlock) void grad_kernel(const float* logits, int64_t stride, RowSpace s, int64_t first, int64_t size,
                                                      uint32_t per_row, char* out, int64_t plane, float* loss)
{
    __shared__ double lds[kWavesPerBlock];
    if (loss && blockIdx.x == 0) sum_loss(s.loss, s.live, loss, lds);
    const int64_t live = *s.live;
    for (RowWalk w(per_row); w.row < live; w.next()) {
        const int64_t c = static_cast<int64_t>(w.col) * kUnit, label = s.label[w.row] - first - c;
        const f32x4* from = reinterpret_cast<const f32x4*>(logits + w.row * stride + c);
        const f32x4 lo = from[0], hi = from[1];
        const float top = s.top[w.row], factor = s.factor[w.row], slope = s.slope[w.row];
        float x[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            x[i] = grad_at<kParts>(i < 4 ? lo[i % 4] : hi[i % 4], top, factor);
            x[i] = c + i < size ? (label == i ? x[i] - slope : x[i]) : 0.0f;
        }
        u32x4* to = reinterpret_cast<u32x4*>(out + (w.row * stride + c) * 2);
        if (kParts == 1) {
            *to = u32x4{bf16_pack2(x[0], x[1]), bf16_pack2(x[2], x[3]), bf16_pack2(x[4], x[5]), bf16_pack2(x[6], x[7])};
        } else {
            u32x4 part[3];
            split(x, part);
#pragma unroll
            for (int k = 0; k < 3; ++k) to[k * (plane / 16)] = part[k];
        }
    }
}

// A bf16 g from the exponentials that kExp left in its place, under the largest logit of their stretch of 128 entries.
__global__ __launch_bounds__(kBlock) void scale_kernel(const float2* stats, int64_t padded, RowSpace s, int64_t first, int64_t size,
                                                       uint32_t per_row, int64_t stride, char* g)
{
    const int64_t live = *s.live;
    for (RowWalk w(per_row); w.row < live; w.next()) {
        const int64_t c = static_cast<int64_t>(w.col) * kUnit, label = s.label[w.row] - first - c;
        u32x4* at = reinterpret_cast<u32x4*>(g + (w.row * stride + c) * 2);
        const u32x4 codes = *at;
        const float top = s.top[w.row], factor = s.factor[w.row];
        const float under = log2_below(stats[c / 128 * padded + w.row].x, top);
        float x[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const uint32_t code = i % 2 ? codes[i / 2] >> 16 : codes[i / 2] & 0xffffu;
            x[i] = c + i < size ? factor * log_value(code, under) : 0.0f;
        }
        if (label >= 0 && label < kUnit) {
            const float at_label = grad_at<1>(s.label_logit[w.row], top, factor) - s.slope[w.row];
#pragma unroll
            for (int i = 0; i < kUnit; ++i) x[i] = label == i ? at_label : x[i];
        }
        *at = u32x4{bf16_pack2(x[0], x[1]), bf16_pack2(x[2], x[3]), bf16_pack2(x[4], x[5]), bf16_pack2(x[6], x[7])};
    }
}

__global__ __launch_bounds__(kBlock) void loss_kernel(const double* rows, const int32_t* live, float* loss)
{
    __shared__ double lds[kWavesPerBlock];
    sum_loss(rows, live, loss, lds);
}

// dh from its packed rows' partial sums, and for bf16 what g lost at the label; zeros for the tokens left out.
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void hidden_kernel(const float* partials, int splits, int64_t plane, int64_t stride, RowSpace s,
                                                        Matrix weight, int64_t tokens, int64_t cols, uint32_t per_row, MatrixOut out)
{
    for (RowWalk w(per_row); w.row < tokens; w.next()) {
        const int64_t row = s.slot[w.row], c = static_cast<int64_t>(w.col) * kUnit;
        float x[kUnit] = {};
        if (row >= 0) {
            for (int i = 0; i < splits; ++i) {
                const f32x4* p = reinterpret_cast<const f32x4*>(partials + i * plane + row * stride + c);
                const f32x4 lo = p[0], hi = p[1];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] += lo[j];
                    x[4 + j] += hi[j];
                }
            }
            if (kBf16) {
                float of_label[kUnit];
                widen<kBf16>(load8<kBf16>(weight.data, s.label[row] * weight.stride + c, cols - c), of_label);
                const float lost = s.lost[row];
#pragma unroll
                for (int j = 0; j < kUnit; ++j) x[j] = __builtin_fmaf(lost, of_label[j], x[j]);
            }
        }
        store8<kBf16>(x, out.data, w.row * out.stride + c, cols - c);
    }
}

// ------------------------------------------------------------- the plan ---

// Of a piece: its g, with fp32 operands and few tokens its logits too, and of the weight what is packed.  Half of what all
// logits would take in the operands' type, so that the call stays an alternative to making them; at least kLeastPieceBytes,
// where the logits are not worth the time, and at most kMostPieceBytes.  What is behind it is made twice: 8192 x 128256 x
// 4096 (2.1 GB of logits) takes 22.1 ms, with all of it kept 19.5; 8192 x 32000 x 4096 (0.5 GB, all kept) 4.9, with half 5.9.
constexpr int64_t kLeastPieceBytes = 512ll << 20, kMostPieceBytes = 2ll << 30;
constexpr int64_t kPackedBytes = 512ll << 20; // of a packed piece of the weight
constexpr int64_t kStatBytes = 128ll << 20;   // of the statistics of a part of the first pass
constexpr int64_t kLeastPiece = 2048;
constexpr int64_t kMostPiece = 1ll << 20;     // keeps a tile's offsets below 2^32 bytes
constexpr int64_t kBlocks = 256;              // that fill the device

// Tiles of 256 x 256 up to which the statistics' are 64 x 64, since those leave most CUs idle.  Log-probabilities of 250 x
// 64 n x 1024, n a quarter of the tiles, in us by tiles of 256 and of 64: bf16 with 32 tiles 40 and 26, with 64 41 and 36, with
// 96 41 and 48, with 256 51 and 109; fp32 136 and 47, 153 and 79, 181 and 107, 291 and 260.  With 4096 features, 500 x 8192
// (64 tiles) bf16 89 and 72, fp32 496 and 253; 500 x 16384 101 and 162, 576 and 482.  So fp32 would gain up to 256 of them.
constexpr int64_t kSmallTiles = 64;

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// The vocabulary in pieces: `others` of at most `piece` entries each up to entry `last`, then one as large as there is room
// for.  The first pass ends with that one, whose logits (or their exponentials) stay for the second, which begins with it:
// the others' are made again.
struct Plan {
    int parts;
    int64_t rows, cols;           // padded tokens and features
    int64_t vocab, others, piece, last, largest;
    int64_t first_piece;          // of the first pass over the others, where nothing is packed
    int splits;                   // of a piece, for dh
    bool packed;                  // the weight goes through the workspace
    bool few;                     // kernels for few tokens
    bool small;                   // their statistics for all tokens
    bool any;                     // which read any weight as it lies
    bool logits;                  // what stays are logits

    int64_t first(int64_t i) const { return i < others ? i * piece : last; }
    int64_t size(int64_t i) const { return i < others ? (last - i * piece < piece ? last - i * piece : piece) : vocab - last; }
};

Plan plan_of(int64_t tokens, int64_t vocab, int64_t cols, bool bf16, bool packed, bool gradients)
{
    Plan p;
    p.parts = bf16 ? 1 : 3;
    p.rows = up(tokens, kTile);
    p.cols = up(cols, kStage);
    p.vocab = vocab;
    p.few = tokens <= kFewTokens;
    p.small = p.few || p.rows / kTile * ((vocab + kTile - 1) / kTile) <= kSmallTiles;
    p.packed = packed && !p.few && (gradients || !p.small);
    p.any = packed && !p.packed;
    p.logits = gradients && (!bf16 || p.small);
    auto within = [](int64_t most, int64_t bytes, int64_t of_entry) {
        const int64_t n = bytes / of_entry / kTile * kTile;
        return n < kLeastPiece ? (most < kLeastPiece ? most : kLeastPiece) : (n < most ? n : most);
    };
    // A float2 a row and stretch, two stretches a tile, four of the small ones.
    const int64_t all = up(vocab, kTile), by_stats = within(all, kStatBytes, (p.small ? 32 : 16) * p.rows / kTile);
    int64_t most = all;
    if (p.packed) most = within(most, kPackedBytes, 2 * p.parts * p.cols);
    if (gradients) {
        const int64_t half = tokens * vocab * (bf16 ? 1 : 2);  // bytes
        const int64_t room = half < kLeastPieceBytes ? kLeastPieceBytes : (half < kMostPieceBytes ? half : kMostPieceBytes);
        const int64_t of_entry = (2 * p.parts + (p.logits ? 4 : 0)) * p.rows + (p.packed ? 2 * p.parts * p.cols : 0);
        most = within(most < kMostPiece ? most : kMostPiece, room, of_entry);
    }
    if (most > by_stats && !gradients) most = by_stats;
    p.last = all - most;
    p.others = (p.last + most - 1) / most;
    p.piece = p.others > 0 ? up((p.last + p.others - 1) / p.others, kTile) : 0;
    if (p.others > 0) p.others = (p.last + p.piece - 1) / p.piece;
    p.largest = most;
    p.first_piece = by_stats < p.last ? by_stats : p.last;
    const int64_t tiles = p.any ? (cols + 127) / 128 : p.rows / kTile * ((cols + kTile - 1) / kTile), stages = most / kStage;
    const int64_t blocks = p.any ? 2 * kBlocks : kBlocks;
    int64_t splits = tiles >= blocks ? 1 : blocks / tiles;
    if (splits > stages / 8) splits = stages / 8 > 0 ? stages / 8 : 1;
    p.splits = static_cast<int>(splits);
    return p;
}

// Where everything lies in the workspace.
struct Space {
    RowSpace rows;
    float2* stats;
    char *sort, *hidden, *weight, *grad;
    float *dh, *logits;
    int64_t hidden_plane, weight_plane, grad_plane, dh_plane;  // bytes, bytes, elements, elements
    size_t bytes;
};

Space space_of(const Plan& p, int64_t tokens, bool gradients, char* base)
{
    Space s = {};
    size_t at = 0;
    auto take = [&](auto*& out, int64_t count) {
        out = reinterpret_cast<std::remove_reference_t<decltype(out)>>(base + at);
        at += static_cast<size_t>(up(count * static_cast<int64_t>(sizeof(*out)), 256));
    };
    take(s.rows.live, 1);
    take(s.rows.slot, tokens);
    take(s.rows.token, p.rows);
    take(s.rows.label, p.rows);
    take(s.rows.tile_rows, (p.vocab + kTile - 1) / kTile + 1);
    take(s.rows.label_logit, p.rows);
    take(s.rows.top, p.rows);
    take(s.rows.sum, p.rows);
    take(s.rows.factor, p.rows);
    take(s.rows.slope, p.rows);
    take(s.rows.lost, p.rows);
    take(s.rows.loss, p.rows);
    take(s.sort, static_cast<int64_t>(sort_scratch(tokens, p.vocab)));
    take(s.stats, (p.largest > p.first_piece ? p.largest : p.first_piece) / kTile * (p.small ? 4 : 2) * p.rows);
    s.hidden_plane = p.rows * p.cols * 2;
    take(s.hidden, p.parts * s.hidden_plane);
    if (p.packed) {
        s.weight_plane = p.largest * p.cols * 2;
        take(s.weight, p.parts * s.weight_plane);
    }
    if (gradients) {
        s.grad_plane = p.rows * p.largest;
        take(s.grad, p.parts * s.grad_plane * 2);
        if (p.logits) take(s.logits, p.rows * p.largest);
        s.dh_plane = p.rows * p.cols;
        take(s.dh, p.splits * s.dh_plane);
    }
    s.bytes = at;
    return s;
}

int grid_for(int64_t units)
{
    const int64_t blocks = (units + kBlock - 1) / kBlock;
    return static_cast<int>(blocks < 1 << 16 ? blocks : 1 << 16);
}

// Whether the products can read the weight where it lies.
bool direct(const Matrix& w, bool bf16, int64_t cols)
{
    return bf16 && cols % kStage == 0 && w.stride % 8 == 0 && w.stride <= 1 << 21 && reinterpret_cast<uintptr_t>(w.data) % 16 == 0;
}

uint32_t blocks_of(const Product& p)  // a multiple of the XCDs
{
    return static_cast<uint32_t>(up((p.m + kTile - 1) / kTile * ((p.n + kTile - 1) / kTile), 8));
}

// The logits' statistics and what `keep` says; the stretches that the statistics are of.
hipError_t run_stats(const Plan& plan, const Product& p, const Matrix& w, int64_t cols, const Target& to, Keep keep, int64_t* stretches,
                     hipStream_t stream)
{
    *stretches = plan.small ? (p.m + 63) / 64 : (p.m + kTile - 1) / kTile * 2;
    auto run = [&](auto kernel) { kernel<<<blocks_of(p), kBlock, 0, stream>>>(p, to); };
    if (plan.small) {
        const dim3 few(static_cast<uint32_t>(up(*stretches, p.splits)), static_cast<uint32_t>((p.n + 63) / 64));
        auto run_few = [&](auto kernel) { kernel<<<few, kBlock, 0, stream>>>(p, w, cols, to); };
        if (p.parts == 3) p.n <= 32 ? run_few(few_stats_f32_kernel<1>) : run_few(few_stats_f32_kernel<2>);
        else if (plan.any) p.n <= 32 ? run_few(few_stats_kernel<1, true>) : run_few(few_stats_kernel<2, true>);
        else p.n <= 32 ? run_few(few_stats_kernel<1, false>) : run_few(few_stats_kernel<2, false>);
    } else if (keep == Keep::kExp) {
        run(product_kernel<Kind::kExp, 1>);
    } else if (keep == Keep::kLogits) {
        run(product_kernel<Kind::kKept, 3>);
    } else {
        p.parts == 1 ? run(product_kernel<Kind::kStats, 1>) : run(product_kernel<Kind::kStats, 3>);
    }
    return hipGetLastError();
}

}  // namespace

// For a weight that can be read where it lies and for one that cannot.
size_t head_scratch(int64_t tokens, int64_t vocab, int64_t cols, bool bf16, bool gradients)
{
    size_t most = 0;
    for (const bool packed : {false, true}) {
        if (!packed && (!bf16 || cols % kStage != 0)) continue;  // such a weight is packed
        const Plan p = plan_of(tokens, vocab, cols, bf16, packed, gradients);
        const size_t need = space_of(p, tokens, gradients, nullptr).bytes;
        if (need > most) most = need;
    }
    return most;
}

hipError_t launch_head(const HeadArgs& a, bool bf16, void* scratch, hipStream_t stream)
{
    const bool gradients = a.dhidden.data || a.dweight;
    hipError_t e;
    if (a.tokens == 0) {
        if (a.loss) loss_kernel<<<1, kBlock, 0, stream>>>(nullptr, nullptr, a.loss);
        if ((e = hipGetLastError()) != hipSuccess || !a.dweight || a.accumulate) return e;
        const int64_t values = a.vocab * a.cols;
        if (!a.dweight_bf16) return launch_zero(static_cast<float*>(a.dweight), values, stream);
        return launch_zero_bf16(a.dweight, values, stream);
    }
    const Plan plan = plan_of(a.tokens, a.vocab, a.cols, bf16, !direct(a.weight, bf16, a.cols), gradients);
    const Space s = space_of(plan, a.tokens, gradients, static_cast<char*>(scratch));
    const uint32_t units = static_cast<uint32_t>(plan.cols / kUnit);

    SortedTokens sorted;
    if ((e = launch_sort(a.labels, a.token_weight, a.tokens, a.vocab, nullptr, s.sort, &sorted, stream)) != hipSuccess) return e;
    const uint32_t tiles = static_cast<uint32_t>((a.vocab + kTile - 1) / kTile), vocab = static_cast<uint32_t>(a.vocab);
    const int rows_grid = grid_for(plan.rows * units > tiles ? plan.rows * units : tiles + 1);
    auto run_rows = [&](auto kernel) {
        kernel<<<rows_grid, kBlock, 0, stream>>>(sorted, a.tokens, vocab, tiles, s.rows, a.token_logp, a.hidden, plan.rows, a.cols, units,
                                                 s.hidden, s.hidden_plane);
    };
    bf16 ? run_rows(rows_kernel<true>) : run_rows(rows_kernel<false>);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    const Side hidden = {s.hidden, s.hidden_plane, static_cast<uint32_t>(plan.cols * 2)};
    const int elem = bf16 ? 2 : 4;
    int64_t in_workspace = -1;  // first entry of the piece of the weight that is packed there
    auto piece_of = [&](int64_t first) { return Matrix{static_cast<const char*>(a.weight.data) + first * a.weight.stride * elem, a.weight.stride}; };
    auto weight_at = [&](int64_t first, int64_t size, Side& w) {
        if (!plan.packed) {
            w = {static_cast<const char*>(piece_of(first).data), 0, static_cast<uint32_t>(a.weight.stride * 2)};
            return hipSuccess;
        }
        w = {s.weight, s.weight_plane, static_cast<uint32_t>(plan.cols * 2)};
        if (in_workspace == first) return hipSuccess;
        in_workspace = first;
        auto run = [&](auto kernel) {
            kernel<<<grid_for(size * units), kBlock, 0, stream>>>(piece_of(first), size, a.cols, units, s.weight, s.weight_plane);
        };
        bf16 ? run(pack_kernel<true>) : run(pack_kernel<false>);
        return hipGetLastError();
    };
    // The logits of `size` entries from `first` on; `keep` what stays of them, in s.logits or s.grad.
    auto make_logits = [&](int64_t first, int64_t size, Keep keep, int64_t* stretches) {
        Side w;
        if ((e = weight_at(first, size, w)) != hipSuccess) return e;
        Target to = {};
        to.stats = s.stats;
        to.label_logit = s.rows.label_logit;
        to.labels = s.rows.label;
        to.first = first;
        to.rows = plan.rows;
        if (keep == Keep::kLogits) to.out = s.logits;
        if (keep == Keep::kExp) to.out = s.grad;
        to.out_stride = plan.largest;
        const Product p = {w, hidden, size, a.tokens, plan.cols, s.rows.live, plan.parts, plan.splits};
        return run_stats(plan, p, piece_of(first), a.cols, to, keep, stretches, stream);
    };
    auto first_pass = [&](int64_t first, int64_t size, Keep keep) {
        int64_t stretches;
        if ((e = make_logits(first, size, keep, &stretches)) != hipSuccess) return e;
        auto join = [&](auto kernel, int64_t rows) {
            kernel<<<static_cast<uint32_t>(plan.rows / rows), kJoinThreads, 0, stream>>>(s.stats, stretches, plan.rows, s.rows,
                                                                                         first + size == a.vocab, a.token_weight, a.token_logp);
        };
        if (plan.few) join(join_kernel<4>, 4);
        else join(join_kernel<16>, 16);
        return hipGetLastError();
    };
    const Keep keep = !gradients ? Keep::kNone : (plan.logits ? Keep::kLogits : Keep::kExp);
    if (plan.packed) {
        for (int64_t i = 0; i < plan.others; ++i) {
            if ((e = first_pass(plan.first(i), plan.size(i), Keep::kNone)) != hipSuccess) return e;
        }
    } else {
        for (int64_t first = 0; first < plan.last; first += plan.first_piece) {
            const int64_t size = plan.last - first < plan.first_piece ? plan.last - first : plan.first_piece;
            if ((e = first_pass(first, size, Keep::kNone)) != hipSuccess) return e;
        }
    }
    if ((e = first_pass(plan.last, a.vocab - plan.last, keep)) != hipSuccess) return e;
    if (!gradients) {
        if (a.loss) loss_kernel<<<1, kBlock, 0, stream>>>(s.rows.loss, s.rows.live, a.loss);
        return hipGetLastError();
    }

    for (int64_t i = plan.others; i >= 0; --i) {
        const int64_t first = plan.first(i), size = plan.size(i);
        const bool kept = i == plan.others;
        Side w;
        if ((e = weight_at(first, size, w)) != hipSuccess) return e;
        const uint32_t per_row = static_cast<uint32_t>(up(size, kTile) / kUnit);
        const int grid = grid_for(a.tokens * per_row);
        if (plan.logits) {
            int64_t stretches;  // of statistics that the rows have already
            if (!kept && (e = make_logits(first, size, Keep::kLogits, &stretches)) != hipSuccess) return e;
            auto run = [&](auto kernel) {
                kernel<<<grid, kBlock, 0, stream>>>(s.logits, plan.largest, s.rows, first, size, per_row, s.grad, s.grad_plane * 2, kept ? a.loss : nullptr);
            };
            bf16 ? run(grad_kernel<1>) : run(grad_kernel<3>);
        } else if (kept) {
            scale_kernel<<<grid, kBlock, 0, stream>>>(s.stats, plan.rows, s.rows, first, size, per_row, plan.largest, s.grad);
        } else {
            Target to = {};
            to.labels = s.rows.label;
            to.first = first;
            to.top = s.rows.top;
            to.factor = s.rows.factor;
            to.slope = s.rows.slope;
            to.out = s.grad;
            to.out_stride = plan.largest;
            const Product logits = {w, hidden, size, a.tokens, plan.cols, s.rows.live, plan.parts, 1};
            product_kernel<Kind::kGrad, 1><<<blocks_of(logits), kBlock, 0, stream>>>(logits, to);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;

        const Side grad = {s.grad, s.grad_plane * 2, static_cast<uint32_t>(plan.largest * 2)};
        Target dh_to = {}, dw_to = {};
        dh_to.out = s.dh;
        dh_to.out_stride = plan.cols;
        dh_to.out_plane = s.dh_plane;
        dh_to.accumulate = !kept;
        const Product dh = {grad, w, a.tokens, plan.cols, size, s.rows.live, plan.parts, plan.splits};
        dw_to.out = static_cast<char*>(a.dweight) + first * a.cols * (a.dweight_bf16 ? 2 : 4);
        dw_to.out_stride = a.cols;
        dw_to.labels = s.rows.label;
        dw_to.first = first;
        dw_to.tile_rows = s.rows.tile_rows;
        dw_to.lost = s.rows.lost;
        dw_to.accumulate = a.accumulate;
        dw_to.bf16 = a.dweight_bf16;
        const Product dw = {grad, hidden, size, a.cols, a.tokens, s.rows.live, plan.parts, 1};
        if (plan.any && a.dhidden.data) {
            const uint32_t few = static_cast<uint32_t>((a.cols + 127) / 128 * plan.splits);
            auto run_any = [&](auto kernel) { kernel<<<few, kBlock, 0, stream>>>(dh, piece_of(first), a.cols, dh_to); };
            if (bf16) a.tokens <= 32 ? run_any(few_hidden_any_kernel<1, 1>) : run_any(few_hidden_any_kernel<1, 2>);
            else a.tokens <= 32 ? run_any(few_hidden_any_kernel<3, 1>) : run_any(few_hidden_any_kernel<3, 2>);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        const uint32_t hidden_blocks = a.dhidden.data && !plan.any ? blocks_of(dh) * plan.splits : 0;
        const uint32_t weight_blocks = a.dweight && !plan.few ? blocks_of(dw) : 0;
        float* loss = kept && !plan.logits ? a.loss : nullptr;
        const uint32_t blocks = hidden_blocks + weight_blocks + (loss ? 1 : 0);
        auto run = [&](auto kernel) { kernel<<<blocks, kBlock, 0, stream>>>(dh, dh_to, hidden_blocks, dw, dw_to, s.rows.loss, loss); };
        if (blocks > 0) plan.parts == 1 ? run(gradients_kernel<1>) : run(gradients_kernel<3>);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (!a.dweight || !plan.few) continue;
        const int64_t across = (a.cols + (bf16 ? 256 : 128) - 1) / (bf16 ? 256 : 128), down = (size + 63) / 64;
        int64_t per_block = across * down / (8 * kBlocks);  // tiles; at least eight blocks a CU
        per_block = per_block < 1 ? 1 : (per_block > 16 ? 16 : per_block);
        const uint32_t few = static_cast<uint32_t>((down + per_block - 1) / per_block * across);
        auto run_few = [&](auto kernel) { kernel<<<few, kBlock, 0, stream>>>(dw, dw_to, static_cast<uint32_t>(per_block)); };
        auto of_length = [&](auto parts, auto type, auto accumulate) {
            if (a.tokens <= 32) run_few(few_weight_kernel<parts.value, 32, type.value, accumulate.value>);
            else run_few(few_weight_kernel<parts.value, 64, type.value, accumulate.value>);
        };
        auto of_type = [&](auto parts, auto type) {
            a.accumulate ? of_length(parts, type, std::true_type()) : of_length(parts, type, std::false_type());
        };
        const std::integral_constant<int, 1> one;
        const std::integral_constant<int, 3> three;
        if (bf16) a.dweight_bf16 ? of_type(one, std::true_type()) : of_type(one, std::false_type());
        else a.dweight_bf16 ? of_type(three, std::true_type()) : of_type(three, std::false_type());
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!a.dhidden.data) return hipSuccess;
    const uint32_t out_units = static_cast<uint32_t>((a.cols + kUnit - 1) / kUnit);
    const int grid = grid_for(a.tokens * out_units);
    if (bf16) hidden_kernel<true><<<grid, kBlock, 0, stream>>>(s.dh, plan.splits, s.dh_plane, plan.cols, s.rows, a.weight, a.tokens, a.cols, out_units, a.dhidden);
    else hidden_kernel<false><<<grid, kBlock, 0, stream>>>(s.dh, plan.splits, s.dh_plane, plan.cols, s.rows, a.weight, a.tokens, a.cols, out_units, a.dhidden);
    return hipGetLastError();
}

}  // namespace mps
