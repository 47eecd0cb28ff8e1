// gfx950 kernels of the embedding lookup, its gradient, and dropout.
#include <hip/hip_runtime.h>

#include "model_kernels.h"
#include "rows.h"

namespace mps {
namespace {

int grid_for(int64_t units, int64_t most)
{
    const int64_t blocks = (units + kBlock - 1) / kBlock;
    return static_cast<int>(blocks < most ? blocks : most);
}

constexpr int64_t kStreamBlocks = 1 << 16;

// ------------------------------------------------------------ embedding ---

// out[t] = scale * table[id_t], rounded once; zeros for an id outside the
// vocabulary.  Bound by memory: a row is read where it lies and written once
// (16384 x 8192 bf16 88 us, 6.1 TB/s with rows read again from the cache; one
// token 5.2 us, the call's host time).
template <bool kBf16>
__global__ __launch_bounds__(kBlock) void embedding_kernel(const int64_t* ids, int64_t tokens, Matrix table, int64_t vocab, int64_t cols,
                                                           uint32_t per_row, float scale, MatrixOut out)
{
    for (RowWalk w(per_row); w.row < tokens; w.next()) {
        const int64_t id = ids[w.row], c = static_cast<int64_t>(w.col) * kUnit;
        const bool known = id >= 0 && id < vocab;
        float x[kUnit];
        widen<kBf16>(load8<kBf16>(table.data, (known ? id : 0) * table.stride + c, known ? cols - c : 0), x);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) x[i] = known ? x[i] * scale : 0.0f;
        store8<kBf16>(x, out.data, w.row * out.stride + c, cols - c);
    }
}

// ------------------------------------------- tokens in the order of their ids ---
//
// A stable radix sort, least significant digit first: what is left of a
// token's place is its number, so that every row's sum has one order.  An id
// outside the vocabulary counts as `vocab`, behind all others.  Bound by its
// launches: two a digit of 9 bits (65536 ids of 15 bits 23 us).  Up to 8192
// tokens are counted against each other instead, in one launch.

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kMostDigit = 9;                 // bits
constexpr int kBins = 1 << kMostDigit;
constexpr int64_t kSortBlocks = 512;          // at most: each reads all blocks' counts

struct SortPass {
    const int64_t* ids;        // of the first pass; else NULL
    const float* weight;       // or NULL; a token whose weight is 0 counts as one outside the vocabulary
    const uint32_t *keys_in, *tokens_in;
    uint32_t *keys, *tokens;   // out
    uint32_t* counts;          // [block][kBins]
    int64_t n, per_block;      // per_block: whole rounds of kSortThreads
    uint32_t vocab;
    int shift;
    uint8_t* touched;          // rows of the table that have tokens: cleared by the first pass's count, set by the last pass
    bool last;
};

__device__ __forceinline__ uint32_t key_of(const SortPass& p, int64_t i)
{
    if (!p.ids) return p.keys_in[i];
    const int64_t id = p.ids[i];
    const bool in = id >= 0 && id < static_cast<int64_t>(p.vocab) && !(p.weight && p.weight[i] == 0.0f);
    return in ? static_cast<uint32_t>(id) : p.vocab;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortPass p)
{
    __shared__ uint32_t bins[kBins];
    if (p.ids && p.touched) {
        for (int64_t v = static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; v < p.vocab; v += static_cast<int64_t>(gridDim.x) * kSortThreads) {
            p.touched[v] = 0;
        }
    }
    if (threadIdx.x < kBins) bins[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * p.per_block, end = min(first + p.per_block, p.n);
    for (int64_t i = first + threadIdx.x; i < end; i += kSortThreads) atomicAdd(&bins[(key_of(p, i) >> p.shift) % kBins], 1u);
    __syncthreads();
    if (threadIdx.x < kBins) p.counts[static_cast<int64_t>(blockIdx.x) * kBins + threadIdx.x] = bins[threadIdx.x];
}

// LDS of a block that moves tokens to their places.
struct SortSpace {
    uint32_t next[kBins];       // where the digit's next token goes
    uint32_t scan[2][kBins];
    uint32_t of_wave[kSortWaves][kBins];
};

// next[d] = before[d] + all tokens of smaller digits, where thread d < kBins has the count of digit d (`all`) and what
// comes before its own tokens of d.
__device__ __forceinline__ void sort_starts(SortSpace& s, uint32_t all, uint32_t before)
{
    const int tid = threadIdx.x;
    if (tid < kBins) s.scan[0][tid] = all;
    __syncthreads();
    int buf = 0;
    for (int off = 1; off < kBins; off <<= 1, buf ^= 1) {
        if (tid < kBins) s.scan[buf ^ 1][tid] = s.scan[buf][tid] + (tid >= off ? s.scan[buf][tid - off] : 0);
        __syncthreads();
    }
    if (tid < kBins) s.next[tid] = s.scan[buf][tid] - all + before;
}

// The place of this thread's token among kSortThreads consecutive ones with these digits; `next` moves on behind them.
__device__ __forceinline__ uint32_t sort_place(SortSpace& s, bool some, uint32_t digit)
{
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    for (int i = tid; i < kSortWaves * kBins; i += kSortThreads) (&s.of_wave[0][0])[i] = 0;
    __syncthreads();
    // Lanes of this wavefront with the same digit.
    uint64_t same = __ballot(some);
#pragma unroll
    for (int b = 0; b < kMostDigit; ++b) {
        const uint64_t votes = __ballot((digit >> b) & 1);
        same &= (digit >> b) & 1 ? votes : ~votes;
    }
    const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
    if (some && rank == 0) s.of_wave[wave][digit] = __popcll(same);
    __syncthreads();
    if (tid < kBins) {
        uint32_t at = s.next[tid];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = s.of_wave[w][tid];
            s.of_wave[w][tid] = at;
            at += c;
        }
        s.next[tid] = at;
    }
    __syncthreads();
    const uint32_t place = s.of_wave[wave][digit] + rank;
    __syncthreads();
    return place;
}

__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(SortPass p)
{
    __shared__ SortSpace space;
    const int tid = threadIdx.x, digit = tid % kBins;
    // Before this block's tokens of a digit: all tokens of smaller digits, and the earlier blocks' of the same.  Half of
    // the threads count the even blocks, half the odd ones.
    uint32_t before = 0, all = 0;
#pragma unroll 8
    for (uint32_t b = tid / kBins; b < gridDim.x; b += kSortThreads / kBins) {
        const uint32_t c = p.counts[static_cast<int64_t>(b) * kBins + digit];
        before += b < blockIdx.x ? c : 0;
        all += c;
    }
    if (tid >= kBins) {
        space.of_wave[0][digit] = before;
        space.of_wave[1][digit] = all;
    }
    __syncthreads();
    before += space.of_wave[0][digit];
    all += space.of_wave[1][digit];
    sort_starts(space, all, before);
    const int64_t first = blockIdx.x * p.per_block, end = min(first + p.per_block, p.n);
    for (int64_t i0 = first; i0 < end; i0 += kSortThreads) {
        const int64_t i = i0 + tid;
        const bool some = i < end;
        const uint32_t key = some ? key_of(p, i) : 0;
        const uint32_t to = sort_place(space, some, (key >> p.shift) % kBins);
        if (some) {
            p.keys[to] = key;
            p.tokens[to] = p.ids ? static_cast<uint32_t>(i) : p.tokens_in[i];
            if (p.last && p.touched && key < p.vocab) p.touched[key] = 1;
        }
    }
}
static_assert(kSortThreads == 2 * kBins, "two threads a digit");

// At most kRankMost tokens, in one launch: a token's place is the number of tokens before it, counted over all keys in LDS.
// A block places kRankTokens, each with kRankTokens groups of threads that have a share of the keys; and it has the flags of
// kRankFlags rows of the table.  The gradient of 256 features into 32003 rows, in us with it and with two launches a digit:
// 512 tokens 22 and 33, 2048 25 and 35, 4096 28 and 37, 8192 33 and 39, 10000 41 and 40, 16384 50 and 38 (with LDS for as
// many keys).
constexpr int kRankMost = 8192, kRankTokens = 32, kRankFlags = 4096;

__global__ __launch_bounds__(kSortThreads) void rank_kernel(SortPass p)
{
    __shared__ __attribute__((aligned(16))) uint32_t keys[kRankMost];
    __shared__ uint32_t places[kRankTokens];
    const int tid = threadIdx.x, mine = tid % kRankTokens, group = tid / kRankTokens;
    const int n = static_cast<int>(p.n), padded = (n + kRankTokens - 1) / kRankTokens * kRankTokens;
    for (int i = tid; i < padded; i += kSortThreads) keys[i] = i < n ? key_of(p, i) : ~0u;
    if (tid < kRankTokens) places[tid] = 0;
    __syncthreads();
    if (p.touched) {
        __shared__ __attribute__((aligned(16))) uint8_t flags[kRankFlags];
        const uint32_t v0 = blockIdx.x * kRankFlags;
        if (v0 < p.vocab) {
            if (tid < kRankFlags / 16) reinterpret_cast<u32x4*>(flags)[tid] = u32x4{0, 0, 0, 0};
            __syncthreads();
            for (int i = tid; i < n; i += kSortThreads) {
                if (keys[i] - v0 < kRankFlags) flags[keys[i] - v0] = 1;
            }
            __syncthreads();
            // The flags' memory ends in a multiple of 256.
            const uint32_t v = v0 + tid * 16;
            if (tid < kRankFlags / 16 && v < p.vocab) *reinterpret_cast<u32x4*>(p.touched + v) = reinterpret_cast<const u32x4*>(flags)[tid];
        }
    }
    const int base = blockIdx.x * kRankTokens, token = base + mine;
    if (base >= n) return;
    const uint32_t key = keys[token];
    const int per = (padded / kRankTokens + kRankTokens - 1) / kRankTokens * kRankTokens;
    const int first = min(group * per, padded), end = min(first + per, padded);
    uint32_t before = 0;
    auto count = [&](int from, int to, uint32_t below) __attribute__((always_inline)) {
#pragma unroll 4
        for (int j = from; j < to; j += 4) {
            const u32x4 k = *reinterpret_cast<const u32x4*>(keys + j);
#pragma unroll
            for (int i = 0; i < 4; ++i) before += k[i] < below;
        }
    };
    // Of equal keys the earlier token comes first.
    count(first, min(end, base), key + 1);
    if (first <= base && base < end) {
        for (int j = 0; j < kRankTokens; ++j) before += keys[base + j] < key + (j < mine);
    }
    count(max(first, base + kRankTokens), end, key);
    atomicAdd(&places[mine], before);
    __syncthreads();
    if (tid < kRankTokens && token < n) {
        const uint32_t to = places[tid];
        p.keys[to] = key;
        p.tokens[to] = token;
    }
}
static_assert(kRankTokens * kRankTokens == kSortThreads, "as many groups as tokens");

// --------------------------------------------------- the table's gradient ---
//
// dtable[v] = [dtable[v] +] scale * sum of dout over the tokens of v, in their
// order.  The sorted tokens are cut into equal chunks, whatever their ids: a
// block sums the runs of one id in its chunk.  A run that lies in one chunk is
// stored at once; the pieces of longer ones go to the workspace and are
// joined, in order, by a second launch.  Rows without tokens are zeros, written
// by further blocks of the first.  Bound by memory where the whole gradient is
// written (8192 x 4096 into 128256 rows in fp32 400 us, 2.17 GB; one launch of
// it 370 us, 5.9 TB/s), by the sort and the join where the table is small
// (65536 x 1024 into 32003 rows 94 us, of which the sums take 60).

struct RowSums {
    Matrix dout;
    const uint32_t *keys, *tokens;  // sorted
    int64_t n, chunk, chunks;
    uint32_t vocab;
    int64_t cols;
    float scale;
    void* dtable;
    bool bf16, accumulate;          // of dtable
    float* pieces;                  // [chunk][first run, last run][width]
    int64_t width;                  // of a piece: cols in whole units
    const uint8_t* touched;
    int64_t slabs, fill_rows;       // blocks that share a chunk's columns; rows that a filling block has
};

__device__ __forceinline__ void store_row(const RowSums& a, uint32_t key, int64_t c, const float (&sum)[kUnit])
{
    float x[kUnit];
    const int64_t at = static_cast<int64_t>(key) * a.cols + c, n = a.cols - c;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) x[i] = sum[i] * a.scale;
    if (a.accumulate) {
        float old[kUnit];
        if (a.bf16) widen<true>(load8<true>(a.dtable, at, n), old);
        else widen<false>(load8<false>(a.dtable, at, n), old);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) x[i] = old[i] + x[i];
    }
    if (a.bf16) store8<true>(x, a.dtable, at, n);
    else store8<false>(x, a.dtable, at, n);
}

__device__ __forceinline__ float* piece_of(const RowSums& a, int64_t chunk, int last, int64_t c)
{
    return a.pieces + (chunk * 2 + last) * a.width + c;
}

// Zeros for the rows without tokens among the `fill_rows` (at most a wavefront's lanes) of filling block b: a lane looks
// up one row each, then each wavefront takes whole rows, 1 KB a store.
__device__ __forceinline__ void zero_rows(const RowSums& a, int64_t b)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
    const int64_t v0 = b * a.fill_rows, v1 = min(v0 + a.fill_rows, static_cast<int64_t>(a.vocab));
    const bool mine = v0 + lane < v1 && a.touched[v0 + lane] == 0;
    uint64_t rows = __ballot(mine);
    const int64_t elem = a.bf16 ? 2 : 4, bytes = a.cols * elem, whole = bytes / 16;
    for (int i = 0; rows; ++i) {
        const int at = __builtin_ctzll(rows);
        rows &= rows - 1;
        if (i % waves != wave) continue;
        char* row = static_cast<char*>(a.dtable) + (v0 + at) * bytes;
        for (int64_t c = lane; c < whole; c += kWave) *reinterpret_cast<u32x4_at2*>(row + c * 16) = u32x4_at2{0, 0, 0, 0};
        const int64_t rest = whole * 16 + lane * elem;
        if (rest < bytes) {
            if (a.bf16) *reinterpret_cast<uint16_t*>(row + rest) = 0;
            else *reinterpret_cast<float*>(row + rest) = 0.0f;
        }
    }
}

template <bool kBf16>
__global__ __launch_bounds__(kBlock) void row_sums_kernel(RowSums a)
{
    const int64_t b = blockIdx.x;
    if (b >= a.chunks * a.slabs) return zero_rows(a, b - a.chunks * a.slabs);
    const int64_t chunk = b / a.slabs, first = chunk * a.chunk, end = min(first + a.chunk, a.n);
    const int64_t c = ((b % a.slabs) * blockDim.x + threadIdx.x) * kUnit;
    if (c >= a.cols) return;
    uint32_t key = a.keys[first];
    bool from_before = first > 0 && a.keys[first - 1] == key;
    float sum[kUnit] = {};
    constexpr int kDeep = 4;
    for (int64_t p = first; p < end; p += kDeep) {
        Raw8<kBf16> raw[kDeep];
        uint32_t keys[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int64_t q = min(p + j, end - 1);
            keys[j] = a.keys[q];
            raw[j] = load8<kBf16>(a.dout.data, static_cast<int64_t>(a.tokens[q]) * a.dout.stride + c, keys[j] < a.vocab ? a.cols - c : 0);
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            if (p + j >= end) break;
            if (keys[j] != key) {  // the run before ends in this chunk
                if (from_before) {
                    float* to = piece_of(a, chunk, 0, c);
#pragma unroll
                    for (int i = 0; i < kUnit; ++i) to[i] = sum[i];
                } else {
                    store_row(a, key, c, sum);
                }
                key = keys[j];
                from_before = false;
#pragma unroll
                for (int i = 0; i < kUnit; ++i) sum[i] = 0.0f;
            }
            float x[kUnit];
            widen<kBf16>(raw[j], x);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) sum[i] += x[i];
        }
    }
    if (key >= a.vocab) return;
    const bool goes_on = end < a.n && a.keys[end] == key;
    if (!from_before && !goes_on) return store_row(a, key, c, sum);
    float* to = piece_of(a, chunk, from_before ? 0 : 1, c);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) to[i] = sum[i];
}

// The run that begins in this block's chunk and goes on behind it; `threads` of the block to a slab of columns.
constexpr int kJoinThreads = 1024;

__global__ __launch_bounds__(kJoinThreads) void join_rows_kernel(RowSums a, int threads)
{
    const int64_t chunk = blockIdx.x / a.slabs, first = chunk * a.chunk, end = first + a.chunk;
    if (end >= a.n) return;
    const uint32_t key = a.keys[end - 1];
    if (key >= a.vocab || a.keys[end] != key) return;
    if (a.keys[first] == key && first > 0 && a.keys[first - 1] == key) return;  // it began before
    // The last chunk with a piece: those between are whole.
    int64_t last = chunk + 1;
    for (;;) {
        const int64_t mine = last + threadIdx.x, behind = (mine + 1) * a.chunk;
        const int whole = __syncthreads_count(behind < a.n && a.keys[min(behind, a.n - 1)] == key);
        last += whole;
        if (whole < static_cast<int>(blockDim.x)) break;
    }
    // Each of the block's groups of threads sums an equal stretch of the pieces; then the groups' sums, in order.
    __shared__ float of_group[kJoinThreads * kUnit];
    const int group = threadIdx.x / threads, groups = blockDim.x / threads, at = threadIdx.x % threads;
    const int64_t c = ((blockIdx.x % a.slabs) * threads + at) * kUnit;
    float sum[kUnit] = {};
    if (c < a.cols) {
        const int64_t count = last - chunk + 1, each = (count + groups - 1) / groups;  // the first one is the chunk's last run
        const int64_t k0 = chunk + group * each, k1 = min(k0 + each, last + 1);
#pragma unroll 8
        for (int64_t k = k0; k < k1; ++k) {
            const f32x4* p = reinterpret_cast<const f32x4*>(piece_of(a, k, k == chunk ? 1 : 0, c));
            const f32x4 lo = p[0], hi = p[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[i] += lo[i];
                sum[4 + i] += hi[i];
            }
        }
    }
    if (group > 0) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) of_group[i * blockDim.x + threadIdx.x] = sum[i];
    }
    __syncthreads();
    if (group > 0 || c >= a.cols) return;
    for (int g = 1; g < groups; ++g) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) sum[i] += of_group[i * blockDim.x + g * threads + at];
    }
    store_row(a, key, c, sum);
}

__global__ __launch_bounds__(kBlock) void zero_bf16_kernel(uint16_t* x, int64_t n)
{
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * kBlock) x[i] = 0;
}

struct SortPlan {
    int64_t blocks, per_block, list;  // list: elements between the two arrays of keys, and of tokens
    int passes;
    size_t tokens, counts, bytes;     // offsets; the keys come first
};

SortPlan sort_plan(int64_t tokens, int64_t vocab)
{
    SortPlan p;
    const int64_t rounds = (tokens + kSortThreads - 1) / kSortThreads;
    p.per_block = (rounds + kSortBlocks - 1) / kSortBlocks * kSortThreads;
    p.blocks = (tokens + p.per_block - 1) / p.per_block;
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;
    p.passes = (bits + kMostDigit - 1) / kMostDigit;
    p.list = (tokens + 63) / 64 * 64;
    p.tokens = static_cast<size_t>(p.list) * 8;
    p.counts = 2 * p.tokens;
    p.bytes = p.counts + static_cast<size_t>(p.blocks) * kBins * 4;
    return p;
}

struct EmbedPlan {
    int64_t chunk, chunks, width;
    size_t touched, pieces, bytes;  // offsets
};

// 65536 x 1024 takes 94 us with at most 2048 chunks, 105 with 4096 and 110 with 1024.
constexpr int64_t kMostChunks = 2048, kLeastChunk = 16;
// Of a filling block: 128256 x 4096 in fp32 405 us, with 64 KB 433, with 256 KB 427 (a wavefront writes a row; all of a
// block on one row after the other 415; past the cache 423, and a table of 262 MB 84 us, not 79).
constexpr int64_t kFillBytes = 16 << 10;

EmbedPlan embed_plan(int64_t tokens, int64_t vocab, int64_t cols)
{
    EmbedPlan p;
    p.chunk = (tokens + kMostChunks - 1) / kMostChunks;
    if (p.chunk < kLeastChunk) p.chunk = kLeastChunk;
    p.chunks = (tokens + p.chunk - 1) / p.chunk;
    p.width = (cols + kUnit - 1) / kUnit * kUnit;
    p.touched = (sort_plan(tokens, vocab).bytes + 255) / 256 * 256;
    p.pieces = (p.touched + static_cast<size_t>(vocab) + 255) / 256 * 256;
    p.bytes = p.pieces + (p.chunks > 1 ? static_cast<size_t>(p.chunks * 2 * p.width * 4) : 0);
    return p;
}

// -------------------------------------------------------------- dropout ---

// Philox4x32-10: ten rounds of two 32 x 32 -> 64 bit products (Salmon, Moraes,
// Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; 2011).
__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = static_cast<uint64_t>(c[0]) * 0xD2511F53u, p1 = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
        c[0] = static_cast<uint32_t>(p1 >> 32) ^ c[1] ^ k0;
        c[1] = static_cast<uint32_t>(p1);
        c[2] = static_cast<uint32_t>(p0 >> 32) ^ c[3] ^ k1;
        c[3] = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// out = [residual +] (dropped ? 0 : x * scale).  A unit of eight elements has
// one call of the generator, 16 bits an element, made again in the backward
// pass from the same counter: no mask is stored.  Bound by memory:
// 16384 x 8192 bf16 with a residual 134 us, 6.0 TB/s; fp32 333 x 5001 5.7 us,
// the call's host time.
template <bool kBf16, bool kResidual>
__global__ __launch_bounds__(kBlock) void dropout_kernel(DropoutArgs a, uint32_t per_row)
{
    const uint32_t k0 = static_cast<uint32_t>(a.seed), k1 = static_cast<uint32_t>(a.seed >> 32);
    const uint32_t step = a.step ? static_cast<uint32_t>(*a.step) : 0;
    for (RowWalk w(per_row); w.row < a.rows; w.next()) {
        const int64_t c = static_cast<int64_t>(w.col) * kUnit;
        const Raw8<kBf16> raw = load8<kBf16>(a.x.data, w.row * a.x.stride + c, a.cols - c);
        Raw8<kBf16> res;
        if (kResidual) res = load8<kBf16>(a.residual.data, w.row * a.residual.stride + c, a.cols - c);
        const uint64_t unit = static_cast<uint64_t>(w.unit());
        uint32_t word[4] = {static_cast<uint32_t>(unit), static_cast<uint32_t>(unit >> 32), a.site, step};
        philox(word, k0, k1);
        float x[kUnit], r[kUnit];
        widen<kBf16>(raw, x);
        if (kResidual) widen<kBf16>(res, r);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const uint32_t bits = i % 2 ? word[i / 2] >> 16 : word[i / 2] & 0xffffu;
            x[i] = bits < a.threshold ? 0.0f : x[i] * a.scale;
            if (kResidual) x[i] = r[i] + x[i];
        }
        store8<kBf16>(x, a.out.data, w.row * a.out.stride + c, a.cols - c);
    }
}

uint32_t units_per_row(int64_t cols) { return static_cast<uint32_t>((cols + kUnit - 1) / kUnit); }

}  // namespace

hipError_t launch_zero_bf16(void* x, int64_t n, hipStream_t stream)
{
    zero_bf16_kernel<<<grid_for(n, kStreamBlocks), kBlock, 0, stream>>>(static_cast<uint16_t*>(x), n);
    return hipGetLastError();
}

hipError_t launch_embedding(const int64_t* ids, int64_t tokens, Matrix table, bool bf16, int64_t vocab, int64_t cols, float scale,
                            MatrixOut out, hipStream_t stream)
{
    const uint32_t per_row = units_per_row(cols);
    const int grid = grid_for(tokens * per_row, kStreamBlocks);
    if (bf16) embedding_kernel<true><<<grid, kBlock, 0, stream>>>(ids, tokens, table, vocab, cols, per_row, scale, out);
    else embedding_kernel<false><<<grid, kBlock, 0, stream>>>(ids, tokens, table, vocab, cols, per_row, scale, out);
    return hipGetLastError();
}

size_t sort_scratch(int64_t tokens, int64_t vocab) { return sort_plan(tokens, vocab).bytes; }

hipError_t launch_sort(const int64_t* ids, const float* weight, int64_t tokens, int64_t vocab, uint8_t* touched, void* scratch,
                       SortedTokens* sorted, hipStream_t stream)
{
    const SortPlan plan = sort_plan(tokens, vocab);
    char* base = static_cast<char*>(scratch);
    uint32_t* keys = reinterpret_cast<uint32_t*>(base);
    uint32_t* order = reinterpret_cast<uint32_t*>(base + plan.tokens);
    if (tokens <= kRankMost) {
        SortPass p = {};
        p.ids = ids;
        p.weight = weight;
        p.keys = keys;
        p.tokens = order;
        p.n = tokens;
        p.vocab = static_cast<uint32_t>(vocab);
        p.touched = touched;
        const int64_t blocks = (tokens + kRankTokens - 1) / kRankTokens, of_flags = touched ? (vocab + kRankFlags - 1) / kRankFlags : 0;
        rank_kernel<<<static_cast<uint32_t>(blocks > of_flags ? blocks : of_flags), kSortThreads, 0, stream>>>(p);
        sorted->keys = keys;
        sorted->tokens = order;
        return hipGetLastError();
    }
    for (int i = 0; i < plan.passes; ++i) {
        SortPass p = {};
        p.ids = i == 0 ? ids : nullptr;
        p.weight = weight;
        p.keys_in = keys + (i % 2 ? 0 : plan.list);
        p.tokens_in = order + (i % 2 ? 0 : plan.list);
        p.keys = keys + (i % 2 ? plan.list : 0);
        p.tokens = order + (i % 2 ? plan.list : 0);
        p.counts = reinterpret_cast<uint32_t*>(base + plan.counts);
        p.n = tokens;
        p.per_block = plan.per_block;
        p.vocab = static_cast<uint32_t>(vocab);
        p.shift = i * kMostDigit;
        p.touched = touched;
        p.last = i + 1 == plan.passes;
        sort_count_kernel<<<static_cast<uint32_t>(plan.blocks), kSortThreads, 0, stream>>>(p);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        sort_move_kernel<<<static_cast<uint32_t>(plan.blocks), kSortThreads, 0, stream>>>(p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        sorted->keys = p.keys;
        sorted->tokens = p.tokens;
    }
    return hipSuccess;
}

size_t embedding_backward_scratch(int64_t tokens, int64_t vocab, int64_t cols) { return embed_plan(tokens, vocab, cols).bytes; }

hipError_t launch_embedding_backward(Matrix dout, bool bf16, const int64_t* ids, int64_t tokens, int64_t vocab, int64_t cols, float scale,
                                     void* dtable, bool dtable_bf16, bool accumulate, void* scratch, hipStream_t stream)
{
    if (tokens == 0) {
        if (accumulate) return hipSuccess;
        return dtable_bf16 ? launch_zero_bf16(dtable, vocab * cols, stream) : launch_zero(static_cast<float*>(dtable), vocab * cols, stream);
    }
    const EmbedPlan plan = embed_plan(tokens, vocab, cols);
    char* base = static_cast<char*>(scratch);
    uint8_t* touched = reinterpret_cast<uint8_t*>(base + plan.touched);
    SortedTokens sorted;
    hipError_t e = launch_sort(ids, nullptr, tokens, vocab, accumulate ? nullptr : touched, scratch, &sorted, stream);
    if (e != hipSuccess) return e;
    const int64_t units = plan.width / kUnit;
    const int64_t threads = units >= kBlock ? kBlock : (units + kWave - 1) / kWave * kWave;
    RowSums a = {};
    a.dout = dout;
    a.keys = sorted.keys;
    a.tokens = sorted.tokens;
    a.n = tokens;
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
    a.vocab = static_cast<uint32_t>(vocab);
    a.cols = cols;
    a.scale = scale;
    a.dtable = dtable;
    a.bf16 = dtable_bf16;
    a.accumulate = accumulate;
    a.pieces = reinterpret_cast<float*>(base + plan.pieces);
    a.width = plan.width;
    a.touched = touched;
    a.slabs = (units + threads - 1) / threads;
    const int64_t row_bytes = cols * (dtable_bf16 ? 2 : 4);
    a.fill_rows = kFillBytes / row_bytes;
    const int64_t least = (vocab * threads >> 31) + 1;  // a launch has less than 2^32 threads; vocab <= 2^27: at most 17 rows
    a.fill_rows = a.fill_rows < least ? least : (a.fill_rows > kWave ? kWave : a.fill_rows);
    const int64_t fill = accumulate ? 0 : (vocab + a.fill_rows - 1) / a.fill_rows;
    const uint32_t grid = static_cast<uint32_t>(plan.chunks * a.slabs + fill);
    if (bf16) row_sums_kernel<true><<<grid, static_cast<uint32_t>(threads), 0, stream>>>(a);
    else row_sums_kernel<false><<<grid, static_cast<uint32_t>(threads), 0, stream>>>(a);
    if ((e = hipGetLastError()) != hipSuccess || plan.chunks == 1) return e;
    int64_t groups = plan.chunks / 256;  // the longest runs have a share of all chunks
    groups = groups < 1 ? 1 : (groups > kJoinThreads / threads ? kJoinThreads / threads : groups);
    join_rows_kernel<<<static_cast<uint32_t>(plan.chunks * a.slabs), static_cast<uint32_t>(groups * threads), 0, stream>>>(
        a, static_cast<int>(threads));
    return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, bool bf16, hipStream_t stream)
{
    const uint32_t per_row = units_per_row(a.cols);
    const int grid = grid_for(a.rows * per_row, kStreamBlocks);
    auto run = [&](auto kernel) { kernel<<<grid, kBlock, 0, stream>>>(a, per_row); };
    if (a.residual.data) {
        if (bf16) run(dropout_kernel<true, true>);
        else run(dropout_kernel<false, true>);
    } else {
        if (bf16) run(dropout_kernel<true, false>);
        else run(dropout_kernel<false, false>);
    }
    return hipGetLastError();
}

}  // namespace mps
