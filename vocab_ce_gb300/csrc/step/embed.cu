// embed.cu -- rows of the token table by id, and the table's gradient.
//
//   forward   X[t] = scale E[ids[t]]                       (ids[t] = -1: zeros)
//   backward  dE[v] = scale sum over the t with ids[t] = v of dX[t],
// the second written whole (rows that no token names are zeros) or added to what
// dE holds, as a table has it that the loss is tied to; then only the rows that
// tokens name are touched. The product and the sums are taken in 32 bits and
// rounded once.
//
// The backward sorts the tokens by id, stably (by counting or by digits: whole
// numbers, no order of atomics in it), and adds up runs of equal ids in the order of the
// tokens, so the result is the same every time. A frequent id's run is long: the
// sorted tokens are cut into chunks of equal length, and a run that crosses a
// cut leaves fp32 sums in the workspace that a last kernel adds in order.
// All of it is bound by HBM.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "host.h"
#include "ptx.cuh"
#include "step/launch.cuh"
#include "step/vec.cuh"

namespace tpce {
namespace {

using namespace step;

constexpr int64_t kMaxTokens = int64_t{1} << 28, kMaxTable = int64_t{1} << 30;
constexpr int kThreads = 256;

// ------------------------------------------------------------------ forward
// `lanes` threads of a block share a piece of lanes * U vectors of a token's row, whose
// loads are under way together (16,384 rows of 8192 bf16: 61 us with four vectors a thread where
// ids are as frequent as words, 6.3 TB/s of rows read and written, 94% of a copy's rate; one
// vector a thread is 6% slower).
template <typename T, int U>
__global__ void __launch_bounds__(kThreads)
    embed_forward_kernel(const T *E, const int32_t *ids, int64_t tokens, int64_t v_valid, int vectors, int lanes,
                         int parts, float scale, T *__restrict__ X, uint32_t *err) {
    const int64_t piece = static_cast<int64_t>(blockIdx.x) * (kThreads / lanes) + threadIdx.x / lanes;
    const int64_t t = piece / parts;
    const int c0 = static_cast<int>(piece - t * parts) * lanes * U + (threadIdx.x & (lanes - 1));
    grid_begin();
    if (t >= tokens) return;
    const int32_t id = ids[t];
    const bool known = id >= 0 && id < v_valid;
    if (!known && id != -1) ptx::record_error(err, kErrInvalid | (5u << 8));
    Raw8<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        zero8(r[u]);
        if (known && c0 + u * lanes < vectors)
            r[u] = load8(E + (static_cast<int64_t>(id) * vectors + c0 + u * lanes) * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (c0 + u * lanes >= vectors) continue;
        if (known) {
            float v[8];
            unpack8(r[u], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) mul2(v[2 * i], v[2 * i + 1], scale, scale);
            pack8(v, r[u]);
        }
        store8(X + (t * vectors + c0 + u * lanes) * 8, r[u]);
    }
}

// ------------------------------------------------------------------ the sort
// Passes over up to ten bits, the lowest first. A block takes a chunk of the tokens,
// each of its warps a contiguous run of the chunk. Up to kClusterTokens tokens are
// sorted by the blocks of one cluster in one launch, which read each other's counts of
// digits (16,384 tokens over 129,024 ids: two launches a pass took 22 us, this one
// takes 18); for more the blocks' counts are one launch and their places the next.
// Up to kRankTokens tokens are not sorted by digits: a token's place is the number of those
// before it in the order, which all SMs count at once (embed_rank_kernel).
constexpr int kClusterThreads = 1024;
// What the SMs that do not sort zero meanwhile, of a table that is written whole: about what the sort's
// time is enough for. A cluster's sort: 8192 tokens of 4096 and 51,200 rows 92 us a call, with 48 MB 96, with
// 192 MB 98. By counting, which is shorter: 999 tokens of 1000 fp32 and 30,001 rows 25.5 us, with none 31.9, with
// 24 MB 28.7, with 96 MB 25.5; 4096 of 2048 and 131,072 rows 95, 102, 99 and 91.
constexpr int64_t kZeroed = 96 << 20, kRankZeroed = 48 << 20;
constexpr int64_t kRankTokens = 4096;
constexpr int kMaxBins = 1024, kCluster = 8;
constexpr int kRankEach = 4, kRankChunk = kRankEach * kThreads / 32;  // tokens of a warp, of a block
constexpr int64_t kSortChunk = 1024, kSortBlocks = 256, kClusterTokens = 65536;

struct SortSplit {
    int64_t chunk;
    int blocks, passes, bits;  // bits of a pass
    bool rank;                 // `blocks` blocks that count
    bool cluster;              // one of `blocks` blocks
};
inline SortSplit sort_split(int64_t tokens, int64_t v_pad) {
    SortSplit sp{};
    int all = 1;  // of the keys 0 .. v_pad; v_pad is that of a token without a row
    while ((int64_t{1} << all) <= v_pad) ++all;
    sp.passes = (all + 9) / 10;
    sp.bits = (all + sp.passes - 1) / sp.passes;
    sp.rank = tokens <= kRankTokens && v_pad < (1 << 24);  // keys up to v_pad, and one more, as fp32
    sp.cluster = !sp.rank && tokens <= kClusterTokens;
    sp.chunk = std::max<int64_t>(kSortChunk, (tokens + kSortBlocks - 1) / kSortBlocks);
    if (sp.rank) {
        sp.chunk = kRankChunk;
        sp.blocks = static_cast<int>((tokens + kRankChunk - 1) / kRankChunk);
        sp.passes = 0;  // the result lies in key[0], token[0]
    } else if (sp.cluster) {
        sp.blocks = 1;
        while (sp.blocks < kCluster && sp.blocks * kSortChunk < tokens) sp.blocks *= 2;
        sp.chunk = (tokens + sp.blocks - 1) / sp.blocks;
    } else {
        sp.blocks = static_cast<int>((tokens + sp.chunk - 1) / sp.chunk);
    }
    return sp;
}

// The key of a token in the first pass, where ids are the keys.
__device__ __forceinline__ int32_t key_of(int32_t id, int32_t v_valid, int32_t v_pad, uint32_t *err) {
    if (id >= 0 && id < v_valid) return id;
    if (id != -1) ptx::record_error(err, kErrInvalid | (5u << 8));
    return v_pad;
}

__global__ void __launch_bounds__(kThreads)
    embed_count_kernel(const int32_t *keys, int64_t n, int64_t chunk, int shift, int bins, bool ids, int32_t v_valid,
                       int32_t v_pad, uint32_t *__restrict__ counts) {
    extern __shared__ uint32_t count[];  // [bins]
    for (int b = threadIdx.x; b < bins; b += kThreads) count[b] = 0u;
    grid_begin();
    __syncthreads();
    const int64_t first = blockIdx.x * chunk, last = min(n, first + chunk);
#pragma unroll 4
    for (int64_t i = first + threadIdx.x; i < last; i += kThreads) {
        const int32_t k = ids ? key_of(keys[i], v_valid, v_pad, nullptr) : keys[i];
        atomicAdd(&count[(k >> shift) & (bins - 1)], 1u);  // whole numbers: any order gives the same
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads)
        counts[static_cast<int64_t>(blockIdx.x) * bins + b] = count[b];
}

__device__ __forceinline__ uint32_t load_cluster(uint32_t addr) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
    return x;
}

// One pass of block `block` of `blocks`: from keys (of the tokens from[i], or of i itself) to key_out and
// token_out. counts: of all blocks' digits, from the launch before; NULL: the blocks are a cluster (or one).
// C holds a warp's counts and places; a cluster's tokens fit 16 bits.
template <int THREADS, typename C>
__host__ __device__ constexpr size_t sort_smem(int bits) {
    return (size_t{THREADS / 32} * sizeof(C) + 3 * sizeof(uint32_t)) << bits;
}
template <int THREADS, typename C>
__device__ void sort_pass(const int32_t *keys, const int32_t *from, int64_t n, int64_t chunk, int block, int blocks,
                          int shift, int bits, const uint32_t *counts, int32_t v_valid, int32_t v_pad,
                          int32_t *key_out, int32_t *token_out, uint32_t *smem, uint32_t *scan, uint32_t *err) {
    constexpr int kWarps = THREADS / 32, kInWord = 4 / sizeof(C);
    const int bins = 1 << bits;
    uint32_t *all = smem;                        // [bins] of all blocks
    uint32_t *below = all + bins;                // [bins] of the blocks before
    uint32_t *total = below + bins;              // [bins] of this block
    uint32_t *words = total + bins;              // [kWarps][bins], then the next place of each warp's digits
    C *count = reinterpret_cast<C *>(words);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool ids = from == nullptr;
    for (int b = threadIdx.x; b < 2 * bins; b += THREADS) smem[b] = 0u;
    for (int b = threadIdx.x; b < kWarps * bins / kInWord; b += THREADS) words[b] = 0u;
    __syncthreads();
    if (counts) {
        int width = 1;
        while (width < bins && width < THREADS) width *= 2;
        const int parts = THREADS / width, part = threadIdx.x / width;
        for (int b = threadIdx.x & (width - 1); b < bins; b += width) {
            uint32_t sum = 0u, before = 0u;
#pragma unroll 8
            for (int q = part; q < blocks; q += parts) {
                const uint32_t c = counts[static_cast<int64_t>(q) * bins + b];
                sum += c;
                before += q < block ? c : 0u;
            }
            atomicAdd(&all[b], sum);
            atomicAdd(&below[b], before);
        }
    }
    const int64_t begin = min(n, block * chunk), end = min(n, begin + chunk);
    const int64_t run = ((end - begin + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int64_t first = min(end, begin + warp * run), last = min(end, first + run);
    C *mine = count + warp * bins;
    auto digit = [&](int32_t k) { return (k >> shift) & (bins - 1); };
#pragma unroll 4
    for (int64_t i = first + lane; i < last; i += 32) {
        const int at = warp * bins + digit(ids ? key_of(keys[i], v_valid, v_pad, err) : keys[i]);
        atomicAdd(&words[at / kInWord], 1u << (at % kInWord * (8 * sizeof(C) % 32)));
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += THREADS) {
        uint32_t sum = 0u;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
            const uint32_t c = count[q * bins + b];
            count[q * bins + b] = static_cast<C>(sum);
            sum += c;
        }
        total[b] = sum;
        if (!counts && blocks == 1) all[b] = sum;
    }
    __syncthreads();
    if (!counts && blocks > 1) {
        ptx::cluster_sync();
        for (int b = threadIdx.x; b < bins; b += THREADS) {
            uint32_t sum = 0u, before = 0u;
            const uint32_t at = ptx::smem_u32(&total[b]);
            uint32_t c[kCluster];
#pragma unroll
            for (int q = 0; q < kCluster; ++q) c[q] = q < blocks ? load_cluster(ptx::mapa_shared(at, q)) : 0u;
#pragma unroll
            for (int q = 0; q < kCluster; ++q) {
                sum += c[q];
                before += q < block ? c[q] : 0u;
            }
            all[b] = sum;
            below[b] = before;
        }
        __syncthreads();
    }
    // first places: a scan over the digits, adjacent ones a thread
    constexpr int kEach = kMaxBins / THREADS;
    uint32_t own[kEach], sum = 0u;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int b = threadIdx.x * kEach + u;
        own[u] = b < bins ? all[b] : 0u;
        sum += own[u];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    uint32_t at = incl - sum;
    for (int q = 0; q < warp; ++q) at += scan[q];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int b = threadIdx.x * kEach + u;
        if (b < bins) {
            const uint32_t place = at + below[b];
            at += own[u];
#pragma unroll 8
            for (int q = 0; q < kWarps; ++q) count[q * bins + b] = static_cast<C>(count[q * bins + b] + place);
        }
    }
    __syncthreads();
    constexpr int kBatch = 4;
    for (int64_t i0 = first; i0 < last; i0 += 32 * kBatch) {
        int32_t k[kBatch], t[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32 + lane;
            k[u] = i < last ? (ids ? key_of(keys[i], v_valid, v_pad, nullptr) : keys[i]) : 0;
            t[u] = i >= last ? 0 : ids ? static_cast<int32_t>(i) : from[i];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i0 + u * 32 >= last) break;
            const bool there = i0 + u * 32 + lane < last;
            const int d = there ? digit(k[u]) : bins;
            const uint32_t same = same_value(d, bits + 1);
            const uint32_t before = __popc(same & ((1u << lane) - 1u));
            uint32_t p = UINT_MAX;
            if (there) p = mine[d] + before;
            __syncwarp();
            if (there && before == 0u) mine[d] = static_cast<C>(mine[d] + __popc(same));
            __syncwarp();
            // an id that changes while it is sorted must lead nowhere
            if (there && p < n) {
                key_out[p] = k[u];
                token_out[p] = t[u];
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads)
    embed_place_kernel(const int32_t *keys, const int32_t *from, int64_t n, int64_t chunk, int shift, int bits,
                       const uint32_t *counts, int32_t v_valid, int32_t v_pad, int32_t *key_out, int32_t *token_out,
                       uint32_t *err) {
    extern __shared__ uint32_t smem[];
    __shared__ uint32_t scan[kThreads / 32];
    grid_begin();
    sort_pass<kThreads, uint32_t>(keys, from, n, chunk, blockIdx.x, gridDim.x, shift, bits, counts, v_valid, v_pad,
                                  key_out, token_out, smem, scan, err);
}

// Place of each of a block's tokens, kRankEach a warp: how many keys are smaller, or equal and of
// an earlier token. The keys lie in shared memory as fp32, so that a comparison and its sum
// are a subtraction that saturates at 0 and 1 and an addition; a key that is read is compared
// with all of the warp's (calls added to a table: 999 tokens of 1000 18.3 us with digits, 9.4
// so; 4096 of 1024 25.5 and 20.8; 8192 27 and 31, since all pairs are compared). The blocks
// after the first `blocks` write zeros as in embed_sort_kernel.
__global__ void __launch_bounds__(kThreads)
    embed_rank_kernel(const int32_t *ids, int n, int blocks, int32_t v_valid, int32_t v_pad, int32_t *key,
                      int32_t *token, uint4 *table, int64_t vectors, uint32_t *err) {
    extern __shared__ float4 keys4[];  // of n tokens, rounded up to whole blocks
    grid_begin();
    if (static_cast<int>(blockIdx.x) >= blocks) {
        const int64_t stride = static_cast<int64_t>(gridDim.x - blocks) * kThreads;
        for (int64_t i = static_cast<int64_t>(blockIdx.x - blocks) * kThreads + threadIdx.x; i < vectors; i += stride)
            table[i] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    float *keys = reinterpret_cast<float *>(keys4);
    const int all = blocks * kRankChunk, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kBatch = 16;  // loads under way together
    for (int i0 = threadIdx.x; i0 < all; i0 += kBatch * kThreads) {
        int32_t id[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) id[u] = i0 + u * kThreads < n ? ids[i0 + u * kThreads] : 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kThreads;
            if (i >= all) break;
            // those past the end are greater than any and come after all
            uint32_t *const report = i / kRankChunk == static_cast<int>(blockIdx.x) ? err : nullptr;
            keys[i] = i < n ? static_cast<float>(key_of(id[u], v_valid, v_pad, report)) : INFINITY;
        }
    }
    __syncthreads();
    const int t0 = blockIdx.x * kRankChunk + warp * kRankEach;  // the warp's first token
    float mine[kRankEach], before[kRankEach];
#pragma unroll
    for (int u = 0; u < kRankEach; ++u) {
        mine[u] = keys[t0 + u];
        before[u] = 0.0f;
    }
    // all tokens before the warp's count if not greater, all behind them if smaller
#pragma unroll 2
    for (int j = lane; j < t0 / 4; j += 32) {
        const float4 k = keys4[j];
#pragma unroll
        for (int u = 0; u < kRankEach; ++u) {
            const float least = mine[u] + 1.0f;
            before[u] += (__saturatef(least - k.x) + __saturatef(least - k.y)) +
                         (__saturatef(least - k.z) + __saturatef(least - k.w));
        }
    }
#pragma unroll 2
    for (int j = (t0 + kRankEach) / 4 + lane; j < all / 4; j += 32) {
        const float4 k = keys4[j];
#pragma unroll
        for (int u = 0; u < kRankEach; ++u)
            before[u] += (__saturatef(mine[u] - k.x) + __saturatef(mine[u] - k.y)) +
                         (__saturatef(mine[u] - k.z) + __saturatef(mine[u] - k.w));
    }
#pragma unroll
    for (int u = 0; u < kRankEach; ++u) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) before[u] += __shfl_xor_sync(0xffffffffu, before[u], d);
#pragma unroll
        for (int w = 0; w < kRankEach; ++w)
            if (w != u) before[u] += mine[w] < mine[u] || (mine[w] == mine[u] && w < u) ? 1.0f : 0.0f;
        if (lane == u && t0 + u < n) {
            const int place = static_cast<int>(before[u]);
            key[place] = static_cast<int32_t>(mine[u]);
            token[place] = t0 + u;
        }
    }
}

// All passes of a cluster's tokens; the last one ends in key[1], token[1] (odd passes) or key[0], token[0].
// The blocks after the first `blocks`, if there are any, write zeros to the table's first rows meanwhile, as many
// as the sort leaves time for (kZeroed bytes), whether tokens name them or not: that is not known yet.
struct SortBuffers {
    int32_t *key[2], *token[2];
};
__global__ void __launch_bounds__(kClusterThreads)
    embed_sort_kernel(const int32_t *ids, int64_t n, int64_t chunk, int blocks, int passes, int bits, int32_t v_valid,
                      int32_t v_pad, SortBuffers buf, uint4 *table, int64_t vectors, uint32_t *err) {
    extern __shared__ uint32_t smem[];
    __shared__ uint32_t scan[kClusterThreads / 32];
    grid_begin();
    if (static_cast<int>(blockIdx.x) >= blocks) {
        const int64_t stride = static_cast<int64_t>(gridDim.x - blocks) * kClusterThreads;
        for (int64_t i = static_cast<int64_t>(blockIdx.x - blocks) * kClusterThreads + threadIdx.x; i < vectors;
             i += stride)
            table[i] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    for (int p = 0; p < passes; ++p) {
        const int to = (p + 1) & 1;
        sort_pass<kClusterThreads, uint16_t>(p ? buf.key[to ^ 1] : ids, p ? buf.token[to ^ 1] : nullptr, n, chunk,
                                             blockIdx.x, blocks, p * bits, bits, nullptr, v_valid, v_pad, buf.key[to],
                                             buf.token[to], smem, scan, err);
        // the next pass reads what all blocks have written, and writes counts that they have read
        if (blocks > 1)
            ptx::cluster_sync();
        else
            __syncthreads();
    }
}

// ------------------------------------------------------------------ the sums
// Chunks of sorted tokens. A chunk's first run may have begun before it, and its
// last may go on after it: their sums go to the workspace, the first's to row 2 c,
// the last's to row 2 c + 1 (a run that does both is the chunk's only one: row 2 c).
struct SumSplit {
    int64_t chunk;
    int chunks, lanes;  // threads of a row's piece of lanes vectors of eight columns
    int parts;          // pieces of a row
};
inline SumSplit sum_split(int64_t tokens, int64_t h) {
    SumSplit sp{};
    // shorter chains where there are few (999 tokens of 1000 bf16: 9.4 us a call, with sixteen 10.4;
    // one id for all 18.6 and 14.8, its run crosses more cuts)
    sp.chunk = std::max<int64_t>(tokens <= 2048 ? 8 : 16, (tokens + 1023) / 1024);
    sp.chunks = static_cast<int>((tokens + sp.chunk - 1) / sp.chunk);
    const int64_t vectors = h / 8;
    sp.lanes = 8;
    while (sp.lanes < kThreads && sp.lanes < vectors) sp.lanes *= 2;
    sp.parts = static_cast<int>((vectors + sp.lanes - 1) / sp.lanes);
    return sp;
}

template <typename T>
__device__ __forceinline__ void finish_row(const float (&sum)[8], const Raw8<T> &old, bool add, float scale,
                                           T *__restrict__ to) {
    float v[8] = {};
    if (add) unpack8(old, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = add ? fmaf(sum[i], scale, v[i]) : sum[i] * scale;
    Raw8<T> r;
    pack8(v, r);
    store8(to, r);
}

// Whether a row is among the sorted keys.
__device__ __forceinline__ bool among(const int32_t *key, int64_t n, int32_t v) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (key[mid] < v)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < n && key[lo] == v;
}

// Rows of a block that fills: 128 KB of them, each looked up by one thread (8192 tokens,
// 262,144 rows of 1024 bf16: 104 us; 32 rows a block, one after the other, 138; 64 KB, 118;
// a million rows of 64: 41, 126 and 43).
inline int fill_rows(size_t row) {
    return static_cast<int>(std::clamp<size_t>((size_t{128} << 10) / row, 32, kThreads));
}

// The first `fill` blocks write zeros to the rows from `zeroed` on that no token names,
// fill_rows of them each; the others add up chunks. Loads are issued four tokens at a time, with
// the old row where a run ends, and the next four's ids with them (2 to 4% less). Bound by HBM:
// 16,384 tokens of 8192 bf16 into a tied table of 129,024 rows (494 MB) in 90 us of the call's
// 120, 70% of DRAM's peak by its counters; with two blocks an SM instead of three 104.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
    embed_sum_kernel(const T *dX, const int32_t *key, const int32_t *token, int64_t n, int64_t v_pad, int vectors,
                     SumSplit sp, unsigned fill, int fill_rows, int64_t zeroed, bool add, float scale,
                     float *__restrict__ partial, T *dE) {
    grid_begin();
    if (blockIdx.x < fill) {
        __shared__ bool named[kThreads];
        const int64_t v0 = zeroed + static_cast<int64_t>(blockIdx.x) * fill_rows;
        if (static_cast<int>(threadIdx.x) < fill_rows) {
            const int64_t v = v0 + threadIdx.x;
            named[threadIdx.x] = v >= v_pad || among(key, n, static_cast<int32_t>(v));
        }
        __syncthreads();
        Raw8<T> zero;
        zero8(zero);
        for (int64_t i = threadIdx.x; i < static_cast<int64_t>(fill_rows) * vectors; i += kThreads) {
            const int r = static_cast<int>(i / vectors);
            if (!named[r]) store8(dE + (v0 * vectors + i) * 8, zero);
        }
        return;
    }
    const int64_t piece = static_cast<int64_t>(blockIdx.x - fill) * (kThreads / sp.lanes) + threadIdx.x / sp.lanes;
    const int64_t c = piece / sp.parts;
    const int at = static_cast<int>(piece - c * sp.parts) * sp.lanes + (threadIdx.x & (sp.lanes - 1));
    if (c >= sp.chunks || at >= vectors) return;
    const int64_t p0 = c * sp.chunk, p1 = min(n, p0 + sp.chunk);
    int32_t now = key[p0];
    bool open = p0 > 0 && key[p0 - 1] == now;  // the run at hand began in a chunk before
    float sum[8] = {};
    constexpr int kBatch = 4;
    int32_t next_k[kBatch + 1], next_t[kBatch];
    auto fetch = [&](int64_t p) {
#pragma unroll
        for (int u = 0; u <= kBatch; ++u) next_k[u] = p + u < n ? key[p + u] : -1;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) next_t[u] = p + u < p1 ? token[p + u] : -1;
    };
    fetch(p0);
    for (int64_t p = p0; p < p1 && static_cast<uint32_t>(now) < v_pad; p += kBatch) {
        int32_t k[kBatch + 1];
        Raw8<T> x[kBatch], old[kBatch];
        bool there[kBatch];
#pragma unroll
        for (int u = 0; u <= kBatch; ++u) k[u] = next_k[u];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            // places that the sort has not written (ids that changed under it) lead nowhere
            const int32_t t = next_t[u];
            there[u] = static_cast<uint32_t>(k[u]) < v_pad && static_cast<uint32_t>(t) < n;
            if (there[u]) x[u] = load8(dX + (static_cast<int64_t>(t) * vectors + at) * 8);
            if (add && there[u] && k[u + 1] != k[u])
                old[u] = load8(dE + (static_cast<int64_t>(k[u]) * vectors + at) * 8);
        }
        fetch(p + kBatch);  // during this batch's rows
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (!there[u]) {
                now = static_cast<int32_t>(v_pad);
                break;
            }
            float v[8];
            unpack8(x[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += v[i];
            const bool ends = k[u + 1] != k[u], cut = p + u + 1 == p1;
            if (!ends && !cut) continue;
            if (ends && !open) {
                finish_row(sum, old[u], add, scale, dE + (static_cast<int64_t>(k[u]) * vectors + at) * 8);
            } else {
                float4 *to = reinterpret_cast<float4 *>(partial + ((2 * c + (open ? 0 : 1)) * vectors + at) * 8);
                to[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
                to[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
            }
            open = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
        }
    }
}

// The runs that cross a cut, by the chunk that they begin in: a block looks at
// kJoinChunks chunks, a lane at one, and adds up the runs that it finds for its columns.
// (A warp for each chunk and 256 columns took 52 us for 1024 chunks of 8192 columns,
// nearly all of it warps that found nothing; this takes 13 to 22.)
constexpr int kJoinChunks = 8;
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    embed_join_kernel(const int32_t *key, int64_t n, int64_t v_pad, int vectors, SumSplit sp, unsigned groups,
                      bool add, float scale, const float *partial, T *dE) {
    const int lane = threadIdx.x & 31;
    const int at = static_cast<int>(blockIdx.x / groups) * kThreads + threadIdx.x;
    grid_begin();
    const int64_t c0 = static_cast<int64_t>(blockIdx.x % groups) * kJoinChunks, mine = c0 + lane;
    int32_t k = -1;
    if (lane < kJoinChunks && mine < sp.chunks - 1) {  // not the last chunk: p1 < n
        const int64_t p0 = mine * sp.chunk, p1 = p0 + sp.chunk;
        const int32_t next = key[p1], last = key[p1 - 1], first = key[p0], before = p0 > 0 ? key[p0 - 1] : -1;
        if (static_cast<uint32_t>(next) < v_pad && last == next && !(first == next && before == next)) k = next;
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, k >= 0); left != 0; left &= left - 1) {
        const int who = __ffs(left) - 1;
        const int32_t id = __shfl_sync(0xffffffffu, k, who);
        const int64_t c = c0 + who;
        const bool there = at < vectors;
        T *row = dE + (static_cast<int64_t>(id) * vectors + at) * 8;
        Raw8<T> old;
        zero8(old);
        float sum[8] = {};
        if (there) {
            if (add) old = load8(row);
            load8f(partial + ((2 * c + 1) * vectors + at) * 8, sum);
        }
        // the chunks after it that begin with the run, kBatch at a time
        constexpr int kBatch = 8;
        for (int64_t m = c + 1; m < sp.chunks; m += 32) {
            const bool on = m + lane < sp.chunks && key[(m + lane) * sp.chunk] == id;
            const uint32_t which = __ballot_sync(0xffffffffu, on);
            const int count = which == 0xffffffffu ? 32 : __ffs(~which) - 1;
            for (int j0 = 0; j0 < count && there; j0 += kBatch) {
                float v[kBatch][8];
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (j0 + j < count) load8f(partial + (2 * (m + j0 + j) * vectors + at) * 8, v[j]);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (j0 + j >= count) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] += v[j][i];
                }
            }
            if (count < 32) break;
        }
        if (there) finish_row(sum, old, add, scale, row);
    }
}

// ------------------------------------------------------------------ host
tpce_status check_shape(const char *name, int64_t T, int64_t h, int64_t v_pad, int64_t v_valid, float scale,
                        int dtype) {
    if (dtype != TPCE_BF16 && dtype != TPCE_F32) return fail(TPCE_ERR_INVALID, "%s: dtype %d", name, dtype);
    if (!std::isfinite(scale)) return fail(TPCE_ERR_INVALID, "%s: scale is not finite", name);
    if (T < 0 || T > kMaxTokens || h < 8 || h % 8 != 0 || h > (1 << 20) || v_pad < 1 || v_pad > kMaxTable ||
        v_valid < 1 || v_valid > v_pad || T > (int64_t{1} << 40) / h || v_pad > (int64_t{1} << 40) / h)
        return fail(TPCE_ERR_SHAPE,
                    "%s: T = %lld (up to 2^28), h = %lld (a multiple of 8 up to 2^20), v_pad = %lld (up to 2^30), "
                    "v_valid = %lld (1 .. v_pad), T h and v_pad h up to 2^40",
                    name, static_cast<long long>(T), static_cast<long long>(h), static_cast<long long>(v_pad),
                    static_cast<long long>(v_valid));
    return TPCE_OK;
}

tpce_status check_pointers(const char *name, std::initializer_list<const void *> need) {
    for (const void *p : need)
        if (!p) return fail(TPCE_ERR_INVALID, "%s: null pointer", name);
    for (const void *p : need)
        if (!aligned16(p)) return fail(TPCE_ERR_ALIGN, "%s: a pointer is not 16-byte aligned", name);
    return TPCE_OK;
}

inline bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a_bytes && b_bytes && x < y + b_bytes && y < x + a_bytes;
}

inline size_t bytes_of(int64_t rows, int64_t h, int dtype) {
    return static_cast<size_t>(rows) * static_cast<size_t>(h) * (dtype == TPCE_BF16 ? 2 : 4);
}

// The workspace: keys and tokens twice, the blocks' counts, the cut runs' sums.
struct Layout {
    size_t each, counts, partial, total;
};
inline Layout layout_of(int64_t T, int64_t h, int64_t v_pad) {
    const SortSplit so = sort_split(T, v_pad);
    const SumSplit su = sum_split(T, h);
    Layout l{};
    l.each = round_up(static_cast<size_t>(T) * sizeof(int32_t), 256);
    l.counts = 4 * l.each;
    l.partial = l.counts +
                round_up(!so.cluster && !so.rank ? static_cast<size_t>(so.blocks) * (size_t{4} << so.bits) : 0, 256);
    l.total = l.partial + (su.chunks > 1 ? 2 * static_cast<size_t>(su.chunks) * static_cast<size_t>(h) * 4 : 0);
    return l;
}

template <typename T>
tpce_status embed_forward(const int32_t *ids, const void *E, int64_t tokens, int64_t h, int64_t v_valid, float scale,
                          void *X, cudaStream_t s) {
    const int vectors = static_cast<int>(h / 8);
    int lanes = 8;
    while (lanes < kThreads && lanes * 2 < vectors) lanes *= 2;
    // four vectors a thread (16,384 rows of 8192 bf16, all ids equally frequent: 79 us, with two 81), one where
    // that would leave SMs idle
    const bool few = tokens * vectors < int64_t{4} * kThreads * 2 * num_sms();
    const int each = lanes * (few ? 1 : 4);
    const int parts = (vectors + each - 1) / each;
    const unsigned blocks = static_cast<unsigned>((tokens * parts + kThreads / lanes - 1) / (kThreads / lanes));
    KernelTimer timer("embed_forward", s);
    auto go = [&](auto kernel) {
        return launch(kernel, blocks, kThreads, 0, s, static_cast<const T *>(E), ids, tokens, v_valid, vectors, lanes,
                      parts, scale, static_cast<T *>(X), device_error_word());
    };
    const cudaError_t e = few ? go(embed_forward_kernel<T, 1>) : go(embed_forward_kernel<T, 4>);
    return e == cudaSuccess ? check_launch("embed_forward", s) : fail_cuda(e, "embed_forward");
}

// table_bytes of the table are zeroed meanwhile, by the two sorts of one launch; 0 for the third
tpce_status embed_sort(const int32_t *ids, int64_t T, int64_t v_pad, int64_t v_valid, const SortSplit &sp,
                       const SortBuffers &buf, uint32_t *counts, void *table, size_t table_bytes, cudaStream_t s) {
    const int32_t valid = static_cast<int32_t>(v_valid), pad = static_cast<int32_t>(v_pad);
    KernelTimer timer("embed_sort", s);
    if (sp.rank) {
        const int64_t vectors = static_cast<int64_t>(table_bytes / 16);
        const int64_t fill = std::min<int64_t>((vectors + 4 * kThreads - 1) / (4 * kThreads), int64_t{8} * num_sms());
        const cudaError_t e =
            launch(embed_rank_kernel, static_cast<unsigned>(sp.blocks + fill), kThreads,
                   static_cast<size_t>(sp.blocks) * kRankChunk * sizeof(float), s, ids, static_cast<int>(T), sp.blocks,
                   valid, pad, buf.key[0], buf.token[0], static_cast<uint4 *>(table), vectors, device_error_word());
        return e == cudaSuccess ? check_launch("embed_sort", s) : fail_cuda(e, "embed_sort");
    }
    if (sp.cluster) {
        static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may have more than 48 KB
        const size_t smem = sort_smem<kClusterThreads, uint16_t>(sp.bits);
        int dev = 0;
        cudaError_t e = taken(cudaGetDevice(&dev));
        const uint64_t bit = uint64_t{1} << (dev & 63);
        if (e == cudaSuccess && !(allowed.load() & bit)) {
            e = taken(cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(sort_smem<kClusterThreads, uint16_t>(10))));
            if (e == cudaSuccess) allowed.fetch_or(bit);
        }
        if (e != cudaSuccess) return fail_cuda(e, "embed_sort");
        // a block an SM zeroes the table, or fewer
        const int64_t vectors = static_cast<int64_t>(table_bytes / 16);
        const int64_t fill = std::min<int64_t>((vectors + 4 * kClusterThreads - 1) / (4 * kClusterThreads),
                                               int64_t{2} * num_sms());
        const unsigned blocks = static_cast<unsigned>((sp.blocks + fill + sp.blocks - 1) / sp.blocks * sp.blocks);
        e = launch_clusters(sp.blocks, embed_sort_kernel, blocks, kClusterThreads, smem, s, ids, T, sp.chunk, sp.blocks,
                            sp.passes, sp.bits, valid, pad, buf, static_cast<uint4 *>(table), vectors,
                            device_error_word());
        return e == cudaSuccess ? check_launch("embed_sort", s) : fail_cuda(e, "embed_sort");
    }
    for (int p = 0; p < sp.passes; ++p) {
        const int to = (p + 1) & 1;
        const int32_t *keys = p ? buf.key[to ^ 1] : ids, *from = p ? buf.token[to ^ 1] : nullptr;
        cudaError_t e = launch(embed_count_kernel, sp.blocks, kThreads, size_t{4} << sp.bits, s, keys, T, sp.chunk,
                               p * sp.bits, 1 << sp.bits, p == 0, valid, pad, counts);
        if (e != cudaSuccess) return fail_cuda(e, "embed_count");
        tpce_status st = check_launch("embed_count", s);
        if (st != TPCE_OK) return st;
        e = launch(embed_place_kernel, sp.blocks, kThreads, sort_smem<kThreads, uint32_t>(sp.bits), s, keys, from, T,
                   sp.chunk, p * sp.bits, sp.bits, counts, valid, pad, buf.key[to], buf.token[to],
                   device_error_word());
        if (e != cudaSuccess) return fail_cuda(e, "embed_place");
        if ((st = check_launch("embed_place", s)) != TPCE_OK) return st;
    }
    return TPCE_OK;
}

template <typename T>
tpce_status embed_sums(const void *dX, int64_t tokens, int64_t h, int64_t v_pad, const int32_t *key,
                       const int32_t *token, float scale, bool add, int64_t zeroed, float *partial, void *dE,
                       cudaStream_t s) {
    const SumSplit sp = sum_split(tokens, h);
    const int vectors = static_cast<int>(h / 8);
    const int64_t of_block = kThreads / sp.lanes;
    const int64_t blocks = (static_cast<int64_t>(sp.chunks) * sp.parts + of_block - 1) / of_block;
    const int rows = fill_rows(static_cast<size_t>(h) * sizeof(T));
    const unsigned fill = add ? 0u : static_cast<unsigned>((v_pad - zeroed + rows - 1) / rows);
    {
        KernelTimer timer("embed_sum", s);
        const cudaError_t e =
            launch(embed_sum_kernel<T>, fill + static_cast<unsigned>(blocks), kThreads, 0, s,
                   static_cast<const T *>(dX), key, token, tokens, v_pad, vectors, sp, fill, rows, zeroed, add, scale,
                   partial, static_cast<T *>(dE));
        if (e != cudaSuccess) return fail_cuda(e, "embed_sum");
        const tpce_status st = check_launch("embed_sum", s);
        if (st != TPCE_OK || sp.chunks == 1) return st;
    }
    KernelTimer timer("embed_join", s);
    const unsigned groups = static_cast<unsigned>((sp.chunks + kJoinChunks - 1) / kJoinChunks);
    const unsigned columns = static_cast<unsigned>((vectors + kThreads - 1) / kThreads);
    const cudaError_t e = launch(embed_join_kernel<T>, groups * columns, kThreads, 0, s, key, tokens, v_pad, vectors,
                                 sp, groups, add, scale, partial, static_cast<T *>(dE));
    return e == cudaSuccess ? check_launch("embed_join", s) : fail_cuda(e, "embed_join");
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" tpce_status tp_embedding_forward(const int32_t *ids, const void *E, int64_t T, int64_t h, int64_t v_pad,
                                            int64_t v_valid, float scale, int dtype, void *X, void *stream) {
    tpce_status st = check_shape("tp_embedding_forward", T, h, v_pad, v_valid, scale, dtype);
    if (st != TPCE_OK || T == 0) return st;
    if ((st = check_pointers("tp_embedding_forward", {ids, E, X})) != TPCE_OK) return st;
    const size_t rows = bytes_of(T, h, dtype);
    if (overlap(X, rows, E, bytes_of(v_pad, h, dtype)) || overlap(X, rows, ids, static_cast<size_t>(T) * 4))
        return fail(TPCE_ERR_INVALID, "tp_embedding_forward: X overlaps E or ids");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == TPCE_BF16 ? embed_forward<__nv_bfloat16>(ids, E, T, h, v_valid, scale, X, s)
                              : embed_forward<float>(ids, E, T, h, v_valid, scale, X, s);
}

extern "C" size_t tpce_embedding_workspace_bytes(int64_t T, int64_t h, int64_t v_pad) {
    if (check_shape("embedding", T, h, v_pad, 1, 1.0f, TPCE_BF16) != TPCE_OK || T == 0) return 0;
    return layout_of(T, h, v_pad).total;
}

extern "C" tpce_status tp_embedding_backward(const void *dX, const int32_t *ids, int64_t T, int64_t h, int64_t v_pad,
                                             int64_t v_valid, float scale, int dtype, int accumulate, void *dE,
                                             void *ws, size_t ws_bytes, void *stream) {
    const char *name = "tp_embedding_backward";
    tpce_status st = check_shape(name, T, h, v_pad, v_valid, scale, dtype);
    if (st != TPCE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t table = bytes_of(v_pad, h, dtype);
    if (T == 0) {
        if (accumulate) return TPCE_OK;
        if ((st = check_pointers(name, {dE})) != TPCE_OK) return st;
        const cudaError_t e = taken(cudaMemsetAsync(dE, 0, table, s));
        return e == cudaSuccess ? TPCE_OK : fail_cuda(e, name);
    }
    if ((st = check_pointers(name, {dX, ids, dE})) != TPCE_OK) return st;
    const Layout l = layout_of(T, h, v_pad);
    if (!ws || ws_bytes < l.total)
        return fail(TPCE_ERR_WORKSPACE, "%s: %zu bytes of workspace needed, %zu given", name, l.total,
                    ws ? ws_bytes : size_t{0});
    if (!aligned16(ws)) return fail(TPCE_ERR_ALIGN, "%s: a pointer is not 16-byte aligned", name);
    const std::pair<const void *, size_t> parts[] = {
        {dX, bytes_of(T, h, dtype)}, {ids, static_cast<size_t>(T) * 4}, {dE, table}, {ws, l.total}};
    for (const auto &a : parts)
        for (const auto &b : parts)
            // dX and ids are only read
            if (&a < &b && &b > &parts[1] && overlap(a.first, a.second, b.first, b.second))
                return fail(TPCE_ERR_INVALID, "%s: dE or ws overlaps another argument", name);
    char *base = static_cast<char *>(ws);
    SortBuffers buf;
    for (int i = 0; i < 2; ++i) {
        buf.key[i] = reinterpret_cast<int32_t *>(base + 2 * i * l.each);
        buf.token[i] = reinterpret_cast<int32_t *>(base + (2 * i + 1) * l.each);
    }
    uint32_t *counts = reinterpret_cast<uint32_t *>(base + l.counts);
    float *partial = reinterpret_cast<float *>(base + l.partial);
    const SortSplit sp = sort_split(T, v_pad);
    const size_t row = table / static_cast<size_t>(v_pad);
    const int64_t meanwhile = sp.rank ? kRankZeroed : sp.cluster ? kZeroed : 0;  // bytes zeroed during the sort
    const int64_t zeroed = accumulate ? 0 : std::min(v_pad, meanwhile / static_cast<int64_t>(row));
    if ((st = embed_sort(ids, T, v_pad, v_valid, sp, buf, counts, dE, static_cast<size_t>(zeroed) * row, s)) != TPCE_OK)
        return st;
    const int last = sp.passes & 1;
    return dtype == TPCE_BF16
               ? embed_sums<__nv_bfloat16>(dX, T, h, v_pad, buf.key[last], buf.token[last], scale, accumulate != 0,
                                           zeroed, partial, dE, s)
               : embed_sums<float>(dX, T, h, v_pad, buf.key[last], buf.token[last], scale, accumulate != 0, zeroed,
                                   partial, dE, s);
}
