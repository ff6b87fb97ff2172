// experts.cu -- tokens sorted by expert and back.
//
// T tokens choose k experts each: ids [T, k], an id in [0, E) or -1 (the
// assignment is dropped). The plan is a stable counting sort of the T k
// assignments i = t k + j by expert: row[i] is the place of assignment i among
// the sorted ones (-1: dropped), source[p] the assignment at place p (-1 past
// the last one), offsets[e] .. offsets[e + 1] the places of expert e. With it
//   dispatch          Xs[row[t, j]] = X[t]                  (rows past the last: 0)
//   combine           Z[t] = sum_j weights[t, j] Ys[row[t, j]]
// and their gradients
//   dispatch backward dX[t] = sum_j dXs[row[t, j]]
//   combine backward  dYs[row[t, j]] = weights[t, j] dZ[t]  (rows past the last: 0)
//                     dweights[t, j] = sum_c dZ[t, c] Ys[row[t, j], c]
// All four go by token: a token's row is read (or written) once and meets its k
// rows there, so that no sum is split over blocks and nothing needs an atomic.
// Sums are taken in 32 bits in the order j = 0, 1, .. and rounded once.
#include <algorithm>
#include <climits>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "host.h"
#include "ptx.cuh"
#include "step/launch.cuh"
#include "step/vec.cuh"

namespace tpce {
namespace {

using namespace step;

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;
constexpr int kMaxHeld = 8;  // choices of a token in a thread's registers

// ------------------------------------------------------------------ the plan
// A block takes a chunk of the assignments, each of its warps a contiguous run
// of the chunk. expert_count_kernel counts the chunks' assignments per expert;
// expert_place_kernel adds up the counts of the chunks before its own, counts
// its own per warp and gives each assignment its rank among the equal ones of
// its run (kept in row[]), and then writes the places. Few assignments are one
// block's, and need no counting before. Many blocks, because the places of
// source[] are scattered: one SM stores only about a word of them in a cycle
// (131,072 assignments over 64 experts took eight SMs 20 us, and take 128 blocks
// 7 us in both launches, nearly all of it the launches' own).
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBatch = 4;  // vectors of 32 assignments whose loads are under way at once
constexpr int64_t kPlanChunk = 1024, kPlanBlocks = 256;

struct PlanSplit {
    int64_t chunk;
    int blocks;
};
inline PlanSplit plan_split(int64_t n) {
    const int64_t chunk = std::max<int64_t>(kPlanChunk, (n + kPlanBlocks - 1) / kPlanBlocks);
    if (n <= 2 * chunk) return {n, 1};
    return {chunk, static_cast<int>((n + chunk - 1) / chunk)};
}

__global__ void __launch_bounds__(kPlanThreads)
    expert_count_kernel(const int32_t *ids, int64_t n, int64_t chunk, int E, uint32_t *__restrict__ counts) {
    extern __shared__ uint32_t count[];  // [E]
    for (int e = threadIdx.x; e < E; e += kPlanThreads) count[e] = 0u;
    grid_begin();
    __syncthreads();
    const int64_t first = blockIdx.x * chunk, last = min(n, first + chunk);
    for (int64_t i0 = first + threadIdx.x; i0 < last; i0 += kPlanThreads * kBatch) {
        int e[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * kPlanThreads;
            e[u] = i < last ? ids[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (e[u] >= 0 && e[u] < E) atomicAdd(&count[e[u]], 1u);  // whole numbers: any order gives the same
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kPlanThreads) counts[static_cast<int64_t>(blockIdx.x) * E + e] = count[e];
}

// The lanes whose value equals this lane's, from one ballot for each of its bits.
__device__ __forceinline__ uint32_t same_value(int v, int bits) {
    uint32_t same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const bool one = (v >> b) & 1;
        const uint32_t with = __ballot_sync(0xffffffffu, one);
        same &= one ? with : ~with;
    }
    return same;
}

// counts NULL: this block is the only one.
__global__ void __launch_bounds__(kPlanThreads)
    expert_place_kernel(const int32_t *ids, int64_t n, int64_t chunk, int E,
                        const uint32_t *counts, int32_t *row, int32_t *source, int32_t *offsets,
                        uint32_t *err) {
    extern __shared__ uint32_t smem[];
    uint32_t *count = smem;                   // [kPlanWarps][E], then prefix sums over the warps
    uint32_t *all = smem + kPlanWarps * E;    // [E] assignments of an expert, then the first place of this block's
    uint32_t *below = all + E;                // [E] those of the blocks before
    __shared__ uint32_t scan[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < (kPlanWarps + 2) * E; e += kPlanThreads) smem[e] = 0u;
    grid_begin();
    __syncthreads();
    if (counts) {
        // E counts a block: a thread adds those of one expert over some of the blocks
        int width = 1;
        while (width < E && width < kPlanThreads) width *= 2;
        const int parts = kPlanThreads / width, part = threadIdx.x / width;
        for (int e = threadIdx.x & (width - 1); e < E; e += width) {
            uint32_t sum = 0u, before = 0u;
#pragma unroll 8
            for (int q = part; q < static_cast<int>(gridDim.x); q += parts) {
                const uint32_t c = counts[static_cast<int64_t>(q) * E + e];
                sum += c;
                before += q < static_cast<int>(blockIdx.x) ? c : 0u;
            }
            atomicAdd(&all[e], sum);
            atomicAdd(&below[e], before);
        }
    }

    const int64_t begin = blockIdx.x * chunk, end = min(n, begin + chunk);
    const int64_t run = ((end - begin + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int64_t first = begin + warp * run, last = min(end, first + run);
    uint32_t *mine = count + warp * E;
    const int bits = 32 - __clz(E);  // of the values 0 .. E - 1 and of E, which stands for a dropped one
    for (int64_t i0 = first; i0 < last; i0 += 32 * kBatch) {
        int e[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32 + lane;
            e[u] = i < last ? ids[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32 + lane;
            if (e[u] < 0 || e[u] >= E) {
                if (e[u] != -1) ptx::record_error(err, kErrInvalid | (2u << 8));
                e[u] = E;
            }
            const bool kept = e[u] < E;
            const uint32_t same = same_value(e[u], bits);
            const uint32_t before = __popc(same & ((1u << lane) - 1u));
            uint32_t seen = 0u;
            if (kept) seen = mine[e[u]];
            __syncwarp();
            if (kept && before == 0u) mine[e[u]] = seen + __popc(same);
            __syncwarp();
            if (i < last) row[i] = kept ? static_cast<int32_t>(seen + before) : -1;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kPlanThreads) {
        uint32_t sum = 0u;
#pragma unroll
        for (int q = 0; q < kPlanWarps; ++q) {
            const uint32_t c = count[q * E + e];
            count[q * E + e] = sum;
            sum += c;
        }
        if (!counts) all[e] = sum;
    }
    __syncthreads();
    // first places: a scan over the experts, four adjacent ones a thread
    constexpr int kEach = kMaxExperts / kPlanThreads;
    uint32_t own[kEach], sum = 0u;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int e = threadIdx.x * kEach + u;
        own[u] = e < E ? all[e] : 0u;
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
    uint32_t at = incl - sum, kept = 0u;
#pragma unroll
    for (int q = 0; q < kPlanWarps; ++q) {
        at += q < warp ? scan[q] : 0u;
        kept += scan[q];
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int e = threadIdx.x * kEach + u;
        if (e < E) {
            all[e] = at + below[e];
            at += own[u];
            if (blockIdx.x == 0) {
                offsets[e + 1] = static_cast<int32_t>(at);
                if (e == 0) offsets[0] = 0;
            }
        }
    }
    __syncthreads();
    for (int64_t i0 = first + lane; i0 < last; i0 += 32 * kBatch) {
        int32_t r[kBatch];
        int x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32;
            r[u] = i < last ? row[i] : -1;
            x[u] = i < last ? ids[i] : 0;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32;
            if (r[u] < 0) continue;  // past the run, or dropped: row[i] is -1 already
            // ids read a second time: one that has changed meanwhile must lead nowhere
            const bool known = static_cast<uint32_t>(x[u]) < static_cast<uint32_t>(E);
            const uint32_t p = known ? all[x[u]] + mine[x[u]] + static_cast<uint32_t>(r[u]) : UINT_MAX;
            if (p >= n) {
                ptx::record_error(err, kErrInvalid | (4u << 8));
                row[i] = -1;
                continue;
            }
            row[i] = static_cast<int32_t>(p);
            source[p] = static_cast<int32_t>(i);
        }
    }
    for (int64_t p = kept + static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x; p < n;
         p += static_cast<int64_t>(gridDim.x) * kPlanThreads)
        source[p] = -1;
}

// ------------------------------------------------------------------ rows by token
// `lanes` threads of a block share a token; each handles 16-byte vectors.
struct Split {
    int lanes;   // a power of two, 8 .. 256
    int tokens;  // of a block
};
// Four vectors a thread, and eight of rows of less than 8 KB: a thread that reads
// its token's places for one or two vectors waits for them as long as for the
// vectors (13,152 tokens of 864 bf16, k = 6, backward: 106, 87, 82 and 79 us with
// one, two, four and eight; 16,384 of 4096, k = 8: 375 us with four, 381 with
// eight). As many threads as there are vectors where that would leave an SM with
// fewer than `blocks`: 512 tokens of 4096, k = 8, take 23 us with four, 28 with
// one. The combine's backward, which adds over a token's lanes, is faster with two
// (3551 of 792 fp32, k = 5: 34.6 and 36.8 us).
inline Split split_of(int64_t vectors, int64_t T, int blocks = 4) {
    int lanes = 8;
    const int each = vectors < 512 ? 8 : 4;
    const int64_t enough = int64_t{256} * blocks * num_sms();
    while (lanes < 256 && (lanes * each < vectors || (lanes < vectors && T * lanes < enough))) lanes *= 2;
    return {lanes, 256 / lanes};
}

// A place read from the plan; one outside the rows is reported and skipped.
__device__ __forceinline__ int32_t place(const int32_t *row, int64_t i, int64_t n, uint32_t *err) {
    const int32_t p = row[i];
    if (p < -1 || p >= n) {
        ptx::record_error(err, kErrInvalid | (3u << 8));
        return -1;
    }
    return p;
}

// The places of K of token t's choices from `row` on, -1 beyond the `left` that it has.
template <int K>
__device__ __forceinline__ void places(const int32_t *row, int64_t t, int k, int64_t n, uint32_t *err,
                                       int32_t (&p)[K], int left) {
#pragma unroll
    for (int j = 0; j < K; ++j) p[j] = j < left ? place(row, t * k + j, n, err) : -1;
}

// Rows `kept` .. n of out are zeros: the threads of the grid take their vectors in
// turn. (With a row a block in turn, 15,938 tokens of 168 bf16 of which half are
// dropped, k = 7, took 37 us instead of 21 in the combine's backward.)
__device__ __forceinline__ void zero_rest(uint4 *out, int64_t kept, int64_t n, int vectors) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = max(int64_t{0}, kept) * vectors + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
         i < n * vectors; i += stride)
        out[i] = make_uint4(0u, 0u, 0u, 0u);
}

// The kernels hold the places of a token's K choices in registers: K is k, or the
// largest, and then they take the choices K at a time. (With one kernel for 5 to 8
// choices 7728 tokens of 776 fp32, k = 7, half of them dropped, took 98 us
// backward instead of 92; with blocks for three of them on an SM instead of two,
// 82.) All three are bound by HBM: the loads of a thread's vectors are issued
// together, before anything is done with them.
//
// Dispatch: 16,384 tokens of 4096 bf16 to 8 experts each, 1.2 GB, 178 us,
// 6.8 TB/s, as fast as a copy.
template <int K>
__global__ void __launch_bounds__(256)
    expert_dispatch_kernel(const uint4 *X, const int32_t *row,
                           const int32_t *offsets, int E, int64_t T, int k, int vectors, int lanes,
                           uint4 *__restrict__ out, uint32_t *err) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t n = T * k;
    grid_begin();
    const int64_t kept = offsets[E];
    if (t < T) {
        for (int j0 = 0; j0 < k; j0 += K) {
            int32_t p[K];
            places(row + j0, t, k, n, err, p, k - j0);
            for (int c0 = lane; c0 < vectors; c0 += 4 * lanes) {
                uint4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c0 + u * lanes < vectors) v[u] = X[t * vectors + c0 + u * lanes];
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (p[j] < 0) continue;
                    uint4 *to = out + static_cast<int64_t>(p[j]) * vectors + c0;
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (c0 + u * lanes < vectors) to[u * lanes] = v[u];
                }
            }
        }
    }
    zero_rest(out, kept, n, vectors);
}

// The values of one 16-byte vector.
__device__ __forceinline__ void widen(const uint4 &u, float (&v)[8]) {
    unpack8(Raw8<__nv_bfloat16>{u}, v);
}
__device__ __forceinline__ void widen(const uint4 &u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
    Raw8<__nv_bfloat16> r;
    pack8(v, r);
    return r.a;
}
__device__ __forceinline__ uint4 narrow(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// Combine, and the dispatch's backward. NV values a vector: 8 (bf16) or 4 (fp32).
// weights NULL: all one. The same 1.2 GB as above: 186 us, 6.5 TB/s (206 us where
// a thread read its places again for each vector).
// Blocks that an SM must have room for, and with them the registers (8192 tokens of
// 4096 bf16, us): six for one and two choices (22.2 and 31.7; with four 23.1 and
// 34.7), four for three and four (42.4, 50.7; with three 42.6, 53.5), three for five
// (61.7; with four 70.3, though 4000 of 1000 fp32 take 16.8 instead of 17.6), four
// for six to eight, which costs eight some spilled registers (71.1, 80.3, 92.8; with
// three 71.1, 84.6, 92.9, and 3783 of 768, half dropped, k = 7, 8.6 instead of 7.1).
// Vectors at a time: one for six and more (two: 88.3, 110, 143), two for three to
// five (one: 42.4, 52.4, 62.9; fp32 k = 3 14.2 instead of 12.1), four and two for one
// and two (two and one: 23.7, 34.4).
template <int NV, int K>
__global__ void __launch_bounds__(256, K == 5 ? 3 : K > 2 ? 4 : 6)
    expert_combine_kernel(const uint4 *Ys, const int32_t *row,
                          const float *weights, int64_t T, int k, int vectors, int lanes,
                          uint4 *__restrict__ Z, uint32_t *err) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    grid_begin();
    if (t >= T) return;
    const int64_t n = T * k;
    constexpr int U = K > 5 ? 1 : K > 2 ? 2 : 4 / K;  // vectors at a time: four to ten loads under way
    int32_t p[K];
    float w[K];
    auto choices = [&](int j0) {
        places(row + j0, t, k, n, err, p, k - j0);
#pragma unroll
        for (int j = 0; j < K; ++j) w[j] = weights && j0 + j < k ? weights[t * k + j0 + j] : 1.0f;
    };
    auto add = [&](const uint4 (&y)[K], float (&z)[NV]) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (p[j] < 0) continue;
            float v[NV];
            widen(y[j], v);
#pragma unroll
            for (int i = 0; i < NV; ++i) z[i] += w[j] * v[i];
        }
    };
    auto load = [&](int c, uint4 (&y)[K]) {
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (p[j] >= 0) y[j] = Ys[static_cast<int64_t>(p[j]) * vectors + c];
    };
    if (K == kMaxHeld && k > K) {
        for (int c = lane; c < vectors; c += lanes) {
            float z[NV] = {};
            for (int j0 = 0; j0 < k; j0 += K) {
                uint4 y[K];
                choices(j0);
                load(c, y);
                add(y, z);
            }
            Z[t * vectors + c] = narrow(z);
        }
        return;
    }
    choices(0);
    for (int c0 = lane; c0 < vectors; c0 += U * lanes) {
        uint4 y[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * lanes < vectors) load(c0 + u * lanes, y[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float z[NV] = {};
            add(y[u], z);
            if (c0 + u * lanes < vectors) Z[t * vectors + c0 + u * lanes] = narrow(z);
        }
    }
}

// The combine's backward: dZ is read once for all of a token's rows. 4096 tokens
// of 8192 bf16 and 2 experts, 10% dropped, 0.32 GB: 50 us, 6.4 TB/s. Three blocks an
// SM from five choices on (8192 of 4096 bf16, k = 7 and 8: 155 and 176 us, with four
// 173 and 206; five take 114 and with four 112, six 132 and 141), four below (k = 4:
// 92, with three 96). One vector at a time from four choices on (92; two: 96), four
// and two for one and two (33 and 52; one: 41 and 57).
template <int NV, int K>
__global__ void __launch_bounds__(256, K > 4 ? 3 : 4)
    expert_combine_backward_kernel(const uint4 *dZ, const uint4 *Ys,
                                   const int32_t *row, const int32_t *offsets, int E,
                                   const float *weights, int64_t T, int k, int vectors, int lanes,
                                   uint4 *__restrict__ dYs, float *__restrict__ dweights, uint32_t *err) {
    __shared__ float red[8][K];
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t n = T * k;
    constexpr int U = K >= 4 ? 1 : 4 / K;
    grid_begin();
    const int64_t kept = offsets[E];
    for (int j0 = 0; j0 < k; j0 += K) {
        int32_t p[K];
        float w[K], dot[K] = {};
#pragma unroll
        for (int j = 0; j < K; ++j) p[j] = -1, w[j] = 0.0f;
        if (t < T) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j] = j0 + j < k ? weights[t * k + j0 + j] : 0.0f;
            places(row + j0, t, k, n, err, p, k - j0);
            for (int c0 = lane; c0 < vectors; c0 += U * lanes) {
                uint4 d[U], y[U][K];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * lanes;
                    if (c >= vectors) continue;
                    d[u] = dZ[t * vectors + c];
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (p[j] >= 0) y[u][j] = Ys[static_cast<int64_t>(p[j]) * vectors + c];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * lanes;
                    if (c >= vectors) continue;
                    float dv[NV];
                    widen(d[u], dv);
#pragma unroll
                    for (int j = 0; j < K; ++j) {
                        if (p[j] < 0) continue;
                        float yv[NV], o[NV];
                        widen(y[u][j], yv);
#pragma unroll
                        for (int i = 0; i < NV; ++i) {
                            dot[j] += dv[i] * yv[i];
                            o[i] = dv[i] * w[j];
                        }
                        dYs[static_cast<int64_t>(p[j]) * vectors + c] = narrow(o);
                    }
                }
            }
        }
        // over the token's lanes: within a warp, then over its warps
#pragma unroll
        for (int j = 0; j < K; ++j)
            for (int d = min(lanes, 32) / 2; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
        if (lanes > 32) {
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int j = 0; j < K; ++j) red[warp][j] = dot[j];
            }
            __syncthreads();
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    for (int q = 1; q < lanes / 32; ++q) dot[j] += red[warp + q][j];
            }
            __syncthreads();
        }
        if (lane == 0 && t < T) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (j0 + j < k) dweights[t * k + j0 + j] = dot[j];
        }
    }
    zero_rest(dYs, kept, n, vectors);
}

// ------------------------------------------------------------------ host
tpce_status check_plan_shape(int64_t T, int k, int E) {
    if (T < 0 || k < 1 || k > kMaxChoices || E < 1 || E > kMaxExperts || T > (INT_MAX - 1024) / k)
        return fail(TPCE_ERR_SHAPE, "experts: T = %lld, k = %d (1 .. %d), E = %d (1 .. %d), T k below 2^31",
                    static_cast<long long>(T), k, kMaxChoices, E, kMaxExperts);
    return TPCE_OK;
}

tpce_status check_rows_shape(int64_t T, int64_t h, int k, int E, int dtype) {
    if (dtype != TPCE_BF16 && dtype != TPCE_F32) return fail(TPCE_ERR_INVALID, "experts: dtype %d", dtype);
    tpce_status st = check_plan_shape(T, k, E);
    if (st != TPCE_OK) return st;
    if (h < 8 || h % 8 != 0 || h > (1 << 20))
        return fail(TPCE_ERR_SHAPE, "experts: h = %lld (a multiple of 8 up to 2^20)", static_cast<long long>(h));
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

inline int vectors_of(int64_t h, int dtype) { return static_cast<int>(h * (dtype == TPCE_BF16 ? 2 : 4) / 16); }

inline unsigned blocks_of(int64_t T, const Split &sp) { return static_cast<unsigned>((T + sp.tokens - 1) / sp.tokens); }

// f(integral constant): k choices held, kMaxHeld at a time for more
template <int K = 1, typename F>
void with_choices(int k, F f) {
    if constexpr (K < kMaxHeld) {
        if (k > K) return with_choices<K + 1>(k, f);
    }
    f(std::integral_constant<int, K>{});
}

tpce_status combine(const char *name, const void *Ys, const int32_t *row, const float *weights, int64_t T, int64_t h,
                    int k, int dtype, void *Z, cudaStream_t s) {
    const int v = vectors_of(h, dtype);
    const Split sp = split_of(v, T);
    KernelTimer timer(name, s);
    cudaError_t e = cudaSuccess;
    with_choices(k, [&](auto K) {
        auto go = [&](auto kernel) {
            e = launch(kernel, blocks_of(T, sp), 256, 0, s, static_cast<const uint4 *>(Ys), row, weights, T, k, v,
                       sp.lanes, static_cast<uint4 *>(Z), device_error_word());
        };
        if (dtype == TPCE_BF16)
            go(expert_combine_kernel<8, decltype(K)::value>);
        else
            go(expert_combine_kernel<4, decltype(K)::value>);
    });
    return e == cudaSuccess ? check_launch(name, s) : fail_cuda(e, name);
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" size_t tpce_expert_plan_workspace_bytes(int64_t T, int k, int E) {
    if (check_plan_shape(T, k, E) != TPCE_OK) return 0;
    const PlanSplit sp = plan_split(T * k);
    return sp.blocks > 1 ? static_cast<size_t>(sp.blocks) * E * sizeof(uint32_t) : 0;
}

extern "C" tpce_status tp_expert_plan(const int32_t *ids, int64_t T, int k, int E, int32_t *row, int32_t *source,
                                      int32_t *offsets, void *ws, size_t ws_bytes, void *stream) {
    tpce_status st = check_plan_shape(T, k, E);
    if (st != TPCE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if ((st = check_pointers("tp_expert_plan", {offsets})) != TPCE_OK) return st;
        const cudaError_t e = taken(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), s));
        return e == cudaSuccess ? TPCE_OK : fail_cuda(e, "tp_expert_plan");
    }
    if ((st = check_pointers("tp_expert_plan", {ids, row, source, offsets})) != TPCE_OK) return st;
    const int64_t n = T * k;
    const PlanSplit sp = plan_split(n);
    uint32_t *counts = nullptr;
    cudaError_t e;
    const size_t need = tpce_expert_plan_workspace_bytes(T, k, E);
    if (sp.blocks > 1) {
        if (!ws || ws_bytes < need)
            return fail(TPCE_ERR_WORKSPACE, "tp_expert_plan: %zu bytes of workspace needed, %zu given", need,
                        ws ? ws_bytes : size_t{0});
        if (!aligned16(ws)) return fail(TPCE_ERR_ALIGN, "tp_expert_plan: a pointer is not 16-byte aligned");
        counts = static_cast<uint32_t *>(ws);
    }
    // ids are read again after places and counts have been written
    const size_t each = static_cast<size_t>(n) * sizeof(int32_t);
    const std::pair<const void *, size_t> parts[] = {
        {ids, each}, {row, each}, {source, each}, {offsets, sizeof(int32_t) * (E + 1)}, {counts, need}};
    for (const auto &a : parts)
        for (const auto &b : parts)
            if (&a < &b && overlap(a.first, a.second, b.first, b.second))
                return fail(TPCE_ERR_INVALID, "tp_expert_plan: ids, row, source, offsets or ws overlap");
    if (counts) {
        KernelTimer timer("expert_count", s);
        e = launch(expert_count_kernel, sp.blocks, kPlanThreads, E * sizeof(uint32_t), s, ids, n, sp.chunk, E, counts);
        if (e != cudaSuccess) return fail_cuda(e, "expert_count");
        if ((st = check_launch("expert_count", s)) != TPCE_OK) return st;
    }
    KernelTimer timer("expert_place", s);
    e = launch(expert_place_kernel, sp.blocks, kPlanThreads, (kPlanWarps + 2) * E * sizeof(uint32_t), s, ids, n,
               sp.chunk, E, counts, row, source, offsets, device_error_word());
    if (e != cudaSuccess) return fail_cuda(e, "expert_place");
    return check_launch("expert_place", s);
}

extern "C" tpce_status tp_expert_dispatch_forward(const void *X, const int32_t *row, const int32_t *offsets, int64_t T,
                                                  int64_t h, int k, int E, int dtype, void *Xs, void *stream) {
    tpce_status st = check_rows_shape(T, h, k, E, dtype);
    if (st != TPCE_OK || T == 0) return st;
    if ((st = check_pointers("tp_expert_dispatch_forward", {X, row, offsets, Xs})) != TPCE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int v = vectors_of(h, dtype);
    const Split sp = split_of(v, T);
    KernelTimer timer("expert_dispatch", s);
    cudaError_t e = cudaSuccess;
    with_choices(k, [&](auto K) {
        e = launch(expert_dispatch_kernel<decltype(K)::value>, blocks_of(T, sp), 256, 0, s,
                   static_cast<const uint4 *>(X), row, offsets, E, T, k, v, sp.lanes, static_cast<uint4 *>(Xs),
                   device_error_word());
    });
    return e == cudaSuccess ? check_launch("expert_dispatch", s) : fail_cuda(e, "expert_dispatch");
}

extern "C" tpce_status tp_expert_dispatch_backward(const void *dXs, const int32_t *row, int64_t T, int64_t h, int k,
                                                   int dtype, void *dX, void *stream) {
    tpce_status st = check_rows_shape(T, h, k, 1, dtype);
    if (st != TPCE_OK || T == 0) return st;
    if ((st = check_pointers("tp_expert_dispatch_backward", {dXs, row, dX})) != TPCE_OK) return st;
    return combine("expert_dispatch_backward", dXs, row, nullptr, T, h, k, dtype, dX,
                   static_cast<cudaStream_t>(stream));
}

extern "C" tpce_status tp_expert_combine_forward(const void *Ys, const int32_t *row, const float *weights, int64_t T,
                                                 int64_t h, int k, int dtype, void *Z, void *stream) {
    tpce_status st = check_rows_shape(T, h, k, 1, dtype);
    if (st != TPCE_OK || T == 0) return st;
    if ((st = check_pointers("tp_expert_combine_forward", {Ys, row, weights, Z})) != TPCE_OK) return st;
    return combine("expert_combine", Ys, row, weights, T, h, k, dtype, Z, static_cast<cudaStream_t>(stream));
}

extern "C" tpce_status tp_expert_combine_backward(const void *dZ, const void *Ys, const int32_t *row,
                                                  const int32_t *offsets, const float *weights, int64_t T, int64_t h,
                                                  int k, int E, int dtype, void *dYs, float *dweights, void *stream) {
    tpce_status st = check_rows_shape(T, h, k, E, dtype);
    if (st != TPCE_OK || T == 0) return st;
    if ((st = check_pointers("tp_expert_combine_backward", {dZ, Ys, row, offsets, weights, dYs, dweights})) != TPCE_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int v = vectors_of(h, dtype);
    const Split sp = split_of(v, T, 2);
    KernelTimer timer("expert_combine_backward", s);
    cudaError_t e = cudaSuccess;
    with_choices(k, [&](auto K) {
        auto go = [&](auto kernel) {
            e = launch(kernel, blocks_of(T, sp), 256, 0, s, static_cast<const uint4 *>(dZ),
                       static_cast<const uint4 *>(Ys), row, offsets, E, weights, T, k, v, sp.lanes,
                       static_cast<uint4 *>(dYs), dweights, device_error_word());
        };
        if (dtype == TPCE_BF16)
            go(expert_combine_backward_kernel<8, decltype(K)::value>);
        else
            go(expert_combine_backward_kernel<4, decltype(K)::value>);
    });
    return e == cudaSuccess ? check_launch("expert_combine_backward", s) : fail_cuda(e, "expert_combine_backward");
}
