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

#include "host.h"
#include "ptx.cuh"
#include "step/vec.cuh"

namespace tpce {
namespace {

using namespace step;

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;

// ------------------------------------------------------------------ the plan
// One launch: a cluster of CTAs, one warp of 32 x CTAs for each contiguous run
// of assignments. Pass 1 counts the run's assignments per expert and gives each
// its rank among the run's equal ones (kept in row[]); the counts are then
// summed over the block's warps, over the cluster's blocks (distributed shared
// memory) and over the experts; pass 2 adds them to the rank.
constexpr int kPlanWarps = 32;
constexpr int kBatch = 8;  // vectors of 32 assignments whose loads are under way at once

__device__ __forceinline__ uint32_t read_cluster_u32(const uint32_t *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(ptx::mapa_shared(ptx::smem_u32(p), rank)) : "memory");
    return v;
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

__global__ void __launch_bounds__(32 * kPlanWarps)
    expert_plan_kernel(const int32_t *__restrict__ ids, int64_t n, int E, int ctas, int32_t *row, int32_t *source,
                       int32_t *offsets, uint32_t *err) {
    extern __shared__ uint32_t smem[];
    uint32_t *count = smem;                      // [kPlanWarps][E], then prefix sums over the warps
    uint32_t *total = smem + kPlanWarps * E;     // [E] this block's counts
    uint32_t *base = total + E;                  // [E] first place of this block's share of an expert
    __shared__ uint32_t scan[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ctas > 1 ? ptx::cluster_ctarank() : 0u;

    const int64_t warps = static_cast<int64_t>(ctas) * kPlanWarps;
    const int64_t run = ((n + warps - 1) / warps + 31) / 32 * 32;
    const int64_t first = (static_cast<int64_t>(rank) * kPlanWarps + warp) * run;
    const int64_t last = min(n, first + run);

    uint32_t *mine = count + warp * E;
    for (int e = lane; e < E; e += 32) mine[e] = 0u;
    __syncwarp();
    const int bits = 32 - __clz(E);  // of the values 0 .. E - 1 and of E, which stands for a dropped one
    for (int64_t i0 = first; i0 < last; i0 += 32 * kBatch) {
        int e[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32 + lane;
            e[u] = i < last ? __ldg(ids + i) : -1;  // dropped, as far as counting goes
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
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        uint32_t sum = 0u;
#pragma unroll 8
        for (int q = 0; q < kPlanWarps; ++q) {
            const uint32_t c = count[q * E + e];
            count[q * E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    if (ctas > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    // E <= 1024: one expert a thread
    uint32_t all = 0u, below = 0u;
    const int e = threadIdx.x;
    if (e < E) {
        if (ctas > 1) {
            for (int q = 0; q < ctas; ++q) {
                const uint32_t c = read_cluster_u32(total + e, q);
                below += q < static_cast<int>(rank) ? c : 0u;
                all += c;
            }
        } else {
            all = total[e];
        }
    }
    uint32_t incl = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    uint32_t prior = 0u, kept = 0u;
    for (int q = 0; q < kPlanWarps; ++q) {
        const uint32_t c = scan[q];
        prior += q < warp ? c : 0u;
        kept += c;
    }
    if (e < E) {
        base[e] = prior + incl - all + below;
        if (rank == 0) {
            offsets[e + 1] = static_cast<int32_t>(prior + incl);
            if (e == 0) offsets[0] = 0;
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
            x[u] = i < last ? __ldg(ids + i) : 0;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32;
            if (r[u] < 0) continue;  // past the run, or dropped: row[i] is -1 already
            const uint32_t p = base[x[u]] + mine[x[u]] + static_cast<uint32_t>(r[u]);
            row[i] = static_cast<int32_t>(p);
            source[p] = static_cast<int32_t>(i);
        }
    }
    for (int64_t p = kept + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; p < n;
         p += static_cast<int64_t>(ctas) * blockDim.x)
        source[p] = -1;
    if (ctas > 1) ptx::cluster_sync();  // no block leaves while another reads its counts
}

// ------------------------------------------------------------------ rows by token
// `lanes` threads of a block share a token; each handles 16-byte vectors.
struct Split {
    int lanes;   // a power of two, 8 .. 256
    int tokens;  // of a block
};
// Four vectors a thread keep enough loads under way; where that would leave
// SMs without a block, as many threads as there are vectors.
inline Split split_of(int64_t vectors, int64_t T) {
    int lanes = 8;
    while (lanes < 256 && lanes * 4 < vectors) lanes *= 2;
    if (T * lanes < int64_t{256} * num_sms())
        while (lanes < 256 && lanes < vectors) lanes *= 2;
    return {lanes, 256 / lanes};
}

// A place read from the plan; one outside the rows is reported and skipped.
__device__ __forceinline__ int32_t place(const int32_t *row, int64_t i, int64_t n, uint32_t *err) {
    const int32_t p = __ldg(row + i);
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

// Rows offsets[E] .. n of out are zeros: the blocks take them in turn.
__device__ __forceinline__ void zero_rest(uint4 *out, const int32_t *offsets, int E, int64_t n, int vectors) {
    const int64_t kept = max(0, __ldg(offsets + E));
    for (int64_t p = kept + blockIdx.x; p < n; p += gridDim.x)
        for (int c = threadIdx.x; c < vectors; c += blockDim.x) out[p * vectors + c] = make_uint4(0u, 0u, 0u, 0u);
}

// The kernels hold the places of a token's K choices in registers; for k > K
// (K is the largest then) they take the choices K at a time.
template <int K>
__global__ void __launch_bounds__(256)
    expert_dispatch_kernel(const uint4 *__restrict__ X, const int32_t *__restrict__ row,
                           const int32_t *__restrict__ offsets, int E, int64_t T, int k, int vectors, int lanes,
                           uint4 *__restrict__ out, uint32_t *err) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t n = T * k;
    if (t < T) {
        for (int j0 = 0; j0 < k; j0 += K) {
            int32_t p[K];
            places(row + j0, t, k, n, err, p, k - j0);
#pragma unroll 4
            for (int c = lane; c < vectors; c += lanes) {
                const uint4 v = __ldg(X + t * vectors + c);
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (p[j] >= 0) out[static_cast<int64_t>(p[j]) * vectors + c] = v;
            }
        }
    }
    zero_rest(out, offsets, E, n, vectors);
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

// NV values a vector: 8 (bf16) or 4 (fp32). weights NULL: all one.
template <int NV, int K>
__global__ void __launch_bounds__(256)
    expert_combine_kernel(const uint4 *__restrict__ Ys, const int32_t *__restrict__ row,
                          const float *__restrict__ weights, int64_t T, int k, int vectors, int lanes,
                          uint4 *__restrict__ Z, uint32_t *err) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    if (t >= T) return;
    const int64_t n = T * k;
    constexpr int U = K >= 4 ? 1 : 4 / K;  // vectors at a time: at least four loads under way
    int32_t p[K];
    float w[K];
    auto choices = [&](int j0) {
        places(row + j0, t, k, n, err, p, k - j0);
#pragma unroll
        for (int j = 0; j < K; ++j) w[j] = weights && j0 + j < k ? __ldg(weights + t * k + j0 + j) : 1.0f;
    };
    if (k <= K) choices(0);
    for (int c0 = lane; c0 < vectors; c0 += U * lanes) {
        float z[U][NV] = {};
        for (int j0 = 0; j0 < k; j0 += K) {
            if (k > K) choices(j0);
            uint4 y[U][K];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (p[j] >= 0 && c0 + u * lanes < vectors)
                        y[u][j] = __ldg(Ys + static_cast<int64_t>(p[j]) * vectors + c0 + u * lanes);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (p[j] < 0) continue;
                    float v[NV];
                    widen(y[u][j], v);
#pragma unroll
                    for (int i = 0; i < NV; ++i) z[u][i] += w[j] * v[i];
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * lanes < vectors) Z[t * vectors + c0 + u * lanes] = narrow(z[u]);
    }
}

template <int NV, int K>
__global__ void __launch_bounds__(256)
    expert_combine_backward_kernel(const uint4 *__restrict__ dZ, const uint4 *__restrict__ Ys,
                                   const int32_t *__restrict__ row, const int32_t *__restrict__ offsets, int E,
                                   const float *__restrict__ weights, int64_t T, int k, int vectors, int lanes,
                                   uint4 *__restrict__ dYs, float *__restrict__ dweights, uint32_t *err) {
    __shared__ float red[8][K];
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t n = T * k;
    constexpr int U = K >= 4 ? 1 : 4 / K;
    for (int j0 = 0; j0 < k; j0 += K) {
        int32_t p[K];
        float w[K], dot[K] = {};
#pragma unroll
        for (int j = 0; j < K; ++j) p[j] = -1, w[j] = 0.0f;
        if (t < T) {
            places(row + j0, t, k, n, err, p, k - j0);
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (p[j] >= 0) w[j] = __ldg(weights + t * k + j0 + j);
            for (int c0 = lane; c0 < vectors; c0 += U * lanes) {
                uint4 d[U], y[U][K];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + u * lanes;
                    if (c >= vectors) continue;
                    d[u] = __ldg(dZ + t * vectors + c);
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (p[j] >= 0) y[u][j] = __ldg(Ys + static_cast<int64_t>(p[j]) * vectors + c);
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
    zero_rest(dYs, offsets, E, n, vectors);
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

inline int vectors_of(int64_t h, int dtype) { return static_cast<int>(h * (dtype == TPCE_BF16 ? 2 : 4) / 16); }

inline unsigned blocks_of(int64_t T, const Split &sp) { return static_cast<unsigned>((T + sp.tokens - 1) / sp.tokens); }

// f(integral constant): the fewest of 1, 2, 4, 8 choices held that cover k (8 for more)
template <typename F>
void with_choices(int k, F f) {
    if (k == 1) f(std::integral_constant<int, 1>{});
    else if (k == 2) f(std::integral_constant<int, 2>{});
    else if (k <= 4) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 8>{});
}

tpce_status combine(const char *name, const void *Ys, const int32_t *row, const float *weights, int64_t T, int64_t h,
                    int k, int dtype, void *Z, cudaStream_t s) {
    const int v = vectors_of(h, dtype);
    const Split sp = split_of(v, T);
    KernelTimer timer(name, s);
    with_choices(k, [&](auto K) {
        auto go = [&](auto kernel) {
            kernel<<<blocks_of(T, sp), 256, 0, s>>>(static_cast<const uint4 *>(Ys), row, weights, T, k, v, sp.lanes,
                                                    static_cast<uint4 *>(Z), device_error_word());
        };
        if (dtype == TPCE_BF16)
            go(expert_combine_kernel<8, decltype(K)::value>);
        else
            go(expert_combine_kernel<4, decltype(K)::value>);
    });
    return check_launch(name, s);
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" tpce_status tp_expert_plan(const int32_t *ids, int64_t T, int k, int E, int32_t *row, int32_t *source,
                                      int32_t *offsets, void *stream) {
    tpce_status st = check_plan_shape(T, k, E);
    if (st != TPCE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if ((st = check_pointers("tp_expert_plan", {offsets})) != TPCE_OK) return st;
        return cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), s) == cudaSuccess ? TPCE_OK : TPCE_ERR_CUDA;
    }
    if ((st = check_pointers("tp_expert_plan", {ids, row, source, offsets})) != TPCE_OK) return st;
    const int64_t n = T * k;
    const int ctas = n <= 4096 ? 1 : 8;
    const size_t smem = static_cast<size_t>(kPlanWarps + 2) * E * sizeof(uint32_t);
    cudaError_t e;
    if (smem > 48 * 1024) {  // more than a launch has without asking: from 362 experts on
        e = cudaFuncSetAttribute(expert_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (kPlanWarps + 2) * kMaxExperts * static_cast<int>(sizeof(uint32_t)));
        if (e != cudaSuccess) return fail_cuda(e, "expert_plan");
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(32 * kPlanWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    KernelTimer timer("expert_plan", s);
    e = cudaLaunchKernelEx(&cfg, expert_plan_kernel, ids, n, E, ctas, row, source, offsets, device_error_word());
    if (e != cudaSuccess) return fail_cuda(e, "expert_plan");
    return check_launch("expert_plan", s);
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
    with_choices(k, [&](auto K) {
        expert_dispatch_kernel<decltype(K)::value>
            <<<blocks_of(T, sp), 256, 0, s>>>(static_cast<const uint4 *>(X), row, offsets, E, T, k, v, sp.lanes,
                                              static_cast<uint4 *>(Xs), device_error_word());
    });
    return check_launch("expert_dispatch", s);
}

extern "C" tpce_status tp_expert_dispatch_backward(const void *dXs, const int32_t *row, int64_t T, int64_t h, int k,
                                                   int dtype, void *dX, void *stream) {
    tpce_status st = check_rows_shape(T, h, k, 1, dtype);
    if (st != TPCE_OK || T == 0) return st;
    if ((st = check_pointers("tp_expert_dispatch_backward", {dXs, row, dX})) != TPCE_OK) return st;
    return combine("expert_dispatch_backward", dXs, row, nullptr, T, h, k, dtype, dX, static_cast<cudaStream_t>(stream));
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
    const Split sp = split_of(v, T);
    KernelTimer timer("expert_combine_backward", s);
    with_choices(k, [&](auto K) {
        auto go = [&](auto kernel) {
            kernel<<<blocks_of(T, sp), 256, 0, s>>>(static_cast<const uint4 *>(dZ), static_cast<const uint4 *>(Ys),
                                                    row, offsets, E, weights, T, k, v, sp.lanes,
                                                    static_cast<uint4 *>(dYs), dweights, device_error_word());
        };
        if (dtype == TPCE_BF16)
            go(expert_combine_backward_kernel<8, decltype(K)::value>);
        else
            go(expert_combine_backward_kernel<4, decltype(K)::value>);
    });
    return check_launch("expert_combine_backward", s);
}
