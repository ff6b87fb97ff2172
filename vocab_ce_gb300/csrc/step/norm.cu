// norm.cu -- RMS norm with the residual's addition, forward and backward.
//
//   S = X + R (rounded to the tensors' type: S is the residual stream that the
//   next layers add to, and what is normalised is that stored value, so that
//   the backward, which reads S, differentiates exactly this function),
//   rstd = (sum_c S^2 / h + eps)^-1/2,  Y = S rstd w.
// The optional 8-bit output holds Y before its rounding to bf16, in groups of
// 128 columns (vec.cuh). Backward, with g = dY w and xh = S rstd:
//   dX = rstd (g - xh sum_c(g xh) / h) + dS,   dw = sum_t dY xh.
// X and R enter as a sum, so dX is the gradient of both.
//
// Both passes read each row once: its values stay in registers between the
// sum over the row and the output. They are bound by HBM (8 bytes a value in
// bf16 with the residual), so what matters is the bytes on their way: wide rows
// come through a ring in shared memory that bulk copies fill some rows ahead,
// whatever the threads wait for; narrow ones are some lanes of a warp, which has
// its next rows in registers (forward) or in a ring of its own (backward).
#include <algorithm>
#include <atomic>

#include "host.h"
#include "ptx.cuh"
#include "step/launch.cuh"
#include "step/vec.cuh"

namespace tpce {
namespace {

using namespace step;

constexpr int64_t kMaxWidth = 16384;  // 2 vectors of 8 values for each of 1024 threads
constexpr int64_t kMaxRows = int64_t{1} << 40;
constexpr int kLanesThreads = 256;    // of a block where a row is some lanes of a warp
constexpr int64_t kSms = 152;         // fixed, so that the workspace's size is known on the host
constexpr int kMaxStages = 4, kPairStages = 6;
// Rows of a block of the forward, where there are enough, with a residual and
// without. Blocks that take all their rows from one launch to the end wait for the
// SM that gets its bytes last: 8192 x 8192 bf16 took 95 us with one round of
// blocks, 87 with four; with three rows a block the ring is filled too often (4096
// x 8192 and 8 bits: 53 and 56 us). Without a residual a row is half as long:
// 4096 x 8192 take 19.7 us with nine, 22.3 with six; 16,384 84.3 and 82.7.
constexpr int kRowsOfBlock[2] = {6, 9};
constexpr int kSmemPerSm = 228 * 1024;

// A row of up to 256 values is 8, 16 or 32 lanes of a warp (no barrier in its
// sum), a wider one a block's. At h = 512 a warp with two vectors a lane took
// 45 us forward and 55 backward for 65,536 rows, a block of 64 threads 42 and 47;
// at h = 64 a whole warp a row took 86 and 87 us for 262,144 fp32 rows, 8 lanes
// 51 and 46.
inline bool lane_rows(int64_t h) { return h <= 256; }
inline bool pair_rows(int64_t h) { return h > 8192; }  // in the backward
inline int lanes_of(int64_t h) { return h <= 64 ? 8 : h <= 128 ? 16 : 32; }
inline int64_t lane_blocks(int64_t rows, int64_t h) {
    const int64_t of_block = kLanesThreads / lanes_of(h);
    return (rows + of_block - 1) / of_block;
}

// Eight columns from c on; zeros past the row's end.
template <typename T>
__device__ __forceinline__ void load_vector(const T *x, int c, int h, Raw8<T> &v) {
    if (c < h)
        v = load8(x + c);
    else
        zero8(v);
}
__device__ __forceinline__ void load_weights(const float *w, int c, int h, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (c < h) load8f(w + c, v);
}
// The vectors of a row that are this thread's.
template <typename T, int VPT>
__device__ __forceinline__ void load_row(const T *x, int h, int lane, int lanes, Raw8<T> (&v)[VPT]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) load_vector(x, (lane + i * lanes) * 8, h, v[i]);
}
template <int VPT>
__device__ __forceinline__ void load_row_weights(const float *w, int h, int lane, int lanes, float (&v)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) load_weights(w, (lane + i * lanes) * 8, h, v[i]);
}

// ------------------------------------------------------------------ the ring
// Stage n % stages holds the n-th row of this block: the rows of up to three
// tensors, each of `bytes`. Thread 0 fills a stage again after a barrier that
// every thread passes when it has read the stage. Waits are bounded (ptx.cuh):
// after one that ran out nothing more is copied, and the block stays for the time
// that a drain may take, in which what is under way to its shared memory lands.
// (Which stages are still being filled is not counted: the counter cost wide rows
// in fp32 2% of their time in every launch.)
struct Ring {
    uint8_t *data;
    uint64_t *full;
    volatile int *abort;
    uint32_t *err;
    int stages, bytes, tensors;

    // withhold: block 0 counts bytes on its first row that nothing copies, so that the wait
    // for it runs out (tpce_debug_withhold_next_load)
    __device__ void init(int withhold) {
        if (threadIdx.x == 0) {
            *abort = 0;
            for (int i = 0; i < stages; ++i) ptx::mbar_init(full + i, 1);
            if (withhold && blockIdx.x == 0)
                asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(ptx::smem_u32(full))
                             : "memory");
            ptx::fence_mbar_init();
        }
        __syncthreads();
    }
    // thread 0 only: the rows at `offset` bytes of the tensors into a stage
    __device__ void fill(int stage, const void *a, const void *b, const void *c, int64_t offset) {
        if (*abort) return;
        ptx::mbar_arrive_expect_tx(full + stage, static_cast<uint32_t>(bytes) * tensors);
        uint8_t *to = data + stage * bytes * tensors;
        copy(to, a, offset, stage);
        if (tensors > 1) copy(to + bytes, b, offset, stage);
        if (tensors > 2) copy(to + 2 * bytes, c, offset, stage);
    }
    __device__ void copy(void *dst, const void *src, int64_t offset, int stage) {
        // read once: first to leave L2
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
            "%4;" ::"r"(ptx::smem_u32(dst)),
            "l"(static_cast<const uint8_t *>(src) + offset), "r"(bytes), "r"(ptx::smem_u32(full + stage)),
            "l"(ptx::l2_policy_evict_first())
            : "memory");
    }
    __device__ void wait(int stage, int phase) { ptx::mbar_wait(full + stage, phase, abort, err, 20u); }
    // one thread, after the last row
    __device__ void leave() {
        if (!*abort) return;
        for (const uint64_t t0 = ptx::globaltimer(); ptx::globaltimer() - t0 < kDrainLimitNs;) {
        }
    }
};

// ------------------------------------------------------------------ forward
template <typename T, int VPT, int GROUP_LANES>
struct ForwardRow {
    float s[VPT][8];

    // S of this thread's vectors, to S + off of the row; returns the sum of their squares
    __device__ __forceinline__ float add(const Raw8<T> (&x)[VPT], const Raw8<T> (&r)[VPT], bool residual, T *S,
                                         int64_t off, int h, int lane, int lanes) {
        float sq = 0.0f, sq1 = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (residual) {
                Raw8<T> o;
                add8(x[i], r[i], o);
                const int c = (lane + i * lanes) * 8;
                if (c < h) stream8(S + off + c, o);
                unpack8(o, s[i]);
            } else {
                unpack8(x[i], s[i]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) fma2(sq, sq1, s[i][2 * j], s[i][2 * j + 1], s[i][2 * j], s[i][2 * j + 1]);
        }
        return sq + sq1;
    }

    // the row's columns up to h; its scales begin at Qs
    __device__ __forceinline__ void finish(float rstd, const float (&w)[VPT][8], T *Y, uint8_t *Q, float *Qs,
                                           int64_t off, int h, int lane, int lanes) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (lane + i * lanes) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mul2(s[i][2 * j], s[i][2 * j + 1], rstd, rstd);
                mul2(s[i][2 * j], s[i][2 * j + 1], w[i][2 * j], w[i][2 * j + 1]);
            }
            if (Y && c < h) {
                Raw8<T> o;
                pack8(s[i], o);
                store8(Y + off + c, o);
            }
            if (Q) {
                // lanes past the row's end bring zeros
                if (c >= h) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[i][j] = 0.0f;
                }
                float scale;
                const uint2 q = quantize8<GROUP_LANES>(s[i], scale);
                if (c < h) {
                    *reinterpret_cast<uint2 *>(Q + off + c) = q;
                    if (lane % GROUP_LANES == 0) Qs[c / kGroup] = scale;
                }
            }
        }
    }
};

__device__ __forceinline__ float rstd_of(float total, float inv_h, float eps) { return rsqrtf(total * inv_h + eps); }

// LANES lanes a row, 256 / LANES rows a block at a time. The lanes of a warp
// leave together: a row past the last has no columns. 131,072 x 256 bf16 with the
// residual: 43 us, 6.3 TB/s.
template <typename T, int LANES>
__global__ void __launch_bounds__(kLanesThreads, 4)
    rmsnorm_forward_lanes_kernel(const T *X, const T *R, const float *w, int64_t rows, int h, float eps, T *S, T *Y,
                                 uint8_t *Q, float *Qs, float *__restrict__ rstd) {
    grid_begin();
    const int lane = threadIdx.x % LANES;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kLanesThreads / LANES);
    const float inv_h = 1.0f / static_cast<float>(h);
    const int groups = (h + kGroup - 1) / kGroup;
    int64_t first = (static_cast<int64_t>(blockIdx.x) * kLanesThreads + (threadIdx.x & ~31u)) / LANES;  // the warp's
    int64_t row = first + (threadIdx.x & 31) / LANES;
    float wv[1][8];
    load_row_weights(w, h, lane, LANES, wv);
    Raw8<T> x[1], r[1];
    auto load = [&](int64_t at) {
        const int end = at < rows ? h : 0;
        load_row(X + at * h, end, lane, LANES, x);
        if (R) load_row(R + at * h, end, lane, LANES, r);
    };
    load(row);
    for (; first < rows; first += stride, row += stride) {
        const int end = row < rows ? h : 0;
        ForwardRow<T, 1, LANES < 16 ? LANES : 16> f;
        const float sq = f.add(x, r, R, S, row * h, end, lane, LANES);
        load(row + stride);  // the next row is on its way while this one is summed and written
        const float v = rstd_of(warp_sum<LANES>(sq), inv_h, eps);
        if (lane == 0 && end) rstd[row] = v;
        f.finish(v, wv, Y, Q, Qs + row * groups, row * h, end, lane, LANES);
    }
}

// A row a block. RING where a block has several rows to come; with one row there
// is nothing to fetch ahead, and the ring would only add its latency. One token
// of 8192 takes 6 us a call, the host's part; 16,384 x 8192 bf16 with the
// residual 157 us, 6.8 TB/s, as fast as a copy; 4096 of them with the 8-bit
// output 50 us, 6.0 TB/s (what is lost is the start and the end of the launch).
// What is read once and S, which waits for the end of the block, are marked to
// leave L2 first (57 us without, for the last); Y is what the next product reads.
template <typename T, int VPT, bool RING>
__global__ void __launch_bounds__(1024)
    rmsnorm_forward_block_kernel(const T *X, const T *R, const float *w, int64_t rows, int h, float eps,
                                 T *S, T *Y, uint8_t *Q, float *Qs, float *__restrict__ rstd, int stages,
                                 int withhold, uint32_t *err) {
    extern __shared__ __align__(128) uint8_t data[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ int abort;
    __shared__ float red[2][32];
    const int lane = threadIdx.x, lanes = blockDim.x;
    const int groups = (h + kGroup - 1) / kGroup;
    const float inv_h = 1.0f / static_cast<float>(h);
    const int64_t stride = gridDim.x, row_bytes = static_cast<int64_t>(h) * sizeof(T);
    Ring ring{data, full, &abort, err, stages, static_cast<int>(row_bytes), R ? 2 : 1};
    if (RING) ring.init(withhold);
    grid_begin();
    if (RING) {
        int64_t r = blockIdx.x;
        if (lane == 0)
            for (int i = 0; i < stages && r < rows; ++i, r += stride) ring.fill(i, X, R, nullptr, r * row_bytes);
    }
    float wv[VPT][8];
    load_row_weights(w, h, lane, lanes, wv);
    int stage = 0, phase = 0, turn = 0;
    const int64_t step = stride * h;
    int64_t off = static_cast<int64_t>(blockIdx.x) * h;
    for (int64_t row = blockIdx.x; row < rows; row += stride, off += step, turn ^= 1) {
        Raw8<T> x[VPT], r[VPT];
        if (RING) {
            ring.wait(stage, phase);
            const uint8_t *at = data + stage * ring.bytes * ring.tensors;
            load_row(reinterpret_cast<const T *>(at), h, lane, lanes, x);
            if (R) load_row(reinterpret_cast<const T *>(at + ring.bytes), h, lane, lanes, r);
        } else {
            load_row(X + off, h, lane, lanes, x);
            if (R) load_row(R + off, h, lane, lanes, r);
        }
        ForwardRow<T, VPT, 16> f;
        const float sq = f.add(x, r, R, S, off, h, lane, lanes);
        const float total = block_sum(sq, red[turn]);  // its barrier: every thread has read the stage
        if (RING) {
            if (lane == 0 && row + stages * stride < rows)
                ring.fill(stage, X, R, nullptr, (row + stages * stride) * row_bytes);
            if (++stage == stages) stage = 0, phase ^= 1;
        }
        const float v = rstd_of(total, inv_h, eps);
        if (lane == 0) rstd[row] = v;
        f.finish(v, wv, Y, Q, Qs + row * groups, off, h, lane, lanes);
    }
    if (RING && lane == 0) ring.leave();
}

// ------------------------------------------------------------------ backward
// dY xh goes to dw; returns this thread's part of sum g xh.
template <typename T>
__device__ __forceinline__ float backward_dots(const Raw8<T> &y, const Raw8<T> &x, const float (&w)[8], float rstd,
                                               float (&dw)[8]) {
    float c0 = 0.0f, c1 = 0.0f;
    float g[8], xh[8];
    unpack8(y, g);
    unpack8(x, xh);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        mul2(xh[j], xh[j + 1], rstd, rstd);
        fma2(dw[j], dw[j + 1], g[j], g[j + 1], xh[j], xh[j + 1]);
        mul2(g[j], g[j + 1], w[j], w[j + 1]);
        fma2(c0, c1, g[j], g[j + 1], xh[j], xh[j + 1]);
    }
    return c0 + c1;
}

// c = sum g xh / h; to dX where the columns are inside
template <typename T>
__device__ __forceinline__ void backward_finish(float c, float rstd, const Raw8<T> &y, const Raw8<T> &x,
                                                const float (&w)[8], const Raw8<T> &d, bool residual, T *dX,
                                                bool inside) {
    float g[8], xh[8];
    unpack8(y, g);
    unpack8(x, xh);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        mul2(xh[j], xh[j + 1], rstd, rstd);
        mul2(g[j], g[j + 1], w[j], w[j + 1]);
        mul2(g[j], g[j + 1], rstd, rstd);
        fma2(g[j], g[j + 1], xh[j], xh[j + 1], -c * rstd, -c * rstd);
    }
    if (residual) {
        float b[8];
        unpack8(d, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] += b[j];
    }
    Raw8<T> out;
    pack8(g, out);
    if (inside) stream8(dX, out);
}

__device__ __forceinline__ void store_partial(float *part, const float (&dw)[8]) {
    float4 *o = reinterpret_cast<float4 *>(part);
    o[0] = make_float4(dw[0], dw[1], dw[2], dw[3]);
    o[1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
}

// Narrow rows. The values of the rows ahead are a warp's own in shared memory, so
// that its lanes wait for one another only: 131,072 x 256 bf16 take 45 us,
// 6.0 TB/s; with one row ahead in registers instead it was 57.
// Four rows of bf16 or two of fp32 are 52 KB: four blocks an SM either way.
template <typename T>
constexpr int kAhead = 8 / static_cast<int>(sizeof(T));
template <typename T>
constexpr int lanes_stage_bytes() {
    return kLanesThreads * (3 * 8 * static_cast<int>(sizeof(T)) + 4);
}
// `bytes` (4 or 16) from global to shared memory, zeros where there is nothing to read
template <int BYTES>
__device__ __forceinline__ void copy_async(void *to, const void *from, bool there) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(to)), "l"(from),
                     "r"(there ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(to)), "l"(from),
                     "r"(there ? 4 : 0)
                     : "memory");
}

template <typename T, int LANES>
__global__ void __launch_bounds__(kLanesThreads, 4)
    rmsnorm_backward_lanes_kernel(const T *dY, const T *S, const float *w, const float *rstd, const T *dS,
                                  int64_t rows, int h, T *dX, float *__restrict__ part) {
    extern __shared__ __align__(128) uint8_t data[];
    grid_begin();
    const int lane = threadIdx.x % LANES;
    const float inv_h = 1.0f / static_cast<float>(h);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kLanesThreads / LANES);
    int64_t first = (static_cast<int64_t>(blockIdx.x) * kLanesThreads + (threadIdx.x & ~31u)) / LANES;  // the warp's
    int64_t row = first + (threadIdx.x & 31) / LANES;
    float wv[8], dw[8] = {};
    load_weights(w, lane * 8, h, wv);
    // [stage][tensor][thread][16-byte piece], then the statistic: [thread]
    constexpr int kPieces = sizeof(T) / 2, kStage = lanes_stage_bytes<T>();
    const int warp = threadIdx.x & ~31, of_warp = threadIdx.x & 31;
    auto slot = [&](int stage, int i, int thread) {
        const int tensor = i / kPieces, piece = i % kPieces;
        return reinterpret_cast<uint4 *>(data + stage * kStage +
                                         ((tensor * kLanesThreads + thread) * kPieces + piece) * 16);
    };
    auto statistic = [&](int stage) {
        return reinterpret_cast<float *>(data + stage * kStage + 3 * kPieces * kLanesThreads * 16) + threadIdx.x;
    };
    // the rows from `at` on of this warp; adjacent lanes copy adjacent pieces, whichever lane they are for
    auto fill = [&](int stage, int64_t at) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int q = of_warp + i * 32, owner = q / kPieces, piece = q % kPieces;
            const int64_t mine = at + owner / LANES;
            const int c = owner % LANES * 8;
            const bool there = mine < rows && c < h;
            const int64_t off = there ? mine * h + c + piece * (16 / static_cast<int>(sizeof(T))) : 0;
            copy_async<16>(slot(stage, piece, warp + owner), dY + off, there);
            copy_async<16>(slot(stage, kPieces + piece, warp + owner), S + off, there);
            if (dS) copy_async<16>(slot(stage, 2 * kPieces + piece, warp + owner), dS + off, there);
        }
        const int64_t mine = at + of_warp / LANES;
        copy_async<4>(statistic(stage), rstd + (mine < rows ? mine : 0), mine < rows);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](int stage, int t, Raw8<T> &v) {
        uint4 *to = reinterpret_cast<uint4 *>(&v);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) to[i] = *slot(stage, t * kPieces + i, threadIdx.x);
    };
#pragma unroll
    for (int i = 0; i < kAhead<T>; ++i) fill(i, first + i * stride);
    int stage = 0;
    for (; first < rows; first += stride, row += stride) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead<T> - 1) : "memory");
        __syncwarp();
        Raw8<T> y, x, d;
        take(stage, 0, y);
        take(stage, 1, x);
        if (dS) take(stage, 2, d);
        const float r = *statistic(stage);
        const float c = warp_sum<LANES>(backward_dots(y, x, wv, r, dw)) * inv_h;
        backward_finish(c, r, y, x, wv, d, dS, dX + row * h + lane * 8, row < rows && lane * 8 < h);
        __syncwarp();  // every lane has read the stage
        fill(stage, first + kAhead<T> * stride);
        if (++stage == kAhead<T>) stage = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!part) return;
    // the block's rows hold the same columns: add them in their order
    constexpr int kColumns = LANES * 8;
    float *fold = reinterpret_cast<float *>(data);  // 8 KB: less than a stage, and no copy is under way
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) fold[threadIdx.x / LANES * kColumns + lane * 8 + j] = dw[j];
    __syncthreads();
    const int c = threadIdx.x;  // 256 threads, up to 256 columns
    if (c < h) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kLanesThreads / LANES; ++q) s += fold[q * kColumns + c];
        part[static_cast<int64_t>(blockIdx.x) * h + c] = s;
    }
}

// A row a block, eight columns a thread and the sums of their dw in its registers
// over all its rows, so the blocks are as many as have a place and their rows are
// divided evenly. 16,384 x 8192 bf16 with the residual path: 158 us with the sum
// of the blocks' dw, 6.8 TB/s, as fast as a copy; 8192 x 4096 44 us, 6.0 TB/s;
// 65,536 x 512 47 us, 5.7 TB/s, where every row's sum costs its two warps as much
// as its values.
template <typename T, bool RING>
__global__ void __launch_bounds__(1024)
    rmsnorm_backward_block_kernel(const T *dY, const T *S, const float *w, const float *rstd,
                                  const T *dS, int64_t rows, int h, T *dX, float *__restrict__ part, int stages,
                                  int withhold, uint32_t *err) {
    extern __shared__ __align__(128) uint8_t data[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ int abort;
    __shared__ float red[2][32];
    const int col = threadIdx.x * 8;
    const int64_t stride = gridDim.x, row_bytes = static_cast<int64_t>(h) * sizeof(T);
    Ring ring{data, full, &abort, err, stages, static_cast<int>(row_bytes), dS ? 3 : 2};
    if (RING) ring.init(withhold);
    grid_begin();
    if (RING) {
        int64_t r = blockIdx.x;
        if (threadIdx.x == 0)
            for (int i = 0; i < stages && r < rows; ++i, r += stride) ring.fill(i, dY, S, dS, r * row_bytes);
    }
    float wv[8], dw[8] = {};
    load_weights(w, col, h, wv);
    const float inv_h = 1.0f / static_cast<float>(h);
    int stage = 0, phase = 0, turn = 0;
    const int64_t step = stride * h;
    int64_t off = static_cast<int64_t>(blockIdx.x) * h;
    for (int64_t row = blockIdx.x; row < rows; row += stride, off += step, turn ^= 1) {
        const float r = rstd[row];
        Raw8<T> y, x, d;
        if (RING) {
            ring.wait(stage, phase);
            const uint8_t *at = data + stage * ring.bytes * ring.tensors;
            load_vector(reinterpret_cast<const T *>(at), col, h, y);
            load_vector(reinterpret_cast<const T *>(at + ring.bytes), col, h, x);
            if (dS) load_vector(reinterpret_cast<const T *>(at + 2 * ring.bytes), col, h, d);
        } else {
            load_vector(dY + off, col, h, y);
            load_vector(S + off, col, h, x);
            if (dS) load_vector(dS + off, col, h, d);
        }
        // its barrier: every thread has read the stage
        const float total = block_sum(backward_dots(y, x, wv, r, dw), red[turn]);
        if (RING) {
            if (threadIdx.x == 0 && row + stages * stride < rows)
                ring.fill(stage, dY, S, dS, (row + stages * stride) * row_bytes);
            if (++stage == stages) stage = 0, phase ^= 1;
        }
        backward_finish(total * inv_h, r, y, x, wv, d, dS, dX + off + col, col < h);
    }
    if (RING && threadIdx.x == 0) ring.leave();
    if (part && col < h) store_partial(part + static_cast<int64_t>(blockIdx.x) * h + col, dw);
}

// Rows of more than 8192 values are shared by the two blocks of a cluster, still
// eight columns a thread: in one block a thread would hold four vectors, whose
// sums leave its registers no room for the weights, and reading those from L2 for
// each row costs as much as the row (121 us for 4096 x 16384).
//
// Each warp sends its sum to both blocks, as a store that the receiver's barrier
// counts: a barrier of the cluster, or a fence, would wait for the rows' stores as
// well (122 and 162 us). Row n + 1's products are summed before row n is finished,
// so that its sum is on the way meanwhile, and row n is read from its stage again
// for that. The last warp fills a stage when every warp has finished its row.
// A warp sends row n's sum after it has finished row n - 2, and so after every
// warp of both blocks has sent that of row n - 2, having read that of row n - 4:
// four buffers.
//
// 4096 x 16384 bf16 with the residual path: 104 us, 5.2 TB/s (110 where a row is
// finished before the next is begun); 16,384 rows 385 us, 5.6 TB/s. Bound by the
// 0.9 us that a warp takes from a row's wait to its store, whatever the width
// (each SM has twice the rows here), and by its instructions, 69% of the cycles.
__host__ __device__ __forceinline__ int half_of_row(int h) { return (h / 8 + 1) / 2 * 8; }

// x to shared memory of a block of the cluster, whose barrier counts the bytes
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, float x) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to),
                 "r"(__float_as_uint(x)), "r"(bar)
                 : "memory");
}
// ptx::mbar_wait for what the other block sends
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t *err) {
    auto test = [&] {
        uint32_t there;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(there)
            : "r"(ptx::smem_u32(bar)), "r"(parity)
            : "memory");
        return there != 0;
    };
    return test() || (ptx::mbar_wait(bar, parity, abort, err, 21u) && test());
}

template <typename T>
__global__ void __launch_bounds__(1024)
    rmsnorm_backward_pair_kernel(const T *dY, const T *S, const float *w, const float *rstd, const T *dS, int64_t rows,
                                 int h, T *dX, float *__restrict__ part, int stages, int tensors, int withhold,
                                 uint32_t *err) {
    extern __shared__ __align__(128) uint8_t data[];
    __shared__ uint64_t full[kPairStages], empty[kPairStages], ready[4];
    __shared__ float sums[4][64];  // [row % 4][block][warp]
    __shared__ int abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, col = threadIdx.x * 8;
    const bool filler = threadIdx.x == blockDim.x - 32;
    const uint32_t rank = ptx::cluster_ctarank();
    // this block's columns, from `begin` on
    const int half = half_of_row(h), begin = rank ? half : 0, columns = rank ? h - half : half;
    const int64_t pairs = gridDim.x / 2, first = blockIdx.x / 2;
    const int64_t mine = first < rows ? (rows - first + pairs - 1) / pairs : 0;
    Ring ring{data, full, &abort, err, stages, columns * static_cast<int>(sizeof(T)), tensors};
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) ptx::mbar_init(empty + i, warps);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(ready + i, 1);
    }
    ring.init(withhold);
    ptx::cluster_sync();  // the other block's barriers are there before anything is sent to them
    grid_begin();
    int64_t filled = 0;
    auto fill = [&](int stage) {
        ring.fill(stage, dY, S, dS, ((first + filled * pairs) * h + begin) * sizeof(T));
        ++filled;
    };
    if (filler)
        while (filled < stages && filled < mine) fill(static_cast<int>(filled));
    float wv[8], dw[8] = {};
    load_weights(w + begin, col, columns, wv);
    const float inv_h = 1.0f / static_cast<float>(h);
    const float *statistic = rstd + first;
    float next = mine > 0 ? *statistic : 0.0f, r = 0.0f;
    const int64_t step = pairs * h;
    int64_t off = first * h + begin + col;
    int in = 0, in_phase = 0, out = 0, out_phase = 0;
    for (int64_t n = 0; n <= mine; ++n) {
        Raw8<T> y, x, d;
        const float before = r;
        if (n < mine) {  // row n: its products
            r = next;
            statistic += pairs;
            if (n + 1 < mine) next = *statistic;
            ring.wait(in, in_phase);
            const uint8_t *at = data + in * ring.bytes * ring.tensors;
            load_vector(reinterpret_cast<const T *>(at), col, columns, y);
            load_vector(reinterpret_cast<const T *>(at + ring.bytes), col, columns, x);
            const float sum = warp_sum(backward_dots(y, x, wv, r, dw));
            const int turn = static_cast<int>(n & 3);
            if (threadIdx.x == 0) ptx::mbar_arrive_expect_tx(ready + turn, static_cast<uint32_t>(2 * warps) * 4u);
            if (lane < 2)
                send(ptx::mapa_shared(ptx::smem_u32(&sums[turn][rank * 32 + warp]), lane),
                     ptx::mapa_shared(ptx::smem_u32(ready + turn), lane), sum);
            if (++in == stages) in = 0, in_phase ^= 1;
        }
        if (n == 0) continue;
        // row n - 1: its dX
        if (dS && tensors < 3) {
            if (col < columns) d = load8(dS + off);
        }
        const int turn = static_cast<int>((n - 1) & 3);
        // (a whole warp leaves, and a block in which a wait ran out sends nothing more)
        if (!__all_sync(0xffffffffu, wait_cluster(ready + turn, ((n - 1) >> 2) & 1, &abort, err))) break;
        const float c = warp_sum(lane < warps ? sums[turn][lane] + sums[turn][32 + lane] : 0.0f) * inv_h;
        const uint8_t *at = data + out * ring.bytes * ring.tensors;
        load_vector(reinterpret_cast<const T *>(at), col, columns, y);
        load_vector(reinterpret_cast<const T *>(at + ring.bytes), col, columns, x);
        if (tensors == 3) load_vector(reinterpret_cast<const T *>(at + 2 * ring.bytes), col, columns, d);
        backward_finish(c, before, y, x, wv, d, dS, dX + off, col < columns);
        off += step;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty + out);
        if (filler && filled < mine) {
            ptx::mbar_wait(empty + out, out_phase, &abort, err, 22u);
            fill(out);
        }
        if (++out == stages) out = 0, out_phase ^= 1;
    }
    ptx::cluster_sync();  // neither block leaves while the other may send to it
    // A block that has waited for every row's sums has received all that was sent to it;
    // to one that gave up, what was sent before the barrier may still be on its way.
    if (threadIdx.x == 0) ring.leave();
    if (part && col < columns) store_partial(part + first * h + begin + col, dw);
}

// dw[c] = the blocks' partial sums, always in the same order: COLS columns a block,
// its threads adding every 1024 / COLS-th row, then lanes and warps. 2 us, mostly
// the launch's; a row of partial sums for each block is 0.5% of what 16,384 x 8192
// reads. 8 columns a block up to 2048 of them (10,273 x 728 bf16 backward 17.5 us
// instead of 20.1), 32 beyond (8192 x 4096 44.9 instead of 46.5). A launch after it
// that began before its end made the next backward 57 us instead of 46 at 32,768 x
// 1024, and a forward and a backward of 65,536 x 512 131 instead of 99.
template <int COLS>
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float *part, int rows, int h,
                                                          float *__restrict__ dw) {
    __shared__ float red[32][COLS];
    grid_begin_alone();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * COLS + lane % COLS;
    float s = 0.0f;
    if (c < h) {
#pragma unroll 8
        for (int r = threadIdx.x / COLS; r < rows; r += 1024 / COLS) s += part[static_cast<int64_t>(r) * h + c];
    }
#pragma unroll
    for (int d = COLS; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane < COLS) red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && lane < COLS && c < h) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += red[i][lane];
        dw[c] = s;
    }
}

// ------------------------------------------------------------------ host
// Vectors a thread holds, threads of a block, blocks of an SM. `halves`: the
// forward of bf16 rows without a residual, of which one vector is 16 bytes a thread
// and row; two a thread, and with them twice as many rows at a time on an SM: 8192
// x 4096 bf16 and 8 bits 30 us instead of 37, 65,536 x 512 21 instead of 28. Where
// a vector is 32 bytes already two take longer (10,146 x 3768 with the residual 59
// and 57 us, 16,384 x 1000 fp32 24.4 and 22.9).
// The backward's blocks each leave a row to the sum of dw: up to 8 on an SM, and 12
// where that is little beside their own rows, from 32,768 of them on, where both take
// the same (512 values: 28.5 us either way; 4000 rows 8.8 with 8 and 9.2 with 12,
// 16,384 17.6 and 18.5, 131,072 91.0 and 87.7; 264 values: 27.5 and 26.5, 16.9 and
// 17.1 for 16,384 rows, 88.5 and 80.1 for 131,072).
struct Layout {
    int vpt, threads, blocks;
};
inline Layout layout_of(int64_t h, int64_t rows, bool backward, bool halves = false) {
    if (lane_rows(h)) return {1, kLanesThreads, 4};
    const int v = static_cast<int>(backward && pair_rows(h) ? half_of_row(static_cast<int>(h)) / 8 : h / 8);
    const int vpt = backward || (v <= 512 && !halves) ? 1 : 2;
    const int threads = ((v + vpt - 1) / vpt + 31) / 32 * 32;
    return {vpt, threads, std::min(!backward ? 16 : rows < 32768 ? 8 : 12, 1024 / threads)};
}

// Stages of the ring where `blocks` blocks share an SM; fewer blocks where two
// stages would not fit, 0 stages where they do not fit even then. A block of the
// backward asks for its whole share, so that no SM takes more than `blocks` of
// them: its rows are divided evenly, and blocks that begin while the kernel
// before them ends would pile up on the SMs that were free first (1.6 times the
// time at h = 512). The forward's blocks are more than have a place.
inline int share_of(int blocks) { return kSmemPerSm / blocks - 2048; }
inline int stages_of(int64_t stage_bytes, int &blocks) {
    for (; blocks >= 1; --blocks) {
        const int64_t n = share_of(blocks) / stage_bytes;
        if (n >= 2) return static_cast<int>(std::min<int64_t>(n, kMaxStages));
    }
    blocks = 1;
    return 0;
}

// Blocks of the backward at most (pairs of blocks), and so rows of its partial sums.
inline int64_t backward_blocks(int64_t T, int64_t h) {
    if (pair_rows(h)) return std::min<int64_t>(T, kSms / 2);
    return std::min<int64_t>(lane_rows(h) ? lane_blocks(T, h) : T, layout_of(h, T, true).blocks * kSms);
}

// More than 48 KB of shared memory, what the kernel declares among it, has to be
// asked for (`most`, what any launch of the kernel takes), once for each kernel
// and device.
template <auto Kernel>
struct Fn {
    static cudaError_t allow(int bytes, int most) {
        static std::atomic<uint64_t> done{0};
        int dev = 0;
        cudaError_t e = taken(cudaGetDevice(&dev));
        if (e != cudaSuccess || bytes <= 40 * 1024) return e;
        const uint64_t bit = uint64_t{1} << (dev & 63);
        if (done.load() & bit) return cudaSuccess;
        e = taken(cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
        if (e == cudaSuccess) done.fetch_or(bit);
        return e;
    }
    static constexpr auto fn = Kernel;
};

tpce_status check_shape(int64_t T, int64_t h, int dtype) {
    if (dtype != TPCE_BF16 && dtype != TPCE_F32) return fail(TPCE_ERR_INVALID, "rmsnorm: dtype %d", dtype);
    if (T < 0 || T > kMaxRows || h < 8 || h % 8 != 0 || h > kMaxWidth)
        return fail(TPCE_ERR_SHAPE, "rmsnorm: T = %lld, h = %lld (h a multiple of 8 up to %lld)",
                    static_cast<long long>(T), static_cast<long long>(h), static_cast<long long>(kMaxWidth));
    return TPCE_OK;
}

template <typename T>
tpce_status forward(const void *X, const void *R, const float *w, int64_t rows, int h, float eps, void *S, void *Y,
                    void *Q, float *Qs, float *rstd, cudaStream_t s) {
    Layout L = layout_of(h, rows, false, sizeof(T) == 2 && !R);
    const T *x = static_cast<const T *>(X), *r = static_cast<const T *>(R);
    T *so = static_cast<T *>(S), *yo = static_cast<T *>(Y);
    uint8_t *q = static_cast<uint8_t *>(Q);
    // the grids below are multiples of it, and rows are divided by it
    const int sms = num_sms();
    if (sms <= 0) return fail(TPCE_ERR_CUDA, "rmsnorm_forward: no usable device");
    KernelTimer timer("rmsnorm_forward", s);
    if (lane_rows(h)) {
        const unsigned grid = static_cast<unsigned>(
            std::min<int64_t>(lane_blocks(rows, h), static_cast<int64_t>(sms) * L.blocks));
        auto go = [&](auto kernel) {
            return launch(kernel, grid, L.threads, 0, s, x, r, w, rows, h, eps, so, yo, q, Qs, rstd);
        };
        const int lanes = lanes_of(h);
        const cudaError_t e = lanes == 8    ? go(rmsnorm_forward_lanes_kernel<T, 8>)
                              : lanes == 16 ? go(rmsnorm_forward_lanes_kernel<T, 16>)
                                            : go(rmsnorm_forward_lanes_kernel<T, 32>);
        if (e != cudaSuccess) return fail_cuda(e, "rmsnorm_forward");
        return check_launch("rmsnorm_forward", s);
    }
    const int64_t stage_bytes = static_cast<int64_t>(h) * sizeof(T) * (R ? 2 : 1);
    const int stages = stages_of(stage_bytes, L.blocks);
    const int64_t fit = static_cast<int64_t>(sms) * L.blocks;
    const int of_block = kRowsOfBlock[R ? 0 : 1];
    // whole rounds of blocks with that many rows each or more: an SM that gets its bytes sooner takes more blocks
    const unsigned grid =
        static_cast<unsigned>(std::min<int64_t>(rows, std::max<int64_t>(1, rows / (of_block * fit)) * fit));
    // with one row a block there is nothing to fetch ahead
    const bool ring = stages > 0 && rows > fit;
    const int smem = ring ? static_cast<int>(stage_bytes * stages) : 0;
    auto go = [&](auto k) -> cudaError_t {
        const cudaError_t e = decltype(k)::allow(smem, share_of(1));
        if (e != cudaSuccess) return e;
        return launch(decltype(k)::fn, grid, L.threads, smem, s, x, r, w, rows, h, eps, so, yo, q, Qs, rstd, stages,
                      ring ? take_debug_withhold() : 0, device_error_word());
    };
    cudaError_t e;
    if (L.vpt == 1)
        e = ring ? go(Fn<rmsnorm_forward_block_kernel<T, 1, true>>{})
                 : go(Fn<rmsnorm_forward_block_kernel<T, 1, false>>{});
    else
        e = ring ? go(Fn<rmsnorm_forward_block_kernel<T, 2, true>>{})
                 : go(Fn<rmsnorm_forward_block_kernel<T, 2, false>>{});
    if (e != cudaSuccess) return fail_cuda(e, "rmsnorm_forward");
    return check_launch("rmsnorm_forward", s);
}

template <typename T>
tpce_status backward(const void *dY, const void *S, const float *w, const float *rstd, const void *dS, int64_t rows,
                     int h, void *dX, float *dw, float *part, cudaStream_t s) {
    Layout L = layout_of(h, rows, true);
    const T *y = static_cast<const T *>(dY), *x = static_cast<const T *>(S), *d = static_cast<const T *>(dS);
    T *out = static_cast<T *>(dX);
    if (!dw) part = nullptr;
    int64_t blocks = backward_blocks(rows, h);
    {
        KernelTimer timer("rmsnorm_backward", s);
        if (lane_rows(h)) {
            const int smem = kAhead<T> * lanes_stage_bytes<T>();
            blocks = std::min<int64_t>(blocks, kSms * (share_of(1) / smem));  // as many as have a place
            auto go = [&](auto k) -> cudaError_t {
                const cudaError_t e = decltype(k)::allow(smem, smem);
                if (e != cudaSuccess) return e;
                return launch(decltype(k)::fn, static_cast<unsigned>(blocks), L.threads, smem, s, y, x, w, rstd, d,
                              rows, h, out, part);
            };
            const int lanes = lanes_of(h);
            const cudaError_t e = lanes == 8    ? go(Fn<rmsnorm_backward_lanes_kernel<T, 8>>{})
                                  : lanes == 16 ? go(Fn<rmsnorm_backward_lanes_kernel<T, 16>>{})
                                                : go(Fn<rmsnorm_backward_lanes_kernel<T, 32>>{});
            if (e != cudaSuccess) return fail_cuda(e, "rmsnorm_backward");
        } else if (pair_rows(h)) {
            // a row in work, one of which the sum is on the way, and one ahead: three stages or more. For that
            // dS of wide fp32 rows stays out of the ring.
            const int bytes = half_of_row(h) * static_cast<int>(sizeof(T)), room = share_of(1) - 2048;
            const int tensors = dS && 3 * 3 * bytes <= room ? 3 : 2;
            const int stages = std::min(kPairStages, room / (tensors * bytes));
            const int smem = stages * tensors * bytes;
            using Pair = Fn<rmsnorm_backward_pair_kernel<T>>;
            cudaError_t e = Pair::allow(smem, room);
            if (e == cudaSuccess)
                e = launch_clusters(2, Pair::fn, static_cast<unsigned>(2 * blocks), L.threads, smem, s, y, x, w, rstd,
                                    d, rows, h, out, part, stages, tensors, take_debug_withhold(),
                                    device_error_word());
            if (e != cudaSuccess) return fail_cuda(e, "rmsnorm_backward");
        } else {
            const int64_t stage_bytes = static_cast<int64_t>(h) * sizeof(T) * (dS ? 3 : 2);
            const int stages = stages_of(stage_bytes, L.blocks);
            blocks = std::min<int64_t>(blocks, L.blocks * kSms);
            const bool ring = stages > 0 && rows > blocks;
            const int smem = ring ? share_of(L.blocks) : 0;
            auto go = [&](auto k) -> cudaError_t {
                const cudaError_t e = decltype(k)::allow(smem, share_of(1));
                if (e != cudaSuccess) return e;
                return launch(decltype(k)::fn, static_cast<unsigned>(blocks), L.threads, smem, s, y, x, w, rstd, d,
                              rows, h, out, part, stages, ring ? take_debug_withhold() : 0,
                              device_error_word());
            };
            const cudaError_t e = ring ? go(Fn<rmsnorm_backward_block_kernel<T, true>>{})
                                       : go(Fn<rmsnorm_backward_block_kernel<T, false>>{});
            if (e != cudaSuccess) return fail_cuda(e, "rmsnorm_backward");
        }
        tpce_status st = check_launch("rmsnorm_backward", s);
        if (st != TPCE_OK) return st;
    }
    if (!dw) return TPCE_OK;
    KernelTimer timer("rmsnorm_dw", s);
    const int columns = h <= 2048 ? 8 : 32;
    const cudaError_t e = launch(columns == 8 ? rmsnorm_dw_kernel<8> : rmsnorm_dw_kernel<32>,
                                 static_cast<unsigned>((h + columns - 1) / columns), 1024, 0, s, part,
                                 static_cast<int>(blocks), h, dw);
    if (e != cudaSuccess) return fail_cuda(e, "rmsnorm_dw");
    return check_launch("rmsnorm_dw", s);
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" size_t tpce_rmsnorm_workspace_bytes(int64_t T, int64_t h) {
    if (check_shape(T, h, TPCE_BF16) != TPCE_OK) return 0;
    return static_cast<size_t>(backward_blocks(T, h)) * h * sizeof(float);
}

extern "C" tpce_status tp_rmsnorm_forward(const void *X, const void *R, const float *w, int64_t T, int64_t h,
                                          float eps, int dtype, void *S, void *Y, void *Q, float *Q_scale,
                                          float *rstd, void *stream) {
    tpce_status st = check_shape(T, h, dtype);
    if (st != TPCE_OK) return st;
    if (!(eps >= 0.0f)) return fail(TPCE_ERR_INVALID, "tp_rmsnorm_forward: eps must be >= 0");
    if (T == 0) return TPCE_OK;
    if (!X || !w || !rstd || (R && !S) || (!Y && !Q) || (Q && !Q_scale))
        return fail(TPCE_ERR_INVALID, "tp_rmsnorm_forward: null pointer");
    for (const void *p : {X, R, static_cast<const void *>(w), static_cast<const void *>(S),
                          static_cast<const void *>(Y), static_cast<const void *>(Q),
                          static_cast<const void *>(Q_scale), static_cast<const void *>(rstd)})
        if (!aligned16(p)) return fail(TPCE_ERR_ALIGN, "tp_rmsnorm_forward: a pointer is not 16-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int hi = static_cast<int>(h);
    return dtype == TPCE_BF16 ? forward<__nv_bfloat16>(X, R, w, T, hi, eps, S, Y, Q, Q_scale, rstd, s)
                              : forward<float>(X, R, w, T, hi, eps, S, Y, Q, Q_scale, rstd, s);
}

extern "C" tpce_status tp_rmsnorm_backward(const void *dY, const void *S, const float *w, const float *rstd,
                                           const void *dS, int64_t T, int64_t h, int dtype, void *dX, float *dw,
                                           void *ws, size_t ws_bytes, void *stream) {
    tpce_status st = check_shape(T, h, dtype);
    if (st != TPCE_OK) return st;
    if (T > 0 && (!dY || !S || !w || !rstd || !dX))
        return fail(TPCE_ERR_INVALID, "tp_rmsnorm_backward: null pointer");
    for (const void *p : {dY, S, static_cast<const void *>(w), static_cast<const void *>(rstd), dS,
                          static_cast<const void *>(dX), static_cast<const void *>(dw), static_cast<const void *>(ws)})
        if (!aligned16(p)) return fail(TPCE_ERR_ALIGN, "tp_rmsnorm_backward: a pointer is not 16-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        // no tokens: an empty sum
        const cudaError_t e = dw ? taken(cudaMemsetAsync(dw, 0, sizeof(float) * h, s)) : cudaSuccess;
        return e == cudaSuccess ? TPCE_OK : fail_cuda(e, "tp_rmsnorm_backward");
    }
    if (dw && (!ws || ws_bytes < tpce_rmsnorm_workspace_bytes(T, h)))
        return fail(TPCE_ERR_WORKSPACE, "tp_rmsnorm_backward: %zu bytes of workspace needed, %zu given",
                    tpce_rmsnorm_workspace_bytes(T, h), ws ? ws_bytes : size_t{0});
    const int hi = static_cast<int>(h);
    float *part = static_cast<float *>(ws);
    return dtype == TPCE_BF16 ? backward<__nv_bfloat16>(dY, S, w, rstd, dS, T, hi, dX, dw, part, s)
                              : backward<float>(dY, S, w, rstd, dS, T, hi, dX, dw, part, s);
}
