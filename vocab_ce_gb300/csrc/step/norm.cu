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
// sum over the row and the output.
#include <algorithm>

#include "host.h"
#include "step/vec.cuh"

namespace tpce {
namespace {

using namespace step;

constexpr int64_t kMaxWidth = 16384;  // 4 vectors of 8 values for each of 512 threads
constexpr int64_t kMaxRows = int64_t{1} << 40;
constexpr int kWarps = 8;             // rows of a block where a warp takes a row
constexpr int64_t kBlocks = 304;      // blocks of the backward: two for each of 152 SMs (fixed, so that the
                                      // workspace's size is known on the host)

// A row of up to 1024 values is a warp's (no barrier in its sum), a wider one a block's.
inline bool warp_rows(int64_t h) { return h <= 1024; }

// Where a thread's row is and which of its vectors are the thread's.
template <bool WARP>
struct Place {
    int lane, lanes;       // this thread's place among those that share the row
    int64_t row, stride;   // first row, rows between
    __device__ Place() {
        if (WARP) {
            lane = threadIdx.x & 31;
            lanes = 32;
            row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
            stride = static_cast<int64_t>(gridDim.x) * kWarps;
        } else {
            lane = threadIdx.x;
            lanes = blockDim.x;
            row = blockIdx.x;
            stride = gridDim.x;
        }
    }
};

template <bool WARP>
__device__ __forceinline__ float row_sum(float x, float *buf) {
    return WARP ? warp_sum(x) : block_sum(x, buf);
}

// The vectors of row r of X that are this thread's; zeros past the row's end.
template <typename T, int VPT>
__device__ __forceinline__ void load_row(const T *X, int64_t r, int h, int lane, int lanes, Raw8<T> (&v)[VPT]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (lane + i * lanes) * 8;
        if (c < h)
            v[i] = load8(X + r * h + c);
        else
            zero8(v[i]);
    }
}

template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : 512)
    rmsnorm_forward_kernel(const T *X, const T *R, const float *__restrict__ w, int64_t rows, int h, float eps, T *S,
                           T *Y, uint8_t *Q, float *Qs, float *__restrict__ rstd_out) {
    __shared__ float red[2][32];
    Place<WARP> at;
    const int groups = (h + kGroup - 1) / kGroup;
    int turn = 0;
    Raw8<T> x[VPT], r[VPT];
    if (at.row < rows) {
        load_row(X, at.row, h, at.lane, at.lanes, x);
        if (R) load_row(R, at.row, h, at.lane, at.lanes, r);
    }
    for (int64_t row = at.row; row < rows; row += at.stride) {
        float s[VPT][8], sq = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            unpack8(x[i], s[i]);
            if (R) {
                float b[8];
                unpack8(r[i], b);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i][j] += b[j];
                Raw8<T> o;
                pack8(s[i], o);
                const int c = (at.lane + i * at.lanes) * 8;
                if (c < h) store8(S + row * h + c, o);
                unpack8(o, s[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sq += s[i][j] * s[i][j];
        }
        // the next row is on its way while this one is summed and written
        if (row + at.stride < rows) {
            load_row(X, row + at.stride, h, at.lane, at.lanes, x);
            if (R) load_row(R, row + at.stride, h, at.lane, at.lanes, r);
        }
        const float total = row_sum<WARP>(sq, red[turn & 1]);
        ++turn;
        const float rstd = 1.0f / sqrtf(total * (1.0f / static_cast<float>(h)) + eps);
        if (at.lane == 0) rstd_out[row] = rstd;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (at.lane + i * at.lanes) * 8;
            float wv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (c < h) load8f(w + c, wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] = s[i][j] * rstd * wv[j];
            if (Y && c < h) {
                Raw8<T> o;
                pack8(s[i], o);
                store8(Y + row * h + c, o);
            }
            if (Q) {
                const float scale = group_scale(group_amax(s[i]));  // lanes past the row's end bring zeros
                if (c < h) {
                    *reinterpret_cast<uint2 *>(Q + row * h + c) = encode8(s[i], 1.0f / scale);
                    if ((at.lane & 15) == 0) Qs[row * groups + c / kGroup] = scale;
                }
            }
        }
    }
}

template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarps : 512)
    rmsnorm_backward_kernel(const T *dY, const T *S, const float *__restrict__ w, const float *__restrict__ rstd_in,
                            const T *dS, int64_t rows, int h, T *dX, float *__restrict__ part) {
    __shared__ float red[2][32];
    __shared__ float fold[WARP ? kWarps * 32 * 8 : 1];
    Place<WARP> at;
    int turn = 0;
    float dw[VPT][8] = {};
    Raw8<T> y[VPT], x[VPT], d[VPT];
    if (at.row < rows) {
        load_row(dY, at.row, h, at.lane, at.lanes, y);
        load_row(S, at.row, h, at.lane, at.lanes, x);
        if (dS) load_row(dS, at.row, h, at.lane, at.lanes, d);
    }
    for (int64_t row = at.row; row < rows; row += at.stride) {
        const float rstd = __ldg(rstd_in + row);
        float g[VPT][8], xh[VPT][8], c = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (at.lane + i * at.lanes) * 8;
            float wv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (col < h) load8f(w + col, wv);
            unpack8(y[i], g[i]);
            unpack8(x[i], xh[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] *= rstd;
                dw[i][j] += g[i][j] * xh[i][j];
                g[i][j] *= wv[j];
                c += g[i][j] * xh[i][j];
            }
        }
        c = row_sum<WARP>(c, red[turn & 1]) * (1.0f / static_cast<float>(h));
        ++turn;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int col = (at.lane + i * at.lanes) * 8;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = (g[i][j] - xh[i][j] * c) * rstd;
            if (dS) {
                float b[8];
                unpack8(d[i], b);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += b[j];
            }
            Raw8<T> out;
            pack8(o, out);
            if (col < h) store8(dX + row * h + col, out);
        }
        if (row + at.stride < rows) {
            load_row(dY, row + at.stride, h, at.lane, at.lanes, y);
            load_row(S, row + at.stride, h, at.lane, at.lanes, x);
            if (dS) load_row(dS, row + at.stride, h, at.lane, at.lanes, d);
        }
    }
    if (!part) return;
    float *mine = part + static_cast<int64_t>(blockIdx.x) * h;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int col = (at.lane + i * at.lanes) * 8;
        if (WARP) {
            // the block's warps hold the same columns: add them in warp order
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) fold[(threadIdx.x >> 5) * 256 + at.lane * 8 + j] = dw[i][j];
            __syncthreads();
            const int cc = i * 256 + threadIdx.x;  // 256 threads, the 256 columns of vector i
            if (cc < h) {
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) s += fold[q * 256 + threadIdx.x];
                mine[cc] = s;
            }
        } else if (col < h) {
            float4 *o = reinterpret_cast<float4 *>(mine + col);
            o[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            o[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dw[c] = the blocks' partial sums, always in the same order: 32 columns a block,
// each of 8 warps adding every eighth row.
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float *__restrict__ part, int rows, int h,
                                                         float *__restrict__ dw) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < h) {
#pragma unroll 4
        for (int r = warp; r < rows; r += 8) s += __ldg(part + static_cast<int64_t>(r) * h + c);
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < h) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        dw[c] = s;
    }
}

// Blocks of the backward and so rows of its partial sums.
inline int64_t backward_blocks(int64_t T, int64_t h) {
    return std::min<int64_t>(warp_rows(h) ? (T + kWarps - 1) / kWarps : T, kBlocks);
}

tpce_status check_shape(int64_t T, int64_t h, int dtype) {
    if (dtype != TPCE_BF16 && dtype != TPCE_F32) return fail(TPCE_ERR_INVALID, "rmsnorm: dtype %d", dtype);
    if (T < 0 || T > kMaxRows || h < 8 || h % 8 != 0 || h > kMaxWidth)
        return fail(TPCE_ERR_SHAPE, "rmsnorm: T = %lld, h = %lld (h a multiple of 8 up to %lld)",
                    static_cast<long long>(T), static_cast<long long>(h), static_cast<long long>(kMaxWidth));
    return TPCE_OK;
}

// Vectors a thread holds, and threads of a block.
struct Launch {
    int vpt, threads;
};
inline Launch launch_of(int64_t h) {
    const int v = static_cast<int>(h / 8);
    if (warp_rows(h)) return {v <= 32 ? 1 : v <= 64 ? 2 : 4, 32 * kWarps};
    const int vpt = v <= 512 ? 1 : v <= 1024 ? 2 : 4;
    return {vpt, ((v + vpt - 1) / vpt + 31) / 32 * 32};
}

template <typename T>
tpce_status forward(const void *X, const void *R, const float *w, int64_t rows, int h, float eps, void *S, void *Y,
                    void *Q, float *Qs, float *rstd, cudaStream_t s) {
    const Launch L = launch_of(h);
    const bool warp = warp_rows(h);
    const int64_t need = warp ? (rows + kWarps - 1) / kWarps : rows;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(need, static_cast<int64_t>(num_sms()) * (2048 / L.threads)));
    KernelTimer timer("rmsnorm_forward", s);
    auto go = [&](auto kernel) {
        kernel<<<grid, L.threads, 0, s>>>(static_cast<const T *>(X), static_cast<const T *>(R), w, rows, h, eps,
                                          static_cast<T *>(S), static_cast<T *>(Y), static_cast<uint8_t *>(Q), Qs,
                                          rstd);
    };
    if (warp) {
        if (L.vpt == 1) go(rmsnorm_forward_kernel<T, 1, true>);
        else if (L.vpt == 2) go(rmsnorm_forward_kernel<T, 2, true>);
        else go(rmsnorm_forward_kernel<T, 4, true>);
    } else {
        if (L.vpt == 1) go(rmsnorm_forward_kernel<T, 1, false>);
        else if (L.vpt == 2) go(rmsnorm_forward_kernel<T, 2, false>);
        else go(rmsnorm_forward_kernel<T, 4, false>);
    }
    return check_launch("rmsnorm_forward", s);
}

template <typename T>
tpce_status backward(const void *dY, const void *S, const float *w, const float *rstd, const void *dS, int64_t rows,
                     int h, void *dX, float *dw, float *part, cudaStream_t s) {
    const Launch L = launch_of(h);
    const unsigned grid = static_cast<unsigned>(backward_blocks(rows, h));
    {
        KernelTimer timer("rmsnorm_backward", s);
        auto go = [&](auto kernel) {
            kernel<<<grid, L.threads, 0, s>>>(static_cast<const T *>(dY), static_cast<const T *>(S), w, rstd,
                                              static_cast<const T *>(dS), rows, h, static_cast<T *>(dX),
                                              dw ? part : nullptr);
        };
        if (warp_rows(h)) {
            if (L.vpt == 1) go(rmsnorm_backward_kernel<T, 1, true>);
            else if (L.vpt == 2) go(rmsnorm_backward_kernel<T, 2, true>);
            else go(rmsnorm_backward_kernel<T, 4, true>);
        } else {
            if (L.vpt == 1) go(rmsnorm_backward_kernel<T, 1, false>);
            else if (L.vpt == 2) go(rmsnorm_backward_kernel<T, 2, false>);
            else go(rmsnorm_backward_kernel<T, 4, false>);
        }
        tpce_status st = check_launch("rmsnorm_backward", s);
        if (st != TPCE_OK) return st;
    }
    if (!dw) return TPCE_OK;
    KernelTimer timer("rmsnorm_dw", s);
    rmsnorm_dw_kernel<<<(h + 31) / 32, 256, 0, s>>>(part, static_cast<int>(grid), h, dw);
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
        if (dw && cudaMemsetAsync(dw, 0, sizeof(float) * h, s) != cudaSuccess) return TPCE_ERR_CUDA;
        return TPCE_OK;
    }
    if (dw && (!ws || ws_bytes < tpce_rmsnorm_workspace_bytes(T, h)))
        return fail(TPCE_ERR_WORKSPACE, "tp_rmsnorm_backward: %zu bytes of workspace needed, %zu given",
                    tpce_rmsnorm_workspace_bytes(T, h), ws ? ws_bytes : size_t{0});
    const int hi = static_cast<int>(h);
    float *part = static_cast<float *>(ws);
    return dtype == TPCE_BF16 ? backward<__nv_bfloat16>(dY, S, w, rstd, dS, T, hi, dX, dw, part, s)
                              : backward<float>(dY, S, w, rstd, dS, T, hi, dX, dw, part, s);
}
