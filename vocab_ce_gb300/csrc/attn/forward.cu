// forward.cu -- the attention core, forward: O = softmax(scale Q K^T) V over the
// keys that a query sees, and lse (attn.cuh has the formulas).
#include "attn/attn.cuh"
#include "attn/host.cuh"

namespace tpce {
namespace {

using namespace attn;

// ------------------------------------------------------------------ plain tiles
// Queries q0 .. q0 + 63 of one head. One pass over the keys with the running maximum
// m and sum l of each row: when m grows, what has been added so far is scaled down.
template <typename T>
__device__ __noinline__ void plain_forward_tile(const Shape &s, const T *QKV, int64_t row0, int n, int q0, int h,
                                                T *O, float *lse, float *smem) {
    const PlainSmem lay(s.d);
    float *Q = smem, *K = Q + lay.rows(), *V = K + lay.rows(), *P = V + lay.rows();
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int d = s.d, kv = h / s.group;
    const T *base = QKV + row0 * s.ld;
    const T *q = base + static_cast<int64_t>(s.q_head(h)) * d, *k = base + static_cast<int64_t>(s.k_head(kv)) * d,
            *v = base + static_cast<int64_t>(s.v_head(kv)) * d;
    const int q1 = min(n, q0 + kRows);
    const KeyTiles tiles = key_tiles(s, q0, q1, kRows);
    float m[4], l[4], o[4][2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) o[i][a][b] = 0.0f;
    }
    const float c = s.scale * kLog2e;
    plain_load(Q, lay.pitch, q, s.ld, q0, n, d);
    for (int u = 0; u < tiles.count(); ++u) {
        const int k0 = tiles.at(u) * kRows;
        plain_sync();
        plain_load(K, lay.pitch, k, s.ld, k0, n, d);
        plain_load(V, lay.pitch, v, s.ld, k0, n, d);
        plain_sync();
        float x[4][4];
        plain_dots(Q, K, lay.pitch, d, x);
        const bool masked = !all_seen(s, q0, q0 + kRows, k0, k0 + kRows);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = q0 + 4 * ty + i;
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] *= c;
                if (masked && !sees(s, row, k0 + tx + 16 * j)) x[i][j] = -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
            top = max16(top);
            const float at = top == -INFINITY ? 0.0f : top;  // no key yet: 2^-inf
            const float shrink = exp2f(m[i] - at);
            m[i] = top;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(x[i][j] - at);
                sum += p;
                P[(4 * ty + i) * kPitchP + tx + 16 * j] = p;
            }
            l[i] = l[i] * shrink + sum16(sum);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) o[i][a][b] *= shrink;
        }
        plain_sync();
        if (masked)
            plain_add<true, false>(P, V, lay.pitch, d, o);
        else
            plain_add<false, false>(P, V, lay.pitch, d, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = q0 + 4 * ty + i;
        if (row >= n) continue;
        const float inv = 1.0f / l[i];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int col = 4 * tx + 64 * a;
            if (col >= d) continue;
            float y[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) y[b] = o[i][a][b] * inv;
            store4(O + (row0 + row) * s.n_q * d + static_cast<int64_t>(h) * d + col, y);
        }
        if (tx == 0) lse[h * s.T + row0 + row] = (m[i] + log2f(l[i])) * kLn2;
    }
}

// The rows without a sequence: zeros in O and lse.
template <typename T>
__device__ __forceinline__ void forward_rest(const Shape &s, const Tile &t, int h, T *O, float *lse) {
    zero_rest(s, t, O, static_cast<int64_t>(s.n_q) * s.d, static_cast<int64_t>(h) * s.d);
    const int64_t rows = t.head_rows + (s.T - t.tail_row);
    for (int64_t r = static_cast<int64_t>(t.part) * blockDim.x + threadIdx.x; r < rows;
         r += static_cast<int64_t>(t.parts) * blockDim.x)
        lse[h * s.T + (r < t.head_rows ? r : t.tail_row + r - t.head_rows)] = 0.0f;
}

template <typename T>
__global__ void __launch_bounds__(kPlainThreads)
    plain_forward_kernel(const Shape s, const T *QKV, int tiles, T *O, float *lse) {
    extern __shared__ float4 smem4[];
    grid_begin();
    const int h = blockIdx.x % s.n_q;
    const Tile t = find_tile(s, blockIdx.x / s.n_q, kRows, tiles);
    if (t.n == 0) {
        forward_rest(s, t, h, O, lse);
        return;
    }
    // the last queries see the most keys: they come first
    plain_forward_tile(s, QKV, t.row0, t.n, (t.tiles - 1 - t.tile) * kRows, h, O, lse,
                       reinterpret_cast<float *>(smem4));
}

template <typename T>
tpce_status plain_forward(const Shape &s, const void *QKV, void *O, float *lse, cudaStream_t stream) {
    KernelTimer timer("attn_forward", stream);
    const int tiles = static_cast<int>(grid_tiles(s, kRows));
    const size_t smem = PlainSmem(s.d).forward();
    cudaError_t e = allow_smem<plain_forward_kernel<T>>();
    if (e == cudaSuccess)
        e = step::launch(plain_forward_kernel<T>, static_cast<unsigned>(tiles) * s.n_q, kPlainThreads, smem, stream, s,
                         static_cast<const T *>(QKV), tiles, static_cast<T *>(O), lse);
    return e == cudaSuccess ? check_launch("attn_forward", stream) : fail_cuda(e, "attn_forward");
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" tpce_status tp_attn_core_forward(const void *QKV, const int32_t *offsets, int sequences, int64_t T,
                                            int64_t n_heads, int64_t n_kv_heads, int64_t head_dim, int64_t window,
                                            int64_t sinks, float scale, int dtype, void *O, float *lse, void *stream) {
    const char *name = "tp_attn_core_forward";
    attn::Shape s;
    tpce_status st = attn::make_shape(name, offsets, sequences, T, n_heads, n_kv_heads, head_dim, window, sinks, scale,
                                      dtype, s);
    if (st != TPCE_OK || T == 0) return st;
    const size_t e = dtype == TPCE_BF16 ? 2 : 4;
    const attn::Arg args[] = {{QKV, static_cast<size_t>(T * s.ld) * e, false},
                              {offsets, offsets ? (static_cast<size_t>(sequences) + 1) * 4 : 0, false},
                              {O, static_cast<size_t>(T * n_heads * head_dim) * e, true},
                              {lse, static_cast<size_t>(T * n_heads) * 4, true}};
    if ((st = attn::check_args(name, args)) != TPCE_OK) return st;
    cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
    return dtype == TPCE_BF16 ? plain_forward<__nv_bfloat16>(s, QKV, O, lse, stream_)
                              : plain_forward<float>(s, QKV, O, lse, stream_);
}
