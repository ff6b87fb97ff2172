// backward.cu -- the attention core, backward (attn.cuh has the formulas).
//
// Three kernels: delta of every query and head; dQ by tiles of queries; dK and dV
// by tiles of keys, over all queries of all heads that share them. S and dP are
// computed in both of the last two, which is seven products for the five that the
// formulas name, and in return every gradient is summed in one place, in registers
// or tensor memory: nothing is added by atomics and results are the same every time.
#include "attn/attn.cuh"
#include "attn/host.cuh"

namespace tpce {
namespace {

using namespace attn;

// ------------------------------------------------------------------ delta
// stats[h, t] = (lse log2(e), delta): what the tiles need of a query. 16 lanes a row of
// one head; bound by reading O and dO.
template <typename T>
__global__ void __launch_bounds__(256) delta_kernel(const Shape s, const T *dO, const T *O, const float *lse,
                                                    float2 *__restrict__ stats) {
    grid_begin();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x / 16;
    const int lane = threadIdx.x & 15;
    const int64_t t = i / s.n_q;
    const int h = static_cast<int>(i - t * s.n_q);
    float sum = 0.0f;
    if (t < s.T && lane * 8 < s.d) {
        float a[8], b[8];
        unpack8(load8(dO + i * s.d + lane * 8), a);
        unpack8(load8(O + i * s.d + lane * 8), b);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum = fmaf(a[c], b[c], sum);
    }
    sum = sum16(sum);
    if (t < s.T && lane == 0) stats[h * s.T + t] = make_float2(lse[h * s.T + t] * kLog2e, sum);
}

// ------------------------------------------------------------------ plain tiles
// P and dS of 64 queries by 64 keys, into shared memory (P may be NULL).
__device__ __forceinline__ void plain_scores(const Shape &s, const float *Q, const float *K, const float *dO,
                                             const float *V, int pitch, const float2 *stats, int q0, int k0, int n,
                                             bool masked, float *P, float *dS) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const float c = s.scale * kLog2e;
    float x[4][4], y[4][4];
    plain_dots(Q, K, pitch, s.d, x);
    plain_dots(dO, V, pitch, s.d, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = q0 + 4 * ty + i;
        const float2 st = row < n ? stats[row] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool seen = !masked || (row < n && sees(s, row, k0 + tx + 16 * j));
            const float p = seen ? exp2f(x[i][j] * c - st.x) : 0.0f;
            const float ds = seen ? p * (y[i][j] - st.y) : 0.0f;
            if (P) P[(4 * ty + i) * kPitchP + tx + 16 * j] = p;
            dS[(4 * ty + i) * kPitchP + tx + 16 * j] = ds;
        }
    }
}

__device__ __forceinline__ void clear(float (&o)[4][2][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) o[i][a][b] = 0.0f;
}

// Rows r0 + 4 ty .. of the accumulator, times f, to rows of one head's columns.
template <typename T>
__device__ __forceinline__ void plain_store(const Shape &s, const float (&o)[4][2][4], float f, T *to, int r0, int n) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = r0 + 4 * ty + i;
        if (row >= n) continue;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int col = 4 * tx + 64 * a;
            if (col >= s.d) continue;
            float y[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) y[b] = o[i][a][b] * f;
            store4(to + row * s.ld + col, y);
        }
    }
}

// dQ of queries q0 .. q0 + 63 of one head.
template <typename T>
__device__ __noinline__ void plain_dq_tile(const Shape &s, const T *QKV, const T *dO, const float2 *stats,
                                           int64_t row0, int n, int q0, int h, T *dQKV, float *smem) {
    const PlainSmem lay(s.d);
    float *Q = smem, *K = Q + lay.rows(), *V = K + lay.rows(), *G = V + lay.rows(), *dS = G + lay.rows();
    const int d = s.d, kv = h / s.group;
    const int64_t qc = static_cast<int64_t>(s.q_head(h)) * d, kc = static_cast<int64_t>(s.k_head(kv)) * d,
                  vc = static_cast<int64_t>(s.v_head(kv)) * d, ldo = static_cast<int64_t>(s.n_q) * d;
    const T *base = QKV + row0 * s.ld;
    const KeyTiles tiles = key_tiles(s, q0, min(n, q0 + kRows), kRows);
    float o[4][2][4];
    clear(o);
    plain_load(Q, lay.pitch, base + qc, s.ld, q0, n, d);
    plain_load(G, lay.pitch, dO + row0 * ldo + static_cast<int64_t>(h) * d, ldo, q0, n, d);
    for (int u = 0; u < tiles.count(); ++u) {
        const int k0 = tiles.at(u) * kRows;
        plain_sync();
        plain_load(K, lay.pitch, base + kc, s.ld, k0, n, d);
        plain_load(V, lay.pitch, base + vc, s.ld, k0, n, d);
        plain_sync();
        const bool masked = !all_seen(s, q0, q0 + kRows, k0, k0 + kRows) || q0 + kRows > n;
        plain_scores(s, Q, K, G, V, lay.pitch, stats + h * s.T + row0, q0, k0, n, masked, nullptr, dS);
        plain_sync();
        if (masked)
            plain_add<true, false>(dS, K, lay.pitch, d, o);
        else
            plain_add<false, false>(dS, K, lay.pitch, d, o);
    }
    plain_store(s, o, s.scale, dQKV + row0 * s.ld + qc, q0, n);
}

// dK and dV of keys k0 .. k0 + 63 of one key/value head.
template <typename T>
__device__ __noinline__ void plain_dkv_tile(const Shape &s, const T *QKV, const T *dO, const float2 *stats,
                                            int64_t row0, int n, int k0, int kv, T *dQKV, float *smem) {
    const PlainSmem lay(s.d);
    float *Q = smem, *K = Q + lay.rows(), *V = K + lay.rows(), *G = V + lay.rows(), *P = G + lay.rows(),
          *dS = P + kRows * kPitchP;
    const int d = s.d;
    const int64_t kc = static_cast<int64_t>(s.k_head(kv)) * d, vc = static_cast<int64_t>(s.v_head(kv)) * d,
                  ldo = static_cast<int64_t>(s.n_q) * d;
    const T *base = QKV + row0 * s.ld;
    float ok[4][2][4], ov[4][2][4];
    clear(ok);
    clear(ov);
    plain_load(K, lay.pitch, base + kc, s.ld, k0, n, d);
    plain_load(V, lay.pitch, base + vc, s.ld, k0, n, d);
    const int end = query_end(s, k0, min(n, k0 + kRows), n);
    for (int g = 0; g < s.group; ++g) {
        const int h = kv * s.group + g;
        for (int q0 = k0; q0 < end; q0 += kRows) {
            plain_sync();
            plain_load(Q, lay.pitch, base + static_cast<int64_t>(s.q_head(h)) * d, s.ld, q0, n, d);
            plain_load(G, lay.pitch, dO + row0 * ldo + static_cast<int64_t>(h) * d, ldo, q0, n, d);
            plain_sync();
            const bool masked = !all_seen(s, q0, q0 + kRows, k0, k0 + kRows) || q0 + kRows > n;
            plain_scores(s, Q, K, G, V, lay.pitch, stats + h * s.T + row0, q0, k0, n, masked, P, dS);
            plain_sync();
            if (masked) {
                plain_add<true, true>(P, G, lay.pitch, d, ov);
                plain_add<true, true>(dS, Q, lay.pitch, d, ok);
            } else {
                plain_add<false, true>(P, G, lay.pitch, d, ov);
                plain_add<false, true>(dS, Q, lay.pitch, d, ok);
            }
        }
    }
    plain_store(s, ok, s.scale, dQKV + row0 * s.ld + kc, k0, n);
    plain_store(s, ov, 1.0f, dQKV + row0 * s.ld + vc, k0, n);
}

template <typename T>
__global__ void __launch_bounds__(kPlainThreads)
    plain_dq_kernel(const Shape s, const T *QKV, const T *dO, const float2 *stats, int tiles, T *dQKV) {
    extern __shared__ float4 smem4[];
    grid_begin();
    const int h = blockIdx.x % s.n_q;
    const Tile t = find_tile(s, blockIdx.x / s.n_q, kRows, tiles);
    if (t.n == 0) {
        zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(s.q_head(h)) * s.d);
        return;
    }
    plain_dq_tile(s, QKV, dO, stats, t.row0, t.n, (t.tiles - 1 - t.tile) * kRows, h, dQKV,
                  reinterpret_cast<float *>(smem4));
}

template <typename T>
__global__ void __launch_bounds__(kPlainThreads)
    plain_dkv_kernel(const Shape s, const T *QKV, const T *dO, const float2 *stats, int tiles, T *dQKV) {
    extern __shared__ float4 smem4[];
    grid_begin();
    const int kv = blockIdx.x % s.n_kv;
    const Tile t = find_tile(s, blockIdx.x / s.n_kv, kRows, tiles);
    if (t.n == 0) {
        zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(s.k_head(kv)) * s.d);
        zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(s.v_head(kv)) * s.d);
        return;
    }
    // the first keys are seen by the most queries: they come first
    plain_dkv_tile(s, QKV, dO, stats, t.row0, t.n, t.tile * kRows, kv, dQKV, reinterpret_cast<float *>(smem4));
}

// ------------------------------------------------------------------ host
template <typename T>
tpce_status plain_backward(const Shape &s, const void *QKV, const void *dO, const float2 *stats, void *dQKV,
                           cudaStream_t stream) {
    const int tiles = static_cast<int>(grid_tiles(s, kRows));
    const size_t smem = PlainSmem(s.d).backward();
    auto go = [&](auto kernel, const char *name, int heads) {
        KernelTimer timer(name, stream);
        const cudaError_t e = step::launch(kernel, static_cast<unsigned>(tiles) * heads, kPlainThreads, smem, stream, s,
                                           static_cast<const T *>(QKV), static_cast<const T *>(dO), stats, tiles,
                                           static_cast<T *>(dQKV));
        return e == cudaSuccess ? check_launch(name, stream) : fail_cuda(e, name);
    };
    cudaError_t e = allow_smem<plain_dq_kernel<T>>();
    if (e == cudaSuccess) e = allow_smem<plain_dkv_kernel<T>>();
    if (e != cudaSuccess) return fail_cuda(e, "attn_backward");
    const tpce_status st = go(plain_dkv_kernel<T>, "attn_dkv", s.n_kv);
    return st != TPCE_OK ? st : go(plain_dq_kernel<T>, "attn_dq", s.n_q);
}

template <typename T>
tpce_status delta(const Shape &s, const void *dO, const void *O, const float *lse, float2 *stats,
                  cudaStream_t stream) {
    KernelTimer timer("attn_delta", stream);
    const cudaError_t e =
        step::launch(delta_kernel<T>, static_cast<unsigned>((s.T * s.n_q + 15) / 16), 256, 0, stream, s,
                     static_cast<const T *>(dO), static_cast<const T *>(O), lse, stats);
    return e == cudaSuccess ? check_launch("attn_delta", stream) : fail_cuda(e, "attn_delta");
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" size_t tpce_attn_core_workspace_bytes(int64_t T, int64_t n_heads) {
    if (T <= 0 || T > (int64_t{1} << 30) || n_heads < 1 || n_heads > 4096) return 0;
    return static_cast<size_t>(T * n_heads) * sizeof(float2);
}

extern "C" tpce_status tp_attn_core_backward(const void *dO, const void *QKV, const void *O, const float *lse,
                                             const int32_t *offsets, int sequences, int64_t T, int64_t n_heads,
                                             int64_t n_kv_heads, int64_t head_dim, int64_t window, int64_t sinks,
                                             float scale, int dtype, void *dQKV, void *ws, size_t ws_bytes,
                                             void *stream) {
    const char *name = "tp_attn_core_backward";
    attn::Shape s;
    tpce_status st = attn::make_shape(name, offsets, sequences, T, n_heads, n_kv_heads, head_dim, window, sinks, scale,
                                      dtype, s);
    if (st != TPCE_OK || T == 0) return st;
    const size_t e = dtype == TPCE_BF16 ? 2 : 4, need = tpce_attn_core_workspace_bytes(T, n_heads);
    if (!ws || ws_bytes < need)
        return fail(TPCE_ERR_WORKSPACE, "%s: %zu bytes of workspace needed, %zu given", name, need,
                    ws ? ws_bytes : size_t{0});
    const size_t rows = static_cast<size_t>(T * n_heads * head_dim) * e;
    const attn::Arg args[] = {{dO, rows, false},
                              {QKV, static_cast<size_t>(T * s.ld) * e, false},
                              {O, rows, false},
                              {lse, static_cast<size_t>(T * n_heads) * 4, false},
                              {offsets, offsets ? (static_cast<size_t>(sequences) + 1) * 4 : 0, false},
                              {dQKV, static_cast<size_t>(T * s.ld) * e, true},
                              {ws, need, true}};
    if ((st = attn::check_args(name, args)) != TPCE_OK) return st;
    cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
    float2 *stats = static_cast<float2 *>(ws);
    if (dtype == TPCE_BF16) {
        if ((st = delta<__nv_bfloat16>(s, dO, O, lse, stats, stream_)) != TPCE_OK) return st;
        return plain_backward<__nv_bfloat16>(s, QKV, dO, stats, dQKV, stream_);
    }
    if ((st = delta<float>(s, dO, O, lse, stats, stream_)) != TPCE_OK) return st;
    return plain_backward<float>(s, QKV, dO, stats, dQKV, stream_);
}
