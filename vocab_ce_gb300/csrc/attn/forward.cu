// forward.cu -- the attention core, forward: O = softmax(scale Q K^T) V over the
// keys that a query sees, and lse (attn.cuh has the formulas).
#include "attn/attn.cuh"
#include "attn/host.cuh"
#include "attn/tc.cuh"

namespace tpce {
namespace {

using namespace attn;

// ------------------------------------------------------------------ plain tiles
// Queries q0 .. q0 + 63 of one head. One pass over the keys with the running maximum
// m and sum l of each row: when m grows, what has been added so far is scaled down.
template <typename T>
__device__ __forceinline__ void plain_forward_tile(const Shape &s, const T *QKV, int64_t row0, int n, int q0, int h,
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

// ------------------------------------------------------------------ tiles on the tensor cores
// A block has two tiles of 128 queries that read the same keys: two heads of a group
// where it is even, else two neighbouring tiles of one head. Twelve warps,
// of which the last two only lend their registers:
//   warps 0 - 3, 4 - 7   the softmax of tile 0 and of tile 1, a thread a query
//   warp 8               loads: Q once, then K and V tiles through a ring
//   warp 9               issues the products
// Tensor memory: the scores S of both tiles (128 columns each; P overwrites the first
// half of S in bf16) and both O. For each key tile
//   S = Q K^T  ->  softmax threads: running maximum, P = 2^(S c - m), row sums  ->  O += P V
// with tile 1's products under way while tile 0's threads work, and the other way
// round. The products of a tile are issued in this order and run in it, so that S of
// the next keys is written only after P has been used, and when S has arrived O is
// complete up to the keys before. A thread raises its maximum (and scales its O in
// tensor memory) only when a score is more than 2^8 above it: P then stays below 2^8,
// and O, l and lse are as exact.
constexpr int kFwdThreads = 384, kFwdStages = 5;
constexpr float kRaise = 8.0f;  // in powers of two
constexpr uint32_t kFwdSmem = 1024 + 2 * kTileBytes + kFwdStages * kTileBytes + 256;
static_assert(kFwdSmem <= static_cast<uint32_t>(kMaxSmem), "the ring fits");

// The key tiles of both tiles together, and which of the two needs one.
struct PairTiles {
    KeyTiles one[2], both;
    __device__ __forceinline__ bool needs(int i, int k) const {
        const KeyTiles &t = i ? one[1] : one[0];
        return k < t.first || (k >= t.from && k <= t.last);
    }
};

__global__ void __launch_bounds__(kFwdThreads, 1)
    tc_forward_kernel(const __grid_constant__ CUtensorMap map, const Shape s, const __nv_bfloat16 *QKV, bool by_heads,
                      int tiles, __nv_bfloat16 *O, float *lse) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + 2 * kTileBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + kFwdStages * kTileBytes);
    uint64_t *empty = full + kFwdStages, *q_full = empty + kFwdStages, *s_full = q_full + 1, *p_full = s_full + 2,
             *o_full = p_full + 2, *drain = o_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *odd = abort_flag + 1;  // [2] a tile has results that are not finite

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kFwdStages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(q_full, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_full[i], 4);
            ptx::mbar_init(&o_full[i], 1);
            odd[i] = 0;
        }
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map);
    }
    grid_begin();
    const int units = by_heads ? s.n_q / 2 : s.n_q;
    const int unit = blockIdx.x % units;
    const Tile t = find_tile(s, blockIdx.x / units, by_heads ? kTile : 2 * kTile, tiles);
    const int head0 = by_heads ? 2 * unit : unit;
    if (t.n == 0) {
        forward_rest(s, t, head0, O, lse);
        if (by_heads) forward_rest(s, t, head0 + 1, O, lse);
        return;
    }
    // the last queries see the most keys: they come first
    const int first = (t.tiles - 1 - t.tile) * (by_heads ? kTile : 2 * kTile);
    const int head[2] = {head0, by_heads ? head0 + 1 : head0};
    const int q0[2] = {first, by_heads ? first : first + kTile};
    PairTiles kt;
    bool there[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        there[i] = q0[i] < t.n;
        kt.one[i] = there[i] ? key_tiles(s, q0[i], min(t.n, q0[i] + kTile), kTile) : KeyTiles{0, 0, -1};
    }
    kt.both = kt.one[0];
    if (there[1]) {
        kt.both.last = kt.one[1].last;
        // the second tile's window begins later: what only its sinks need is needed by the first anyway
        kt.both.first = max(kt.one[0].first, min(kt.one[1].first, kt.one[0].from));
    }
    const int count = kt.both.count();
    const int kv = head0 / s.group;

    if (warp == 9) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    constexpr uint32_t tmem = 0;  // all columns there are: they begin at 0
    const int blocks = s.d > 64 ? 2 : 1;

    if (warp < 8) {
        ptx::registers_up<208>();  // 2 x 208 + 88 = 3 x 168, the launch's
        // ------------------------------------------------ softmax
        const int i = warp >> 2;
        const int my_q0 = i ? q0[1] : q0[0], my_head = i ? head[1] : head[0];
        const int row = my_q0 + (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + i * 128 + lanes, o_tmem = tmem + 256 + i * 128 + lanes;
        const float c = s.scale * kLog2e;
        const int wide = (width16(s.d) + 31) / 32;  // pieces of 32 columns of O
        float m = -INFINITY, l = 0.0f;
        uint32_t phase = 0;
        bool alive = i ? there[1] : there[0], begun = false;
        for (int u = 0; u < count && alive; ++u) {
            const int k = kt.both.at(u);
            if (!kt.needs(i, k)) continue;
            alive = wait_all(&s_full[i], phase, abort_flag, s.err, 24);
            phase ^= 1;
            if (!alive) break;
            ptx::tc_fence_after();
            float x[4][32];
#pragma unroll
            for (int b = 0; b < 4; ++b) ptx::tmem_ld32_async(s_tmem + b * 32, x[b]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 4; ++b) ptx::tmem_ready(x[b]);
            const int k0 = k * kTile;
            if (!all_seen(s, my_q0, my_q0 + kTile, k0, k0 + kTile)) {
                const int hi = row - k0, lo = s.window ? hi - s.window + 1 : -kTile, sink = s.sinks - k0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t seen = visible(hi - b * 32, lo - b * 32, sink - b * 32);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[b][e] = seen & (1u << e) ? x[b][e] : -INFINITY;
                }
            }
            float top[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                top[b] = x[b][0];
#pragma unroll
                for (int e = 1; e < 32; ++e) top[b] = fmaxf(top[b], x[b][e]);
            }
            const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
            const bool raise = most > m + kRaise;  // the first one, too: m is -inf
            if (__any_sync(0xffffffffu, raise)) {
                const float to = fmaxf(m, most);
                const float shrink = m == -INFINITY ? 0.0f : exp2_fast(m - to);
                if (begun) {
                    for (int b = 0; b < width16(s.d) / 16; ++b) ptx::tmem_scale16(o_tmem + b * 16, shrink);
                }
                l *= shrink;
                m = to;
            }
            begun = true;
            const float at = m == -INFINITY ? 0.0f : m;  // no key seen yet: 2^-inf
            float sum[4] = {};
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t p[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float v = x[2 * b + e / 16][2 * e % 32], w = x[2 * b + e / 16][2 * e % 32 + 1];
                    scale2(v, w, c, -at);
                    v = exp2_fast(v);
                    w = exp2_fast(w);
                    add2(sum[(e & 1) * 2], sum[(e & 1) * 2 + 1], v, w);
                    p[e] = pack2(v, w);
                }
                ptx::tmem_st32_async(s_tmem + b * 32, p);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&p_full[i]);
        }
        if (alive && wait_all(&o_full[i], 0, abort_flag, s.err, 25)) {
            ptx::tc_fence_after();
            const float inv = 1.0f / l;
            const bool mine = row < t.n;
            float check = l * 0.0f;  // stays 0 while everything is finite
            __nv_bfloat16 *to = O + (t.row0 + row) * s.n_q * s.d + static_cast<int64_t>(my_head) * s.d;
            for (int b = 0; b < wide; ++b) {
                float o[32];
                ptx::tmem_ld32_async(o_tmem + b * 32, o);
                ptx::tmem_wait_ld();
                ptx::tmem_ready(o);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if (b * 32 + v * 8 >= s.d) continue;
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        y[e] = o[v * 8 + e] * inv;
                        check = fmaf(y[e], 0.0f, check);
                    }
                    Raw8<__nv_bfloat16> r;
                    pack8(y, r);
                    if (mine) store8(to + b * 32 + v * 8, r);
                }
            }
            if (mine) lse[my_head * s.T + t.row0 + row] = (m + log2f(l)) * kLn2;
            if (mine && check != 0.0f) odd[i] = 1;  // NaN is not 0
        }
    } else {
        ptx::registers_down<88>();
        if (warp == 8) {
            // ------------------------------------------------ loads
            if (lane == 0) {
                const uint32_t bytes = blocks * kBlockBytes;
                ptx::mbar_arrive_expect_tx(q_full, (there[1] ? 2 : 1) * bytes);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (there[i]) load_tile(smem + i * kTileBytes, &map, q_full, s.q_head(head[i]), t.row0 + q0[i], blocks);
                int stage = 0;
                uint32_t phase = 0, issued = 0, parity = 0;
                auto load = [&](int at_head, int k) {
                    if (!ptx::mbar_wait(&empty[stage], phase ^ 1, abort_flag, s.err, 20)) return false;
                    ptx::mbar_arrive_expect_tx(&full[stage], bytes);
                    issued |= 1u << stage;
                    parity = (parity & ~(1u << stage)) | (phase << stage);
                    load_tile(ring + stage * kTileBytes, &map, &full[stage], at_head,
                              t.row0 + static_cast<int64_t>(k) * kTile, blocks);
                    if (++stage == kFwdStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                    return true;
                };
                // in the order of their use: K of a tile, then V of the one before
                for (int u = 0; u <= count; ++u) {
                    if (u < count && !load(s.k_head(kv), kt.both.at(u))) break;
                    if (u > 0 && !load(s.v_head(kv), kt.both.at(u - 1))) break;
                }
                if (*abort_flag) {
                    ptx::mbar_wait_drain(q_full, 0);
                    for (int i = 0; i < kFwdStages; ++i)
                        if (issued & (1u << i)) ptx::mbar_wait_drain(&full[i], (parity >> i) & 1u);
                }
            }
        } else if (warp == 9) {
            // ------------------------------------------------ products
            {
                const bool leader = ptx::elect_one();
                const uint32_t idesc = idesc_weighted(s.d);
                const uint32_t q_tile = ptx::smem_u32(smem), base = ptx::smem_u32(ring);
                int stage = 0;
                uint32_t phase = 0, p_phase[2] = {0, 0};
                bool begun[2] = {false, false};
                bool ok = wait_all(q_full, 0, abort_flag, s.err, 21);
                auto next = [&](int &at) {
                    ok = ok && wait_all(&full[stage], phase, abort_flag, s.err, 22);
                    at = stage;
                    if (++stage == kFwdStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                };
                for (int u = 0; u <= count && ok; ++u) {
                    int k_stage = 0, v_stage = 0;
                    if (u < count) next(k_stage);
                    if (u > 0 && ok) next(v_stage);
                    ptx::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!ok) break;
                        if (u > 0 && kt.needs(i, kt.both.at(u - 1))) {
                            if (!wait_all(&p_full[i], p_phase[i], abort_flag, s.err, 23)) {
                                ok = false;
                                break;
                            }
                            p_phase[i] ^= 1;
                            ptx::tc_fence_after();
                            mma_weighted(leader, tmem + 256 + i * 128, tmem + i * 128, 32, base + v_stage * kTileBytes, idesc,
                                         begun[i]);
                            begun[i] = true;
                            if (kt.both.at(u - 1) == kt.one[i].last) commit(leader, &o_full[i]);
                        }
                        if (u < count && kt.needs(i, kt.both.at(u))) {
                            mma_scores(leader, tmem + i * 128, q_tile + i * kTileBytes, base + k_stage * kTileBytes, s.d);
                            commit(leader, &s_full[i]);
                        }
                    }
                    if (u < count) commit(leader, &empty[k_stage]);
                    if (u > 0) commit(leader, &empty[v_stage]);
                }
                commit(leader, drain);
                ptx::mbar_wait_drain(drain, 0);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    // What is masked has met 0 times its value: a tile with results that are not finite
    // is computed again where masked values are passed over.
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        if (!odd[i] || *abort_flag || threadIdx.x >= kPlainThreads) continue;
        const int begin = i ? q0[1] : q0[0];
        for (int q = begin; q < min(t.n, begin + kTile); q += kRows) {
            plain_sync();
            plain_forward_tile(s, QKV, t.row0, t.n, q, i ? head[1] : head[0], O, lse, reinterpret_cast<float *>(smem));
        }
    }
}

tpce_status tc_forward(const Shape &s, const void *QKV, void *O, float *lse, cudaStream_t stream) {
    const char *name = "attn_forward";
    CUtensorMap map;
    if (!make_tmap_heads(&map, QKV, s.d, s.n_q + 2 * s.n_kv, s.T, s.ld, kTile))
        return fail(TPCE_ERR_CUDA, "%s: tensor map", name);
    const bool by_heads = s.group % 2 == 0;
    const int tiles = static_cast<int>(grid_tiles(s, by_heads ? kTile : 2 * kTile));
    const unsigned blocks = static_cast<unsigned>(tiles) * (by_heads ? s.n_q / 2 : s.n_q);
    cudaError_t e = allow_smem<tc_forward_kernel>();
    if (e != cudaSuccess) return fail_cuda(e, name);
    KernelTimer timer(name, stream);
    e = step::launch(tc_forward_kernel, blocks, kFwdThreads, kFwdSmem, stream, map, s,
                     static_cast<const __nv_bfloat16 *>(QKV), by_heads, tiles, static_cast<__nv_bfloat16 *>(O), lse);
    return e == cudaSuccess ? check_launch(name, stream) : fail_cuda(e, name);
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
    if (dtype == TPCE_F32) return plain_forward<float>(s, QKV, O, lse, stream_);
    // the tensor-core kernel looks for a row's maximum before the scale, which has to be positive for that
    return scale > 0.0f ? tc_forward(s, QKV, O, lse, stream_) : plain_forward<__nv_bfloat16>(s, QKV, O, lse, stream_);
}
