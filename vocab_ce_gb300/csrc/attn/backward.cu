// backward.cu -- the attention core, backward (attn.cuh has the formulas).
//
// Three kernels: delta of every query and head; dQ by tiles of queries; dK and dV
// by tiles of keys, over all queries of all heads that share them. S and dP are
// computed in both of the last two, which is seven products for the five that the
// formulas name, and in return every gradient is summed in one place, in registers
// or tensor memory: nothing is added by atomics and results are the same every time.
#include "attn/attn.cuh"
#include "attn/host.cuh"
#include "attn/tc.cuh"

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
__device__ __forceinline__ void plain_dq_tile(const Shape &s, const T *QKV, const T *dO, const float2 *stats,
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
__device__ __forceinline__ void plain_dkv_tile(const Shape &s, const T *QKV, const T *dO, const float2 *stats,
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

// ------------------------------------------------------------------ tiles on the tensor cores
// Twelve warps: 0 - 7 compute, a thread one row of a 128 x 128 tile and half of its
// columns (warps 4 - 7 the second half); warp 8 loads; warps 9 and 10 issue the
// products (dQ: warp 9 alone); warp 11 fetches the queries' statistics where they go by
// columns. A warp's products run in the order in which they are issued, which is what
// keeps a buffer of tensor memory from being written while one before reads it.
constexpr int kBwdThreads = 384, kBwdRing = 5;
// the two tiles that stay, the ring, statistics of two tiles, barriers
constexpr uint32_t kBwdSmem = 2 * kTileBytes + kBwdRing * kTileBytes + 2 * kTile * 8 + 256;
static_assert(kBwdSmem <= static_cast<uint32_t>(kMaxSmem), "the ring fits");

// The tiles that come and go, two of each step: those that are used from a step's first
// product to its last (Q for dK and dV, K for dQ) have three places, the others (dO, V)
// two. (One ring of five for both in turn made a tile wait for the other kind's last use:
// dQ stood still for 500 of 2400 cycles a step.)
constexpr int kLong = 0, kShort = 1;
struct Ring {
    uint8_t *at;
    uint64_t *full, *empty;
    __device__ __forceinline__ static int slot(int kind, int pos) { return kind == kLong ? pos % 3 : 3 + (pos & 1); }
    __device__ __forceinline__ static uint32_t parity(int kind, int pos) {
        return static_cast<uint32_t>(kind == kLong ? pos / 3 : pos >> 1) & 1u;
    }
};

struct BwdSmem {
    uint8_t *tiles;  // the two that stay
    Ring ring;
    float *stats;  // [2][2][kTile]
    uint64_t *stay, *scores, *dots, *p_ready, *ds_ready, *stats_full, *stats_empty, *done, *drain, *turn;
    uint32_t *tmem_slot;
    volatile int *abort_flag, *odd;
    __device__ __forceinline__ explicit BwdSmem(uint8_t *raw) {
        tiles = raw;  // 1024-byte aligned, as the swizzle needs it
        ring.at = tiles + 2 * kTileBytes;
        stats = reinterpret_cast<float *>(ring.at + kBwdRing * kTileBytes);
        uint64_t *b = reinterpret_cast<uint64_t *>(stats + 4 * kTile);
        ring.full = b;
        ring.empty = b + kBwdRing;
        b += 2 * kBwdRing;
        stay = b;
        scores = b + 1;      // [2]
        dots = b + 3;
        p_ready = b + 4;
        ds_ready = b + 5;
        stats_full = b + 6;  // [2]
        stats_empty = b + 8;  // [2]
        done = b + 10;
        drain = b + 11;
        turn = b + 12;  // [2]
        tmem_slot = reinterpret_cast<uint32_t *>(b + 14);
        abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
        odd = abort_flag + 1;
    }
    // issuers: warps that issue products
    __device__ __forceinline__ void init(int issuers) const {
        for (int i = 0; i < kBwdRing; ++i) {
            ptx::mbar_init(&ring.full[i], 1);
            ptx::mbar_init(&ring.empty[i], issuers);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&turn[i], 1);
            ptx::mbar_init(&scores[i], 1);
            ptx::mbar_init(&stats_full[i], 32);
            ptx::mbar_init(&stats_empty[i], 8);
        }
        ptx::mbar_init(stay, 1);
        ptx::mbar_init(dots, 1);
        ptx::mbar_init(p_ready, 8);
        ptx::mbar_init(ds_ready, 8);
        ptx::mbar_init(done, issuers);
        ptx::mbar_init(drain, issuers);
        *abort_flag = 0;
        *odd = 0;
        ptx::fence_mbar_init();
    }
};

// Loads the tile of step `pos` of its kind (all lanes call it); false when a wait gave up.
__device__ __forceinline__ bool ring_load(const BwdSmem &m, bool leader, int kind, int pos, const CUtensorMap *map,
                                          int head, int64_t row, int blocks, uint32_t *err) {
    const int slot = Ring::slot(kind, pos);
    if (!wait_all<true>(&m.ring.empty[slot], Ring::parity(kind, pos) ^ 1, m.abort_flag, err, 30)) return false;
    if (leader) {
        ptx::mbar_arrive_expect_tx(&m.ring.full[slot], blocks * kBlockBytes);
        load_tile(m.ring.at + slot * kTileBytes, map, &m.ring.full[slot], head, row, blocks);
    }
    return true;
}
// After a wait gave up: the loads of the steps before `pos` land.
__device__ __forceinline__ void ring_drain(const BwdSmem &m, int longs, int shorts) {
    ptx::mbar_wait_drain(m.stay, 0);
    for (int p = max(0, longs - 3); p < longs; ++p)
        ptx::mbar_wait_drain(&m.ring.full[Ring::slot(kLong, p)], Ring::parity(kLong, p));
    for (int p = max(0, shorts - 2); p < shorts; ++p)
        ptx::mbar_wait_drain(&m.ring.full[Ring::slot(kShort, p)], Ring::parity(kShort, p));
}

// This thread's row of an accumulator, times f, from column c0 on (up to 64), to `to`; false if
// something is not finite.
__device__ __forceinline__ bool write_half(uint32_t taddr, float f, int c0, int d, __nv_bfloat16 *to, bool mine) {
    float check = 0.0f;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (c0 + b * 32 >= d) break;
        float o[32];
        ptx::tmem_ld32_async(taddr + b * 32, o);
        ptx::tmem_wait_ld();
        ptx::tmem_ready(o);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int c = c0 + b * 32 + v * 8;
            if (c >= d) continue;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = o[v * 8 + e] * f;
                check = fmaf(y[e], 0.0f, check);
            }
            Raw8<__nv_bfloat16> r;
            pack8(y, r);
            if (mine) store8(to + c, r);
        }
    }
    return !mine || check == 0.0f;  // NaN is not 0
}

// dK and dV of 128 keys. Per tile of 128 queries of a head, with the keys as rows:
//   S^T = K Q^T  ->  P^T = 2^(S^T c - lse)   ->  dV += P^T dO
//   dP^T = V dO^T  ->  dS^T = P^T (dP^T - delta)  ->  dK += dS^T Q
// Tensor memory: S^T, dP^T, dV, dK, 128 columns each; P^T and dS^T overwrite what they
// are made of, in bf16, each half of the columns its own place. One warp issues S and
// dV, the other dP and dK, in turn:
//   S(0), dP(0), dV(0) S(1), dK(0) dP(1), dV(1) S(2), ..
// so that two products are under way while the threads form P or dS, and each warp
// waits for what it needs during the other's.
__global__ void __launch_bounds__(kBwdThreads, 1)
    tc_dkv_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_do, const Shape s,
                  const __nv_bfloat16 *QKV, const __nv_bfloat16 *dO, const float2 *stats, int tiles,
                  __nv_bfloat16 *dQKV) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const BwdSmem m(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        m.init(2);
        ptx::prefetch_tmap(&map);
        ptx::prefetch_tmap(&map_do);
    }
    grid_begin();
    const int kv = blockIdx.x % s.n_kv;
    const Tile t = find_tile(s, blockIdx.x / s.n_kv, kTile, tiles);
    if (t.n == 0) {
        zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(s.k_head(kv)) * s.d);
        zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(s.v_head(kv)) * s.d);
        return;
    }
    // the first keys are seen by the most queries: they come first
    const int k0 = t.tile * kTile;
    const int end = query_end(s, k0, min(t.n, k0 + kTile), t.n);
    const int of_head = (end - k0 + kTile - 1) / kTile, count = of_head * s.group;
    if (warp == 9) {
        ptx::tmem_alloc(m.tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    constexpr uint32_t tmem = 0,  // all columns there are: they begin at 0
                       t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;
    const int blocks = s.d > 64 ? 2 : 1;

    if (warp == 8) {
        {
            const bool leader = ptx::elect_one();
            if (leader) {
                ptx::mbar_arrive_expect_tx(m.stay, 2 * blocks * kBlockBytes);
                load_tile(m.tiles, &map, m.stay, s.k_head(kv), t.row0 + k0, blocks);
                load_tile(m.tiles + kTileBytes, &map, m.stay, s.v_head(kv), t.row0 + k0, blocks);
            }
            int longs = 0, shorts = 0;
            bool ok = true;
            for (int g = 0; g < s.group && ok; ++g)
                for (int q = 0; q < of_head && ok; ++q) {
                    const int64_t row = t.row0 + k0 + q * kTile;
                    const int h = kv * s.group + g;
                    ok = ring_load(m, leader, kLong, longs, &map, s.q_head(h), row, blocks, s.err);
                    longs += ok;
                    ok = ok && ring_load(m, leader, kShort, shorts, &map_do, h, row, blocks, s.err);
                    shorts += ok;
                }
            if (*m.abort_flag && leader) ring_drain(m, longs, shorts);
        }
    } else if (warp == 9 || warp == 10) {
        // step `it`: the sum with tile it - 1, then the scores (or dots) of tile it
        const int i = warp - 9;
        const bool leader = ptx::elect_one();
        const uint32_t idesc = idesc_weighted(s.d), base = ptx::smem_u32(m.ring.at);
        const uint32_t stays = ptx::smem_u32(m.tiles) + i * kTileBytes;  // K, V
        const uint32_t t_in = i ? t_dp : t_s, t_sum = i ? t_dk : t_dv;
        uint64_t *const ready = i ? m.ds_ready : m.p_ready, *const out = i ? m.dots : m.scores;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t where) {
            ok = ok && wait_all<true>(bar, parity, m.abort_flag, s.err, where);
        };
        // Q (long) serves S and dK, dO (short) dP and dV
        const int kind_in = i ? kShort : kLong, kind_of = i ? kLong : kShort;
        auto arrived = [&](int kind, int pos) {
            wait(&m.ring.full[Ring::slot(kind, pos)], Ring::parity(kind, pos), 31);
        };
        auto tile = [&](int kind, int pos) { return base + Ring::slot(kind, pos) * kTileBytes; };
        wait(m.stay, 0, 32);
        for (int it = 0; it <= count && ok; ++it) {
            const bool scores = it < count, sums = it > 0;
            if (scores) arrived(kind_in, it);
            if (sums) arrived(kind_of, it - 1);
            if (i == 1 || it > 0) wait(&m.turn[i], (i == 1 ? it : it - 1) & 1, 33);
            if (sums) wait(ready, (it - 1) & 1, 34);
            if (!ok) break;
            ptx::tc_fence_after();
            if (sums) mma_weighted(leader, t_sum, t_in, 64, tile(kind_of, it - 1), idesc, it > 1);
            if (scores)
                mma_scores(leader, t_in, stays, tile(kind_in, it), s.d, out, &m.turn[i ^ 1]);
            else if (leader)
                ptx::mbar_arrive(&m.turn[i ^ 1]);
            if (sums) commit(leader, &m.ring.empty[Ring::slot(kind_of, it - 1)]);
            if (scores) commit(leader, &m.ring.empty[Ring::slot(kind_in, it)]);
        }
        if (ok) commit(leader, m.done);
        commit(leader, m.drain);
        if (lane == 0) ptx::mbar_wait_drain(m.drain, 0);
        __syncwarp();
    } else if (warp == 11) {
        // the statistics of a tile, when the one two before has been used; queries past the end: P = 2^-inf
        int it = 0;
        bool ok = true;
        for (int g = 0; g < s.group && ok; ++g) {
            const float2 *from = stats + (kv * s.group + g) * s.T + t.row0;
            for (int q = 0; q < of_head && ok; ++q, ++it) {
                float2 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = k0 + q * kTile + e * 32 + lane;
                    v[e] = row < t.n ? from[row] : make_float2(INFINITY, 0.0f);
                }
                ok = wait_all(&m.stats_empty[it & 1], ((it >> 1) & 1) ^ 1, m.abort_flag, s.err, 35);
                if (!ok) break;
                float *to = m.stats + (it & 1) * 2 * kTile;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    to[e * 32 + lane] = -v[e].x;  // both are subtracted
                    to[kTile + e * 32 + lane] = -v[e].y;
                }
                ptx::mbar_arrive(&m.stats_full[it & 1]);
            }
        }
    } else if (warp < 8) {
        const int half = warp >> 2, r = (warp & 3) * 32 + lane, key = k0 + r;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = s.scale * kLog2e;
        const int limit = s.window && key >= s.sinks ? min(t.n, key + s.window) : t.n;  // queries below it see the key
        bool alive = true;
        int q = 0;
        for (int it = 0; it < count && alive; ++it) {
            const int q0 = k0 + q * kTile;
            q = q + 1 == of_head ? 0 : q + 1;
            const bool masked = !all_seen(s, q0, q0 + kTile, k0, k0 + kTile) || q0 + kTile > t.n;
            // queries from the key's own on, below its limit
            auto seen = [&](int b) {
                const int at = q0 + half * 64 + b * 32;
                return below(limit - at) & ~below(key - at);
            };
            const float *lse = m.stats + (it & 1) * 2 * kTile + half * 64, *delta = lse + kTile;
            alive = wait_all<true>(&m.stats_full[it & 1], (it >> 1) & 1, m.abort_flag, s.err, 36) &&
                    wait_all<true>(m.scores, it & 1, m.abort_flag, s.err, 37);
            if (!alive) break;
            ptx::tc_fence_after();
            float x[2][32];
            read_half(t_s + lanes + half * 64, x);
            uint32_t p[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(lse + b * 32 + e);
                    float(&y)[32] = x[b];
                    scale2(y[e], y[e + 1], c, l.x, l.y);
                    scale2(y[e + 2], y[e + 3], c, l.z, l.w);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) x[b][e] = exp2_fast(x[b][e]);
                if (masked) keep(x[b], seen(b), 0.0f);
                pack32(x[b], p + b * 16);
            }
            ptx::tmem_st32_async(t_s + lanes + half * 64, p);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(m.p_ready);
            alive = wait_all<true>(m.dots, it & 1, m.abort_flag, s.err, 38);
            if (!alive) break;
            ptx::tc_fence_after();
            float y[2][32];
            read_half(t_dp + lanes + half * 64, y);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 d = *reinterpret_cast<const float4 *>(delta + b * 32 + e);
                    float(&v)[32] = y[b];
                    add2(v[e], v[e + 1], d.x, d.y);
                    add2(v[e + 2], v[e + 3], d.z, d.w);
                    step::mul2(v[e], v[e + 1], x[b][e], x[b][e + 1]);
                    step::mul2(v[e + 2], v[e + 3], x[b][e + 2], x[b][e + 3]);
                }
                if (masked) keep(y[b], seen(b), 0.0f);  // what is masked may be infinite here
                pack32(y[b], p + b * 16);
            }
            ptx::tmem_st32_async(t_dp + lanes + half * 64, p);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(m.ds_ready);
                ptx::mbar_arrive(&m.stats_empty[it & 1]);
            }
        }
        if (alive) alive = wait_all<true>(m.done, 0, m.abort_flag, s.err, 39);
        if (alive) {
            ptx::tc_fence_after();
            // warps 0 - 3 write dK, 4 - 7 dV
            const bool mine = key < t.n;
            const uint32_t from = (half ? t_dv : t_dk) + lanes;
            __nv_bfloat16 *to = dQKV + (t.row0 + key) * s.ld +
                                static_cast<int64_t>(half ? s.v_head(kv) : s.k_head(kv)) * s.d;
            const float f = half ? 1.0f : s.scale;
            bool fine = write_half(from, f, 0, s.d, to, mine);
            fine = write_half(from + 64, f, 64, s.d, to, mine) && fine;
            if (!fine) *m.odd = 1;
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    // something masked may have been infinite (0 inf is NaN): once more, passing it over
    if (*m.odd && !*m.abort_flag && threadIdx.x < kPlainThreads) {
#pragma unroll 1
        for (int k = k0; k < min(t.n, k0 + kTile); k += kRows) {
            plain_sync();
            plain_dkv_tile(s, QKV, dO, stats, t.row0, t.n, k, kv, dQKV, reinterpret_cast<float *>(m.tiles));
        }
    }
}

// dQ of 128 queries of a head. Per tile of 128 keys, with the queries as rows:
//   S = Q K^T, dP = dO V^T  ->  dS = 2^(S c - lse) (dP - delta)  ->  dQ += dS K
// Tensor memory: two S (dS overwrites the one that it is made of), dP, dQ. In the order
//   S(0) dP(0) | S(1) dP(1) dQ(0) | S(2) dP(2) dQ(1) | ..
// dP of the next keys is begun as soon as the threads have read the one before, and P
// is formed of the next S before dP has come.
__global__ void __launch_bounds__(kBwdThreads, 1)
    tc_dq_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_do, const Shape s,
                 const __nv_bfloat16 *QKV, const __nv_bfloat16 *dO, const float2 *stats, int tiles,
                 __nv_bfloat16 *dQKV) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const BwdSmem m(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        m.init(1);
        ptx::prefetch_tmap(&map);
        ptx::prefetch_tmap(&map_do);
    }
    grid_begin();
    const int h = blockIdx.x % s.n_q, kv = h / s.group;
    const Tile t = find_tile(s, blockIdx.x / s.n_q, kTile, tiles);
    if (t.n == 0) {
        zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(s.q_head(h)) * s.d);
        return;
    }
    const int q0 = (t.tiles - 1 - t.tile) * kTile;
    const KeyTiles kt = key_tiles(s, q0, min(t.n, q0 + kTile), kTile);
    const int count = kt.count();
    if (warp == 9) {
        ptx::tmem_alloc(m.tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    constexpr uint32_t tmem = 0, t_dp = tmem + 256, t_dq = tmem + 384;
    const int blocks = s.d > 64 ? 2 : 1;

    if (warp == 8) {
        {
            const bool leader = ptx::elect_one();
            if (leader) {
                ptx::mbar_arrive_expect_tx(m.stay, 2 * blocks * kBlockBytes);
                load_tile(m.tiles, &map, m.stay, s.q_head(h), t.row0 + q0, blocks);
                load_tile(m.tiles + kTileBytes, &map_do, m.stay, h, t.row0 + q0, blocks);
            }
            int longs = 0, shorts = 0;
            bool ok = true;
            for (int u = 0; u < count && ok; ++u) {
                const int64_t row = t.row0 + static_cast<int64_t>(kt.at(u)) * kTile;
                ok = ring_load(m, leader, kLong, longs, &map, s.k_head(kv), row, blocks, s.err);
                longs += ok;
                ok = ok && ring_load(m, leader, kShort, shorts, &map, s.v_head(kv), row, blocks, s.err);
                shorts += ok;
            }
            if (*m.abort_flag && leader) ring_drain(m, longs, shorts);
        }
    } else if (warp == 9) {
        {
            const bool leader = ptx::elect_one();
            const uint32_t idesc = idesc_weighted(s.d), base = ptx::smem_u32(m.ring.at), q_tile = ptx::smem_u32(m.tiles);
            auto tile = [&](int kind, int pos) { return base + Ring::slot(kind, pos) * kTileBytes; };
            auto arrived = [&](int kind, int pos) {
                return wait_all<true>(&m.ring.full[Ring::slot(kind, pos)], Ring::parity(kind, pos), m.abort_flag, s.err,
                                      41);
            };
            auto scores = [&](int it) {
                if (!arrived(kLong, it)) return false;
                ptx::tc_fence_after();
                mma_scores(leader, tmem + (it & 1) * 128, q_tile, tile(kLong, it), s.d, &m.scores[it & 1]);
                return true;
            };
            auto dots = [&](int it) {
                if (!arrived(kShort, it)) return false;
                if (it > 0 && !wait_all<true>(m.p_ready, (it - 1) & 1, m.abort_flag, s.err, 43)) return false;
                ptx::tc_fence_after();
                mma_scores(leader, t_dp, q_tile + kTileBytes, tile(kShort, it), s.d, m.dots);
                commit(leader, &m.ring.empty[Ring::slot(kShort, it)]);
                return true;
            };
            bool ok = wait_all(m.stay, 0, m.abort_flag, s.err, 42) && scores(0) && dots(0);
            for (int it = 0; it < count && ok; ++it) {
                if (it + 1 < count) ok = scores(it + 1) && dots(it + 1);
                ok = ok && wait_all<true>(m.ds_ready, it & 1, m.abort_flag, s.err, 47);
                if (!ok) break;
                ptx::tc_fence_after();
                mma_weighted(leader, t_dq, tmem + (it & 1) * 128, 64, tile(kLong, it), idesc, it > 0);
                commit(leader, &m.ring.empty[Ring::slot(kLong, it)]);
            }
            if (ok) commit(leader, m.done);
            commit(leader, m.drain);
            ptx::mbar_wait_drain(m.drain, 0);
        }
    } else if (warp < 8) {
        const int half = warp >> 2, row = q0 + (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = s.scale * kLog2e;
        const bool mine = row < t.n;
        const float2 st = mine ? stats[h * s.T + t.row0 + row] : make_float2(INFINITY, 0.0f);
        bool alive = true;
        for (int it = 0; it < count && alive; ++it) {
            const int k0 = kt.at(it) * kTile;
            const bool masked = !all_seen(s, q0, q0 + kTile, k0, k0 + kTile);
            auto seen = [&](int b) {
                const int at = k0 + half * 64 + b * 32, hi = row - at;
                return visible(hi, s.window ? hi - s.window + 1 : -kTile, s.sinks - at);
            };
            const uint32_t t_s = tmem + (it & 1) * 128 + lanes + half * 64;
            alive = wait_all<true>(&m.scores[it & 1], (it >> 1) & 1, m.abort_flag, s.err, 44);
            if (!alive) break;
            ptx::tc_fence_after();
            float x[2][32], y[2][32];
            read_half(t_s, x);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    scale2(x[b][e], x[b][e + 1], c, -st.x, -st.x);
                    x[b][e] = exp2_fast(x[b][e]);
                    x[b][e + 1] = exp2_fast(x[b][e + 1]);
                }
            alive = wait_all<true>(m.dots, it & 1, m.abort_flag, s.err, 45);
            if (!alive) break;
            ptx::tc_fence_after();
            read_half(t_dp + lanes + half * 64, y);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(m.p_ready);  // dP has been read
            uint32_t p[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    add2(y[b][e], y[b][e + 1], -st.y, -st.y);
                    step::mul2(y[b][e], y[b][e + 1], x[b][e], x[b][e + 1]);
                }
                if (masked) keep(y[b], seen(b), 0.0f);
                pack32(y[b], p + b * 16);
            }
            ptx::tmem_st32_async(t_s, p);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(m.ds_ready);
        }
        if (alive) alive = wait_all<true>(m.done, 0, m.abort_flag, s.err, 46);
        if (alive && half * 64 < s.d) {
            ptx::tc_fence_after();
            __nv_bfloat16 *to = dQKV + (t.row0 + row) * s.ld + static_cast<int64_t>(s.q_head(h)) * s.d;
            if (!write_half(t_dq + lanes + half * 64, s.scale, half * 64, s.d, to, mine)) *m.odd = 1;
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    if (*m.odd && !*m.abort_flag && threadIdx.x < kPlainThreads) {
#pragma unroll 1
        for (int q = q0; q < min(t.n, q0 + kTile); q += kRows) {
            plain_sync();
            plain_dq_tile(s, QKV, dO, stats, t.row0, t.n, q, h, dQKV, reinterpret_cast<float *>(m.tiles));
        }
    }
}

// ------------------------------------------------------------------ host
tpce_status tc_backward(const Shape &s, const void *QKV, const void *dO, const float2 *stats, void *dQKV,
                        cudaStream_t stream) {
    CUtensorMap map, map_do;
    if (!make_tmap_heads(&map, QKV, s.d, s.n_q + 2 * s.n_kv, s.T, s.ld, kTile) ||
        !make_tmap_heads(&map_do, dO, s.d, s.n_q, s.T, static_cast<uint64_t>(s.n_q) * s.d, kTile))
        return fail(TPCE_ERR_CUDA, "attn_backward: tensor map");
    const int tiles = static_cast<int>(grid_tiles(s, kTile));
    auto go = [&](auto kernel, const char *name, int heads) {
        KernelTimer timer(name, stream);
        const cudaError_t e = step::launch(kernel, static_cast<unsigned>(tiles) * heads, kBwdThreads, kBwdSmem,
                                           stream, map, map_do, s, static_cast<const __nv_bfloat16 *>(QKV),
                                           static_cast<const __nv_bfloat16 *>(dO), stats, tiles,
                                           static_cast<__nv_bfloat16 *>(dQKV));
        return e == cudaSuccess ? check_launch(name, stream) : fail_cuda(e, name);
    };
    cudaError_t e = allow_smem<tc_dkv_kernel>();
    if (e == cudaSuccess) e = allow_smem<tc_dq_kernel>();
    if (e != cudaSuccess) return fail_cuda(e, "attn_backward");
    const tpce_status st = go(tc_dkv_kernel, "attn_dkv", s.n_kv);
    return st != TPCE_OK ? st : go(tc_dq_kernel, "attn_dq", s.n_q);
}

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
        return tc_backward(s, QKV, dO, stats, dQKV, stream_);
    }
    if ((st = delta<float>(s, dO, O, lse, stats, stream_)) != TPCE_OK) return st;
    return plain_backward<float>(s, QKV, dO, stats, dQKV, stream_);
}
