// backward.cu -- the attention core, backward (attn.cuh has the formulas).
//
// Two kernels: delta of every query and head; and the gradients, dK and dV by tiles
// of keys, over all queries of all heads that share them, and dQ by tiles of queries.
// S and dP are computed for both kinds of tiles, which is seven products for the five
// that the formulas name, and in return every gradient is summed in one place, in
// registers or tensor memory: nothing is added by atomics and results are the same
// every time.
#include "attn/attn.cuh"
#include "attn/host.cuh"
#include "attn/tc.cuh"

namespace tpce {
namespace {

using namespace attn;

// ------------------------------------------------------------------ delta
// stats[h, t] = (lse log2(e), delta): what the tiles need of a query. 16 lanes take
// kDeltaRows rows of one head each, all loads of which are under way together; bound by
// reading O and dO. The counter of the units that follow begins at 0.
constexpr int kDeltaRows = 4;
template <typename T>
__global__ void __launch_bounds__(256) delta_kernel(const Shape s, const T *dO, const T *O, const float *lse,
                                                    float2 *__restrict__ stats, int *counter) {
    grid_begin();
    if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * 16 * kDeltaRows + threadIdx.x / 16, rows = s.T * s.n_q;
    const int lane = threadIdx.x & 15;
    // lane k keeps row k's statistics: its lse is under way with everything else
    const int64_t mine = first + 16 * (lane < kDeltaRows ? lane : 0), t = mine / s.n_q;
    const int64_t at = (mine - t * s.n_q) * s.T + t;
    const bool keeps = lane < kDeltaRows && mine < rows;
    const float own_lse = keeps ? lse[at] : 0.0f;
    float own = 0.0f;
    Raw8<T> a[kDeltaRows], b[kDeltaRows];
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
        const int64_t i = first + 16 * k;
        zero8(a[k]);
        zero8(b[k]);
        if (i < rows && lane * 8 < s.d) {
            a[k] = load8(dO + i * s.d + lane * 8);
            b[k] = load8(O + i * s.d + lane * 8);
        }
    }
#pragma unroll
    for (int k = 0; k < kDeltaRows; ++k) {
        float x[8], y[8], sum = 0.0f;
        unpack8(a[k], x);
        unpack8(b[k], y);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum = fmaf(x[c], y[c], sum);
        sum = sum16(sum);
        if (lane == k) own = sum;
    }
    if (keeps) stats[at] = make_float2(own_lse * kLog2e, own);
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

// The same of all ranks' sums, which they have in shared memory at `sums`.
template <typename T>
__device__ __forceinline__ void plain_store_shared(const Shape &s, const float *sums, int pitch, float f, T *to, int r0,
                                                   int n, Share by) {
    const int rows = kRows / by.ranks, vectors = s.d / 4;
    for (int i = threadIdx.x; i < rows * vectors; i += kPlainThreads) {
        const int row = by.rank * rows + i / vectors, col = i % vectors * 4;
        if (r0 + row >= n) break;
        float4 x[kMaxRanks];
        of_ranks(sums + row * pitch + col, by.ranks, x);
        float y[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
        for (int q = 1; q < kMaxRanks; ++q) {
            y[0] += x[q].x;
            y[1] += x[q].y;
            y[2] += x[q].z;
            y[3] += x[q].w;
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) y[b] *= f;
        store4(to + (r0 + row) * s.ld + col, y);
    }
}

// dQ of queries q0 .. q0 + 63 of one head.
template <typename T>
__device__ __forceinline__ void plain_dq_tile(const Shape &s, const T *QKV, const T *dO, const float2 *stats,
                                           int64_t row0, int n, int q0, int h, T *dQKV, float *smem, Share by) {
    const PlainSmem lay(s.d);
    float *Q = smem, *K = Q + lay.rows(), *V = K + lay.rows(), *G = V + lay.rows(), *dS = G + lay.rows();
    const int d = s.d, kv = h / s.group;
    const int64_t qc = static_cast<int64_t>(s.q_head(h)) * d, kc = static_cast<int64_t>(s.k_head(kv)) * d,
                  vc = static_cast<int64_t>(s.v_head(kv)) * d, ldo = static_cast<int64_t>(s.n_q) * d;
    const T *base = QKV + row0 * s.ld;
    const KeyTiles tiles = key_tiles(s, q0, min(n, q0 + kRows), kRows);
    float o[4][2][4];
    clear(o);
    PlainRows<T> one, two;
    one.fetch(base + qc, s.ld, q0, n, d);
    two.fetch(dO + row0 * ldo + static_cast<int64_t>(h) * d, ldo, q0, n, d);
    one.put(Q, lay.pitch, d);
    two.put(G, lay.pitch, d);
    auto fetch = [&](int u) {
        if (u >= tiles.count()) return;
        one.fetch(base + kc, s.ld, tiles.at(u) * kRows, n, d);
        two.fetch(base + vc, s.ld, tiles.at(u) * kRows, n, d);
    };
    fetch(by.rank);
    for (int u = by.rank; u < tiles.count(); u += by.ranks) {
        const int k0 = tiles.at(u) * kRows;
        plain_sync();
        one.put(K, lay.pitch, d);
        two.put(V, lay.pitch, d);
        fetch(u + by.ranks);
        plain_sync();
        const bool masked = !all_seen(s, q0, q0 + kRows, k0, k0 + kRows) || q0 + kRows > n;
        plain_scores(s, Q, K, G, V, lay.pitch, stats + h * s.T + row0, q0, k0, n, masked, nullptr, dS);
        plain_sync();
        if (masked)
            plain_add<true, false>(dS, K, lay.pitch, d, o);
        else
            plain_add<false, false>(dS, K, lay.pitch, d, o);
    }
    if (by.ranks == 1) {
        plain_store(s, o, s.scale, dQKV + row0 * s.ld + qc, q0, n);
        return;
    }
    plain_sync();  // a rank may have had no step
    plain_put(o, Q, lay.pitch, d);
    ptx::cluster_sync();
    plain_store_shared(s, Q, lay.pitch, s.scale, dQKV + row0 * s.ld + qc, q0, n, by);
    ptx::cluster_sync();  // until all have read
}

// dK and dV of keys k0 .. k0 + 63 of one key/value head.
template <typename T>
__device__ __forceinline__ void plain_dkv_tile(const Shape &s, const T *QKV, const T *dO, const float2 *stats,
                                            int64_t row0, int n, int k0, int kv, T *dQKV, float *smem, Share by) {
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
    PlainRows<T> one, two;
    one.fetch(base + kc, s.ld, k0, n, d);
    two.fetch(base + vc, s.ld, k0, n, d);
    one.put(K, lay.pitch, d);
    two.put(V, lay.pitch, d);
    // steps: the tiles of queries that see the keys, head by head
    const int tiles = (query_end(s, k0, min(n, k0 + kRows), n) - k0 + kRows - 1) / kRows, steps = tiles * s.group;
    auto fetch = [&](int u) {
        if (u >= steps) return;
        const int at = kv * s.group + u / tiles, r0 = k0 + u % tiles * kRows;
        one.fetch(base + static_cast<int64_t>(s.q_head(at)) * d, s.ld, r0, n, d);
        two.fetch(dO + row0 * ldo + static_cast<int64_t>(at) * d, ldo, r0, n, d);
    };
    fetch(by.rank);
    for (int u = by.rank; u < steps; u += by.ranks) {
        const int h = kv * s.group + u / tiles, q0 = k0 + u % tiles * kRows;
        plain_sync();
        one.put(Q, lay.pitch, d);
        two.put(G, lay.pitch, d);
        fetch(u + by.ranks);
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
    if (by.ranks == 1) {
        plain_store(s, ok, s.scale, dQKV + row0 * s.ld + kc, k0, n);
        plain_store(s, ov, 1.0f, dQKV + row0 * s.ld + vc, k0, n);
        return;
    }
    plain_sync();  // a rank may have had no step
    plain_put(ok, K, lay.pitch, d);
    plain_put(ov, V, lay.pitch, d);
    ptx::cluster_sync();
    plain_store_shared(s, K, lay.pitch, s.scale, dQKV + row0 * s.ld + kc, k0, n, by);
    plain_store_shared(s, V, lay.pitch, 1.0f, dQKV + row0 * s.ld + vc, k0, n, by);
    ptx::cluster_sync();  // until all have read
}

template <typename T, bool MANY>
__global__ void __launch_bounds__(kPlainThreads)
    plain_backward_kernel(const Shape s, const T *QKV, const T *dO, const float2 *stats, int tiles, int ranks,
                          T *dQKV) {
    extern __shared__ float4 smem4[];
    float *const smem = reinterpret_cast<float *>(smem4);
    grid_begin();
    const Share by = this_share(ranks);
    const int64_t of_keys = static_cast<int64_t>(tiles) * s.n_kv;
    Scan scan;
    int64_t unit = blockIdx.x / static_cast<unsigned>(ranks);
#pragma unroll 1
    do {
        // dK and dV have the most steps and come first: those of the first keys, seen by the most queries; then dQ,
        // that of the last queries, which see the most keys
        const bool keys = unit < of_keys;
        const int heads = keys ? s.n_kv : s.n_q, at = static_cast<int>(keys ? unit : unit - of_keys), h = at % heads;
        const Tile t = find_tile(s, at / heads, kRows, tiles, scan);
        if (t.n == 0) {
            if (by.rank == 0) {
                zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(keys ? s.k_head(h) : s.q_head(h)) * s.d);
                if (keys) zero_rest(s, t, dQKV, s.ld, static_cast<int64_t>(s.v_head(h)) * s.d);
            }
        } else {
            if (MANY) plain_sync();  // the tile before
            if (keys)
                plain_dkv_tile(s, QKV, dO, stats, t.row0, t.n, t.tile * kRows, h, dQKV, smem, by);
            else
                plain_dq_tile(s, QKV, dO, stats, t.row0, t.n, (t.tiles - 1 - t.tile) * kRows, h, dQKV, smem, by);
        }
        unit += gridDim.x;
    } while (MANY && unit < of_keys + static_cast<int64_t>(tiles) * s.n_q);
}

// ------------------------------------------------------------------ tiles on the tensor cores
// The work is cut into units: dK and dV of 128 keys of a key/value head, and dQ of 128
// queries of a head. One block an SM takes units from a counter until there are none,
// those of dK and dV first and among each kind the ones with the most steps first, so
// that the small ones fill what the large ones leave. Sixteen warps, a warpgroup each of
//   warps 0 - 3, 4 - 7   compute: a thread one row of a 128 x 128 tile and half of its
//                        columns (warps 4 - 7 the second half)
//   warps 8, 11, 12      load tiles; fetch the queries' statistics where they go by
//                        columns; take the next unit, two ahead
//   warps 9, 10          issue the products
// While a unit's results are written the next one's tiles are loaded and its first
// scores formed.
constexpr int kBwdThreads = 512;
// The tiles that come and go, two of each step: those that are used from a step's first
// product to its last (Q for dK and dV, K for dQ) have three places, the others (dO, V)
// two. (One ring of five for both in turn made a tile wait for the other kind's last use:
// dQ stood still for 500 of 2400 cycles a step.)
constexpr int kLong = 0, kShort = 1, kPlaces = 5;
__device__ __forceinline__ int place_of(int kind, int n) { return kind == kLong ? n % 3 : 3 + (n & 1); }
__device__ __forceinline__ uint32_t round_of(int kind, int n) {
    return static_cast<uint32_t>(kind == kLong ? n / 3 : n >> 1) & 1u;
}

enum Kind : int { kKeys, kQueries, kRest, kEnd };  // of a unit; kRest: rows without a sequence
struct Unit {
    Tile t;
    int kind, head, first, steps, id;
};

struct BwdSmem {
    uint8_t stay[2][kTileBytes];  // K and V, or Q and dO
    uint8_t ring[kPlaces][kTileBytes];
    float stats[2][2][kTile];     // -lse log2(e) and -delta of a step's queries
    uint64_t full[kPlaces], empty[kPlaces], stay_full, stay_empty;
    uint64_t scores[2], dots, p_ready, ds_ready, stats_full[2], stats_empty[2], turn[2];
    uint64_t sum_done;            // a step's sum of dQ is complete
    uint64_t done, read;          // a unit's products are complete; its results have been read
    uint64_t unit_full[2], unit_empty[2], drain, aux;
    Unit unit[2];
    uint32_t tmem_slot;
    int abort_flag, odd;          // odd: the last of the block's units that has results which are not finite
};
static_assert(sizeof(BwdSmem) <= static_cast<size_t>(kMaxSmem), "the ring fits");
static_assert(offsetof(BwdSmem, full) >= 4 * (4 * kRows * (kMaxDim + 4) + 2 * kRows * kPitchP), "room for plain tiles");
constexpr int kUnitReaders = 12;  // warps

// What the backward keeps in its workspace beside the statistics.
struct Shared {
    int *counter;  // of units taken; zeroed by the kernel before
    int *next;     // [units] the block's odd unit before this one
};

// Tiles of all sequences, and the rows of none.
__device__ __forceinline__ Tile count_tiles(const Shape &s, int &tiles) {
    Scan scan;
    Tile t = find_tile(s, INT_MAX, kTile, 0, scan);
    tiles = INT_MAX - t.part;
    t.part = blockIdx.x;
    t.parts = gridDim.x;
    return t;
}

// Unit `id` of so many tiles; every lane of a warp calls it.
__device__ __forceinline__ Unit find_unit(const Shape &s, int id, int tiles, Scan &scan) {
    Unit u{};
    u.id = id;
    u.kind = kEnd;
    const int64_t of_keys = static_cast<int64_t>(tiles) * s.n_kv, all = of_keys + static_cast<int64_t>(tiles) * s.n_q;
    if (id >= all) return u;
    u.kind = id < of_keys ? kKeys : kQueries;
    const int heads = u.kind == kKeys ? s.n_kv : s.n_q, at = u.kind == kKeys ? id : static_cast<int>(id - of_keys);
    u.head = at % heads;
    u.t = find_tile(s, at / heads, kTile, 0, scan);
    if (u.kind == kKeys) {
        // the first keys are seen by the most queries, the last queries see the most keys
        u.first = u.t.tile * kTile;
        const int end = query_end(s, u.first, min(u.t.n, u.first + kTile), u.t.n);
        u.steps = (end - u.first + kTile - 1) / kTile * s.group;
    } else {
        u.first = (u.t.tiles - 1 - u.t.tile) * kTile;
        u.steps = key_tiles(s, u.first, min(u.t.n, u.first + kTile), kTile).count();
    }
    return u;
}

// Keys as rows, per tile of 128 queries of a head:
//   S^T = K Q^T  ->  P^T = 2^(S^T c - lse)   ->  dV += P^T dO
//   dP^T = V dO^T  ->  dS^T = P^T (dP^T - delta)  ->  dK += dS^T Q
// Tensor memory: S^T, dP^T, dV, dK, 128 columns each; P^T and dS^T overwrite what they
// are made of, in bf16, each half of the columns its own place. One warp issues S and
// dV, the other dP and dK, in turn:
//   S(0), dP(0), dV(0) S(1), dK(0) dP(1), dV(1) S(2), ..
// so that two products are under way while the threads form P or dS, and each warp
// waits for what it needs during the other's.
//
// Queries as rows, per tile of 128 keys:
//   S = Q K^T, dP = dO V^T  ->  dS = 2^(S c - lse) (dP - delta)  ->  dQ += dS K
// Tensor memory: two S (dS overwrites the one that it is made of), dP, dQ. One warp issues
// S, the other dP and dQ, in the order  S(0), dP(0), S(1), dP(1) dQ(0), S(2), dP(2) dQ(1), ..
// dP of the next keys is begun as soon as the threads have read the one before, and P
// is formed of the next S before dP has come.
//
// Steps are counted through all of a block's units: barriers go by their number.
constexpr uint32_t kSumV = 256, kSumK = 384, kDots = 256, kSumQ = 384;  // and at 0 and 128 S^T and dP^T, or the two S

__global__ void __launch_bounds__(kBwdThreads, 1)
    tc_backward_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_do,
                       const Shape s, const __nv_bfloat16 *QKV, const __nv_bfloat16 *dO, const float2 *stats,
                       Shared shared, int debug_withhold, __nv_bfloat16 *dQKV) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    BwdSmem &m = *reinterpret_cast<BwdSmem *>(smem_raw);
    volatile int *abort_flag = &m.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPlaces; ++i) {
            ptx::mbar_init(&m.full[i], 1);
            ptx::mbar_init(&m.empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&m.scores[i], 1);
            ptx::mbar_init(&m.turn[i], 1);
            ptx::mbar_init(&m.stats_full[i], 32);
            ptx::mbar_init(&m.stats_empty[i], 8);
            ptx::mbar_init(&m.unit_full[i], 1);
            ptx::mbar_init(&m.unit_empty[i], kUnitReaders);
        }
        ptx::mbar_init(&m.stay_full, 1);
        ptx::mbar_init(&m.stay_empty, 2);
        ptx::mbar_init(&m.dots, 1);
        ptx::mbar_init(&m.p_ready, 8);
        ptx::mbar_init(&m.ds_ready, 8);
        ptx::mbar_init(&m.sum_done, 1);
        ptx::mbar_init(&m.done, 2);
        ptx::mbar_init(&m.read, 8);
        ptx::mbar_init(&m.drain, 2);
        ptx::mbar_init(&m.aux, 1);
        m.abort_flag = 0;
        m.odd = -1;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map);
        ptx::prefetch_tmap(&map_do);
    }
    if (warp == 9) {
        ptx::tmem_alloc(&m.tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    grid_begin();
    // the next unit of the warp that calls it, read by all its lanes; false at the end
    int round = 0;
    auto next_unit = [&](Unit &u) {
        const int at = round & 1;
        const uint32_t parity = (round >> 1) & 1;
        ++round;
        if (!wait_all(&m.unit_full[at], parity, abort_flag, s.err, 48)) return false;
        u = m.unit[at];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&m.unit_empty[at]);
        return u.kind != kEnd;
    };
    const int blocks = s.d > 64 ? 2 : 1;
    int n = 0, units = 0;  // steps and units (with steps) so far
    Unit u;

    if (warp < 8) {
        // ------------------------------------------------ compute
        ptx::registers_up<184>();  // 2 x 184 + 2 x 72 = 4 x 128, the launch's
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float c = s.scale * kLog2e;
        int steps_of_keys = 0;
        bool alive = true;
        auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t where) {
            alive = alive && wait_all<true>(bar, parity, abort_flag, s.err, where);
            return alive;
        };
        auto tell = [&](uint64_t *bar) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar);
        };
        while (alive && next_unit(u)) {
            if (u.kind == kRest) {
                for (int h = 0; h < s.n_q + 2 * s.n_kv; ++h)
                    zero_rest(s, u.t, dQKV, s.ld, static_cast<int64_t>(h) * s.d);
                continue;
            }
            const int row = u.first + r;
            const bool mine = row < u.t.n;
            bool fine = true;
            if (u.kind == kKeys) {
                const int limit = s.window && row >= s.sinks ? min(u.t.n, row + s.window) : u.t.n;  // of queries
                const int of_head = u.steps / s.group;
                int q = 0;
                for (int it = 0; it < u.steps; ++it, ++n, ++steps_of_keys) {
                    const int q0 = u.first + q * kTile, k0 = u.first;
                    q = q + 1 == of_head ? 0 : q + 1;
                    const bool masked = !all_seen(s, q0, q0 + kTile, k0, k0 + kTile) || q0 + kTile > u.t.n;
                    // queries from the key's own on, below its limit
                    auto seen = [&](int b) {
                        const int at = q0 + half * 64 + b * 32;
                        return below(limit - at) & ~below(row - at);
                    };
                    const int buf = steps_of_keys & 1;
                    const float *lse = m.stats[buf][0] + half * 64, *delta = m.stats[buf][1] + half * 64;
                    wait(&m.stats_full[buf], (steps_of_keys >> 1) & 1, 36);
                    if (!wait(&m.scores[n & 1], (n >> 1) & 1, 37)) break;
                    ptx::tc_fence_after();
                    float x[2][32], y[2][32];
                    uint32_t p[32];
                    read_half(lanes + half * 64, x);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 l = *reinterpret_cast<const float4 *>(lse + b * 32 + e);
                            float(&v)[32] = x[b];
                            scale2(v[e], v[e + 1], c, l.x, l.y);
                            scale2(v[e + 2], v[e + 3], c, l.z, l.w);
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[b][e] = exp2_fast(x[b][e]);
                        if (masked) keep(x[b], seen(b), 0.0f);
                        pack32(x[b], p + b * 16);
                    }
                    ptx::tmem_st32_async(lanes + half * 64, p);
                    ptx::tmem_wait_st();
                    tell(&m.p_ready);
                    if (!wait(&m.dots, n & 1, 38)) break;
                    ptx::tc_fence_after();
                    read_half(128 + lanes + half * 64, y);
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
                    ptx::tmem_st32_async(128 + lanes + half * 64, p);
                    ptx::tmem_wait_st();
                    tell(&m.ds_ready);
                    if (lane == 0) ptx::mbar_arrive(&m.stats_empty[buf]);
                }
            } else {
                const KeyTiles kt = key_tiles(s, u.first, min(u.t.n, u.first + kTile), kTile);
                const float2 st = mine ? stats[u.head * s.T + u.t.row0 + row] : make_float2(INFINITY, 0.0f);
                for (int it = 0; it < u.steps; ++it, ++n) {
                    const int q0 = u.first, k0 = kt.at(it) * kTile;
                    const bool masked = !all_seen(s, q0, q0 + kTile, k0, k0 + kTile);
                    auto seen = [&](int b) {
                        const int at = k0 + half * 64 + b * 32, hi = row - at;
                        return visible(hi, s.window ? hi - s.window + 1 : -kTile, s.sinks - at);
                    };
                    const uint32_t t_s = (n & 1) * 128 + lanes + half * 64;
                    if (!wait(&m.scores[n & 1], (n >> 1) & 1, 44)) break;
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
                    if (!wait(&m.dots, n & 1, 45)) break;
                    ptx::tc_fence_after();
                    read_half(kDots + lanes + half * 64, y);
                    tell(&m.p_ready);  // dP has been read
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
                    tell(&m.ds_ready);
                }
            }
            if (!wait(&m.done, units & 1, 46)) break;
            ++units;
            ptx::tc_fence_after();
            float o[2][32];
            const int head = u.kind == kQueries ? s.q_head(u.head) : half ? s.v_head(u.head) : s.k_head(u.head);
            const int rows = u.t.n - (row - lane);
            __nv_bfloat16 *to = dQKV + (u.t.row0 + row - lane) * s.ld + static_cast<int64_t>(head) * s.d;
            if (u.kind == kKeys) {
                // both halves of dK by warps 0 - 3, of dV by warps 4 - 7
                const uint32_t from = (half ? kSumV : kSumK) + lanes;
                const float f = half ? 1.0f : s.scale;
                read_half(from, o);
                fine = write_rows(o, f, 0, s.d, to, s.ld, rows);
                read_half(from + 64, o);
                tell(&m.read);
                if (s.d > 64) fine = write_rows(o, f, 64, s.d, to, s.ld, rows) && fine;
            } else {
                read_half(kSumQ + lanes + half * 64, o);
                tell(&m.read);
                if (half * 64 < s.d) fine = write_rows(o, s.scale, half * 64, s.d, to, s.ld, rows);
            }
            // the block's odd units are a list that begins at m.odd
            if (!__all_sync(0xffffffffu, fine) && lane == 0) {
                const int before = atomicExch(&m.odd, u.id);
                if (before != u.id) shared.next[u.id] = before;  // not put there by another warp
            }
        }
    } else {
        ptx::registers_down<72>();
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t where) {
            ok = ok && wait_all<true>(bar, parity, abort_flag, s.err, where);
            return ok;
        };
        if (warp == 8) {
            // ------------------------------------------------ loads
            const bool leader = ptx::elect_one();
            const uint32_t bytes = blocks * kBlockBytes;
            uint32_t aux_phase = 0;
            auto load = [&](int kind, int at, const CUtensorMap *from, int head, int64_t row, int rows) {
                const int place = place_of(kind, at);
                if (!wait(&m.empty[place], round_of(kind, at) ^ 1, 30)) return;
                ok = load_rows(leader, m.ring[place], from, &m.full[place], &m.aux, aux_phase, head, row, blocks, rows,
                               abort_flag, s.err, debug_withhold != 0 && blockIdx.x == 0 && n == 0);
            };
            int longs = 0, shorts = 0;
            while (ok && next_unit(u)) {
                if (u.kind == kRest) continue;
                const bool keys = u.kind == kKeys;
                const int kv = keys ? u.head : u.head / s.group;
                if (!wait(&m.stay_empty, (units & 1) ^ 1, 27)) break;
                ++units;
                const int64_t row = u.t.row0 + u.first;
                if (leader) {
                    ptx::mbar_arrive_expect_tx(&m.stay_full, 2 * bytes);
                    load_tile(m.stay[0], &map, &m.stay_full, keys ? s.k_head(kv) : s.q_head(u.head), row, blocks);
                    load_tile(m.stay[1], keys ? &map : &map_do, &m.stay_full, keys ? s.v_head(kv) : u.head, row,
                              blocks);
                }
                const KeyTiles kt = key_tiles(s, u.first, min(u.t.n, u.first + kTile), kTile);
                const int of_head = u.steps / s.group;
                int g = 0, q = 0;
                for (int it = 0; it < u.steps && ok; ++it, ++n) {
                    if (keys) {
                        const int h = kv * s.group + g;
                        const int64_t at = row + q * kTile;
                        const int left = u.t.n - (u.first + q * kTile), rows = left < kTile ? left : 0;
                        load(kLong, n, &map, s.q_head(h), at, rows);
                        longs = ok ? n + 1 : longs;
                        if (ok) load(kShort, n, &map_do, h, at, rows);
                        if (++q == of_head) {
                            q = 0;
                            ++g;
                        }
                    } else {
                        const int64_t at = u.t.row0 + static_cast<int64_t>(kt.at(it)) * kTile;
                        const int left = u.t.n - kt.at(it) * kTile;
                        load(kLong, n, &map, s.k_head(kv), at, left < kTile ? left : 0);
                        longs = ok ? n + 1 : longs;
                        if (ok) load(kShort, n, &map, s.v_head(kv), at, 0);
                    }
                    shorts = ok ? n + 1 : shorts;
                }
            }
            // copies land before the block ends, also where others give up only after this warp is done
            if (leader) {
                if (units) ptx::mbar_wait_drain(&m.stay_full, (units - 1) & 1);
                for (int i = max(0, longs - 3); i < longs; ++i)
                    ptx::mbar_wait_drain(&m.full[place_of(kLong, i)], round_of(kLong, i));
                for (int i = max(0, shorts - 2); i < shorts; ++i)
                    ptx::mbar_wait_drain(&m.full[place_of(kShort, i)], round_of(kShort, i));
            }
            __syncwarp();
        } else if (warp == 9 || warp == 10) {
            // ------------------------------------------------ products
            const int i = warp - 9;
            const bool leader = ptx::elect_one();
            const uint32_t idesc = idesc_weighted(s.d), base = ptx::smem_u32(m.ring[0]),
                           stays = ptx::smem_u32(m.stay[0]);
            auto wait_for = [&](const auto &phases, uint32_t where) {
                ok = ok && wait_each(phases, abort_flag, s.err, where);
                return ok;
            };
            auto arrived = [&](bool needed, int kind, int at) {
                return Phase{needed ? &m.full[place_of(kind, at)] : nullptr, round_of(kind, at)};
            };
            // a turn of the first warp, then one of the second
            int turns = 0, sums_of_queries = 0;
            auto my_turn = [&] {
                const int before = i == 1 ? turns : turns - 1;
                ++turns;
                return Phase{before >= 0 ? &m.turn[i] : nullptr, before & 1u};
            };
            auto tile = [&](int kind, int at) { return base + place_of(kind, at) * kTileBytes; };
            auto free_place = [&](int kind, int at) { commit(leader, &m.empty[place_of(kind, at)]); };
            while (ok && next_unit(u)) {
                if (u.kind == kRest) continue;
                // the unit before has left tensor memory, but for its results
                const Phase begin[2] = {{units > 0 ? &m.done : nullptr, (units - 1) & 1u}, {&m.stay_full, units & 1u}};
                wait_for(begin, 32);
                if (u.kind == kKeys) {
                    // step `it`: the sum with the tile of step it - 1, then the scores (or dots) of this one
                    const uint32_t t_in = i * 128, t_sum = i ? kSumK : kSumV;
                    const int kind_in = i ? kShort : kLong, kind_of = i ? kLong : kShort;
                    uint64_t *const ready = i ? &m.ds_ready : &m.p_ready;
                    for (int it = 0; it <= u.steps && ok; ++it, ++n) {
                        const bool scores = it < u.steps, sums = it > 0;
                        const Phase phases[4] = {arrived(scores, kind_in, n), arrived(sums, kind_of, n - 1), my_turn(),
                                                 {sums ? ready : nullptr, (n - 1) & 1u}};
                        if (!wait_for(phases, 33)) break;
                        ptx::tc_fence_after();
                        if (sums) mma_weighted(leader, t_sum, t_in, 64, tile(kind_of, n - 1), idesc, it > 1);
                        if (scores)
                            mma_scores(leader, t_in, stays + i * kTileBytes, tile(kind_in, n), s.d,
                                       i ? &m.dots : &m.scores[n & 1], &m.turn[i ^ 1]);
                        else if (leader)
                            ptx::mbar_arrive(&m.turn[i ^ 1]);
                        if (it == u.steps - 1) commit(leader, &m.stay_empty);
                        if (sums) free_place(kind_of, n - 1);
                        if (scores) free_place(kind_in, n);
                    }
                    --n;  // the last turn was one more than there are steps
                } else if (i == 0) {
                    for (int it = 0; it < u.steps && ok; ++it, ++n) {
                        // dS in this S's place has been used
                        const Phase phases[3] = {arrived(true, kLong, n), my_turn(),
                                                 {it > 1 ? &m.sum_done : nullptr, (sums_of_queries - 2) & 1u}};
                        ++sums_of_queries;
                        if (!wait_for(phases, 43)) break;
                        ptx::tc_fence_after();
                        mma_scores(leader, (n & 1) * 128, stays, tile(kLong, n), s.d, &m.scores[n & 1], &m.turn[1]);
                        free_place(kLong, n);
                        if (it == u.steps - 1) commit(leader, &m.stay_empty);
                    }
                } else {
                    auto sum = [&](int at, bool first) {
                        if (!wait(&m.ds_ready, at & 1, 47)) return;
                        ptx::tc_fence_after();
                        mma_weighted(leader, kSumQ, (at & 1) * 128, 64, tile(kLong, at), idesc, !first);
                        free_place(kLong, at);
                        commit(leader, &m.sum_done);
                    };
                    for (int it = 0; it < u.steps && ok; ++it, ++n) {
                        // dP before has been read; of a unit's first: what was in its place before
                        const Phase phases[4] = {arrived(true, kShort, n), arrived(true, kLong, n), my_turn(),
                                                 it > 0          ? Phase{&m.p_ready, (n - 1) & 1u}
                                                 : units > 0     ? Phase{&m.read, (units - 1) & 1u}
                                                                 : Phase{nullptr, 0}};
                        if (!wait_for(phases, 26)) break;
                        ptx::tc_fence_after();
                        mma_scores(leader, kDots, stays + kTileBytes, tile(kShort, n), s.d, &m.dots, &m.turn[0]);
                        // a place is given back by two warps elsewhere
                        free_place(kShort, n);
                        free_place(kShort, n);
                        if (it == u.steps - 1) commit(leader, &m.stay_empty);
                        if (it > 0) sum(n - 1, it == 1);
                    }
                    if (ok) sum(n - 1, u.steps == 1);
                }
                if (!ok) break;
                ++units;
                commit(leader, &m.done);
            }
            commit(leader, &m.drain);
            if (lane == 0) ptx::mbar_wait_drain(&m.drain, 0);
            __syncwarp();
        } else if (warp == 11) {
            // ------------------------------------------------ the queries' statistics; past the end P is 2^-inf
            while (ok && next_unit(u)) {
                if (u.kind != kKeys) continue;
                const int of_head = u.steps / s.group;
                for (int g = 0; g < s.group && ok; ++g) {
                    const float2 *from = stats + (u.head * s.group + g) * s.T + u.t.row0;
                    for (int q = 0; q < of_head; ++q, ++n) {
                        float2 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int row = u.first + q * kTile + e * 32 + lane;
                            v[e] = row < u.t.n ? from[row] : make_float2(INFINITY, 0.0f);
                        }
                        if (!wait(&m.stats_empty[n & 1], ((n >> 1) & 1) ^ 1, 29)) break;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            m.stats[n & 1][0][e * 32 + lane] = -v[e].x;  // both are subtracted
                            m.stats[n & 1][1][e * 32 + lane] = -v[e].y;
                        }
                        ptx::mbar_arrive(&m.stats_full[n & 1]);
                    }
                }
            }
        } else if (warp == 12) {
            // ------------------------------------------------ what comes next
            int tiles;
            const Tile rest = count_tiles(s, tiles);
            Scan scan;
            bool zero = rest.head_rows + (s.T - rest.tail_row) != 0;
            for (int r = 0;; ++r) {
                Unit next{};
                if (zero) {
                    next.t = rest;
                    next.kind = kRest;
                    zero = false;
                } else {
                    int id = lane == 0 ? atomicAdd(shared.counter, 1) : 0;
                    id = __shfl_sync(0xffffffffu, id, 0);
                    next = find_unit(s, id, tiles, scan);
                }
                if (!wait(&m.unit_empty[r & 1], ((r >> 1) & 1) ^ 1, 28)) break;
                if (lane == 0) {
                    m.unit[r & 1] = next;
                    ptx::mbar_arrive(&m.unit_full[r & 1]);
                }
                __syncwarp();
                if (next.kind == kEnd) break;
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(0, kTmemCols);
    }
    // What is masked within a sequence has met 0 times its value: a unit with results that are not finite is
    // computed again where masked values are passed over.
    int odd = m.odd;
    if (odd < 0 || *abort_flag || threadIdx.x >= kPlainThreads) return;
    int tiles;
    count_tiles(s, tiles);
    plain_sync();  // all have read m.odd
    for (; odd >= 0; odd = shared.next[odd]) {
        Scan scan;
        const Unit w = find_unit(s, odd, tiles, scan);
#pragma unroll 1
        for (int at = w.first; at < min(w.t.n, w.first + kTile); at += kRows) {
            plain_sync();
            if (w.kind == kKeys)
                plain_dkv_tile(s, QKV, dO, stats, w.t.row0, w.t.n, at, w.head, dQKV,
                               reinterpret_cast<float *>(smem_raw), Share{0, 1});
            else
                plain_dq_tile(s, QKV, dO, stats, w.t.row0, w.t.n, at, w.head, dQKV,
                              reinterpret_cast<float *>(smem_raw), Share{0, 1});
        }
    }
}

// ------------------------------------------------------------------ host
// The workspace: statistics, the counter, the lists of odd units.
inline int64_t units_of(int64_t T, int64_t n_heads, int64_t n_kv_heads, int64_t sequences) {
    return (T / kTile + sequences) * (n_heads + n_kv_heads);
}
inline size_t stats_bytes(int64_t T, int64_t n_heads) {
    return round_up(static_cast<size_t>(T * n_heads) * sizeof(float2), 256);
}

tpce_status tc_backward(const Shape &s, const void *QKV, const void *dO, const float2 *stats, void *dQKV,
                        cudaStream_t stream) {
    const char *name = "attn_backward";
    CUtensorMap map, map_do;
    if (!make_tmap_heads(&map, QKV, s.d, s.n_q + 2 * s.n_kv, s.T, s.ld, kTile) ||
        !make_tmap_heads(&map_do, dO, s.d, s.n_q, s.T, static_cast<uint64_t>(s.n_q) * s.d, kTile))
        return fail(TPCE_ERR_CUDA, "%s: tensor map", name);
    cudaError_t e = allow_smem<tc_backward_kernel>();
    if (e != cudaSuccess) return fail_cuda(e, name);
    const int64_t units = units_of(s.T, s.n_q, s.n_kv, s.offsets ? s.sequences : 1);
    char *after = reinterpret_cast<char *>(const_cast<float2 *>(stats)) + stats_bytes(s.T, s.n_q);
    const Shared shared{reinterpret_cast<int *>(after), reinterpret_cast<int *>(after + 256)};
    KernelTimer timer(name, stream);
    e = step::launch(tc_backward_kernel, static_cast<unsigned>(std::min<int64_t>(units, num_sms())), kBwdThreads,
                     sizeof(BwdSmem), stream, map, map_do, s, static_cast<const __nv_bfloat16 *>(QKV),
                     static_cast<const __nv_bfloat16 *>(dO), stats, shared, take_debug_withhold(),
                     static_cast<__nv_bfloat16 *>(dQKV));
    return e == cudaSuccess ? check_launch(name, stream) : fail_cuda(e, name);
}

template <typename T>
tpce_status plain_backward(const Shape &s, const void *QKV, const void *dO, const float2 *stats, void *dQKV,
                           cudaStream_t stream) {
    const char *name = "attn_backward";
    const int tiles = static_cast<int>(grid_tiles(s, kRows));
    const size_t smem = PlainSmem(s.d).backward();
    const int64_t units = static_cast<int64_t>(tiles) * (s.n_q + s.n_kv);
    const int ranks = ranks_of(s, units, static_cast<int64_t>(tiles) * s.n_kv, steps_of(s) * s.group, 8);
    KernelTimer timer(name, stream);
    auto go = [&](auto kernel, cudaError_t e, int64_t blocks) {
        if (e != cudaSuccess) return e;
        return step::launch_clusters(ranks, kernel, static_cast<unsigned>(blocks), kPlainThreads, smem, stream, s,
                                     static_cast<const T *>(QKV), static_cast<const T *>(dO), stats, tiles, ranks,
                                     static_cast<T *>(dQKV));
    };
    const cudaError_t e =
        many_sequences(s)
            ? go(plain_backward_kernel<T, true>, allow_smem<plain_backward_kernel<T, true>>(), many_blocks(units))
            : go(plain_backward_kernel<T, false>, allow_smem<plain_backward_kernel<T, false>>(), units * ranks);
    return e == cudaSuccess ? check_launch(name, stream) : fail_cuda(e, name);
}

template <typename T>
tpce_status delta(const Shape &s, const void *dO, const void *O, const float *lse, float2 *stats,
                  cudaStream_t stream) {
    KernelTimer timer("attn_delta", stream);
    const int64_t blocks = (s.T * s.n_q + 16 * kDeltaRows - 1) / (16 * kDeltaRows);
    const cudaError_t e =
        step::launch(delta_kernel<T>, static_cast<unsigned>(blocks), 256, 0, stream, s,
                     static_cast<const T *>(dO), static_cast<const T *>(O), lse, stats,
                     reinterpret_cast<int *>(reinterpret_cast<char *>(stats) + stats_bytes(s.T, s.n_q)));
    return e == cudaSuccess ? check_launch("attn_delta", stream) : fail_cuda(e, "attn_delta");
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" size_t tpce_attn_core_workspace_bytes(int64_t T, int64_t n_heads) {
    if (T <= 0 || T > (int64_t{1} << 30) || n_heads < 1 || n_heads > 4096) return 0;
    // no more tiles than rows, for query and key/value heads
    return stats_bytes(T, n_heads) + 256 + static_cast<size_t>(T * 2 * n_heads) * sizeof(int);
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
