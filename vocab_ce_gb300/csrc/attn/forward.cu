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
                                                T *O, float *lse, float *smem, Share by) {
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
    PlainRows<T> rows_q, rows_k, rows_v;
    auto fetch = [&](int u) {
        if (u >= tiles.count()) return;
        rows_k.fetch(k, s.ld, tiles.at(u) * kRows, n, d);
        rows_v.fetch(v, s.ld, tiles.at(u) * kRows, n, d);
    };
    rows_q.fetch(q, s.ld, q0, n, d);
    fetch(by.rank);
    rows_q.put(Q, lay.pitch, d);
    for (int u = by.rank; u < tiles.count(); u += by.ranks) {
        const int k0 = tiles.at(u) * kRows;
        plain_sync();
        rows_k.put(K, lay.pitch, d);
        rows_v.put(V, lay.pitch, d);
        fetch(u + by.ranks);
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
    if (by.ranks > 1) {
        // each rank's maximum, sum and outputs so far, scaled to the largest maximum
        plain_sync();  // a rank may have had no step
        plain_put(o, Q, lay.pitch, d);
        if (tx == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4 *>(K + (4 * ty + i) * lay.pitch) = make_float4(m[i], l[i], 0.0f, 0.0f);
        }
        ptx::cluster_sync();
        const int rows = kRows / by.ranks, vectors = d / 4;
        for (int i = threadIdx.x; i < rows * vectors; i += kPlainThreads) {
            const int r = by.rank * rows + i / vectors, row = q0 + r, col = i % vectors * 4;
            if (row >= n) break;
            float4 x[kMaxRanks], y[kMaxRanks];
            of_ranks(K + r * lay.pitch, by.ranks, x);
            of_ranks(Q + r * lay.pitch + col, by.ranks, y);
            float top = -INFINITY, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kMaxRanks; ++w)
                if (w < by.ranks) top = fmaxf(top, x[w].x);
            const float at = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < kMaxRanks; ++w) {
                const float f = w < by.ranks ? exp2f(x[w].x - at) : 0.0f;
                sum = fmaf(x[w].y, f, sum);
                v[0] = fmaf(y[w].x, f, v[0]);
                v[1] = fmaf(y[w].y, f, v[1]);
                v[2] = fmaf(y[w].z, f, v[2]);
                v[3] = fmaf(y[w].w, f, v[3]);
            }
            const float inv = 1.0f / sum;
#pragma unroll
            for (int b = 0; b < 4; ++b) v[b] *= inv;
            store4(O + (row0 + row) * s.n_q * d + static_cast<int64_t>(h) * d + col, v);
            if (col == 0) lse[h * s.T + row0 + row] = (top + log2f(sum)) * kLn2;
        }
        ptx::cluster_sync();  // until all have read
        return;
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
    for (int64_t r = static_cast<int64_t>(t.part) * kPlainThreads + threadIdx.x; r < rows;
         r += static_cast<int64_t>(t.parts) * kPlainThreads)
        lse[h * s.T + (r < t.head_rows ? r : t.tail_row + r - t.head_rows)] = 0.0f;
}

template <typename T, bool MANY>
__global__ void __launch_bounds__(kPlainThreads)
    plain_forward_kernel(const Shape s, const T *QKV, int tiles, int ranks, T *O, float *lse) {
    extern __shared__ float4 smem4[];
    grid_begin();
    const Share by = this_share(ranks);
    Scan scan;
    int64_t unit = blockIdx.x / static_cast<unsigned>(ranks);
#pragma unroll 1
    do {
        const int h = static_cast<int>(unit % s.n_q);
        const Tile t = find_tile(s, static_cast<int>(unit / s.n_q), kRows, tiles, scan);
        if (t.n == 0) {
            if (by.rank == 0) forward_rest(s, t, h, O, lse);
        } else {
            if (MANY) plain_sync();  // the tile before
            // the last queries see the most keys: they come first
            plain_forward_tile(s, QKV, t.row0, t.n, (t.tiles - 1 - t.tile) * kRows, h, O, lse,
                               reinterpret_cast<float *>(smem4), by);
        }
        unit += gridDim.x;
    } while (MANY && unit < static_cast<int64_t>(tiles) * s.n_q);
}

template <typename T>
tpce_status plain_forward(const Shape &s, const void *QKV, void *O, float *lse, cudaStream_t stream) {
    KernelTimer timer("attn_forward", stream);
    const int tiles = static_cast<int>(grid_tiles(s, kRows));
    const size_t smem = PlainSmem(s.d).forward();
    const int64_t units = static_cast<int64_t>(tiles) * s.n_q;
    const int ranks = ranks_of(s, units, units, steps_of(s), 4);
    auto go = [&](auto kernel, cudaError_t e, int64_t blocks) {
        if (e != cudaSuccess) return e;
        return step::launch_clusters(ranks, kernel, static_cast<unsigned>(blocks), kPlainThreads, smem, stream, s,
                                     static_cast<const T *>(QKV), tiles, ranks, static_cast<T *>(O), lse);
    };
    const cudaError_t e =
        many_sequences(s)
            ? go(plain_forward_kernel<T, true>, allow_smem<plain_forward_kernel<T, true>>(), many_blocks(units))
            : go(plain_forward_kernel<T, false>, allow_smem<plain_forward_kernel<T, false>>(), units * ranks);
    return e == cudaSuccess ? check_launch("attn_forward", stream) : fail_cuda(e, "attn_forward");
}

// ------------------------------------------------------------------ tiles on the tensor cores
// One block an SM stays for all its work: pairs of 128-query tiles that read the same
// keys, two heads of a group where it is even, else two neighbouring tiles of one head.
// Twenty warps:
//   warps 0 - 7, 8 - 15  the softmax of tile 0 and of tile 1, two threads a query: the
//                        first four warps have the first 64 keys of a tile, the next four
//                        the others (with one thread a query the tensor cores waited for it)
//   warp 16              loads: Q of a pair, K and V tiles through a ring
//   warps 17, 18         issue the products of tile 0 and of tile 1, in turn: while one has
//                        its products under way the other waits for what it needs next
//                        (one warp for both left the tensor cores idle in its waits, a sixth
//                        of the time; two that do not take turns split them when both have
//                        something, so that neither tile's threads have theirs early)
//   warp 19              finds the next pair, two ahead
// so that the next pair's loads and first scores run while results are written.
// Tensor memory: the scores S of both tiles (128 columns each; P overwrites the first
// half of S in bf16) and both O. For each key tile
//   S = Q K^T  ->  softmax threads: running maximum, P = 2^(S c - m), row sums  ->  O += P V
// with tile 1's products under way while tile 0's threads work, and the other way
// round. The products of a tile are issued in this order and run in it, so that S of
// the next keys is written only after P has been used, and when S has arrived O is
// complete up to the keys before. A thread raises its maximum (and scales its O in
// tensor memory) only when a score is more than 2^8 above it: P then stays below 2^8,
// and O, l and lse are as exact.
constexpr int kFwdThreads = 640, kFwdStages = 4;
constexpr int kSoftWarps = 16, kLoadWarp = 16, kMmaWarp = 17, kWorkWarp = 19;
constexpr float kRaise = 8.0f;  // in powers of two
constexpr int kOddBits = 512;

// A pair of tiles, or rows without a sequence (n == 0), or the end (unit < 0).
struct Work {
    Tile t;
    int unit, first;
};
struct FwdSmem {
    uint8_t q[2][kTileBytes];
    uint8_t ring[kFwdStages][kTileBytes];
    uint8_t out[kSoftWarps][32 * 64];  // a warp's rows on their way to O, 32 columns at a time; its rows' maxima
    float row_sum[kSoftWarps][32];
    uint64_t full[kFwdStages], empty[kFwdStages];
    uint64_t q_full, q_empty;
    uint64_t turn[2], s_full[2], p_full[2], o_full[2], o_empty[2];
    uint64_t work_full[2], work_empty[2];
    uint64_t drain, aux;
    Work work[2];
    uint32_t odd[2][kOddBits / 32];  // of the block's pairs: a tile has results that are not finite
    uint32_t tmem_slot;
    int abort_flag;
};
static_assert(sizeof(FwdSmem) <= static_cast<size_t>(kMaxSmem), "the ring fits");
constexpr int kWorkReaders = kSoftWarps + 3;  // warps

// The key tiles of both tiles together, and which of the two needs one.
struct Pair {
    int head[2], q0[2], count;
    KeyTiles one[2], both;
    __device__ __forceinline__ bool there(int i) const { return one[i].last >= 0; }
    __device__ __forceinline__ bool needs(int i, int k) const {
        return k < one[i].first || (k >= one[i].from && k <= one[i].last);
    }
    __device__ __forceinline__ Pair(const Shape &s, const Work &w, bool by_heads) {
        head[0] = by_heads ? 2 * w.unit : w.unit;
        head[1] = head[0] + (by_heads ? 1 : 0);
        q0[0] = w.first;
        q0[1] = w.first + (by_heads ? 0 : kTile);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            one[i] = q0[i] < w.t.n ? key_tiles(s, q0[i], min(w.t.n, q0[i] + kTile), kTile) : KeyTiles{0, 0, -1};
        both = one[0];
        if (there(1)) {
            both.last = one[1].last;
            // the second tile's window begins later: what only its sinks need is needed by the first anyway
            both.first = max(one[0].first, min(one[1].first, one[0].from));
        }
        count = both.count();
    }
};

// The block's r-th pair: neighbouring blocks take neighbouring pairs, in turn from both
// ends, and the pairs with the most keys come first.
__device__ __forceinline__ Work find_work(const Shape &s, int r, int units, int tiles, bool by_heads, Scan &scan) {
    Work w{};
    w.unit = -1;
    const int64_t item = static_cast<int64_t>(r) * gridDim.x + (r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (item >= static_cast<int64_t>(units) * tiles) return w;
    const int rows = by_heads ? kTile : 2 * kTile;
    w.t = find_tile(s, static_cast<int>(item / units), rows, tiles, scan);
    if (w.t.n == 0 && w.t.head_rows + (s.T - w.t.tail_row) == 0) return w;  // no rows left to be zeroed
    w.unit = static_cast<int>(item % units);
    w.first = (w.t.tiles - 1 - w.t.tile) * rows;
    return w;
}

__global__ void __launch_bounds__(kFwdThreads, 1)
    tc_forward_kernel(const __grid_constant__ CUtensorMap map, const Shape s, const __nv_bfloat16 *QKV, bool by_heads,
                      int tiles, int debug_withhold, __nv_bfloat16 *O, float *lse) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    FwdSmem &m = *reinterpret_cast<FwdSmem *>(smem_raw);
    volatile int *abort_flag = &m.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = by_heads ? s.n_q / 2 : s.n_q;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kFwdStages; ++i) {
            ptx::mbar_init(&m.full[i], 1);
            ptx::mbar_init(&m.empty[i], 2);
        }
        ptx::mbar_init(&m.q_full, 1);
        ptx::mbar_init(&m.q_empty, 2);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&m.s_full[i], 1);
            ptx::mbar_init(&m.turn[i], 1);
            ptx::mbar_init(&m.p_full[i], 8);
            ptx::mbar_init(&m.o_full[i], 1);
            ptx::mbar_init(&m.o_empty[i], 8);
            ptx::mbar_init(&m.work_full[i], 1);
            ptx::mbar_init(&m.work_empty[i], kWorkReaders);
        }
        ptx::mbar_init(&m.drain, 2);
        ptx::mbar_init(&m.aux, 1);
        m.abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map);
    }
    if (threadIdx.x < 2 * kOddBits / 32) m.odd[threadIdx.x / (kOddBits / 32)][threadIdx.x % (kOddBits / 32)] = 0u;
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&m.tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    grid_begin();
    constexpr uint32_t tmem = 0;  // all columns there are: they begin at 0
    // the next work of the warp that calls it, read by all its lanes; false at the end, or where all(it is there) is
    int round = 0;
    auto next_work = [&](Work &w, auto all) {
        const int at = round & 1;
        const uint32_t parity = (round >> 1) & 1;
        ++round;
        if (!all(wait_all(&m.work_full[at], parity, abort_flag, s.err, 28))) return false;
        w = m.work[at];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&m.work_empty[at]);
        return w.unit >= 0;
    };
    const auto alone = [](bool ok) { return ok; };

    if (warp < kSoftWarps) {
        // ------------------------------------------------ softmax
        ptx::registers_up<104>();  // 4 x 104 + 64 = 5 x 96, the launch's
        const int i = warp >> 3, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + i * 128 + lanes, o_tmem = tmem + 256 + i * 128 + half * 64 + lanes;
        const float c = s.scale * kLog2e;
        // The two warps that share queries meet. Each waits for itself, and may be the only one whose wait runs out:
        // so neither leaves within a pair, where the other counts on it. They go through all of it with whatever is
        // there, and on to the next pair only if both have seen that it is there. (The two cases of attn_forward
        // that are bound by the tensor cores take 1% longer for it; asking at each meeting took 3%.)
        const int shared_by = 2 + i * 4 + (warp & 3);
        auto meet = [&] { asm volatile("bar.sync %0, 64;" ::"r"(shared_by) : "memory"); };
        auto both = [&](bool yes) {
            uint32_t all;
            __syncwarp();
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
                "bar.red.and.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(all)
                : "r"(shared_by), "r"(static_cast<uint32_t>(yes))
                : "memory");
            return all != 0;
        };
        uint32_t phase = 0, o_phase = 0;
        Work w;
        while (next_work(w, both)) {
            if (w.t.n == 0) {
                const int head0 = by_heads ? 2 * w.unit : w.unit;
                forward_rest(s, w.t, head0, O, lse);
                if (by_heads) forward_rest(s, w.t, head0 + 1, O, lse);
                continue;
            }
            const Pair pr(s, w, by_heads);
            if (!(i ? pr.there(1) : pr.there(0))) continue;
            const KeyTiles my = i ? pr.one[1] : pr.one[0];
            const int my_q0 = i ? pr.q0[1] : pr.q0[0], my_head = i ? pr.head[1] : pr.head[0];
            const int row = my_q0 + r;
            float top = -INFINITY, l = 0.0f;  // the maximum that P is relative to, times c; the sum of P
            const int count = my.count();
            for (int u = 0; u < count; ++u) {
                const int k0 = my.at(u) * kTile;
                wait_all(&m.s_full[i], phase, abort_flag, s.err, 24);
                phase ^= 1;
                ptx::tc_fence_after();
                float x[2][32];
                read_half(s_tmem + half * 64, x);
                if (!all_seen(s, my_q0, my_q0 + kTile, k0, k0 + kTile)) {
                    const int hi = row - k0 - half * 64, lo = s.window ? hi - s.window + 1 : -kTile,
                              sink = s.sinks - k0 - half * 64;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        keep(x[b], visible(hi - b * 32, lo - b * 32, sink - b * 32), -INFINITY);
                }
                float high[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float(&y)[32] = x[b >> 1];
                    high[b] = fmaxf(y[(b & 1) * 16], y[(b & 1) * 16 + 1]);
#pragma unroll
                    for (int e = 2; e < 16; e += 2)
                        high[b] = max3(high[b], y[(b & 1) * 16 + e], y[(b & 1) * 16 + e + 1]);
                }
                float most = fmaxf(max3(high[0], high[1], high[2]), high[3]);
                reinterpret_cast<float *>(m.out[warp])[lane] = most;
                meet();  // and both have read S: P may overwrite it
                most = fmaxf(most, reinterpret_cast<const float *>(m.out[warp ^ 4])[lane]) * c;
                if (__any_sync(0xffffffffu, most > top + kRaise)) {  // the first one, too: top is -inf
                    const float to = fmaxf(top, most);
                    const float shrink = top == -INFINITY ? 0.0f : exp2_fast(top - to);
                    if (u > 0) {
                        for (int b = half * 64; b < min(width16(s.d), half * 64 + 64); b += 16)
                            ptx::tmem_scale16(o_tmem + b - half * 64, shrink);
                    }
                    l *= shrink;
                    top = to;
                }
                const float at = top == -INFINITY ? 0.0f : top;  // no key seen yet: 2^-inf
                float sum[4] = {};
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float v = x[b][2 * e], y = x[b][2 * e + 1];
                        scale2(v, y, c, -at, -at);
                        v = exp2_fast(v);
                        y = exp2_fast(y);
                        add2(sum[(e & 1) * 2], sum[(e & 1) * 2 + 1], v, y);
                        p[e] = pack2(v, y);
                    }
                    ptx::tmem_st16_async(s_tmem + half * 32 + b * 16, p);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&m.p_full[i]);
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            // of both halves (the next pair's sums come after its maxima, when these have been read)
            m.row_sum[warp][lane] = l;
            meet();
            l = m.row_sum[warp & ~4][lane] + m.row_sum[warp | 4][lane];
            const bool there = wait_all(&m.o_full[i], o_phase, abort_flag, s.err, 25);
            o_phase ^= 1;
            if (!there) continue;
            ptx::tc_fence_after();
            const float inv = 1.0f / l;
            const bool mine = row < w.t.n;
            float check = l * 0.0f;  // stays 0 while everything is finite
            // through shared memory, so that four lanes write 64 adjacent bytes of a row (with exchanges between
            // lanes, as the backward has it, and a fifth place in the ring instead: 1.5% slower)
            uint8_t *out = m.out[warp];
            const int rows = min(32, w.t.n - (row - lane));
            __nv_bfloat16 *to = O + (w.t.row0 + row - lane) * s.n_q * s.d + static_cast<int64_t>(my_head) * s.d;
            float o[2][32];
            read_half(o_tmem, o);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&m.o_empty[i]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int c0 = half * 64 + b * 32;
                if (c0 >= s.d) break;
                __syncwarp();  // the columns before have been read
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = o[b][v * 8 + e] * inv;
                    if (c0 + v * 8 < s.d) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) check = fmaf(y[e], 0.0f, check);
                    }
                    Raw8<__nv_bfloat16> p;
                    pack8(y, p);
                    *reinterpret_cast<uint4 *>(out + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) = p.a;
                }
                __syncwarp();
                const int v = lane & 3, col = c0 + v * 8;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = 8 * k + (lane >> 2);
                    const uint4 y = *reinterpret_cast<const uint4 *>(out + at * 64 + ((v ^ ((at >> 1) & 3)) << 4));
                    if (at < rows && col < s.d)
                        *reinterpret_cast<uint4 *>(to + static_cast<int64_t>(at) * s.n_q * s.d + col) = y;
                }
            }
            if (mine && !half) lse[my_head * s.T + w.t.row0 + row] = (top + log2f(l)) * kLn2;
            if (mine && check != 0.0f)  // NaN is not 0
                atomicOr(&m.odd[i][(round - 1) % kOddBits / 32], 1u << ((round - 1) & 31));
        }
    } else {
        ptx::registers_down<64>();
        if (warp == kLoadWarp) {
            // ------------------------------------------------ loads
            const int blocks = s.d > 64 ? 2 : 1;
            const uint32_t bytes = blocks * kBlockBytes;
            int stage = 0;
            uint32_t phase = 0, issued = 0, parity = 0, q_phase = 0;
            const bool leader = ptx::elect_one();
            bool ok = true, any = false;
            uint32_t aux_phase = 0;
            auto load = [&](int at_head, int64_t row, int rows) {
                ok = ok && wait_all(&m.empty[stage], phase ^ 1, abort_flag, s.err, 20);
                if (!ok) return;
                ok = load_rows(leader, m.ring[stage], &map, &m.full[stage], &m.aux, aux_phase, at_head, row, blocks,
                               rows, abort_flag, s.err, debug_withhold == 1 && blockIdx.x == 0 && issued == 0);
                issued |= 1u << stage;
                parity = (parity & ~(1u << stage)) | (phase << stage);
                if (++stage == kFwdStages) {
                    stage = 0;
                    phase ^= 1;
                }
            };
            Work w;
            while (ok && next_work(w, alone)) {
                if (w.t.n == 0) continue;
                const Pair pr(s, w, by_heads);
                const int kv = pr.head[0] / s.group;
                ok = wait_all(&m.q_empty, q_phase ^ 1, abort_flag, s.err, 27);
                if (!ok) break;
                q_phase ^= 1;
                any = true;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(&m.q_full, (pr.there(1) ? 2 : 1) * bytes);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (pr.there(i))
                            load_tile(m.q[i], &map, &m.q_full, s.q_head(pr.head[i]), w.t.row0 + pr.q0[i], blocks);
                }
                __syncwarp();
                // in the order of their use: K of a tile after V of the one before
                for (int u = 0; u <= pr.count && ok; ++u) {
                    const int v0 = u > 0 ? pr.both.at(u - 1) * kTile : 0;
                    if (u > 0) load(s.v_head(kv), w.t.row0 + v0, v0 + kTile > w.t.n ? w.t.n - v0 : 0);
                    if (u < pr.count) load(s.k_head(kv), w.t.row0 + static_cast<int64_t>(pr.both.at(u)) * kTile, 0);
                }
            }
            // copies land before the block ends, also where others give up only after this warp is done
            if (lane == 0) {
                if (any) ptx::mbar_wait_drain(&m.q_full, q_phase ^ 1);
                for (int i = 0; i < kFwdStages; ++i)
                    if (issued & (1u << i)) ptx::mbar_wait_drain(&m.full[i], (parity >> i) & 1u);
            }
        } else if (warp < kWorkWarp) {
            // ------------------------------------------------ products
            const int i = warp - kMmaWarp;
            const bool leader = ptx::elect_one();
            const uint32_t idesc = idesc_weighted(s.d);
            const uint32_t q_tile = ptx::smem_u32(m.q[0]) + i * kTileBytes, base = ptx::smem_u32(m.ring[0]);
            const uint32_t t_s = tmem + i * 128, t_o = tmem + 256 + i * 128;
            int pos = 0;  // tiles of the ring used so far
            int turns = 0;
            uint32_t p_phase = 0, o_phase = 0, q_phase = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t where) {
                ok = ok && wait_all<true>(bar, parity, abort_flag, s.err, where);
            };
            auto arrived = [&](bool needed, int at) {
                return Phase{needed ? &m.full[at % kFwdStages] : nullptr, (at / kFwdStages) & 1u};
            };
            auto tile = [&](int at) { return base + (at % kFwdStages) * kTileBytes; };
            // each turn of tile 0 is followed by one of tile 1, with something to issue or without
            auto my_turn = [&] {
                const int before = i == 1 ? turns : turns - 1;
                ++turns;
                return Phase{before >= 0 ? &m.turn[i] : nullptr, before & 1u};
            };
            Work w;
            while (ok && next_work(w, alone)) {
                if (w.t.n == 0) continue;
                const Pair pr(s, w, by_heads);
                const KeyTiles my = i ? pr.one[1] : pr.one[0];
                wait(&m.q_full, q_phase, 21);
                q_phase ^= 1;
                bool begun = false;
                for (int u = 0; u <= pr.count && ok; ++u) {
                    // V of the tile before at pos, then K of this one
                    const int v_at = pos, k_at = u > 0 ? pos + 1 : pos;
                    const int k_now = u < pr.count ? pr.both.at(u) : -1, k_before = u > 0 ? pr.both.at(u - 1) : -1;
                    const bool sums = u > 0 && pr.needs(i, k_before), scores = u < pr.count && pr.needs(i, k_now);
                    const Phase phases[5] = {arrived(u < pr.count, k_at), arrived(u > 0, v_at), my_turn(),
                                             {sums && !begun ? &m.o_empty[i] : nullptr, o_phase ^ 1},
                                             {sums ? &m.p_full[i] : nullptr, p_phase}};
                    if (sums && !begun) o_phase ^= 1;
                    if (sums) p_phase ^= 1;
                    ok = ok && wait_each(phases, abort_flag, s.err, 23);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (sums) {
                        mma_weighted(leader, t_o, t_s, 32, tile(v_at), idesc, begun);
                        begun = true;
                    }
                    if (scores)
                        mma_scores(leader, t_s, q_tile, tile(k_at), s.d, &m.s_full[i], &m.turn[i ^ 1]);
                    else if (leader)
                        ptx::mbar_arrive(&m.turn[i ^ 1]);
                    if (u > 0 && k_before == my.last) commit(leader, &m.o_full[i]);
                    if (u > 0) commit(leader, &m.empty[v_at % kFwdStages]);
                    if (u < pr.count) commit(leader, &m.empty[k_at % kFwdStages]);
                    if (u == pr.count - 1) commit(leader, &m.q_empty);
                    pos = u < pr.count ? k_at + 1 : v_at + 1;
                }
            }
            commit(leader, &m.drain);
            if (lane == 0) ptx::mbar_wait_drain(&m.drain, 0);
            __syncwarp();
        } else {
            // ------------------------------------------------ what comes next
            Scan scan;
            for (int r = 0;; ++r) {
                if (r == 1 && debug_withhold > 1) {  // gives up after so many ns
                    const uint64_t from = ptx::globaltimer(), ns = min(debug_withhold, 1 << 20);
                    while (ptx::globaltimer() - from < ns) {}
                    ptx::record_error(s.err, kErrTimeout | (29u << 8));
                    *abort_flag = 1;
                }
                const Work w = find_work(s, r, units, tiles, by_heads, scan);
                if (!wait_all(&m.work_empty[r & 1], ((r >> 1) & 1) ^ 1, abort_flag, s.err, 29)) break;
                if (lane == 0) {
                    m.work[r & 1] = w;
                    ptx::mbar_arrive(&m.work_full[r & 1]);
                }
                __syncwarp();
                if (w.unit < 0) break;
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    // What is masked within a sequence has met 0 times its value: a tile with results that
    // are not finite is computed again where masked values are passed over.
    uint32_t any = 0;
    for (int i = 0; i < 2 * kOddBits / 32; ++i) any |= m.odd[i / (kOddBits / 32)][i % (kOddBits / 32)];
    if (any == 0 || *abort_flag || threadIdx.x >= kPlainThreads) return;
    // the bits lie where the tiles below do not reach
    static_assert(offsetof(FwdSmem, odd) >= 4 * (3 * kRows * (kMaxDim + 4) + kRows * kPitchP), "room for plain tiles");
    Scan scan;
#pragma unroll 1
    for (int r = 0;; ++r) {
        const Work w = find_work(s, r, units, tiles, by_heads, scan);
        if (w.unit < 0 || w.t.n == 0) break;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (!(m.odd[i][r % kOddBits / 32] & (1u << (r & 31)))) continue;
            const Pair pr(s, w, by_heads);
            if (!(i ? pr.there(1) : pr.there(0))) continue;
            const int begin = i ? pr.q0[1] : pr.q0[0];
#pragma unroll 1
            for (int q = begin; q < min(w.t.n, begin + kTile); q += kRows) {
                plain_sync();
                plain_forward_tile(s, QKV, w.t.row0, w.t.n, q, i ? pr.head[1] : pr.head[0], O, lse,
                                   reinterpret_cast<float *>(smem_raw), Share{0, 1});
            }
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
    const int64_t pairs = static_cast<int64_t>(tiles) * (by_heads ? s.n_q / 2 : s.n_q);
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(pairs, num_sms()));
    cudaError_t e = allow_smem<tc_forward_kernel>();
    if (e != cudaSuccess) return fail_cuda(e, name);
    KernelTimer timer(name, stream);
    e = step::launch(tc_forward_kernel, blocks, kFwdThreads, sizeof(FwdSmem), stream, map, s,
                     static_cast<const __nv_bfloat16 *>(QKV), by_heads, tiles, take_debug_withhold(),
                     static_cast<__nv_bfloat16 *>(O), lse);
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
