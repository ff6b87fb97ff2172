// attn.cuh -- what the attention core's kernels share: the call's shape, which
// sequence and tile a block has, which keys a query sees, and the tiles that are
// computed without tensor cores.
//
// Queries and keys of one sequence are numbered from 0. Query i sees key j when
//   j <= i  and  (window == 0  or  i - j < window  or  j < sinks).
// With S = scale Q K^T over the visible keys, P = softmax(S), O = P V and
// lse = log sum exp S (natural logarithm). Backward, from dO:
//   delta_i = sum_c dO_ic O_ic,  dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
// the last two summed over the query heads that share the key/value head.
// P is formed as 2^(S log2(e) - m), one product and one exponential of base two.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "host.h"
#include "ptx.cuh"
#include "step/launch.cuh"
#include "step/vec.cuh"

namespace tpce {
namespace attn {

using step::grid_begin;
using step::load8;
using step::pack8;
using step::Raw8;
using step::store8;
using step::unpack8;
using step::zero8;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxDim = 128;

// The fused rows: for each key/value head its group's query heads, then K, then V.
struct Shape {
    int64_t T;
    int n_q, n_kv, group, d;
    int64_t ld;              // (n_q + 2 n_kv) d
    const int32_t *offsets;  // [sequences + 1] or NULL: one sequence of T tokens
    int sequences;
    int window, sinks;
    float scale;
    uint32_t *err;

    __device__ __forceinline__ int q_head(int h) const { return h / group * (group + 2) + h % group; }
    __device__ __forceinline__ int k_head(int kv) const { return kv * (group + 2) + group; }
    __device__ __forceinline__ int v_head(int kv) const { return kv * (group + 2) + group + 1; }
};

__device__ __forceinline__ bool sees(const Shape &s, int i, int j) {
    return j <= i && (s.window == 0 || i - j < s.window || j < s.sinks);
}

// ------------------------------------------------------------------ which tile
// Of a sequence: its first row among the T, its length, the tile of it. n == 0: the
// block has no tile; it may zero the rows that belong to no sequence.
struct Tile {
    int64_t row0;
    int n, tile, tiles;
    int64_t head_rows, tail_row;  // rows before the first sequence, and the first one after the last
    int part, parts;              // of the blocks without a tile
};

// How far a search has come: sequences passed, their last row, their tiles. The next search
// goes on there if it looks for no earlier tile, so that a block which takes tiles in order
// reads the offsets once (4096 sequences of 16 tokens, 32 heads on 8 of 128: from the start
// for each tile 15.3 ms and backward 29; so 1.7 and 7.0).
struct Scan {
    int first = -1, passed, end, before;
};

// Eight sequences a lane from scan.passed on, their loads under way together; true: the tile
// is among them, else they are passed.
__device__ __forceinline__ bool scan_step(const Shape &s, int x, int shift, Scan &scan, Tile &t) {
    constexpr int K = 8;
    const int lane = threadIdx.x & 31, T = static_cast<int>(s.T), b0 = scan.passed + lane * K;
    int given[K], most = scan.end;
#pragma unroll
    for (int k = 0; k < K; ++k) given[k] = b0 + k < s.sequences ? s.offsets[b0 + k + 1] : INT_MIN;
#pragma unroll
    for (int k = 0; k < K; ++k) most = max(most, min(given[k], T));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, most, d);
        if (lane >= d) most = max(most, o);
    }
    const int up = __shfl_up_sync(0xffffffffu, most, 1), begin = lane == 0 ? scan.end : up;
    int sum = 0, e = begin;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int from = e;
        e = max(e, min(given[k], T));
        if (b0 + k < s.sequences && given[k] != e) ptx::record_error(s.err, kErrInvalid | (6u << 8));
        sum += (e - from + (1 << shift) - 1) >> shift;
    }
    int up_to = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, up_to, d);
        if (lane >= d) up_to += o;
    }
    int at = x - scan.before - (up_to - sum);
    const uint32_t found = __ballot_sync(0xffffffffu, at >= 0 && at < sum);
    if (!found) {
        scan.passed += 32 * K;
        scan.end = __shfl_sync(0xffffffffu, most, 31);
        scan.before += __shfl_sync(0xffffffffu, up_to, 31);
        return false;
    }
    // of the lane that has it
    int row0 = begin, n = 0, tiles = 0;
    e = begin;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int from = e;
        e = max(e, min(given[k], T));
        const int here = (e - from + (1 << shift) - 1) >> shift;
        if (tiles <= at) {  // not reached yet
            at -= tiles;
            row0 = from;
            n = e - from;
            tiles = here;
        }
    }
    const int who = __ffs(found) - 1;
    t.row0 = __shfl_sync(0xffffffffu, row0, who);
    t.n = __shfl_sync(0xffffffffu, n, who);
    t.tile = __shfl_sync(0xffffffffu, at, who);
    t.tiles = __shfl_sync(0xffffffffu, tiles, who);
    return true;
}

// Every lane of a warp calls it. `x` counts tiles of `rows` (a power of two) rows over all
// sequences; the grid has grid_tiles of them for each head, more than there are tiles.
// Offsets that fall, or lie outside, are read as the nearest that do not.
__device__ __forceinline__ Tile find_tile(const Shape &s, int x, int rows, int grid_tiles, Scan &scan) {
    Tile t{};
    if (!s.offsets) {
        const int tiles = static_cast<int>((s.T + rows - 1) / rows);
        if (x < tiles) {
            t.n = static_cast<int>(s.T);
            t.tile = x;
            t.tiles = tiles;
            return t;
        }
        t.tail_row = s.T;
        t.part = x - tiles;
        t.parts = grid_tiles - tiles;
        return t;
    }
    if (scan.first < 0 || x < scan.before) {
        const int T = static_cast<int>(s.T);
        int first = s.offsets[0];
        if (first < 0 || first > T) {
            if ((threadIdx.x & 31) == 0) ptx::record_error(s.err, kErrInvalid | (6u << 8));
            first = first < 0 ? 0 : T;
        }
        scan.first = scan.end = first;
        scan.passed = scan.before = 0;
    }
    const int shift = __ffs(rows) - 1;
    while (scan.passed < s.sequences)
        if (scan_step(s, x, shift, scan, t)) return t;
    t.head_rows = scan.first;
    t.tail_row = scan.end;
    t.part = x - scan.before;
    t.parts = grid_tiles - scan.before;
    return t;
}

// Tiles in a grid for each head: all sequences' tiles and one more at least.
inline int64_t grid_tiles(const Shape &s, int rows) { return s.T / rows + (s.offsets ? s.sequences : 1) + 1; }

// ------------------------------------------------------------------ key tiles of queries, query tiles of keys
// The tiles of `rows` keys that queries q0 .. q1 - 1 see: 0 .. first - 1 (sinks), then from .. last.
struct KeyTiles {
    int first, from, last;
    __device__ __forceinline__ int count() const { return first + last - from + 1; }
    __device__ __forceinline__ int at(int u) const { return u < first ? u : from + u - first; }
};
__device__ __forceinline__ KeyTiles key_tiles(const Shape &s, int q0, int q1, int rows) {
    KeyTiles k{};
    const int lo = s.window && q0 >= s.window ? q0 - s.window + 1 : 0;
    k.from = lo / rows;
    k.last = (q1 - 1) / rows;
    k.first = min((min(s.sinks, lo) + rows - 1) / rows, k.from);
    return k;
}

// The end (one past the last) of the queries that see any of the keys k0 .. k1 - 1 of n.
__device__ __forceinline__ int query_end(const Shape &s, int k0, int k1, int n) {
    if (s.window == 0 || k0 < s.sinks) return n;
    return static_cast<int>(min(static_cast<int64_t>(n), static_cast<int64_t>(k1) - 1 + s.window));
}

// Whether every query q0 .. q1 - 1 sees every key k0 .. k1 - 1.
__device__ __forceinline__ bool all_seen(const Shape &s, int q0, int q1, int k0, int k1) {
    return k1 - 1 <= q0 && (s.window == 0 || q1 - 1 - k0 < s.window || k1 <= s.sinks);
}

// ------------------------------------------------------------------ tiles without tensor cores
// 64 queries by 64 keys on 256 threads, all in fp32: the path of fp32 tensors, whose
// products would lose 13 bits as tf32, and of tiles in which something was infinite
// or NaN (a tensor core multiplies what is masked by zero, and 0 inf is NaN: here a
// masked factor is passed over). Thread (ty, tx) of 16 x 16 has the rows 4 ty .. and
// the columns tx + 16 j of a 64 x 64 product, and the columns 4 tx + 64 m of a row of d.
// A thread's four rows take three 16-byte reads of shared memory for eight paired products,
// and an SM has the registers for eight warps: reading keeps shared memory busy for 58 to
// 69% of the time and the multipliers are for 42 to 51% (4096 tokens, 8 heads of 64: 0.65 ms,
// 26 TFLOP/s, backward 1.86 ms; 2048 tokens, 8 heads on 4 of 128: 29 and 26 TFLOP/s).
constexpr int kRows = 64, kPlainThreads = 256;
constexpr int kPitchP = kRows + 4;

struct PlainSmem {
    int pitch;  // of a row of d values: 16-byte aligned, a row's start four banks after the one before
    __host__ __device__ explicit PlainSmem(int d) : pitch(d + 4 + (d % 32 == 0 ? 0 : (32 - d % 32) % 32)) {}
    __host__ __device__ size_t rows() const { return static_cast<size_t>(kRows) * pitch; }
    __host__ __device__ size_t forward() const { return 4 * (3 * rows() + kRows * kPitchP); }
    __host__ __device__ size_t backward() const { return 4 * (4 * rows() + 2 * kRows * kPitchP); }
};

// the threads that compute a tile, which may be some of a larger block's
__device__ __forceinline__ void plain_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The columns c0 .. c0 + d of the rows that belong to no sequence become zeros, by the
// block's first 256 threads.
template <typename T>
__device__ __forceinline__ void zero_rest(const Shape &s, const Tile &t, T *out, int64_t ld, int64_t c0) {
    if (threadIdx.x >= kPlainThreads) return;
    Raw8<T> zero;
    zero8(zero);
    const int vectors = s.d / 8;
    const int64_t rows = t.head_rows + (s.T - t.tail_row);
    for (int64_t i = static_cast<int64_t>(t.part) * kPlainThreads + threadIdx.x; i < rows * vectors;
         i += static_cast<int64_t>(t.parts) * kPlainThreads) {
        const int64_t r = i / vectors;
        store8(out + (r < t.head_rows ? r : t.tail_row + r - t.head_rows) * ld + c0 + (i - r * vectors) * 8, zero);
    }
}

// Rows r0 .. of a tile (zeros from row n on), fetched into registers, all loads of which
// are under way together and during whatever comes before put() writes them to shared
// memory. (With each load waited for a step of 64 x 64 took 12 us, mostly that.)
template <typename T>
struct PlainRows {
    static constexpr int kEach = kRows * kMaxDim / 8 / kPlainThreads;
    Raw8<T> v[kEach];
    __device__ __forceinline__ void fetch(const T *from, int64_t ld, int r0, int n, int d) {
        const int vectors = d / 8;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kPlainThreads, r = i / vectors, c = i - r * vectors;
            zero8(v[k]);
            if (r < kRows && r0 + r < n) v[k] = load8(from + (r0 + r) * ld + c * 8);
        }
    }
    __device__ __forceinline__ void put(float *to, int pitch, int d) const {
        const int vectors = d / 8;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kPlainThreads, r = i / vectors, c = i - r * vectors;
            if (r >= kRows) break;
            float x[8];
            unpack8(v[k], x);
            float4 *p = reinterpret_cast<float4 *>(to + r * pitch + c * 8);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
};

// s[i][j] = sum_c A[4 ty + i][c] B[tx + 16 j][c], even and odd c two sums of one instruction
__device__ __forceinline__ void plain_dots(const float *A, const float *B, int pitch, int d, float (&s)[4][4]) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    float odd[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = odd[i][j] = 0.0f;
#pragma unroll 2
    for (int c = 0; c < d; c += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * pitch + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * pitch + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                step::fma2(s[i][j], odd[i][j], a[i].x, a[i].y, b[j].x, b[j].y);
                step::fma2(s[i][j], odd[i][j], a[i].z, a[i].w, b[j].z, b[j].w);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] += odd[i][j];
}

// o[i][m] += sum_k P[4 ty + i][k] X[k][4 tx + 64 m ..]  (ROWS: P[k][4 ty + i]); a zero factor
// of a masked tile is passed over, whatever it would multiply.
template <bool MASKED, bool ROWS>
__device__ __forceinline__ void plain_add(const float *P, const float *X, int pitch, int d, float (&o)[4][2][4]) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 2
    for (int k = 0; k < kRows; k += 4) {
        float4 p[4];  // four rows (or columns) of P, four k each
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = *reinterpret_cast<const float4 *>(
                P + (ROWS ? (k + i) * kPitchP + 4 * ty : (4 * ty + i) * kPitchP + k));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int c = 4 * tx + 64 * m;
            if (c >= d) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 x = *reinterpret_cast<const float4 *>(X + (k + q) * pitch + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f4 = ROWS ? p[q] : p[i];
                    const int at = ROWS ? i : q;
                    const float f = at == 0 ? f4.x : at == 1 ? f4.y : at == 2 ? f4.z : f4.w;
                    if (MASKED && f == 0.0f) continue;
                    step::fma2(o[i][m][0], o[i][m][1], f, f, x.x, x.y);
                    step::fma2(o[i][m][2], o[i][m][3], f, f, x.z, x.w);
                }
            }
        }
    }
}

// Four adjacent values in the tensors' type.
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Where there are fewer tiles than the SMs have room for, the blocks of a cluster share
// one: rank r of `ranks` takes its steps r, r + ranks, .., and the sums of all are added in
// the order of the ranks, by each rank those of 64 / ranks rows. (rank, ranks) = (0, 1): alone.
struct Share {
    int rank, ranks;
};
constexpr int kMaxRanks = 8;
__device__ __forceinline__ Share this_share(int ranks) {
    return Share{static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks)), ranks};
}
// One block (or cluster) for each tile, so that the SMs take them as they become free; of
// many sequences fewer blocks, which take several tiles each, in order (see Scan).
inline bool many_sequences(const Shape &s) { return s.offsets && s.sequences > 256; }
inline int64_t many_blocks(int64_t units) { return std::min<int64_t>(units, 8 * num_sms()); }
// For `units` tiles, `longest` of which have about `steps` steps each; an SM has the
// registers for one block. As long as all blocks run at once more ranks cost nothing (a
// sequence of 200 tokens, one head: forward 39 -> 14 us, backward 69 -> 24). Beyond that,
// where the last queries see many more keys than the first ones, up to four that keep
// `least` / 2 steps pay while the longest tiles hold up the rest (1024 tokens, 4 heads on 2,
// width 64: forward 92 -> 36 us, backward 312 -> 88; 2048 tokens, 8 heads on 4, width 128,
// backward 1018 -> 828). Eight did not (60 and 131 us in the first of these: a cluster waits
// for as many SMs of one group), nor do any where a window makes all tiles alike (window
// 128: 28 -> 44 and 92 -> 103 us).
inline int ranks_of(const Shape &s, int64_t units, int64_t longest, int64_t steps, int64_t least) {
    if (many_sequences(s)) return 1;
    const int64_t room = num_sms();
    const bool uneven = s.window == 0 || 2 * int64_t{s.window} >= s.T;
    int ranks = 1;
    while (ranks < kMaxRanks && ranks < steps) {
        const bool fits = 2 * ranks * units <= room;
        const bool pays = uneven && ranks < 4 && steps >= least * ranks && 2 * ranks * longest < 3 * room;
        if (!fits && !pays) break;
        ranks *= 2;
    }
    return ranks;
}
// About the most steps of 64 keys that a tile of queries has; the lengths of sequences are
// not known here, and taken as up to twice their mean.
inline int64_t steps_of(const Shape &s) {
    const int64_t n = std::min(s.T, s.offsets ? 2 * s.T / s.sequences + 1 : s.T);
    return (std::min<int64_t>(n, s.window ? int64_t{s.window} + s.sinks + 2 * kRows : n) + kRows - 1) / kRows;
}

// A thread's accumulator to rows of d in shared memory.
__device__ __forceinline__ void plain_put(const float (&o)[4][2][4], float *to, int pitch, int d) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int col = 4 * tx + 64 * a;
            if (col < d)
                *reinterpret_cast<float4 *>(to + (4 * ty + i) * pitch + col) =
                    make_float4(o[i][a][0], o[i][a][1], o[i][a][2], o[i][a][3]);
        }
}
// What each rank has at `p` in its shared memory.
__device__ __forceinline__ void of_ranks(const float *p, int ranks, float4 (&x)[kMaxRanks]) {
    const uint32_t at = ptx::smem_u32(p);
#pragma unroll
    for (int q = 0; q < kMaxRanks; ++q)
        x[q] = q < ranks ? ptx::ld_cluster4(ptx::mapa_shared(at, q)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

}  // namespace attn
}  // namespace tpce
