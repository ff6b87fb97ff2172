// tc.cuh -- what the attention kernels on the tensor cores share: 128 x 128 tiles in
// shared memory as TMA leaves them, their descriptors, and the products.
//
// A tile of 128 rows of one head is one or two blocks of 64 columns, a block 128 rows
// of 128 bytes with the 128-byte swizzle. The same tile serves as an operand by rows
// (K-major: a sum over the head's d columns) and by columns (MN-major: a sum over the
// tile's rows). Columns past d are zeros.
#pragma once

#include "attn/attn.cuh"
#include "attn/host.cuh"

namespace tpce {
namespace attn {

constexpr int kTile = 128;
constexpr uint32_t kBlockBytes = kTile * 128, kTileBytes = 2 * kBlockBytes;
constexpr uint32_t kTmemCols = 512;

__device__ __forceinline__ uint64_t desc_rows(uint32_t tile) { return ptx::sdesc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t desc_cols(uint32_t tile) { return ptx::sdesc_sw128(tile, kBlockBytes, 1024); }
// sixteen of the summed index further
__device__ __forceinline__ uint64_t step_rows(uint64_t desc, int k) {
    return desc + static_cast<uint32_t>(((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4);
}
__device__ __forceinline__ uint64_t step_cols(uint64_t desc, int k) {
    return desc + static_cast<uint32_t>((k * 16 * 128) >> 4);
}

// The columns of one row that are visible, as bits of 32 columns each: those up to hi,
// from lo on or below sink (all relative to the tile's first column).
__device__ __forceinline__ uint32_t below(int n) {  // bits 0 .. n - 1
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
__device__ __forceinline__ uint32_t visible(int hi, int lo, int sink) {
    return below(hi + 1) & (~below(lo) | below(sink));
}

// All lanes of the warp that issues products call these; `leader` is the one that does.
// D = A B^T over d: 128 x 128 scores of two tiles' rows, and the barrier that they arrive
// on; `turn` is told when most of them are issued.
__device__ __forceinline__ void mma_scores(bool leader, uint32_t d_tmem, uint32_t a_tile, uint32_t b_tile, int d,
                                           uint64_t *done, uint64_t *turn = nullptr) {
    constexpr uint32_t kIdesc = ptx::idesc_f32acc(kTile, kTile, 1, false, false);
    const uint64_t a = desc_rows(a_tile), b = desc_rows(b_tile);
    const int steps = (d + 15) / 16;
    if (leader) {
#pragma unroll
        for (int k = 0; k < kMaxDim / 16; ++k)
            if (k < steps) {
                if (turn && k == max(0, steps - 3)) ptx::mbar_arrive(turn);
                ptx::mma_bf16(d_tmem, step_rows(a, k), step_rows(b, k), kIdesc, k != 0);
            }
        ptx::mma_commit(done);
    }
}

// D (+)= A X: A (bf16 in tensor memory from a_tmem on, its second 64 columns second_half
// further) times a tile's 128 rows of d columns. (With fewer columns or rows where a tile
// has fewer keys that anything sees, the instructions that this takes in front of every
// product cost 3 to 4% of everything, and a window with four sinks gained nothing.)
__device__ __forceinline__ void mma_weighted(bool leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t second_half,
                                             uint32_t x_tile, uint32_t idesc, bool accumulate) {
    const uint64_t x = desc_cols(x_tile);
    if (leader) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
            ptx::mma_bf16_ts(d_tmem, a_tmem + (k & 3) * 8 + (k >> 2) * second_half, step_cols(x, k), idesc,
                             (accumulate || k > 0) ? 1u : 0u);
    }
}
// the width of such a product: d, rounded up to what the instruction takes
__host__ __device__ inline int width16(int d) { return (d + 15) / 16 * 16; }
__device__ __forceinline__ uint32_t idesc_weighted(int d) {
    return ptx::idesc_f32acc(kTile, 16, 1, false, true) +
           (static_cast<uint32_t>((width16(d) - 16) >> 3) << 17);
}

// (x, y) = (x, y) * f + (a, b); 2^x to 2 units in the last place, results below 2^-126 zero
__device__ __forceinline__ void scale2(float &x, float &y, float f, float a, float b) {
    asm("{\n\t.reg .b64 p, q, r;\n\t"
        "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %4};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(f), "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {
    asm("{\n\t.reg .b64 p, q;\n\t"
        "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 64 columns of this thread's row, waited for.
__device__ __forceinline__ void read_half(uint32_t taddr, float (&x)[2][32]) {
    ptx::tmem_ld32_async(taddr, x[0]);
    ptx::tmem_ld32_async(taddr + 32, x[1]);
    ptx::tmem_wait_ld();
    ptx::tmem_ready(x[0]);
    ptx::tmem_ready(x[1]);
}

// The columns of 32 that are not in `seen` become `other`. One branch around all of it
// where a tile may be visible as a whole: one a value makes a phase three times as long.
__device__ __forceinline__ void keep(float (&x)[32], uint32_t seen, float other) {
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = seen & (1u << e) ? x[e] : other;
}
__device__ __forceinline__ void pack32(const float (&x)[32], uint32_t *p) {
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] = pack2(x[2 * e], x[2 * e + 1]);
}

// Columns c0 .. c0 + 63 (below d) of a warp's 32 rows, a row a lane, times each lane's f,
// as bf16 to the first `rows` rows from `to` on. Eight lanes exchange their rows' pieces of
// eight columns, so that they write 128 adjacent bytes of one row after the other: with
// each lane writing its own row the stores of a tile took 4000 cycles. Returns whether
// everything of this lane's row is finite.
__device__ __forceinline__ bool write_rows(const float (&o)[2][32], float f, int c0, int d, __nv_bfloat16 *to,
                                           int64_t ld, int rows) {
    const int lane = threadIdx.x & 31, j = lane & 7;
    uint4 v[8];
    float check = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = o[i >> 2][(i & 3) * 8 + e] * f;
        if (c0 + i * 8 < d) {
#pragma unroll
            for (int e = 0; e < 8; ++e) check = fmaf(y[e], 0.0f, check);
        }
        Raw8<__nv_bfloat16> p;
        pack8(y, p);
        v[i] = p.a;
    }
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) {
        const bool high = (j & s) != 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i & s) continue;
            uint4 &a = v[i], &b = v[i | s];
            uint4 x = high ? a : b;
            x.x = __shfl_xor_sync(0xffffffffu, x.x, s);
            x.y = __shfl_xor_sync(0xffffffffu, x.y, s);
            x.z = __shfl_xor_sync(0xffffffffu, x.z, s);
            x.w = __shfl_xor_sync(0xffffffffu, x.w, s);
            if (high)
                a = x;
            else
                b = x;
        }
    }
    const int col = c0 + j * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = (lane & ~7) + i;
        if (row < rows && col < d) *reinterpret_cast<uint4 *>(to + row * ld + col) = v[i];
    }
    return lane >= rows || check == 0.0f;  // NaN is not 0
}

// A wait of all lanes, which all get the same answer; bounded as mbar_wait() is. Reading
// the timer takes a while: with it in each round the many warps that wait do not crowd
// out those that work, and the few that issue products look at it now and then only
// (EAGER). (Sleeping in the try, trying from one lane, or trying without a pause cost the
// forward 7, 20 and 13%.)
template <bool EAGER = false>
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint32_t *err,
                                         uint32_t where) {
    const uint32_t a = ptx::smem_u32(bar);
    uint64_t since = 0;
#pragma unroll 1
    for (uint32_t i = 1; !__all_sync(0xffffffffu, ptx::mbar_try_wait(a, parity)); ++i) {
        if (EAGER && i % 64 != 0) continue;
        const uint64_t now = ptx::globaltimer();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
        if (__any_sync(0xffffffffu, now - since > kWaitLimitNs)) {
            ptx::record_error(err, kErrTimeout | (where << 8));
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// The same for several barriers at once, eagerly: the tries of all are under way together
// (one after the other each took 200 cycles, even where nothing had to be waited for).
// A null one is passed over.
struct Phase {
    uint64_t *bar;
    uint32_t parity;
};
template <int N>
__device__ __forceinline__ bool wait_each(const Phase (&phases)[N], volatile int *abort_flag, uint32_t *err,
                                          uint32_t where) {
    uint64_t since = 0;
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        bool done = true;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (phases[k].bar) done &= ptx::mbar_try_wait(ptx::smem_u32(phases[k].bar), phases[k].parity);
        if (__all_sync(0xffffffffu, done)) return true;
        if (i % 64 != 0) continue;
        const uint64_t now = ptx::globaltimer();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
        if (__any_sync(0xffffffffu, now - since > kWaitLimitNs)) {
            ptx::record_error(err, kErrTimeout | (where << 8));
            *abort_flag = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void commit(bool leader, uint64_t *bar) {
    if (leader) ptx::mma_commit(bar);
}

// Rows `from` .. 127 of a tile in shared memory become zeros, by a warp.
__device__ __forceinline__ void zero_tail(uint8_t *tile, int from, int blocks) {
    const int lane = threadIdx.x & 31;
    for (int b = 0; b < blocks; ++b)
        for (int i = from * 8 + lane; i < kTile * 8; i += 32)
            *reinterpret_cast<uint4 *>(tile + b * kBlockBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
    __syncwarp();
}

// The blocks of one head's tile of rows, into one stage.
__device__ __forceinline__ void load_tile(uint8_t *to, const CUtensorMap *m, uint64_t *bar, int head, int64_t row,
                                          int blocks) {
    for (int b = 0; b < blocks; ++b)
        ptx::tma_load_3d(to + b * kBlockBytes, m, bar, b * 64, head, static_cast<int>(row));
}

// The same by the warp that loads, counted on `full`; of a tile that a sequence ends in,
// `rows` of it (0: all 128), the others are zeros: what is there belongs to the next
// sequence or to none, its factors in a sum over rows are zeros, and it may be infinite or
// NaN. Such a tile lands on `aux` first. (Zeroed by the warps that issue products it cost
// the forward 4 to 7%, for the instructions between a wait and its products.) withhold:
// nothing is loaded, for the test of the waits' ends.
__device__ __forceinline__ bool load_rows(bool leader, uint8_t *to, const CUtensorMap *m, uint64_t *full, uint64_t *aux,
                                          uint32_t &aux_phase, int head, int64_t row, int blocks, int rows,
                                          volatile int *abort_flag, uint32_t *err, bool withhold = false) {
    uint64_t *const bar = rows ? aux : full;
    if (leader) {
        ptx::mbar_arrive_expect_tx(bar, blocks * kBlockBytes);
        if (!withhold) load_tile(to, m, bar, head, row, blocks);
    }
    __syncwarp();
    if (!rows) return true;
    const bool ok = wait_all<true>(aux, aux_phase, abort_flag, err, 49);
    if (ok)
        zero_tail(to, rows, blocks);
    else if (leader)
        ptx::mbar_wait_drain(aux, aux_phase);  // the copy may still be under way
    aux_phase ^= 1;
    if (leader) ptx::mbar_arrive(full);
    return ok;
}

}  // namespace attn
}  // namespace tpce
