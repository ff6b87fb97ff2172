// host.cuh -- checks of the attention core's calls, and what their launches share.
#pragma once

#include <atomic>

#include "attn/attn.cuh"

namespace tpce {
namespace attn {

constexpr int64_t kMaxReach = int64_t{1} << 26;
constexpr int kMaxSequences = 1 << 26;

inline tpce_status make_shape(const char *name, const int32_t *offsets, int sequences, int64_t T, int64_t n_heads,
                              int64_t n_kv_heads, int64_t head_dim, int64_t window, int64_t sinks, float scale,
                              int dtype, Shape &s) {
    if (dtype != TPCE_BF16 && dtype != TPCE_F32) return fail(TPCE_ERR_INVALID, "%s: dtype %d", name, dtype);
    if (!std::isfinite(scale * kLog2e))
        return fail(TPCE_ERR_INVALID, "%s: scale is not finite, or not times log2(e)", name);
    if (n_kv_heads < 1 || n_heads < 1 || n_heads > 4096 || n_heads % n_kv_heads != 0)
        return fail(TPCE_ERR_SHAPE, "%s: %lld query heads (up to 4096) over %lld key/value heads", name,
                    static_cast<long long>(n_heads), static_cast<long long>(n_kv_heads));
    if (head_dim < 8 || head_dim % 8 != 0 || head_dim > kMaxDim)
        return fail(TPCE_ERR_SHAPE, "%s: head width %lld (a multiple of 8 up to %d)", name,
                    static_cast<long long>(head_dim), kMaxDim);
    if (window < 0 || sinks < 0) return fail(TPCE_ERR_SHAPE, "%s: a negative window or number of sinks", name);
    if (T < 0 || sequences < (offsets ? 1 : 0))
        return fail(TPCE_ERR_SHAPE, "%s: T = %lld, %d sequences", name, static_cast<long long>(T), sequences);
    // blocks of the largest grid, and rows as 32-bit numbers
    if (T > (int64_t{1} << 30) || T * n_heads > (int64_t{1} << 33) ||
        (T / 32 + 2 * int64_t{sequences} + 2) * n_heads > INT_MAX)
        return fail(TPCE_ERR_SHAPE, "%s: T = %lld, %lld heads, %d sequences: too many tiles", name,
                    static_cast<long long>(T), static_cast<long long>(n_heads), sequences);
    s.T = T;
    s.n_q = static_cast<int>(n_heads);
    s.n_kv = static_cast<int>(n_kv_heads);
    s.group = s.n_q / s.n_kv;
    s.d = static_cast<int>(head_dim);
    s.ld = (n_heads + 2 * n_kv_heads) * head_dim;
    s.offsets = offsets;
    s.sequences = sequences;
    // a window of T keys hides nothing, and then sinks show nothing more
    s.window = window >= T ? 0 : static_cast<int>(window);
    s.sinks = s.window ? static_cast<int>(std::min(sinks, T)) : 0;
    // a unit of work on the tensor cores, 1.3 us for each 128 queries of a head that see its keys, stays well below
    // the limit of the waits for it
    const int64_t reach = s.window && !s.sinks ? std::min(T, window + 256) : T;
    if (dtype == TPCE_BF16 && reach * s.group > kMaxReach)
        return fail(TPCE_ERR_SHAPE, "%s: %lld tokens that see a key, with %d query heads that share it: more than 2^26",
                    name, static_cast<long long>(reach), s.group);
    // and so does the search for one, which may pass all sequences (2^26 of them take 0.23 s, and are passed
    // twice before the backward's first unit)
    if (dtype == TPCE_BF16 && offsets && sequences > kMaxSequences)
        return fail(TPCE_ERR_SHAPE, "%s: %d sequences: more than 2^26", name, sequences);
    s.scale = scale;
    s.err = device_error_word();
    return TPCE_OK;
}

// A pointer of a call: its bytes (0: it may be NULL, and is not checked), whether it is written.
struct Arg {
    const void *p;
    size_t bytes;
    bool written;
};
template <size_t N>
tpce_status check_args(const char *name, const Arg (&args)[N]) {
    for (const Arg &a : args)
        if (a.bytes && !a.p) return fail(TPCE_ERR_INVALID, "%s: null pointer", name);
    for (const Arg &a : args)
        if (a.bytes && !aligned16(a.p)) return fail(TPCE_ERR_ALIGN, "%s: a pointer is not 16-byte aligned", name);
    for (const Arg &a : args)
        for (const Arg &b : args) {
            const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
            if (&a != &b && a.written && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes)
                return fail(TPCE_ERR_INVALID, "%s: what is written overlaps another argument", name);
        }
    return TPCE_OK;
}

// Kernel may take all of an SM's shared memory; set once a device.
constexpr int kMaxSmem = 227 * 1024;
template <auto Kernel>
cudaError_t allow_smem() {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    cudaError_t e = step::taken(cudaGetDevice(&dev));
    if (e != cudaSuccess) return e;
    if (dev < kDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = step::taken(cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem));
    if (e == cudaSuccess && dev < kDevices) done[dev].store(true, std::memory_order_release);
    return e;
}

}  // namespace attn
}  // namespace tpce
