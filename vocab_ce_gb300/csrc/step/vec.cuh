// vec.cuh -- what the row and element kernels of a training step share: eight
// values of a row in registers, the e4m3 codes with one scale per 128 values,
// and sums over a warp or a block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

namespace tpce {
namespace step {

// Eight adjacent values as they lie in memory: one 16-byte vector of bf16, two
// of fp32. Addresses are 16-byte aligned: row widths are multiples of 8.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Raw8<float> {
    float4 a, b;
};

__device__ __forceinline__ Raw8<__nv_bfloat16> load8(const __nv_bfloat16 *p) {
    return {*reinterpret_cast<const uint4 *>(p)};
}
__device__ __forceinline__ Raw8<float> load8(const float *p) {
    const float4 *q = reinterpret_cast<const float4 *>(p);
    return {q[0], q[1]};
}

__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16> &r) { r.a = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void zero8(Raw8<float> &r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }

__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a bf16 is the upper half of an fp32
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&v)[8]) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}

// the one rounding to the stored type (nearest even; none for fp32)
__device__ __forceinline__ void pack8(const float (&v)[8], Raw8<__nv_bfloat16> &r) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack8(const float (&v)[8], Raw8<float> &r) {
    r.a = make_float4(v[0], v[1], v[2], v[3]);
    r.b = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Raw8<__nv_bfloat16> &r) {
    *reinterpret_cast<uint4 *>(p) = r.a;
}
__device__ __forceinline__ void store8(float *p, const Raw8<float> &r) {
    float4 *q = reinterpret_cast<float4 *>(p);
    q[0] = r.a;
    q[1] = r.b;
}

// The same for values that nothing reads again soon: first to leave L2.
__device__ __forceinline__ void stream8(__nv_bfloat16 *p, const Raw8<__nv_bfloat16> &r) {
    __stcs(reinterpret_cast<uint4 *>(p), r.a);
}
__device__ __forceinline__ void stream8(float *p, const Raw8<float> &r) {
    float4 *q = reinterpret_cast<float4 *>(p);
    __stcs(q, r.a);
    __stcs(q + 1, r.b);
}

// (x, y) *= (a, b) and (x, y) += (a, b) * (c, d), two values an instruction; each
// is rounded as by the single form. (A paired product and a paired sum after it
// were fused to one rounding, whatever their rounding modes say: where both
// roundings count, the sum is a single one.)
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b) {
    asm("{\n\t.reg .b64 p, q;\n\t"
        "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float c, float d) {
    asm("{\n\t.reg .b64 p, q, r;\n\t"
        "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\t"
        "fma.rn.f32x2 p, q, r, p;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b), "f"(c), "f"(d));
}

// a + b, rounded once to the stored type. A bf16 sum rounded from fp32 would be
// the same: 24 bits are more than twice 8 and two, so rounding twice never differs.
__device__ __forceinline__ void add8(const Raw8<__nv_bfloat16> &a, const Raw8<__nv_bfloat16> &b,
                                     Raw8<__nv_bfloat16> &r) {
    const uint32_t x[4] = {a.a.x, a.a.y, a.a.z, a.a.w}, y[4] = {b.a.x, b.a.y, b.a.z, b.a.w};
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&x[i]),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&y[i]));
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void add8(const Raw8<float> &a, const Raw8<float> &b, Raw8<float> &r) {
    r.a = make_float4(a.a.x + b.a.x, a.a.y + b.a.y, a.a.z + b.a.z, a.a.w + b.a.w);
    r.b = make_float4(a.b.x + b.b.x, a.b.y + b.b.y, a.b.z + b.b.z, a.b.w + b.b.w);
}

__device__ __forceinline__ void load8f(const float *p, float (&v)[8]) {
    const float4 a = *(reinterpret_cast<const float4 *>(p)), b = *(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// ------------------------------------------------------------------ e4m3 with scales
// A group of 128 values shares scale = max(amax / 448, 2^-126), amax over its
// finite values, and holds code = e4m3(x / scale), rounded to nearest even. The
// lower bound keeps 1 / scale finite (a group of zeros needs no special case).
// NaN and infinity become the NaN code: a saturated code would hide them.
constexpr int kGroup = 128;
constexpr float kE4m3Max = 448.0f, kE4m3Least = 1.0f / 512.0f;

__device__ __forceinline__ float group_scale(float amax) { return fmaxf(__fmul_rn(amax, 1.0f / kE4m3Max), FLT_MIN); }

// 20 bits that depend on all bits of a value and of its place: products and shifted
// exclusive ors, twice. The multipliers are 2^32 times the golden ratio's fraction and
// that of the root of 3, odd. The same value in the same place and step always gives
// the same bits.
__device__ __forceinline__ uint32_t noise20(uint32_t value, uint32_t place) {
    uint32_t x = value ^ (place * 0x9E3779B9u);
    x = (x ^ (x >> 16)) * 0xBB67AE85u;
    x = (x ^ (x >> 15)) * 0x9E3779B9u;
    return x >> 12;
}

// x (0 .. 448) to one of the two e4m3 values around it, the upper one where the 20 bits
// of x that e4m3 does not hold and `noise` carry: with the probability of x's place
// between them. Below 2^-6 the codes are 2^-9 apart, as fp32's are after 2^-6 is added
// and 20 bits are cleared. Other values (NaN) stay.
__device__ __forceinline__ float round_randomly(float x, uint32_t noise) {
    const float below = x < 0.015625f ? 0.015625f : 0.0f;
    const float r = __uint_as_float((__float_as_uint(x + below) + noise) & 0xfff00000u) - below;
    return x <= 512.0f ? r : x;
}

// Codes and scale of a group whose 128 values lie in 16 adjacent lanes, eight
// each (LANES: in fewer, the rest being another group's); every lane of the warp
// calls it (values past an end: zeros). fmaxf
// passes over NaN, whose product and code are NaN by themselves; infinities,
// which would spoil the scale and saturate, are looked for only in a warp
// whose maximum shows one. DIVISOR: none of the values is negative, and one that is
// not zero gets no code below the smallest, 2^-9: what divides by it stays bounded.
// RANDOM: a value between two codes becomes either, the nearer one more often, so that
// its expectation is the value; `seed` differs by 8 from eight values to the next.
template <int LANES = 16, bool DIVISOR = false, bool RANDOM = false>
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float &scale, uint32_t seed = 0u) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    const bool infinite = __any_sync(0xffffffffu, a > FLT_MAX);
    if (infinite) {
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]) <= FLT_MAX ? fabsf(v[i]) : 0.0f);
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    }
    scale = group_scale(a);
    const float inv = __frcp_rn(scale);
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) mul2(t[2 * i], t[2 * i + 1], inv, inv);
    if (RANDOM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = round_randomly(fabsf(t[i]), noise20(__float_as_uint(v[i]), seed + i));
            t[i] = DIVISOR ? r : copysignf(r, t[i]);
        }
    }
    if (infinite) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(fabsf(v[i]) <= FLT_MAX)) t[i] = __int_as_float(0x7fffffff);
    }
    if (DIVISOR) {
        float least = t[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) least = fminf(least, t[i]);
        if (least < kE4m3Least) {  // few threads: a value below 4e-6 of the group's largest, or none
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (v[i] > 0.0f && t[i] < kE4m3Least) t[i] = kE4m3Least;
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(t[2 * i], t[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ void decode8(uint2 q, float scale, float (&v)[8]) {
    const uint32_t w[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i]), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
        mul2(v[2 * i], v[2 * i + 1], scale, scale);
    }
}

// ------------------------------------------------------------------ sums
// over groups of LANES adjacent lanes
template <int LANES = 32>
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Sum over the block's warps with one barrier: `buf` is one of two alternating
// buffers of 32 floats, so that a buffer is written again only after the
// barrier of the sum between, which every reader of it has passed. The warps'
// sums are added in the same order in every thread.
__device__ __forceinline__ float block_sum(float x, float *buf) {
    x = warp_sum(x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) buf[warp] = x;
    __syncthreads();
    return warp_sum(lane < warps ? buf[lane] : 0.0f);
}

}  // namespace step
}  // namespace tpce
