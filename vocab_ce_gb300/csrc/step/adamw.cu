// adamw.cu -- one AdamW step over many tensors in one launch.
//
// Per value, with g = grad * grad_scale and t the step's number (from 1):
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps).
// States in 32 bits hold m and v. States in 8 bits hold m and the root
// r = sqrt(v), each in e4m3 with one scale per 128 values of the flat tensor
// (vec.cuh). The root, not v: e4m3 spans a factor of 2^18 between a group's
// largest and smallest value, which in v would leave only 2^9 in the root that
// the update divides by. The update uses the new moments before they are rounded.
// A root that is not zero gets no code of zero: its m has a scale of its own and may
// survive, and the next step would divide it by that step's gradient alone, or by eps
// (gradients present one step in twenty, spread over three decades: steps of 2.1 lr in
// 32 bits, and of 8.5, 85 and 850 lr at gradients of 0.1, 1 and 10 without this).
//
// Codes are rounded to nearest, or at random where asked. To nearest, what a step
// moves by less than half a code stays, while its group's scale does:
// - a root does not grow with its gradients until they are
//   sqrt(((17/16)^2 - b2) / (1 - b2)) times it (11.4 at b2 = 0.999, 3.7 at 0.99, 1.9 at
//   0.95), and its updates are too large by up to that. (Gradients that grow by 5
//   beside a larger one, b2 = 0.999: 3000 steps later the roots are 0.38 of what they
//   should be, rounded at random 0.98.) It shrinks no sooner, which makes steps small.
// - a moment without gradients does not shrink below 1 / (2 - 2 b1) steps of its codes:
//   at b1 = 0.9 four of the smallest, which are nothing beside the others; from 15/16
//   on any, and its parameter goes on moving (b1 = 0.95 beside a steady moment: 74 lr in
//   1000 steps, 2.1 in 32 bits and at random).
// At random it is a hash of the value, its place and the step that decides, so a step
// repeats its bits. Two hashes a value, 34 instructions of 100, bind it to those: 134
// million with masters 427 us instead of 338, 42 million without 134 instead of 98.
//
// Every product and sum is rounded on its own (no contraction to a fused
// multiply-add), so that a step gives the same bits wherever a tensor lies in
// the list and however its tail is handled, and the same as elementary 32-bit
// operations in the order above: an 8-bit state rounds next to a border the
// same way everywhere.
//
// Bound by HBM: 134 million bf16 weights with fp32 masters and bf16 gradients
// take 538 us with 32-bit states (28 bytes a value, 7.0 TB/s, a little above the
// copy rate, as reads and writes meet the same lines) and 338 us with 8-bit ones
// (16.1 bytes, 6.4 TB/s, 94% of the copy rate). There the arithmetic, 66
// instructions a value, takes two thirds of the time that the bytes take, so it
// is done beside the next chunk's loads (448 us without) and products in pairs.
//
// A parameter is fp32, or bf16, or bf16 with an fp32 master copy (then the
// master is read and written, and the bf16 weight only written, rounded from
// it). The tensors' addresses travel in the kernel's parameters: no table is
// copied to the device, and a captured step keeps them.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <memory>

#include "host.h"
#include "step/launch.cuh"
#include "step/vec.cuh"

namespace tpce {
namespace {

using namespace step;

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;  // values that a block takes at a time: 16 groups

// Chunks of a tensor with 8-bit states that a block takes one after the other,
// and the list's number of chunks from which on it does (below it a chunk each
// keeps more SMs busy). A tensor with 32-bit states has a block for each chunk.
constexpr int kSpan = 4;
constexpr int64_t kSpanFrom = 152 * 32;

enum : uint32_t { kParamBf16 = 1u, kMaster = 2u, kGradBf16 = 4u, kState8 = 8u, kRandom = 16u };

struct Entry {
    void *p, *master;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    uint32_t block0;  // blocks of the tensors before it
    uint32_t kind;
    float decay;      // 1 - lr wd
    float wd;
    uint32_t span;    // chunks of a block
    uint32_t unused;
};
static_assert(sizeof(Entry) == 88, "the table's size is what a launch's parameters hold");

// Parameters of a launch: up to 4 KB for a short list, up to 32,764 bytes for a
// long one (more take more launches); what is not used is copied all the same.
constexpr int kShort = 44, kMiddle = 136, kLong = 368;
template <int N>
struct Table {
    Entry t[N];
    int count;
};

struct Scalars {
    float b1, one_b1, b2, one_b2, eps;
    float step_size;   // lr / (1 - b1^t)
    float root_scale;  // 1 / sqrt(1 - b2^t)
    float grad_scale;
    uint32_t step;        // of the seed of random rounding
    const float *device;  // {step_size, root_scale, lr, grad_scale} on the device, or NULL
};

struct Rates {
    float step_size, root_scale, grad_scale, decay;
    uint32_t seed;
};

// Two values' step; r becomes the root of the new v.
__device__ __forceinline__ void update2(const Scalars &k, const Rates &c, const float *grad, float *p, float *m,
                                        float *v, float *r) {
    float g0 = grad[0], g1 = grad[1];
    mul2(g0, g1, c.grad_scale, c.grad_scale);
    float s0 = g0, s1 = g1;
    mul2(m[0], m[1], k.b1, k.b1);
    mul2(s0, s1, k.one_b1, k.one_b1);
    m[0] = __fadd_rn(m[0], s0);
    m[1] = __fadd_rn(m[1], s1);
    mul2(g0, g1, g0, g1);
    mul2(v[0], v[1], k.b2, k.b2);
    mul2(g0, g1, k.one_b2, k.one_b2);
    v[0] = __fadd_rn(v[0], g0);
    v[1] = __fadd_rn(v[1], g1);
    r[0] = __fsqrt_rn(v[0]);
    r[1] = __fsqrt_rn(v[1]);
    float d0 = r[0], d1 = r[1];
    mul2(d0, d1, c.root_scale, c.root_scale);
    float u0 = __fdiv_rn(m[0], __fadd_rn(d0, k.eps)), u1 = __fdiv_rn(m[1], __fadd_rn(d1, k.eps));
    mul2(u0, u1, c.step_size, c.step_size);
    mul2(p[0], p[1], c.decay, c.decay);
    p[0] = __fsub_rn(p[0], u0);
    p[1] = __fsub_rn(p[1], u1);
}

// Eight values from i on as they lie in memory; those from n on are zeros, and
// are not stored.
template <typename T>
__device__ __forceinline__ Raw8<T> fetch(const void *base, int64_t i, int64_t n) {
    const T *p = static_cast<const T *>(base) + i;
    if (i + 8 <= n) return load8(p);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < n ? static_cast<float>(p[j]) : 0.0f;
    Raw8<T> r;
    pack8(v, r);  // exact: the values are T's
    return r;
}
template <typename T>
__device__ __forceinline__ void put(void *base, int64_t i, int64_t n, const float (&v)[8]) {
    T *p = static_cast<T *>(base) + i;
    if (i + 8 <= n) {
        Raw8<T> o;
        pack8(v, o);
        store8(p, o);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) p[j] = static_cast<T>(v[j]);
    }
}
__device__ __forceinline__ uint2 fetch_codes(const void *base, int64_t i, int64_t n) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + i;
    if (i + 8 <= n) return *reinterpret_cast<const uint2 *>(p);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (i + j < n) w[j / 4] |= static_cast<uint32_t>(p[j]) << (8 * (j % 4));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(void *base, int64_t i, int64_t n, uint2 q) {
    uint8_t *p = static_cast<uint8_t *>(base) + i;
    if (i + 8 <= n) {
        *reinterpret_cast<uint2 *>(p) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) p[j] = static_cast<uint8_t>((j < 4 ? q.x : q.y) >> (8 * (j % 4)));
    }
}

// What a thread reads for its eight values: P is the type that is updated (the
// master's, where there is one), G the gradient's.
template <typename P, typename G, bool S8>
struct Inputs;
template <typename P, typename G>
struct Inputs<P, G, false> {
    Raw8<P> p;
    Raw8<G> g;
    Raw8<float> m, v;
    __device__ __forceinline__ void load(const Entry &e, const void *base, int64_t i, int64_t n) {
        p = fetch<P>(base, i, n);
        g = fetch<G>(e.g, i, n);
        m = fetch<float>(e.m, i, n);
        v = fetch<float>(e.v, i, n);
    }
    __device__ __forceinline__ void moments(float (&mm)[8], float (&vv)[8]) const {
        unpack8(m, mm);
        unpack8(v, vv);
    }
};
template <typename P, typename G>
struct Inputs<P, G, true> {
    Raw8<P> p;
    Raw8<G> g;
    uint2 m, r;
    float ms, rs;
    __device__ __forceinline__ void load(const Entry &e, const void *base, int64_t i, int64_t n) {
        p = fetch<P>(base, i, n);
        g = fetch<G>(e.g, i, n);
        m = fetch_codes(e.m, i, n);
        r = fetch_codes(e.v, i, n);
        ms = rs = 0.0f;
        if (i < n) {
            ms = e.m_scale[i / kGroup];
            rs = e.v_scale[i / kGroup];
        }
    }
    __device__ __forceinline__ void moments(float (&mm)[8], float (&vv)[8]) const {
        decode8(m, ms, mm);
        decode8(r, rs, vv);
#pragma unroll
        for (int j = 0; j < 8; j += 2) mul2(vv[j], vv[j + 1], vv[j], vv[j + 1]);
    }
};

// The chunks from value i of this thread on, `left` of them. With 8-bit states
// the arithmetic takes about as long as the bytes, so the next chunk's values are
// on their way while one is computed.
template <typename P, typename G, bool S8, bool RANDOM>
__device__ __forceinline__ void run_state(const Scalars &k, const Rates &c, const Entry &e, int64_t i, int left) {
    const int64_t n = e.n;
    const bool master = e.kind & kMaster;
    void *base = master ? e.master : e.p;
    Inputs<P, G, S8> next;
    next.load(e, base, i, n);
    for (; left > 0; --left, i += kChunk) {
        const Inputs<P, G, S8> in = next;
        if (left > 1) next.load(e, base, i + kChunk, n);
        float p[8], g[8], m[8], v[8], r[8];
        unpack8(in.p, p);
        unpack8(in.g, g);
        in.moments(m, v);
#pragma unroll
        for (int j = 0; j < 8; j += 2) update2(k, c, g + j, p + j, m + j, v + j, r + j);
        if (S8) {
            // values past the end have no gradient and no moments: they stay zero and leave the scale alone
            float ms, rs;
            const uint32_t place = c.seed + static_cast<uint32_t>(i);
            const uint2 mq = quantize8<16, false, RANDOM>(m, ms, place + 0x40000000u),
                        rq = quantize8<16, true, RANDOM>(r, rs, place);
            if (i < n) {
                put_codes(e.m, i, n, mq);
                put_codes(e.v, i, n, rq);
                if ((threadIdx.x & 15) == 0) {
                    e.m_scale[i / kGroup] = ms;
                    e.v_scale[i / kGroup] = rs;
                }
            }
        } else {
            put<float>(e.m, i, n, m);
            put<float>(e.v, i, n, v);
        }
        put<P>(base, i, n, p);
        if (master) put<__nv_bfloat16>(e.p, i, n, p);
    }
}

template <typename P, typename G, bool RANDOM>
__device__ __forceinline__ void run(const Scalars &k, const Rates &c, const Entry &e, int64_t i, int left) {
    if (RANDOM && (e.kind & kRandom))
        run_state<P, G, true, true>(k, c, e, i, left);
    else if (e.kind & kState8)
        run_state<P, G, true, false>(k, c, e, i, left);
    else
        run_state<P, G, false, false>(k, c, e, i, left);
}

// RANDOM: some tensor of the list rounds at random; a kernel of its own, so that the
// others' have no registers for it.
template <int N, bool RANDOM>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<N> table,
                                                         const __grid_constant__ Scalars k) {
    // this block's tensor: the last one that starts at or before it
    int lo = 0, hi = table.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (table.t[mid].block0 <= blockIdx.x)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Entry &e = table.t[lo];
    const int64_t first = static_cast<int64_t>(blockIdx.x - e.block0) * e.span * kChunk;
    const int64_t chunks = (e.n - first + kChunk - 1) / kChunk;
    const int left = chunks < e.span ? static_cast<int>(chunks) : static_cast<int>(e.span);
    const int64_t i = first + threadIdx.x * 8;
    grid_begin();
    Rates c{k.step_size, k.root_scale, k.grad_scale, e.decay, 0u};
    if (k.device) {
        c.step_size = k.device[0];
        c.root_scale = k.device[1];
        c.decay = __fsub_rn(1.0f, __fmul_rn(k.device[2], e.wd));
        c.grad_scale = k.device[3];
    }
    // a captured step repeats k.step; its rates differ from step to step
    if (RANDOM)
        c.seed = (k.step + __float_as_uint(c.step_size) * 3u + __float_as_uint(c.root_scale) * 5u) * 0xBB67AE85u;
    const bool narrow = (e.kind & kParamBf16) && !(e.kind & kMaster);
    if (e.kind & kGradBf16) {
        if (narrow)
            run<__nv_bfloat16, __nv_bfloat16, RANDOM>(k, c, e, i, left);
        else
            run<float, __nv_bfloat16, RANDOM>(k, c, e, i, left);
    } else {
        if (narrow)
            run<__nv_bfloat16, float, RANDOM>(k, c, e, i, left);
        else
            run<float, float, RANDOM>(k, c, e, i, left);
    }
}

template <int N>
tpce_status launch_table(const Entry *entries, int count, uint32_t blocks, bool random, const Scalars &k,
                         cudaStream_t s) {
    Table<N> table;
    std::copy(entries, entries + count, table.t);
    table.count = count;
    KernelTimer timer("adamw_step", s);
    const cudaError_t e =
        launch(random ? adamw_kernel<N, true> : adamw_kernel<N, false>, blocks, kThreads, 0, s, table, k);
    if (e != cudaSuccess) return fail_cuda(e, "adamw_step");
    return check_launch("adamw_step", s);
}

inline bool state8(const tpce_adamw_tensor &t) { return (t.state_bits & ~TPCE_ADAMW_RANDOM) == 8; }

// ------------------------------------------------------------------ overlaps
// Blocks of a launch run in any order, so nothing that a step writes may be written
// or read by another tensor's step too: a state or master given twice, a parameter
// inside another, a gradient in a moment's place. (Gradients are only read, and may
// be shared.)
struct Range {
    uintptr_t begin, end;  // a gradient's begin is odd; addresses are 16-byte aligned
};
constexpr int kParts = 7;
const char *const kPartNames[kParts] = {"p", "master", "m", "v", "m_scale", "v_scale", "g"};

// take(part, range) for each part of a tensor.
template <typename F>
inline void ranges_of(const tpce_adamw_tensor &t, F take) {
    const uint64_t n = static_cast<uint64_t>(t.n);
    if (n == 0) return;
    auto part = [&](int q, const void *at, uint64_t bytes, uintptr_t odd) {
        const uintptr_t begin = reinterpret_cast<uintptr_t>(at);
        take(q, Range{begin | odd, begin + bytes});
    };
    part(0, t.p, n * (t.p_dtype == TPCE_BF16 ? 2 : 4), 0);
    if (t.master) part(1, t.master, n * 4, 0);
    const uint64_t state = state8(t) ? 1 : 4;
    part(2, t.m, n * state, 0);
    part(3, t.v, n * state, 0);
    if (state8(t)) {
        part(4, t.m_scale, (n + kGroup - 1) / kGroup * 4, 0);
        part(5, t.v_scale, (n + kGroup - 1) / kGroup * 4, 0);
    }
    part(6, t.g, n * (t.g_dtype == TPCE_BF16 ? 2 : 4), 1);
}

// Ranges in the order of their begin, from or to `a`: neighbouring runs that rise are
// merged until one is left, which for tensors made in the list's order are few steps.
// `other` is as long as `a`.
inline Range *sorted(Range *a, Range *other, int64_t n) {
    auto before = [](const Range &x, const Range &y) { return x.begin < y.begin; };
    for (;;) {
        for (int64_t i = 0; i < n;) {
            const int64_t j = std::is_sorted_until(a + i, a + n, before) - a;
            if (i == 0 && j == n) return a;
            const int64_t k = j < n ? std::is_sorted_until(a + j, a + n, before) - a : n;
            std::merge(a + i, a + j, a + j, a + k, other + i, before);
            i = k;
        }
        std::swap(a, other);
    }
}

// Whether the ranges are in a few dense runs of rising addresses that do not meet, as
// where the tensors of a kind lie in one buffer: one pass over them shows that none
// overlap. Of part q there are count[q], from part[q] on.
inline bool apart(Range *const (&part)[kParts], const int64_t (&count)[kParts]) {
    constexpr uintptr_t kGap = 4096;  // (a begin below the end is a gap of nearly 2^64)
    Range runs[16];
    int n = 0;
    for (int q = 0; q < kParts; ++q) {
        for (int64_t i = 0; i < count[q];) {
            if (n == 16) return false;
            Range run = part[q][i];
            run.begin &= ~uintptr_t{1};
            for (++i; i < count[q] && part[q][i].begin - run.end < kGap; ++i) run.end = part[q][i].end;
            runs[n++] = run;
        }
    }
    std::sort(runs, runs + n, [](const Range &x, const Range &y) { return x.begin < y.begin; });
    for (int i = 1; i < n; ++i)
        if (runs[i].begin < runs[i - 1].end) return false;
    return true;
}

tpce_status overlap(const tpce_adamw_tensor *tensors, int count, const Range &x, const Range &y) {
    int at[2] = {-1, -1}, part[2] = {0, 0};
    for (int i = 0; i < count; ++i)
        ranges_of(tensors[i], [&](int q, const Range &r) {
            // two equal ranges are two different places of the list
            if (at[0] < 0 && r.begin == x.begin && r.end == x.end)
                at[0] = i, part[0] = q;
            else if (at[1] < 0 && r.begin == y.begin && r.end == y.end)
                at[1] = i, part[1] = q;
        });
    return fail(TPCE_ERR_INVALID, "tp_adamw_step: tensor %d: %s overlaps tensor %d: %s", at[1], kPartNames[part[1]],
                at[0], kPartNames[part[0]]);
}

// 100 tensors with 8-bit states (600 ranges) on GB300's host: 0.5 us where the tensors
// of a kind lie in buffers, 2.7 us where each was allocated by itself in the list's
// order, 7 us in no order at all.
tpce_status check_overlaps(const tpce_adamw_tensor *tensors, int count) {
    const int64_t most = static_cast<int64_t>(count) * kParts;
    const std::unique_ptr<Range, decltype(&std::free)> held(
        static_cast<Range *>(std::malloc(sizeof(Range) * static_cast<size_t>(2 * most))), &std::free);
    if (!held) return fail(TPCE_ERR_WORKSPACE, "tp_adamw_step: no host memory for %d tensors", count);
    Range *part[kParts];
    int64_t in[kParts] = {};
    for (int q = 0; q < kParts; ++q) part[q] = held.get() + static_cast<int64_t>(q) * count;
    for (int i = 0; i < count; ++i)
        ranges_of(tensors[i], [&](int q, const Range &r) { part[q][in[q]++] = r; });
    if (apart(part, in)) return TPCE_OK;
    int64_t n = 0;
    for (int q = 0; q < kParts; ++q) {
        std::copy(part[q], part[q] + in[q], held.get() + n);  // to the front of where it is
        n += in[q];
    }
    const Range *r = sorted(held.get(), held.get() + most, n);
    // of the ranges before, those that reach farthest: of all, and of the written ones
    Range any{0, 0}, written{0, 0};
    for (int64_t i = 0; i < n; ++i) {
        const bool writes = !(r[i].begin & 1);
        const Range &before = writes ? any : written;
        if ((r[i].begin & ~uintptr_t{1}) < before.end) return overlap(tensors, count, before, r[i]);
        if (r[i].end > any.end) any = r[i];
        if (writes && r[i].end > written.end) written = r[i];
    }
    return TPCE_OK;
}

}  // namespace
}  // namespace tpce

// ====================================================================== C ABI
using namespace tpce;

extern "C" tpce_status tp_adamw_step(const tpce_adamw_tensor *tensors, int count, double lr, double beta1,
                                     double beta2, double eps, int64_t step, double grad_scale,
                                     const float *device_scalars, void *stream) {
    if (count < 0 || (count > 0 && !tensors)) return fail(TPCE_ERR_INVALID, "tp_adamw_step: no tensors");
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(lr) ||
        !std::isfinite(eps) || !std::isfinite(grad_scale) || step < 1)
        return fail(TPCE_ERR_INVALID, "tp_adamw_step: beta1 and beta2 in [0, 1), eps >= 0, step >= 1, finite lr");
    // everything is checked before anything is launched
    int64_t total = 0;
    for (int i = 0; i < count; ++i) {
        const tpce_adamw_tensor &t = tensors[i];
        const bool bf = t.p_dtype == TPCE_BF16;
        if ((!bf && t.p_dtype != TPCE_F32) || (t.g_dtype != TPCE_BF16 && t.g_dtype != TPCE_F32) ||
            (!state8(t) && t.state_bits != 32) || !std::isfinite(t.weight_decay))
            return fail(TPCE_ERR_INVALID,
                        "tp_adamw_step: tensor %d: dtypes, state_bits (8, 32 or 8 | TPCE_ADAMW_RANDOM) or weight_decay",
                        i);
        if (t.n < 0) return fail(TPCE_ERR_SHAPE, "tp_adamw_step: tensor %d: n = %lld", i, static_cast<long long>(t.n));
        if (t.n == 0) continue;
        if (!t.p || !t.g || !t.m || !t.v || (state8(t) && (!t.m_scale || !t.v_scale)) || (t.master && !bf))
            return fail(TPCE_ERR_INVALID, "tp_adamw_step: tensor %d: null pointer, or a master beside fp32 values", i);
        for (const void *p : {static_cast<const void *>(t.p), static_cast<const void *>(t.master), t.g,
                              static_cast<const void *>(t.m), static_cast<const void *>(t.v),
                              static_cast<const void *>(t.m_scale), static_cast<const void *>(t.v_scale)})
            if (!aligned16(p))
                return fail(TPCE_ERR_ALIGN, "tp_adamw_step: tensor %d: a pointer is not 16-byte aligned", i);
        if (t.n > INT64_MAX - kChunk || (t.n + kChunk - 1) / kChunk > INT_MAX - total)
            return fail(TPCE_ERR_SHAPE, "tp_adamw_step: too many values");
        total += (t.n + kChunk - 1) / kChunk;
    }
    if (reinterpret_cast<uintptr_t>(device_scalars) & 3u)
        return fail(TPCE_ERR_ALIGN, "tp_adamw_step: device_scalars is not aligned");
    if (count) {
        const tpce_status st = check_overlaps(tensors, count);
        if (st != TPCE_OK) return st;
    }

    Scalars k{};
    k.b1 = static_cast<float>(beta1);
    k.one_b1 = static_cast<float>(1.0 - beta1);
    k.b2 = static_cast<float>(beta2);
    k.one_b2 = static_cast<float>(1.0 - beta2);
    k.eps = static_cast<float>(eps);
    k.step_size = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
    k.root_scale = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
    k.grad_scale = static_cast<float>(grad_scale);
    k.step = static_cast<uint32_t>(step);
    k.device = device_scalars;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Entry entries[kLong];
    int held = 0;
    uint32_t blocks = 0;
    bool random = false;
    auto flush = [&]() -> tpce_status {
        if (!held) return TPCE_OK;
        tpce_status st = held <= kShort    ? launch_table<kShort>(entries, held, blocks, random, k, s)
                         : held <= kMiddle ? launch_table<kMiddle>(entries, held, blocks, random, k, s)
                                           : launch_table<kLong>(entries, held, blocks, random, k, s);
        held = 0;
        random = false;
        blocks = 0;
        return st;
    };
    for (int i = 0; i < count; ++i) {
        const tpce_adamw_tensor &t = tensors[i];
        if (t.n == 0) continue;
        Entry &e = entries[held++];
        e = Entry{t.p, t.master, t.g, t.m, t.v, t.m_scale, t.v_scale, t.n, blocks, 0u, 0.0f, 0.0f, 1u, 0u};
        e.kind = (t.p_dtype == TPCE_BF16 ? kParamBf16 : 0u) | (t.master ? kMaster : 0u) |
                 (t.g_dtype == TPCE_BF16 ? kGradBf16 : 0u) | (state8(t) ? kState8 : 0u) |
                 (t.state_bits & TPCE_ADAMW_RANDOM ? kRandom : 0u);
        random |= (e.kind & kRandom) != 0u;
        e.decay = static_cast<float>(1.0 - lr * t.weight_decay);
        e.wd = static_cast<float>(t.weight_decay);
        if (state8(t) && total >= kSpanFrom) e.span = kSpan;
        const int64_t block = static_cast<int64_t>(e.span) * kChunk;
        blocks += static_cast<uint32_t>((t.n + block - 1) / block);
        if (held == kLong) {
            tpce_status st = flush();
            if (st != TPCE_OK) return st;
        }
    }
    return flush();
}
