// adamw8_kernels.hip -- the AdamW step with both states in 8 bits (gfx950).
//
//     m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//     w = (1 - lr decay) w - (lr / (1 - b1^t)) m / (sqrt(v / (1 - b2^t)) + eps)
//
// m and v are kept as codes of blocks of 256 elements of a span, each with its
// largest magnitude s in binary32:
//     m = s (k / 127)^2 with k's sign, k = -127 .. 127
//     v = s (k / 255)^4,               k = 0 .. 255
// The powers give the root of v, which the step divides by, the same kind of
// code as m: steps of 2 / k of the value, from 1/16000 (m) or 1/65000 (v's root)
// of the block's largest on.  On gradients whose sizes spread by e the step is
// 10% off that of binary32 states and 7.5% over 3000 steps together; with
// e4m3 values for m and v's root it is 16% and 13%.
//
// A code is the one whose root is nearest to the value's.  Which one that is is
// decided in binary64, where the card is as fast as in binary32, with every term
// rounded as the formula reads: the same step gives the same codes everywhere.  A v
// over 0 keeps at least k = 1: rounded to 0 it would leave eps alone under an m that
// is not 0.
//
// Bound by memory: 16 bytes an element with binary16 gradients and copies, against
// 28 with binary32 states.  300M elements with binary32 gradients and bfloat16
// copies take 895 us (6.0 TB/s of 18 bytes), with binary32 states 1735 us.  A wave
// takes two blocks, so that one row of exchanges finds both largest values and
// enough waves fit to hide memory (four blocks, a block's maxima one after the
// other: 1530 us); elements that binary64 has to decide are done one at a time
// (both blocks whole: 1190 us).
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <limits>
#include <new>
#include <type_traits>

#include "../../include/ddl.h"
#include "optimizer_internal.h"

namespace ddl {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kBlock = DDL_ADAMW8_BLOCK;  // 4 elements of each lane
constexpr uint32_t kWave = 2 * kBlock;         // two blocks a wave
constexpr uint32_t kChunk = kWave * (kThreads / 64);
static_assert(kBlock == 256, "4 elements of each lane");

// A workgroup's part of a span, and the index of its first block.
struct Part {
    uint64_t at;
    uint32_t count;
    uint32_t block;
};

struct States {
    int8_t *m;
    uint8_t *v;
    float *m_scale, *v_scale;
};

struct Adam8Args {
    const Part *parts;
    const void *grad;
    States s;
    float *w;
    void *copy;
    double b1, b2, c1, c2;  // c = 1 - b
    float step, root, eps;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    float keep;             // 1 - lr decay
    int vec;
    int wide;               // the weights meet subnormal numbers (see ddl_adamw8_step)
};

// The largest of x over the wave in its lower half's lanes, and that of y in the
// upper half's: bits of numbers without a sign, so that NaN is over all others;
// NaN where it is not finite.
template <int TURN>
__device__ __forceinline__ uint32_t turn_max(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + TURN, 0xf, 0xf, false));
}
__device__ __forceinline__ float both_max(uint32_t x, uint32_t y) {
    const auto h = __builtin_amdgcn_permlane32_swap(x, y, false, false);  // halves
    x = turn_max<1>(turn_max<2>(turn_max<4>(turn_max<8>(max(h[0], h[1])))));  // rows of 16
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);  // the half's two rows
    x = max(r[0], r[1]);
    return __builtin_bit_cast(float, x >= 0x7f800000u ? 0x7fc00000u : x);
}
__device__ __forceinline__ float of_lane(float x, int lane) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

constexpr double kM = 127.0 * 127.0, kV = 255.0 * 255.0 * 255.0 * 255.0;

// k of y = 127^2 |m| / s: the nearest to y's root, at most 127.  The root in
// binary32 is at most one off.
__device__ __forceinline__ float code_m(double y) {
    const float k = __builtin_rintf(sqrtf((float)y));
    const float h = k + 0.5f, l = fmaxf(k - 0.5f, 0.0f);
    return fminf(k + (y >= (double)(h * h) ? 1.0f : 0.0f) - (y < (double)(l * l) ? 1.0f : 0.0f),
                 127.0f);
}
// k of y = 255^4 v / s, at most 255.
__device__ __forceinline__ float code_v(double y) {
    const float k = __builtin_rintf(sqrtf(sqrtf((float)y)));
    const float h = k + 0.5f, l = fmaxf(k - 0.5f, 0.0f);
    const double hi = (double)(h * h), lo = (double)(l * l);  // exact
    return fminf(k + (y >= hi * hi ? 1.0f : 0.0f) - (y < lo * lo ? 1.0f : 0.0f), 255.0f);
}

// The element e of a lane, within its block: 4 neighbours (VEC), or every 64th.
template <bool VEC>
__device__ __forceinline__ uint32_t place(uint32_t lane, int e) {
    return VEC ? lane * 4 + e : lane + 64 * e;
}

// Every byte is read and written once: all accesses are non-temporal (300M
// elements without the arithmetic: 930 us, otherwise 1020).
// VEC: a lane's elements are all there or none.
template <bool VEC, class X>
__device__ __forceinline__ void load4(const X *p, uint32_t lane, uint32_t count, X (&out)[4]) {
    typedef X X4 __attribute__((ext_vector_type(4)));
    if constexpr (VEC) {
        X4 v = {};
        if (lane * 4 < count)
            v = __builtin_nontemporal_load((const X4 *)(p + lane * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            out[e] = v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            out[e] = place<VEC>(lane, e) < count ? p[place<VEC>(lane, e)] : (X)0;
    }
}
template <bool VEC, class X>
__device__ __forceinline__ void store4(X *p, uint32_t lane, uint32_t count, const X (&in)[4]) {
    typedef X X4 __attribute__((ext_vector_type(4)));
    if constexpr (VEC) {
        X4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = in[e];
        if (lane * 4 < count)
            __builtin_nontemporal_store(v, (X4 *)(p + lane * 4));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (place<VEC>(lane, e) < count)
                p[place<VEC>(lane, e)] = in[e];
    }
}

struct Moments {
    double m, v;
};
// dm, dv: b times the block's scale.  A block's largest m is often from k = 127, as
// b s + c g, and midway between two binary32 numbers (of 0.9 s + 0.1 g with
// binary16 g 1 in 12): which one the scale becomes goes by the last bit
// of binary64.  So terms are rounded one by one, as the formula reads, and the
// share of the largest k is 1.
__device__ __forceinline__ Moments moments(const Adam8Args &a, double dm, double dv, int8_t km,
                                           uint8_t kv, float g) {
    const double ge = (double)g;
    const float k = (float)km, h = (float)kv;
    const double h2 = (double)(h * h);
    return {dm * ((double)(k * fabsf(k)) * (1 / kM)) + a.c1 * ge,
            dv * (h2 * h2 * (1 / kV)) + a.c2 * ge * ge};
}

// A wave's two blocks from element `at` on, `count` elements of them.
template <class G, class C, bool VEC, class R>
__device__ __forceinline__ void step_wave(const Adam8Args &a, const R &r, uint64_t at,
                                          uint32_t count, uint32_t block, uint32_t lane) {
    const uint32_t have[2] = {count, count > kBlock ? count - kBlock : 0};
    G gh[2][4];
    float w[2][4];
    int8_t km[2][4];
    uint8_t kv[2][4];
    double dm[2], dv[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint64_t i = at + b * kBlock;
        load4<VEC>((const G *)a.grad + i, lane, have[b], gh[b]);
        load4<VEC>((const float *)a.w + i, lane, have[b], w[b]);
        load4<VEC>((const int8_t *)a.s.m + i, lane, have[b], km[b]);
        load4<VEC>((const uint8_t *)a.s.v + i, lane, have[b], kv[b]);
        dm[b] = have[b] ? a.b1 * (double)a.s.m_scale[block + b] : 0.0;
        dv[b] = have[b] ? a.b2 * (double)a.s.v_scale[block + b] : 0.0;
    }
    double m[2][4], v[2][4];
    float root[2][4];
    uint32_t top_m[2] = {0, 0}, top_v[2] = {0, 0};
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Moments x = moments(a, dm[b], dv[b], km[b][e], kv[b][e], (float)gh[b][e]);
            m[b][e] = x.m;
            v[b][e] = x.v;
            const float mf = (float)x.m, vf = (float)x.v;
            top_m[b] = max(top_m[b], __builtin_bit_cast(uint32_t, mf) & 0x7fffffffu);
            top_v[b] = max(top_v[b], __builtin_bit_cast(uint32_t, vf));
            // The hardware's root and reciprocal are 1 ulp off (correctly rounded
            // ones: 300M elements 960 us, so 890) and take subnormal numbers for 0.
            root[b][e] = __builtin_amdgcn_sqrtf(vf);
            if (a.wide)
                w[b][e] = a.keep * w[b][e] - a.step * (mf / (sqrtf(vf) * a.root + a.eps));
            else
                w[b][e] = __builtin_fmaf(
                    -a.step,
                    mf * __builtin_amdgcn_rcpf(__builtin_fmaf(root[b][e], a.root, a.eps)),
                    a.keep * w[b][e]);
        }
        const uint64_t i = at + b * kBlock;
        store4<VEC>(a.w + i, lane, have[b], w[b]);
        if constexpr (std::is_same<R, Replicas>::value)
            for (int k = 1; k < r.count; ++k)
                store4<VEC>(r.w[k] + i, lane, have[b], w[b]);
        if (a.copy) {
            C c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c[e] = (C)w[b][e];
            store4<VEC>((C *)a.copy + i, lane, have[b], c);
        }
    }
    const float tm = both_max(top_m[0], top_m[1]), tv = both_max(top_v[0], top_v[1]);
    // The codes by binary32 roots: the hardware's, reciprocals and roots of
    // reciprocals are 1 ulp off, so that 255 times the root is 8.8e-5 off at
    // most.  Where one is closer to a border than 1e-4 (a block in ten), or scales
    // are so small or large that shares lose digits, binary64 decides.
    auto plain = [](float t) { return t == 0.0f || (t >= 0x1p-80f && t <= 0x1p80f); };
    const float im = tm > 0.0f ? __builtin_amdgcn_rcpf(tm) : 0.0f;
    const float iv = tv > 0.0f ? __builtin_amdgcn_rsqf(tv) : 0.0f;
    const bool far = !plain(tm) || !plain(tv);
    float off = far ? 1.0f : 0.0f;
    float x[2][4], y[2][4];
    int8_t cm[2][4];
    uint8_t cv[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const float jm = of_lane(im, b * 32), jv = of_lane(iv, b * 32);
        const float least = jv > 0.0f ? 1.0f : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float mf = (float)m[b][e];
            x[b][e] = 127.0f * __builtin_amdgcn_sqrtf(fabsf(mf) * jm);
            y[b][e] = 255.0f * __builtin_amdgcn_sqrtf(root[b][e] * jv);
            const float k = __builtin_rintf(x[b][e]), h = __builtin_rintf(y[b][e]);
            x[b][e] -= k;
            y[b][e] -= h;
            off = fmaxf(off, fmaxf(fabsf(x[b][e]), fabsf(y[b][e])));
            cm[b][e] = (int8_t)(int)__builtin_copysignf(k, mf);
            cv[b][e] = (uint8_t)(int)(v[b][e] > 0.0 ? fmaxf(h, least) : h);
        }
    }
    if (__any(!(off < 0.4999f))) {
        const bool far_any = __any(far);
        const double em = tm > 0.0f ? kM / (double)tm : 0.0, ev = tv > 0.0f ? kV / (double)tv : 0.0;
        auto of = [](double x, int lane) {
            const uint64_t u = __builtin_bit_cast(uint64_t, x);
            const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
            const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
            return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const double jm = of(em, b * 32), jv = of(ev, b * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!far_any && fmaxf(fabsf(x[b][e]), fabsf(y[b][e])) < 0.4999f)
                    continue;
                const int k = (int)code_m(fabs(m[b][e]) * jm), h = (int)code_v(v[b][e] * jv);
                cm[b][e] = (int8_t)(m[b][e] < 0.0 ? -k : k);
                cv[b][e] = (uint8_t)(v[b][e] > 0.0 && jv > 0.0 ? max(h, 1) : h);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        store4<VEC>(a.s.m + at + b * kBlock, lane, have[b], cm[b]);
        store4<VEC>(a.s.v + at + b * kBlock, lane, have[b], cv[b]);
    }
    if (lane % 32 == 0 && lane / 32 * kBlock < count) {
        a.s.m_scale[block + lane / 32] = tm;
        a.s.v_scale[block + lane / 32] = tv;
    }
}

// A wave's part of workgroup blockIdx.x's part, to f(VEC, element, elements, block).
template <class F>
__device__ __forceinline__ void with_wave(const Part *parts, int vec, F &&f) {
    const Part p = parts[blockIdx.x];
    const uint32_t first = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kWave;
    if (first >= p.count)
        return;
    const uint32_t count = p.count - first, block = p.block + first / kBlock;
    if (vec && p.at % 4 == 0 && (count % 4 == 0 || count >= kWave))
        f(std::true_type(), p.at + first, count, block);
    else
        f(std::false_type(), p.at + first, count, block);
}

// R: Replicas; or int for one, whose launch then carries 1 KB of arguments less.
template <class G, class C, class R>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(Adam8Args a, R r) {
    with_wave(a.parts, a.vec, [&](auto vec, uint64_t at, uint32_t count, uint32_t block) {
        step_wave<G, C, decltype(vec)::value>(a, r, at, count, block, threadIdx.x & 63u);
    });
}

template <bool VEC>
__device__ __forceinline__ void values_wave(const States &s, float *m, float *v, uint64_t at,
                                            uint32_t count, uint32_t block, uint32_t lane) {
    const uint32_t have[2] = {count, count > kBlock ? count - kBlock : 0};
    int8_t km[2][4];
    uint8_t kv[2][4];
    double dm[2], dv[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        load4<VEC>((const int8_t *)s.m + at + b * kBlock, lane, have[b], km[b]);
        load4<VEC>((const uint8_t *)s.v + at + b * kBlock, lane, have[b], kv[b]);
        dm[b] = have[b] ? (double)s.m_scale[block + b] * (1 / kM) : 0.0;
        dv[b] = have[b] ? (double)s.v_scale[block + b] * (1 / kV) : 0.0;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float k = (float)km[b][e], h = (float)kv[b][e];
            const double h2 = (double)(h * h);
            x[e] = (float)(dm[b] * (double)(k * fabsf(k)));
            y[e] = (float)(dv[b] * (h2 * h2));
        }
        store4<VEC>(m + at + b * kBlock, lane, have[b], x);
        store4<VEC>(v + at + b * kBlock, lane, have[b], y);
    }
}

__global__ __launch_bounds__(kThreads) void values8_kernel(const Part *parts, States s, float *m,
                                                           float *v, int vec) {
    with_wave(parts, vec, [&](auto vec_, uint64_t at, uint32_t count, uint32_t block) {
        values_wave<decltype(vec_)::value>(s, m, v, at, count, block, threadIdx.x & 63u);
    });
}

}  // namespace
}  // namespace ddl

using namespace ddl;

struct ddl_adamw8_s {
    std::vector<Part> parts;
    size_t blocks = 0;
    Handle dev;
    Part *d_parts = nullptr;

    int bind(hipStream_t s) {
        return dev.bind(s, [&]() { return upload(parts, &d_parts); });
    }
};

extern "C" {

int ddl_adamw8_create(ddl_adamw8 *out, const size_t *offsets, const size_t *counts, int nspans) {
    if (!out || (nspans > 0 && (!offsets || !counts)))
        return DDL_E_NULL;
    *out = nullptr;
    if (nspans < 0)
        return DDL_E_ARG;
    ddl_adamw8 h = nullptr;
    try {
        std::vector<Span> spans;
        uint64_t all = 0;
        for (int i = 0; i < nspans; ++i)
            spans.push_back({offsets[i], counts[i]});
        if (!disjoint(spans))
            return DDL_E_BUCKETS;
        for (const Span &s : spans)
            all += (s.count + kBlock - 1) / kBlock;
        if (all > kMaxGrid)
            return DDL_E_ARG;
        h = new ddl_adamw8_s;
        for (const Span &s : spans) {
            for (uint64_t x = 0; x < s.count; x += kChunk)
                h->parts.push_back({s.at + x, (uint32_t)std::min<uint64_t>(kChunk, s.count - x),
                                    (uint32_t)(h->blocks + x / kBlock)});
            h->blocks += (s.count + kBlock - 1) / kBlock;
        }
        register_handle(h);
    } catch (...) {
        delete h;
        return DDL_E_NOMEM;
    }
    *out = h;
    return DDL_OK;
}

int ddl_adamw8_destroy(ddl_adamw8 h) {
    if (!h)
        return DDL_E_NULL;
    if (!unregister_handle(h))
        return DDL_E_ARG;
    h->dev.release(h->d_parts);
    delete h;
    return DDL_OK;
}

int ddl_adamw8_blocks(ddl_adamw8 h, size_t *blocks) {
    if (!h || !blocks)
        return DDL_E_NULL;
    std::unique_lock<std::mutex> lk;
    if (!hold_handle(h, lk))
        return DDL_E_ARG;
    *blocks = h->blocks;
    return DDL_OK;
}

int ddl_adamw8_step(ddl_adamw8 h, const void *grad, int grad_dtype, signed char *m,
                    unsigned char *v, float *m_scale, float *v_scale, float *const *weights,
                    int nweights, void *copy, int copy_dtype, double lr, double beta1,
                    double beta2, double eps, double weight_decay, long long step, void *stream) {
    if (!h)
        return DDL_E_NULL;
    std::unique_lock<std::mutex> lk;
    if (!hold_handle(h, lk))
        return DDL_E_ARG;
    if (nweights < 1 || nweights > DDL_MAX_RANKS || !float_type(grad_dtype)
        || (copy && copy_dtype != DDL_F16 && copy_dtype != DDL_BF16) || step < 1
        || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0)
        || !std::isfinite(eps) || !std::isfinite(lr) || !std::isfinite(weight_decay))
        return DDL_E_ARG;
    if (h->parts.empty())
        return DDL_OK;
    Replicas r;
    int rc = take_replicas(weights, nweights, r);
    if (rc)
        return rc;
    if (!grad || !m || !v || !m_scale || !v_scale)
        return DDL_E_NULL;
    if (!aligned_to(grad, grad_dtype) || !aligned_to(m_scale, DDL_F32)
        || !aligned_to(v_scale, DDL_F32) || (copy && !aligned_to(copy, copy_dtype)))
        return DDL_E_ALIGN;
    rc = h->bind((hipStream_t)stream);
    if (rc)
        return rc;
    Adam8Args a;
    a.parts = h->d_parts;
    a.grad = grad;
    a.s = {(int8_t *)m, v, m_scale, v_scale};
    a.w = r.w[0];
    a.copy = copy;
    a.b1 = beta1;
    a.b2 = beta2;
    a.c1 = 1 - beta1;
    a.c2 = 1 - beta2;
    a.step = (float)(lr / (1 - std::pow(beta1, (double)step)));
    a.root = (float)(1 / std::sqrt(1 - std::pow(beta2, (double)step)));
    // an eps over 0 stays over 0: weights without a gradient so far do not move
    a.eps = eps > 0 ? std::max((float)eps, std::numeric_limits<float>::denorm_min()) : 0.0f;
    a.keep = (float)(1 - lr * weight_decay);
    // roots of subnormal v, up to 2^-63, times a.root are more than a rounding of eps,
    // or eps or its reciprocal is subnormal itself
    a.wide = !(eps >= (double)a.root * 0x1p-63 * 0x1p24 && eps <= 0x1p125);
    uintptr_t all = (uintptr_t)grad | (uintptr_t)copy | (uintptr_t)m | (uintptr_t)v;
    for (int i = 0; i < r.count; ++i)
        all |= (uintptr_t)r.w[i];
    a.vec = all % 16 == 0;
    const dim3 grid((uint32_t)h->parts.size()), block(kThreads);
    hipStream_t s = (hipStream_t)stream;
    auto go = [&](auto g) {
        using G = decltype(g);
        const bool half = !copy || copy_dtype == DDL_F16;
        if (r.count > 1)
            return launch(half ? adamw8_kernel<G, _Float16, Replicas>
                               : adamw8_kernel<G, __bf16, Replicas>,
                          grid, block, 0, s, a, r);
        return launch(half ? adamw8_kernel<G, _Float16, int> : adamw8_kernel<G, __bf16, int>, grid,
                      block, 0, s, a, 0);
    };
    return grad_dtype == DDL_F32   ? go(float())
           : grad_dtype == DDL_F16 ? go(_Float16())
                                   : go(__bf16());
}

int ddl_adamw8_values(ddl_adamw8 h, const signed char *m, const unsigned char *v,
                      const float *m_scale, const float *v_scale, float *m_out, float *v_out,
                      void *stream) {
    if (!h)
        return DDL_E_NULL;
    std::unique_lock<std::mutex> lk;
    if (!hold_handle(h, lk))
        return DDL_E_ARG;
    if (h->parts.empty())
        return DDL_OK;
    if (!m || !v || !m_scale || !v_scale || !m_out || !v_out)
        return DDL_E_NULL;
    for (const float *p : {m_scale, v_scale, (const float *)m_out, (const float *)v_out})
        if (!aligned_to(p, DDL_F32))
            return DDL_E_ALIGN;
    const int rc = h->bind((hipStream_t)stream);
    if (rc)
        return rc;
    const int vec =
        ((uintptr_t)m_out | (uintptr_t)v_out | (uintptr_t)m | (uintptr_t)v) % 16 == 0;
    const States st = {(int8_t *)m, (uint8_t *)v, (float *)m_scale, (float *)v_scale};
    return launch(values8_kernel, dim3((uint32_t)h->parts.size()), dim3(kThreads), 0,
                  (hipStream_t)stream, h->d_parts, st, m_out, v_out, vec);
}

}  // extern "C"
