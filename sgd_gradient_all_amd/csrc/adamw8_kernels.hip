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
// decided in binary64, where the card is as fast as in binary32: it then does
// not depend on how sums are contracted, and the same step gives the same codes
// everywhere.  A v over 0 keeps at least k = 1: rounded to 0 it would leave eps
// alone under an m that is not 0.
//
// 16 bytes an element with binary16 gradients and copies, against 28 with
// binary32 states: bound by memory.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "../../include/ddl.h"
#include "optimizer_internal.h"

namespace ddl {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kBlock = DDL_ADAMW8_BLOCK;  // a wave's: 4 elements a lane
constexpr uint32_t kEach = 4;                  // blocks of a wave
constexpr uint32_t kChunk = kBlock * kEach * (kThreads / 64);
static_assert(kBlock == 256, "4 elements a lane");

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
    double b1, b2, c1, c2;  // c = 1 - b; b1 / 127^2 and b2 / 255^4
    float step, root, eps;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    float keep;             // 1 - lr decay
    int vec;
};

// The largest of a wave's values (bits of numbers without a sign, so that NaN
// is over all others), NaN if it is not finite.
__device__ __forceinline__ float wave_max(uint32_t x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        x = max(x, (uint32_t)__shfl_xor((int)x, d));
    return __builtin_bit_cast(float, x >= 0x7f800000u ? 0x7fc00000u : x);
}

// k of y = 127^2 |m| / s: the nearest to y's root, at most 127.  The root in
// binary32 is at most one off.
__device__ __forceinline__ float code_m(double y) {
    float k = __builtin_rintf(__builtin_amdgcn_sqrtf((float)y));
    const float hi = k + 0.5f, lo = k - 0.5f;
    if (y >= (double)(hi * hi))
        k += 1.0f;
    else if (k > 0.0f && y < (double)(lo * lo))
        k -= 1.0f;
    return fminf(k, 127.0f);
}
// k of y = 255^4 v / s, at most 255.
__device__ __forceinline__ float code_v(double y) {
    float k = __builtin_rintf(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf((float)y)));
    const float h = k + 0.5f, l = k - 0.5f;
    const double hi = (double)(h * h), lo = (double)(l * l);  // exact
    if (y >= hi * hi)
        k += 1.0f;
    else if (k > 0.0f && y < lo * lo)
        k -= 1.0f;
    return fminf(k, 255.0f);
}

constexpr double kM = 127.0 * 127.0, kV = 255.0 * 255.0 * 255.0 * 255.0;

// Elements of a lane: 4 neighbours (VEC), or every 64th of the block.
template <bool VEC>
__device__ __forceinline__ uint32_t place(uint32_t lane, int e) {
    return VEC ? lane * 4 + e : lane + 64 * e;
}

template <bool VEC, class X, class F>
__device__ __forceinline__ void load4(const X *p, uint32_t lane, uint32_t count, F (&out)[4]) {
    typedef X X4 __attribute__((ext_vector_type(4)));
    if (VEC && lane * 4 + 4 <= count) {
        const X4 v = *(const X4 *)(p + lane * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            out[e] = (F)v[e];
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        out[e] = place<VEC>(lane, e) < count ? (F)p[place<VEC>(lane, e)] : (F)0;
}
template <bool VEC, class X, class F>
__device__ __forceinline__ void store4(X *p, uint32_t lane, uint32_t count, const F (&in)[4]) {
    typedef X X4 __attribute__((ext_vector_type(4)));
    if (VEC && lane * 4 + 4 <= count) {
        X4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = (X)in[e];
        *(X4 *)(p + lane * 4) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (place<VEC>(lane, e) < count)
            p[place<VEC>(lane, e)] = (X)in[e];
}

// kEach blocks of a wave, from element `at` on, `count` elements; all are
// loaded before the first is computed.
template <class G, class C, bool VEC, bool MANY>
__device__ __forceinline__ void step_blocks(const Adam8Args &a, const Replicas &r, uint64_t at,
                                            uint32_t count, uint32_t block, uint32_t lane) {
    float g[kEach][4], w[kEach][4];
    int km[kEach][4], kv[kEach][4];
    float sm[kEach], sv[kEach];
#pragma unroll
    for (uint32_t b = 0; b < kEach; ++b) {
        const uint64_t i = at + b * kBlock;
        const uint32_t have = count > b * kBlock ? count - b * kBlock : 0;
        load4<VEC>((const G *)a.grad + i, lane, have, g[b]);
        load4<VEC>(a.w + i, lane, have, w[b]);
        load4<VEC>(a.s.m + i, lane, have, km[b]);
        load4<VEC>(a.s.v + i, lane, have, kv[b]);
        sm[b] = have ? a.s.m_scale[block + b] : 0.0f;
        sv[b] = have ? a.s.v_scale[block + b] : 0.0f;
    }
#pragma unroll
    for (uint32_t b = 0; b < kEach; ++b) {
        if (count <= b * kBlock)
            break;
        const uint64_t i = at + b * kBlock;
        const uint32_t have = count - b * kBlock;
        const double dm = a.b1 * (double)sm[b], dv = a.b2 * (double)sv[b];
        double m[4], v[4];
        uint32_t top_m = 0, top_v = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const double ge = (double)g[b][e];
            const double v2 = (double)(kv[b][e] * kv[b][e]);
            const int k2 = km[b][e] * km[b][e];
            m[e] = dm * (double)(km[b][e] < 0 ? -k2 : k2) + a.c1 * ge;
            v[e] = dv * (v2 * v2) + a.c2 * (ge * ge);
            const float mf = (float)m[e], vf = (float)v[e];
            w[b][e] = a.keep * w[b][e] - a.step * (mf / (sqrtf(vf) * a.root + a.eps));
            top_m = max(top_m, __builtin_bit_cast(uint32_t, mf) & 0x7fffffffu);
            top_v = max(top_v, __builtin_bit_cast(uint32_t, vf));
        }
        const float tm = wave_max(top_m), tv = wave_max(top_v);
        const double im = tm > 0.0f ? kM / (double)tm : 0.0, iv = tv > 0.0f ? kV / (double)tv : 0.0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = (int)code_m(fabs(m[e]) * im), q = (int)code_v(v[e] * iv);
            km[b][e] = m[e] < 0.0 ? -p : p;
            kv[b][e] = q == 0 && v[e] * iv > 0.0 ? 1 : q;
        }
        store4<VEC>(a.s.m + i, lane, have, km[b]);
        store4<VEC>(a.s.v + i, lane, have, kv[b]);
        store4<VEC>(a.w + i, lane, have, w[b]);
        if (MANY)
            for (int k = 1; k < r.count; ++k)
                store4<VEC>(r.w[k] + i, lane, have, w[b]);
        if (a.copy)
            store4<VEC>((C *)a.copy + i, lane, have, w[b]);
        if (lane == 0) {
            a.s.m_scale[block + b] = tm;
            a.s.v_scale[block + b] = tv;
        }
    }
}

template <class G, class C, bool MANY>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(Adam8Args a, Replicas r) {
    const Part p = a.parts[blockIdx.x];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    const uint32_t first = wave * kEach * kBlock;
    if (first >= p.count)
        return;
    const uint64_t at = p.at + first;
    const uint32_t count = p.count - first, block = p.block + wave * kEach;
    if (a.vec && p.at % 4 == 0)
        step_blocks<G, C, true, MANY>(a, r, at, count, block, lane);
    else
        step_blocks<G, C, false, MANY>(a, r, at, count, block, lane);
}

template <bool VEC>
__device__ __forceinline__ void values_blocks(const States &s, float *m, float *v, uint64_t at,
                                              uint32_t count, uint32_t block, uint32_t lane) {
#pragma unroll
    for (uint32_t b = 0; b < kEach; ++b) {
        if (count <= b * kBlock)
            break;
        const uint64_t i = at + b * kBlock;
        const uint32_t have = count - b * kBlock;
        int km[4], kv[4];
        load4<VEC>(s.m + i, lane, have, km);
        load4<VEC>(s.v + i, lane, have, kv);
        const double dm = (double)s.m_scale[block + b] / kM, dv = (double)s.v_scale[block + b] / kV;
        float x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const double v2 = (double)(kv[e] * kv[e]);
            const int k2 = km[e] * km[e];
            x[e] = (float)(dm * (double)(km[e] < 0 ? -k2 : k2));
            y[e] = (float)(dv * (v2 * v2));
        }
        store4<VEC>(m + i, lane, have, x);
        store4<VEC>(v + i, lane, have, y);
    }
}

__global__ __launch_bounds__(kThreads) void values8_kernel(const Part *parts, States s, float *m,
                                                           float *v, int vec) {
    const Part p = parts[blockIdx.x];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    const uint32_t first = wave * kEach * kBlock;
    if (first >= p.count)
        return;
    if (vec && p.at % 4 == 0)
        values_blocks<true>(s, m, v, p.at + first, p.count - first, p.block + wave * kEach, lane);
    else
        values_blocks<false>(s, m, v, p.at + first, p.count - first, p.block + wave * kEach, lane);
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
    a.b1 = beta1 / kM;
    a.b2 = beta2 / kV;
    a.c1 = 1 - beta1;
    a.c2 = 1 - beta2;
    a.step = (float)(lr / (1 - std::pow(beta1, (double)step)));
    a.root = (float)(1 / std::sqrt(1 - std::pow(beta2, (double)step)));
    a.eps = (float)eps;
    a.keep = (float)(1 - lr * weight_decay);
    uintptr_t all = (uintptr_t)grad | (uintptr_t)copy;
    for (int i = 0; i < r.count; ++i)
        all |= (uintptr_t)r.w[i];
    a.vec = all % 16 == 0 && ((uintptr_t)m | (uintptr_t)v) % 4 == 0;
    const dim3 grid((uint32_t)h->parts.size()), block(kThreads);
    hipStream_t s = (hipStream_t)stream;
    auto go = [&](auto g) {
        using G = decltype(g);
        const bool half = !copy || copy_dtype == DDL_F16;
        return launch(r.count > 1 ? half ? adamw8_kernel<G, _Float16, true>
                                         : adamw8_kernel<G, __bf16, true>
                      : half      ? adamw8_kernel<G, _Float16, false>
                                  : adamw8_kernel<G, __bf16, false>,
                      grid, block, 0, s, a, r);
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
    const int vec = ((uintptr_t)m_out | (uintptr_t)v_out) % 16 == 0
                    && ((uintptr_t)m | (uintptr_t)v) % 4 == 0;
    const States st = {(int8_t *)m, (uint8_t *)v, (float *)m_scale, (float *)v_scale};
    return launch(values8_kernel, dim3((uint32_t)h->parts.size()), dim3(kThreads), 0,
                  (hipStream_t)stream, h->d_parts, st, m_out, v_out, vec);
}

}  // extern "C"
