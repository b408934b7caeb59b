// adamw_kernels.hip -- the AdamW step over spans of flat buffers (gfx950).
//
//     m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//     w = (1 - lr decay) w - (lr / (1 - b1^t)) m / (sqrt(v / (1 - b2^t)) + eps)
//
// in binary32 (Loshchilov and Hutter's decoupled weight decay).  Every
// element is read and written once, so the step is bound by memory: with
// binary32 gradients 28 bytes an element (25557032 of them: 138 us, 5.2 TB/s).
// The spans are cut into chunks of
// kChunk elements that start on 16-byte boundaries of the buffers, one
// workgroup each, so that 107 short vectors and one long buffer are both one
// launch.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "../../include/ddl.h"
#include "optimizer_internal.h"

namespace ddl {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kChunk = 2048;  // 8 elements a lane

struct AdamArgs {
    const Chunk *chunks;
    const void *grad;
    float *m, *v, *w;
    void *copy;
    float b1, b2, c1, c2;    // c = 1 - b
    float step, root, eps;   // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    float keep;              // 1 - lr decay
    int vec;
};

struct Adam {
    float m, v, w;
};
__device__ __forceinline__ Adam adam1(const AdamArgs &a, float g, Adam s) {
    s.m = a.b1 * s.m + a.c1 * g;
    s.v = a.b2 * s.v + a.c2 * (g * g);
    s.w = a.keep * s.w - a.step * (s.m / (sqrtf(s.v) * a.root + a.eps));
    return s;
}

template <class G, class C>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamArgs a) {
    const Chunk c = a.chunks[blockIdx.x];
    const G *g = (const G *)a.grad + c.at;
    float *m = a.m + c.at, *v = a.v + c.at, *w = a.w + c.at;
    C *copy = a.copy ? (C *)a.copy + c.at : nullptr;
    typedef float V4 __attribute__((ext_vector_type(4)));
    typedef G G4 __attribute__((ext_vector_type(4)));
    typedef C C4 __attribute__((ext_vector_type(4)));
    uint32_t done = 0;
    if (a.vec && c.at % 8 == 0) {
        done = c.count & ~3u;
#pragma unroll
        for (uint32_t x = 0; x < kChunk; x += 4 * kThreads) {
            const uint32_t i = x + threadIdx.x * 4;
            if (i < done) {
                const G4 gv = *(const G4 *)(g + i);
                V4 mv = *(V4 *)(m + i), vv = *(V4 *)(v + i), wv = *(V4 *)(w + i);
                C4 cv;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Adam s = adam1(a, (float)gv[e], {mv[e], vv[e], wv[e]});
                    mv[e] = s.m;
                    vv[e] = s.v;
                    wv[e] = s.w;
                    cv[e] = (C)s.w;
                }
                *(V4 *)(m + i) = mv;
                *(V4 *)(v + i) = vv;
                *(V4 *)(w + i) = wv;
                if (copy)
                    *(C4 *)(copy + i) = cv;
            }
        }
    }
    for (uint32_t i = done + threadIdx.x; i < c.count; i += kThreads) {
        const Adam s = adam1(a, (float)g[i], {m[i], v[i], w[i]});
        m[i] = s.m;
        v[i] = s.v;
        w[i] = s.w;
        if (copy)
            copy[i] = (C)s.w;
    }
}

// The other replicas of each chunk, from replica 0: a second launch that reads
// the new weights back, 4 bytes a lane (ResNet-50's buffer in binary32: 138 us
// with one replica, 312 us with eight, 4.6 TB/s of its 56 bytes an element).
__global__ __launch_bounds__(kThreads) void replica_kernel(const Chunk *chunks, const float *w0,
                                                           Replicas r) {
    const Chunk c = chunks[blockIdx.x];
    for (uint32_t i = threadIdx.x; i < c.count; i += kThreads) {
        const float x = w0[c.at + i];
        for (int k = 1; k < r.count; ++k)
            r.w[k][c.at + i] = x;
    }
}

}  // namespace
}  // namespace ddl

using namespace ddl;

struct ddl_adamw_s {
    std::vector<Chunk> chunks;
    Handle dev;
    Chunk *d_chunks = nullptr;
};

extern "C" {

int ddl_adamw_create(ddl_adamw *out, const size_t *offsets, const size_t *counts, int nspans) {
    if (!out || (nspans > 0 && (!offsets || !counts)))
        return DDL_E_NULL;
    *out = nullptr;
    if (nspans < 0)
        return DDL_E_ARG;
    ddl_adamw h = nullptr;
    try {
        std::vector<Span> spans;
        for (int i = 0; i < nspans; ++i)
            spans.push_back({offsets[i], counts[i]});
        if (!disjoint(spans))
            return DDL_E_BUCKETS;
        h = new ddl_adamw_s;
        for (const Span &s : spans)
            cut_chunks(s, kChunk, h->chunks);
        if (h->chunks.size() > kMaxGrid) {
            delete h;
            return DDL_E_ARG;
        }
        register_handle(h);
    } catch (...) {
        delete h;
        return DDL_E_NOMEM;
    }
    *out = h;
    return DDL_OK;
}

int ddl_adamw_destroy(ddl_adamw h) {
    if (!h)
        return DDL_E_NULL;
    if (!unregister_handle(h))
        return DDL_E_ARG;
    h->dev.release(h->d_chunks);
    delete h;
    return DDL_OK;
}

int ddl_adamw_step(ddl_adamw h, const void *grad, int grad_dtype, float *m, float *v,
                   float *const *weights, int nweights, void *copy, int copy_dtype, double lr,
                   double beta1, double beta2, double eps, double weight_decay, long long step,
                   void *stream) {
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
    if (h->chunks.empty())
        return DDL_OK;
    Replicas r;
    int rc = take_replicas(weights, nweights, r);
    if (rc)
        return rc;
    if (!grad || !m || !v)
        return DDL_E_NULL;
    if (!aligned_to(grad, grad_dtype) || !aligned_to(m, DDL_F32) || !aligned_to(v, DDL_F32)
        || (copy && !aligned_to(copy, copy_dtype)))
        return DDL_E_ALIGN;
    rc = h->dev.bind((hipStream_t)stream, [&]() {
        return upload(h->chunks, &h->d_chunks);
    });
    if (rc)
        return rc;
    AdamArgs a;
    a.chunks = h->d_chunks;
    a.grad = grad;
    a.m = m;
    a.v = v;
    a.w = r.w[0];
    a.copy = copy;
    a.b1 = (float)beta1;
    a.b2 = (float)beta2;
    a.c1 = (float)(1 - beta1);
    a.c2 = (float)(1 - beta2);
    a.step = (float)(lr / (1 - std::pow(beta1, (double)step)));
    a.root = (float)(1 / std::sqrt(1 - std::pow(beta2, (double)step)));
    a.eps = (float)eps;
    a.keep = (float)(1 - lr * weight_decay);
    a.vec = !(((uintptr_t)grad | (uintptr_t)m | (uintptr_t)v | (uintptr_t)r.w[0]
               | (uintptr_t)copy) % 16);
    const dim3 grid((uint32_t)h->chunks.size()), block(kThreads);
    hipStream_t s = (hipStream_t)stream;
    auto go = [&](auto g) {
        using G = decltype(g);
        return launch(copy && copy_dtype == DDL_BF16 ? adamw_kernel<G, __bf16>
                                                     : adamw_kernel<G, _Float16>,
                      grid, block, 0, s, a);
    };
    rc = grad_dtype == DDL_F32   ? go(float())
         : grad_dtype == DDL_F16 ? go(_Float16())
                                 : go(__bf16());
    return rc || r.count == 1
               ? rc
               : launch(replica_kernel, grid, block, 0, s, h->d_chunks, r.w[0], r);
}

}  // extern "C"
