// linear_kernels.hip -- the linear layer of a training step (gfx950):
//
//     forward          z = x w^T + bias,  y = act(z) + residual
//     input gradient   dx = dz w + residual,  dz_prev = dx act'(z_prev)
//     weight gradient  dw = dz^T x,  db = the column sums of dz  (or added)
//
// with x m x k, w n x k, dz m x n.  All three are the product of gemm_core.h
// with both operands as they lie in memory: x and w with k contiguous; dz
// with k contiguous against w row by row; dz and x both row by row.  Bias,
// activation, residual and the second output ride in the epilogue on the
// binary32 sums; every output is rounded once.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>

#include "../../include/ddl.h"
#include "gemm_core.h"

namespace ddl {
namespace {

using gemm::Bfloat;
using gemm::f32x4;
using gemm::Half;
using gemm::Operand;

// The epilogue of C[m, n] (its own m and n, not the layer's).
struct Epilogue {
    uint64_t m, n;
    void *c;  // T, or binary32 (f32out)
    uint64_t ldc;
    const void *bias;  // T[n] or null
    const void *residual;
    uint64_t ldr;
    void *z;  // the sum before act and residual, or null
    uint64_t ldz;
    const void *z_prev;  // input gradient: the activation's argument
    uint64_t ldzp;
    void *dz_prev;
    uint64_t lddzp;
    int act;
    int f32out, add;
    int vec;  // rows of every array above start on 16-byte boundaries
};

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + __expf(-v)); }

constexpr float kGelu = 0.7978845608028654f;  // sqrt(2 / pi)

// __expf (the hardware's 2^x of a scaled argument, 2 ulp near 0 and relative
// error |x| 2^-24 far out) is exact to well under half a step of the 16-bit
// outputs that take it.
__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
    case DDL_ACT_RELU: return v < 0.0f ? 0.0f : v;  // NaN stays NaN
    case DDL_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.7071067811865476f));
    case DDL_ACT_GELU_TANH:
        return v * sigmoid(2.0f * kGelu * (v + 0.044715f * v * v * v));
    case DDL_ACT_SILU: return v * sigmoid(v);
    default: return v;
    }
}

__device__ __forceinline__ float act_slope(float v, int act) {
    switch (act) {
    case DDL_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
    case DDL_ACT_GELU:
        return 0.5f * (1.0f + erff(v * 0.7071067811865476f))
               + v * __expf(-0.5f * v * v) * 0.3989422804014327f;
    case DDL_ACT_GELU_TANH: {
        const float s = sigmoid(2.0f * kGelu * (v + 0.044715f * v * v * v));
        return s + v * s * (1.0f - s) * (2.0f * kGelu) * (1.0f + 0.134145f * v * v);
    }
    case DDL_ACT_SILU: {
        const float s = sigmoid(v);
        return s * (1.0f + v * (1.0f - s));
    }
    default: return 1.0f;
    }
}

template <class E, int N>
__device__ __forceinline__ void load_n(const E *p, uint32_t have, bool vec, float (&out)[N]) {
    typedef E V __attribute__((ext_vector_type(8)));
    if (vec && have >= N) {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const V v = *(const V *)(p + i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                out[i + e] = (float)v[e];
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < N; ++i)
            out[i] = i < have ? (float)p[i] : 0.0f;
    }
}
template <class E, int N>
__device__ __forceinline__ void store_n(E *p, uint32_t have, bool vec, const float (&v)[N]) {
    constexpr int W = 16 / sizeof(E);
    typedef E V __attribute__((ext_vector_type(W)));
    if (vec && have >= N) {
#pragma unroll
        for (int i = 0; i < N; i += W) {
            V o;
#pragma unroll
            for (int e = 0; e < W; ++e)
                o[e] = (E)v[i + e];
            *(V *)(p + i) = o;
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < N; ++i)
            if (i < have)
                p[i] = (E)v[i];
    }
}

// N consecutive results of row m from column n on; n < e.n.
template <class T, int N>
__device__ __forceinline__ void finish(const Epilogue &e, uint64_t m, uint64_t n, float (&v)[N]) {
    using E = typename T::E;
    const uint32_t have = e.n - n < (uint64_t)N ? (uint32_t)(e.n - n) : (uint32_t)N;
    const bool vec = e.vec;
    float t[N];
    if (e.bias) {
        load_n<E, N>((const E *)e.bias + n, have, vec, t);
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += t[i];
    }
    if (e.z)
        store_n<E, N>((E *)e.z + m * e.ldz + n, have, vec, v);
    if (e.act && !e.dz_prev) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = activate(v[i], e.act);
    }
    if (e.residual) {
        load_n<E, N>((const E *)e.residual + m * e.ldr + n, have, vec, t);
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += t[i];
    }
    if (e.f32out) {
        float *c = (float *)e.c + m * e.ldc + n;
        if (e.add) {
#pragma unroll
            for (uint32_t i = 0; i < N; ++i)
                t[i] = 0.0f;
            if (vec && have >= N) {
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    const f32x4 o = *(const f32x4 *)(c + i);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        t[i + x] = o[x];
                }
            } else {
#pragma unroll
                for (uint32_t i = 0; i < N; ++i)
                    t[i] = i < have ? c[i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += t[i];
        }
        store_n<float, N>(c, have, vec, v);
    } else {
        E *c = (E *)e.c + m * e.ldc + n;
        if (e.add) {
            load_n<E, N>(c, have, vec, t);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += t[i];
        }
        store_n<E, N>(c, have, vec, v);
    }
    if (e.dz_prev) {
        load_n<E, N>((const E *)e.z_prev + m * e.ldzp + n, have, vec, t);
#pragma unroll
        for (int i = 0; i < N; ++i)
            t[i] = v[i] * act_slope(t[i], e.act);
        store_n<E, N>((E *)e.dz_prev + m * e.lddzp + n, have, vec, t);
    }
}

struct GemmArgs {
    Operand a, b;
    uint32_t tm, tn;      // tiles of C
    uint32_t kt, splits;  // k tiles; parts that they are dealt to
    float *partial;       // splits > 1: [splits][m][n]
    Epilogue e;
};

constexpr uint32_t kDies = 8;  // accelerator dies, each with an L2 of its own

// The tile of workgroup `id`: workgroups go round the dies, so each die is
// given a run of consecutive tiles, which walk C in bands of 8 tiles of m;
// the band's rows of A and the columns of B in flight then stay in its L2.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tm, uint32_t tn, uint32_t &i,
                                        uint32_t &j) {
    const uint32_t all = tm * tn, per = all / kDies, more = all % kDies;
    const uint32_t die = id % kDies, at = id / kDies;
    id = die * per + (die < more ? die : more) + at;
    constexpr uint32_t kBand = 8;
    const uint32_t band = id / (kBand * tn), first = band * kBand;
    const uint32_t height = tm - first < kBand ? tm - first : kBand;
    const uint32_t in = id - band * kBand * tn;
    i = first + in % height;
    j = in / height;
}

template <class T, class Core>
__global__ __launch_bounds__(Core::THREADS) void linear_kernel(GemmArgs g) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    uint32_t ti, tj;
    tile_of(blockIdx.x, g.tm, g.tn, ti, tj);
    g.a.row0 = ti * Core::BM;
    g.b.row0 = tj * Core::BN;
    const uint32_t s = blockIdx.y;
    const uint32_t t0 = (uint32_t)((uint64_t)g.kt * s / g.splits);
    const uint32_t t1 = (uint32_t)((uint64_t)g.kt * (s + 1) / g.splits);
    f32x4 acc[Core::FM][Core::FN] = {};
    Core::run(g.a, g.b, t0, t1, 0, lds, acc);
    Core::each(acc, lds, [&](uint32_t mi, uint32_t ni, float (&v)[8]) {
        const uint64_t m = (uint64_t)g.a.row0 + mi, n = (uint64_t)g.b.row0 + ni;
        if (m >= g.e.m || n >= g.e.n)
            return;
        if (g.splits > 1) {
            const uint64_t left = g.e.n - n;
            store_n<float, 8>(g.partial + ((uint64_t)s * g.e.m + m) * g.e.n + n,
                              left < 8 ? (uint32_t)left : 8, g.e.n % 4 == 0, v);
        } else {
            finish<T, 8>(g.e, m, n, v);
        }
    });
}

// The sums of the parts, in their order, and the epilogue.  8 columns a lane.
template <class T>
__global__ __launch_bounds__(256) void linear_join(Epilogue e, const float *partial,
                                                   uint32_t splits) {
    const uint64_t groups = (e.n + 7) / 8;
    const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= groups * e.m)
        return;
    const uint64_t m = id / groups, n = id % groups * 8;
    const bool vec = e.n % 8 == 0;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t s = 0; s < splits; ++s) {
        const float *p = partial + ((uint64_t)s * e.m + m) * e.n + n;
        if (vec) {
            const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += a[i];
                v[4 + i] += b[i];
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i)
                if (n + i < e.n)
                    v[i] += p[i];
        }
    }
    finish<T, 8>(e, m, n, v);
}

// Column sums of dz[m, n]: workgroup (c, s) sums columns 512 c .. + 512 over
// the rows of slice s, its four waves every fourth row each.
template <class T>
__global__ __launch_bounds__(256) void column_sums(const typename T::E *dz, uint64_t ld,
                                                   uint64_t m, uint64_t n, uint32_t slices,
                                                   float *partial) {
    using E = typename T::E;
    __shared__ float sum[4][512];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint64_t col = (uint64_t)blockIdx.x * 512 + lane * 8;
    const uint64_t r0 = m * blockIdx.y / slices, r1 = m * (blockIdx.y + 1) / slices;
    const uint32_t have = col >= n ? 0 : n - col < 8 ? (uint32_t)(n - col) : 8;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (have == 8) {
#pragma unroll 4
        for (uint64_t r = r0 + wave; r < r1; r += 4) {
            E h[8];
            __builtin_memcpy(h, dz + r * ld + col, 16);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += (float)h[i];
        }
    } else if (have) {
        for (uint64_t r = r0 + wave; r < r1; r += 4)
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i)
                if (i < have)
                    v[i] += (float)dz[r * ld + col + i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sum[wave][lane * 8 + i] = v[i];
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < 512; c += 256) {
        const uint64_t at = (uint64_t)blockIdx.x * 512 + c;
        if (at < n)
            partial[(uint64_t)blockIdx.y * n + at] = sum[0][c] + sum[1][c] + sum[2][c] + sum[3][c];
    }
}

template <class O>
__global__ __launch_bounds__(256) void column_join(const float *partial, uint32_t slices,
                                                   uint64_t n, O *db, int add) {
    const uint64_t c = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= n)
        return;
    float v = 0.0f;
    for (uint32_t s = 0; s < slices; ++s)
        v += partial[s * n + c];
    db[c] = (O)(add ? (float)db[c] + v : v);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

enum { kForward = DDL_LINEAR_FORWARD, kDgrad = DDL_LINEAR_DGRAD, kWgrad = DDL_LINEAR_WGRAD };
constexpr size_t kMaxExtent = 1u << 22;   // columns and row strides (32-bit tile offsets)
constexpr size_t kMaxRows = 1u << 30;

// How a product is cut: tile size (0: 256 x 256, 1: 128 x 128, 2: 64 x 64)
// and parts of k.
struct Cut {
    int tile;
    uint32_t splits;
};
constexpr uint32_t kTile[3] = {256, 128, 64};

uint64_t tiles(uint64_t m, uint64_t n, int t) {
    return ((m + kTile[t] - 1) / kTile[t]) * ((n + kTile[t] - 1) / kTile[t]);
}

Cut cut(uint64_t m, uint64_t n, uint64_t k) {
    const uint64_t kt = (k + gemm::kBK - 1) / gemm::kBK;
    Cut c{0, 1};
    if (tiles(m, n, 0) < 192)
        c.tile = tiles(m, n, 1) >= 192 ? 1 : 2;
    const uint64_t t = tiles(m, n, c.tile);
    if (t < 256 && kt >= 16)
        c.splits = (uint32_t)std::min<uint64_t>(std::min<uint64_t>(512 / t, kt / 8), 64);
    c.splits = std::max(c.splits, 1u);
    return c;
}

uint32_t db_slices(uint64_t m) {
    return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(m / 64, 64));
}

// C's shape and the length of the sums, by operation.
void product_shape(int op, size_t m, size_t n, size_t k, size_t &cm, size_t &cn, size_t &ck) {
    cm = op == kWgrad ? n : m;
    cn = op == kForward ? n : k;
    ck = op == kForward ? k : op == kDgrad ? n : m;
}

size_t partial_bytes(int op, size_t m, size_t n, size_t k) {
    size_t cm, cn, ck;
    product_shape(op, m, n, k, cm, cn, ck);
    if (!cm || !cn)
        return 0;
    const Cut c = cut(cm, cn, ck);
    return c.splits > 1 ? (c.splits * cm * cn * 4 + 255) / 256 * 256 : 0;
}

size_t workspace_bytes(int op, size_t m, size_t n, size_t k) {
    return partial_bytes(op, m, n, k) + (op == kWgrad ? db_slices(m) * n * 4 : 0);
}

bool sizes_ok(size_t m, size_t n, size_t k) {
    return m <= kMaxRows && n <= kMaxExtent && k <= kMaxExtent;
}

bool aligned16(const void *p, size_t ld, size_t esz) {
    return ((uintptr_t)p | ld * esz) % 16 == 0;
}

template <class T, class Core>
int launch(const GemmArgs &g, hipStream_t stream) {
    const void *f = (const void *)&linear_kernel<T, Core>;
    if (Core::LDS > 65536
        && hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, Core::LDS)
               != hipSuccess)
        return DDL_E_HIP;
    hipLaunchKernelGGL((linear_kernel<T, Core>), dim3(g.tm * g.tn, g.splits),
                       dim3(Core::THREADS), Core::LDS, stream, g);
    return hipGetLastError() == hipSuccess ? DDL_OK : DDL_E_HIP;
}

template <class T, bool TRA, bool TRB, bool STAGED>
int launch_tile(int tile, const GemmArgs &g, hipStream_t s) {
    if (tile == 0)
        return launch<T, gemm::Core<T, 256, 256, 2, 4, TRA, TRB, STAGED>>(g, s);
    if (tile == 1)
        return launch<T, gemm::Core<T, 128, 128, 2, 2, TRA, TRB, STAGED>>(g, s);
    return launch<T, gemm::Core<T, 64, 64, 2, 2, TRA, TRB, STAGED>>(g, s);
}

template <class T, bool TRA, bool TRB>
int product(const Operand &a, const Operand &b, const Epilogue &e, uint64_t k, void *workspace,
            hipStream_t s) {
    GemmArgs g;
    g.a = a;
    g.b = b;
    g.e = e;
    const Cut c = cut(e.m, e.n, k);
    g.tm = (uint32_t)((e.m + kTile[c.tile] - 1) / kTile[c.tile]);
    g.tn = (uint32_t)((e.n + kTile[c.tile] - 1) / kTile[c.tile]);
    g.kt = (uint32_t)((k + gemm::kBK - 1) / gemm::kBK);
    g.splits = g.kt ? c.splits : 0;
    g.partial = (float *)workspace;
    if (g.kt) {
        // straight to LDS where every row of both starts on 16 bytes and the
        // contiguous extents are whole chunks
        const bool direct = aligned16(a.plane[0], a.ld, 2) && aligned16(b.plane[0], b.ld, 2)
                            && (TRA ? a.rows : k) % 8 == 0 && (TRB ? b.rows : k) % 8 == 0;
        const int rc = direct ? launch_tile<T, TRA, TRB, false>(c.tile, g, s)
                              : launch_tile<T, TRA, TRB, true>(c.tile, g, s);
        if (rc || g.splits == 1)
            return rc;
    }
    const uint64_t lanes = (e.n + 7) / 8 * e.m;
    hipLaunchKernelGGL(linear_join<T>, dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, s, e,
                       g.partial, g.splits);
    return hipGetLastError() == hipSuccess ? DDL_OK : DDL_E_HIP;
}

bool row_ok(const void *p, size_t ld, size_t cols, size_t rows) {
    return !p || (ld <= kMaxExtent && (ld >= cols || rows <= 1));
}

// Even addresses: a 16-bit element does not straddle its own size.
bool element_ok(const void *p, size_t esz) { return (uintptr_t)p % esz == 0; }

int check_workspace(int op, size_t m, size_t n, size_t k, const void *ws, size_t bytes) {
    const size_t need = workspace_bytes(op, m, n, k);
    if (!need)
        return DDL_OK;
    if (!ws)
        return DDL_E_NULL;
    if ((uintptr_t)ws % 16)
        return DDL_E_ALIGN;
    return bytes < need ? DDL_E_SCRATCH : DDL_OK;
}

Operand operand(const void *p, size_t ld, size_t rows, size_t k) {
    Operand o;
    o.plane[0] = o.plane[1] = (const uint16_t *)p;
    o.ld = ld;
    o.rows = (uint32_t)rows;
    o.row0 = 0;
    o.k = k;
    return o;
}

bool act_ok(int act) { return act >= DDL_ACT_NONE && act <= DDL_ACT_SILU; }

}  // namespace
}  // namespace ddl

using namespace ddl;

extern "C" {

int ddl_linear_workspace(int op, size_t m, size_t n, size_t k, size_t *bytes) {
    if (!bytes)
        return DDL_E_NULL;
    if ((op != kForward && op != kDgrad && op != kWgrad) || !sizes_ok(m, n, k))
        return DDL_E_ARG;
    *bytes = workspace_bytes(op, m, n, k);
    return DDL_OK;
}

int ddl_linear(const ddl_linear_args *a, void *workspace, size_t workspace_bytes, void *stream) {
    if (!a)
        return DDL_E_NULL;
    const size_t m = a->m, n = a->n, k = a->k;
    if ((a->dtype != DDL_F16 && a->dtype != DDL_BF16) || !act_ok(a->act) || !sizes_ok(m, n, k))
        return DDL_E_ARG;
    if (!m || !n)
        return DDL_OK;
    if (!a->y || (k && (!a->x || !a->w)))
        return DDL_E_NULL;
    if (!row_ok(a->x, a->ldx, k, m) || !row_ok(a->w, a->ldw, k, n) || !row_ok(a->y, a->ldy, n, m)
        || !row_ok(a->residual, a->ldr, n, m) || !row_ok(a->z, a->ldz, n, m))
        return DDL_E_ARG;
    for (const void *p : {a->x, a->w, (const void *)a->y, a->bias, a->residual,
                          (const void *)a->z})
        if (!element_ok(p, 2))
            return DDL_E_ALIGN;
    const int rc = check_workspace(kForward, m, n, k, workspace, workspace_bytes);
    if (rc)
        return rc;
    Epilogue e = {};
    e.m = m;
    e.n = n;
    e.c = a->y;
    e.ldc = a->ldy;
    e.bias = a->bias;
    e.residual = a->residual;
    e.ldr = a->ldr;
    e.z = a->z;
    e.ldz = a->ldz;
    e.act = a->act;
    e.vec = aligned16(a->y, a->ldy, 2) && aligned16(a->bias, 0, 2)
            && (!a->residual || aligned16(a->residual, a->ldr, 2))
            && (!a->z || aligned16(a->z, a->ldz, 2));
    const Operand x = operand(a->x, a->ldx, m, k), w = operand(a->w, a->ldw, n, k);
    return a->dtype == DDL_F16
               ? product<Half, false, false>(x, w, e, k, workspace, (hipStream_t)stream)
               : product<Bfloat, false, false>(x, w, e, k, workspace, (hipStream_t)stream);
}

int ddl_linear_dgrad(const ddl_dgrad_args *a, void *workspace, size_t workspace_bytes,
                     void *stream) {
    if (!a)
        return DDL_E_NULL;
    const size_t m = a->m, n = a->n, k = a->k;
    if ((a->dtype != DDL_F16 && a->dtype != DDL_BF16) || !act_ok(a->act) || !sizes_ok(m, n, k))
        return DDL_E_ARG;
    if (!m || !k)
        return DDL_OK;
    if (!a->dx || (n && (!a->dz || !a->w)))
        return DDL_E_NULL;
    if (!a->z_prev != !a->dz_prev)  // both or neither
        return DDL_E_NULL;
    if (!a->dz_prev && a->act != DDL_ACT_NONE)
        return DDL_E_NULL;
    if (!row_ok(a->dz, a->lddz, n, m) || !row_ok(a->w, a->ldw, k, n)
        || !row_ok(a->dx, a->lddx, k, m) || !row_ok(a->residual, a->ldr, k, m)
        || !row_ok(a->z_prev, a->ldz_prev, k, m) || !row_ok(a->dz_prev, a->lddz_prev, k, m))
        return DDL_E_ARG;
    for (const void *p : {a->dz, a->w, (const void *)a->dx, a->residual, a->z_prev,
                          (const void *)a->dz_prev})
        if (!element_ok(p, 2))
            return DDL_E_ALIGN;
    const int rc = check_workspace(kDgrad, m, n, k, workspace, workspace_bytes);
    if (rc)
        return rc;
    Epilogue e = {};
    e.m = m;
    e.n = k;
    e.c = a->dx;
    e.ldc = a->lddx;
    e.residual = a->residual;
    e.ldr = a->ldr;
    e.act = a->act;
    e.z_prev = a->z_prev;
    e.ldzp = a->ldz_prev;
    e.dz_prev = a->dz_prev;
    e.lddzp = a->lddz_prev;
    e.vec = aligned16(a->dx, a->lddx, 2) && (!a->residual || aligned16(a->residual, a->ldr, 2))
            && (!a->z_prev
                || (aligned16(a->z_prev, a->ldz_prev, 2)
                    && aligned16(a->dz_prev, a->lddz_prev, 2)));
    const Operand dz = operand(a->dz, a->lddz, m, n), w = operand(a->w, a->ldw, k, n);
    return a->dtype == DDL_F16
               ? product<Half, false, true>(dz, w, e, n, workspace, (hipStream_t)stream)
               : product<Bfloat, false, true>(dz, w, e, n, workspace, (hipStream_t)stream);
}

}  // extern "C"

namespace ddl {
namespace {

template <class T>
int weight_gradient(const ddl_wgrad_args *a, uint8_t *ws, hipStream_t s) {
    using E = typename T::E;
    const size_t m = a->m, n = a->n, k = a->k;
    const bool f32 = a->out_dtype == DDL_F32;
    if (a->db && n) {
        float *partial = (float *)(ws + partial_bytes(kWgrad, m, n, k));
        const uint32_t slices = db_slices(m);
        hipLaunchKernelGGL(column_sums<T>, dim3((uint32_t)((n + 511) / 512), slices), dim3(256),
                           0, s, (const E *)a->dz, a->lddz, m, n, slices, partial);
        const dim3 grid((uint32_t)((n + 255) / 256));
        if (f32)
            hipLaunchKernelGGL(column_join<float>, grid, dim3(256), 0, s, partial, slices, n,
                               (float *)a->db, a->accumulate);
        else
            hipLaunchKernelGGL(column_join<E>, grid, dim3(256), 0, s, partial, slices, n,
                               (E *)a->db, a->accumulate);
        if (hipGetLastError() != hipSuccess)
            return DDL_E_HIP;
    }
    if (!n || !k)
        return DDL_OK;
    Epilogue e = {};
    e.m = n;
    e.n = k;
    e.c = a->dw;
    e.ldc = a->lddw;
    e.f32out = f32;
    e.add = a->accumulate;
    e.vec = aligned16(a->dw, a->lddw, f32 ? 4 : 2);
    return product<T, true, true>(operand(a->dz, a->lddz, n, m), operand(a->x, a->ldx, k, m), e,
                                  m, ws, s);
}

}  // namespace
}  // namespace ddl

extern "C" int ddl_linear_wgrad(const ddl_wgrad_args *a, void *workspace, size_t workspace_bytes,
                                void *stream) {
    if (!a)
        return DDL_E_NULL;
    const size_t m = a->m, n = a->n, k = a->k;
    if ((a->dtype != DDL_F16 && a->dtype != DDL_BF16)
        || (a->out_dtype != DDL_F32 && a->out_dtype != a->dtype)
        || (a->accumulate != 0 && a->accumulate != 1) || !sizes_ok(m, n, k))
        return DDL_E_ARG;
    if (!n)
        return DDL_OK;
    if ((k && !a->dw) || (m && (!a->dz || (k && !a->x))))
        return DDL_E_NULL;
    if (!row_ok(a->dz, a->lddz, n, m) || !row_ok(a->x, a->ldx, k, m)
        || !row_ok(a->dw, a->lddw, k, n))
        return DDL_E_ARG;
    const size_t esz = a->out_dtype == DDL_F32 ? 4 : 2;
    if (!element_ok(a->dz, 2) || !element_ok(a->x, 2) || !element_ok(a->dw, esz)
        || !element_ok(a->db, esz))
        return DDL_E_ALIGN;
    const int rc = check_workspace(kWgrad, m, n, k, workspace, workspace_bytes);
    if (rc)
        return rc;
    return a->dtype == DDL_F16
               ? weight_gradient<Half>(a, (uint8_t *)workspace, (hipStream_t)stream)
               : weight_gradient<Bfloat>(a, (uint8_t *)workspace, (hipStream_t)stream);
}
