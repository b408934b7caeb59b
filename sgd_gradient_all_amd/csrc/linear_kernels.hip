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
using gemm::u32x4;

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

// The activations are a good part of a tile's time (a wave's instruction takes
// 4 cycles for its 64 lanes, an exponential or reciprocal 16), so they are
// written with the hardware's 2^x and 1/x (each within 1 ulp of binary32;
// outputs are rounded to 11 bits at most) and fused multiply-adds.
__device__ __forceinline__ float fma(float a, float b, float c) {
    return __builtin_fmaf(a, b, c);
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanh = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// 1 / (1 + 2^-u)
__device__ __forceinline__ float sigmoid2(float u) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u));
}
// tanh's form of GELU is v sigmoid(2 sqrt(2/pi) (v + 0.044715 v^3))
__device__ __forceinline__ float tanh_argument(float v) {
    return v * fma(v * v, 0.044715f * kTanh * kLog2e, kTanh * kLog2e);
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
    case DDL_ACT_RELU: return v < 0.0f ? 0.0f : v;  // NaN stays NaN
    case DDL_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.7071067811865476f));
    case DDL_ACT_GELU_TANH: return v * sigmoid2(tanh_argument(v));
    case DDL_ACT_SILU: return v * sigmoid2(v * kLog2e);
    default: return v;
    }
}

__device__ __forceinline__ float act_slope(float v, int act) {
    switch (act) {
    case DDL_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
    case DDL_ACT_GELU:
        return fma(v * 0.3989422804014327f,
                   __builtin_amdgcn_exp2f(v * v * (-0.5f * kLog2e)),
                   fma(0.5f, erff(v * 0.7071067811865476f), 0.5f));
    case DDL_ACT_GELU_TANH: {
        const float s = sigmoid2(tanh_argument(v));
        const float d = fma(v * v, 3.0f * 0.044715f * kTanh, kTanh);
        return fma(v * d * s, 1.0f - s, s);
    }
    case DDL_ACT_SILU: {
        const float s = sigmoid2(v * kLog2e);
        return s * fma(v, 1.0f - s, 1.0f);
    }
    default: return 1.0f;
    }
}

// 8 elements as they lie; elements past `have` are 0.
// VEC: all of them at a 16-byte boundary.
template <bool VEC, class E>
__device__ __forceinline__ void load8(const E *p, uint32_t have, u32x4 (&out)[sizeof(E) / 2]) {
    constexpr int PARTS = sizeof(E) / 2;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
            out[i] = ((const u32x4 *)p)[i];
    } else {
        E t[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            t[i] = i < have ? p[i] : (E)0.0f;
        __builtin_memcpy(out, t, sizeof(t));
    }
}
template <class E>
__device__ __forceinline__ void widen8(const u32x4 (&in)[sizeof(E) / 2], float (&out)[8]) {
    E t[8];
    __builtin_memcpy(t, in, sizeof(t));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        out[i] = (float)t[i];
}
template <bool VEC, class E>
__device__ __forceinline__ void store8(E *p, uint32_t have, const float (&v)[8]) {
    constexpr int W = 16 / sizeof(E);
    typedef E V __attribute__((ext_vector_type(W)));
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 8; i += W) {
            V o;
#pragma unroll
            for (int e = 0; e < W; ++e)
                o[e] = (E)v[i + e];
            *(V *)(p + i) = o;
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            if (i < have)
                p[i] = (E)v[i];
    }
}

// What the epilogue reads for 8 results.
struct Fetched {
    u32x4 bias[1], residual[1], z_prev[1], old[1], old32[2];
};

template <class T, bool VEC>
__device__ __forceinline__ Fetched fetch8(const Epilogue &e, uint64_t m, uint64_t n) {
    using E = typename T::E;
    Fetched f;
    if (!VEC && (m >= e.m || n >= e.n))
        return f;
    const uint32_t have = !VEC && e.n - n < 8 ? (uint32_t)(e.n - n) : 8u;
    if (e.bias)
        load8<VEC>((const E *)e.bias + n, have, f.bias);
    if (e.residual)
        load8<VEC>((const E *)e.residual + m * e.ldr + n, have, f.residual);
    if (e.dz_prev)
        load8<VEC>((const E *)e.z_prev + m * e.ldzp + n, have, f.z_prev);
    if (e.add) {
        if (e.f32out)
            load8<VEC>((const float *)e.c + m * e.ldc + n, have, f.old32);
        else
            load8<VEC>((const E *)e.c + m * e.ldc + n, have, f.old);
    }
    return f;
}

// 8 consecutive results of row m from column n on.
// VEC: the 8 are inside C and every array's rows start at 16-byte boundaries.
template <class T, bool VEC>
__device__ __forceinline__ void finish8(const Epilogue &e, uint64_t m, uint64_t n, float (&v)[8],
                                        const Fetched &f) {
    using E = typename T::E;
    if (!VEC && (m >= e.m || n >= e.n))
        return;
    const uint32_t have = !VEC && e.n - n < 8 ? (uint32_t)(e.n - n) : 8u;
    float t[8];
    auto plus = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += t[i];
    };
    if (e.bias) {
        widen8<E>(f.bias, t);
        plus();
    }
    if (e.z)
        store8<VEC>((E *)e.z + m * e.ldz + n, have, v);
    if (e.act && !e.dz_prev) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = activate(v[i], e.act);
    }
    if (e.residual) {
        widen8<E>(f.residual, t);
        plus();
    }
    if (e.add) {
        if (e.f32out)
            widen8<float>(f.old32, t);
        else
            widen8<E>(f.old, t);
        plus();
    }
    if (e.f32out)
        store8<VEC>((float *)e.c + m * e.ldc + n, have, v);
    else
        store8<VEC>((E *)e.c + m * e.ldc + n, have, v);
    if (e.dz_prev) {
        widen8<E>(f.z_prev, t);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = v[i] * act_slope(t[i], e.act);
        store8<VEC>((E *)e.dz_prev + m * e.lddzp + n, have, t);
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
    const uint64_t m0 = g.a.row0, n0 = g.b.row0;
    const bool whole = m0 + Core::BM <= g.e.m && n0 + Core::BN <= g.e.n;
    auto nothing = [](uint32_t, uint32_t) { return 0; };
    if (g.splits > 1) {
        float *to = g.partial + ((uint64_t)s * g.e.m + m0) * g.e.n + n0;
        if (whole && g.e.n % 4 == 0)
            Core::each(acc, lds, nothing, [&](uint32_t mi, uint32_t ni, float (&v)[8], int) {
                store8<true>(to + mi * g.e.n + ni, 8, v);
            });
        else
            Core::template each<false, 1>(
                acc, lds, nothing, [&](uint32_t mi, uint32_t ni, float (&v)[8], int) {
                    if (m0 + mi < g.e.m && n0 + ni < g.e.n) {
                        const uint64_t left = g.e.n - n0 - ni;
                        store8<false>(to + mi * g.e.n + ni, left < 8 ? (uint32_t)left : 8u, v);
                    }
                });
    } else if (whole && g.e.vec) {
        Core::each(
            acc, lds,
            [&](uint32_t mi, uint32_t ni) { return fetch8<T, true>(g.e, m0 + mi, n0 + ni); },
            [&](uint32_t mi, uint32_t ni, float (&v)[8], const Fetched &f) {
                finish8<T, true>(g.e, m0 + mi, n0 + ni, v, f);
            });
    } else {
        Core::template each<false, 1>(
            acc, lds,
            [&](uint32_t mi, uint32_t ni) { return fetch8<T, false>(g.e, m0 + mi, n0 + ni); },
            [&](uint32_t mi, uint32_t ni, float (&v)[8], const Fetched &f) {
                finish8<T, false>(g.e, m0 + mi, n0 + ni, v, f);
            });
    }
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
    const Fetched f = vec && e.vec ? fetch8<T, true>(e, m, n) : fetch8<T, false>(e, m, n);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
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
    if (vec && e.vec)
        finish8<T, true>(e, m, n, v, f);
    else
        finish8<T, false>(e, m, n, v, f);
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
    const uint64_t kt = (k + 63) / 64;
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
int launch_tile(int tile, GemmArgs &g, uint64_t k, hipStream_t s) {
    auto go = [&](auto core) {
        using Core = decltype(core);
        g.kt = (uint32_t)((k + Core::BK - 1) / Core::BK);
        return launch<T, Core>(g, s);
    };
    if (tile == 0)
        return go(gemm::Core<T, 256, 256, 2, 4, 64, 2, TRA, TRB, STAGED>());
    if (tile == 1)
        return go(gemm::Core<T, 128, 128, 2, 2, 64, 2, TRA, TRB, STAGED>());
    return go(gemm::Core<T, 64, 64, 2, 2, 64, 3, TRA, TRB, STAGED>());
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
    g.splits = k ? c.splits : 0;
    g.partial = (float *)workspace;
    if (k) {
        // straight to LDS where every row of both starts on 16 bytes and the
        // contiguous extents are whole chunks
        const bool direct = aligned16(a.plane[0], a.ld, 2) && aligned16(b.plane[0], b.ld, 2)
                            && (TRA ? a.rows : k) % 8 == 0 && (TRB ? b.rows : k) % 8 == 0;
        const int rc = direct ? launch_tile<T, TRA, TRB, false>(c.tile, g, k, s)
                              : launch_tile<T, TRA, TRB, true>(c.tile, g, k, s);
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
