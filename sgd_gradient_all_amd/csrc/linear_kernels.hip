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
#include "hip_call.h"
#include "product_parts.h"

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

// Phi(v) by erfc: 1 + erf cancels in the left tail (4% off at -5), though it is
// shorter (8192 x 16384 x 4096 in bfloat16: 1107 us by erfc, 1078 by erf).
__device__ __forceinline__ float normal_cdf(float v) {
    return 0.5f * erfcf(v * -0.7071067811865476f);
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
    case DDL_ACT_RELU: return v < 0.0f ? 0.0f : v;  // NaN stays NaN
    case DDL_ACT_GELU: return v * normal_cdf(v);
    case DDL_ACT_GELU_TANH: return v * sigmoid2(tanh_argument(v));
    case DDL_ACT_SILU: return v * sigmoid2(v * kLog2e);
    default: return v;
    }
}

// Past |v| = 128 every slope is 0 or 1 in binary32; farther out, infinities
// included, its terms pass binary32's range and meet zeros (inf 0 is NaN), so
// the argument stops there.  NaN stays NaN.
__device__ __forceinline__ float act_slope(float v, int act) {
    v = v > 128.0f ? 128.0f : v < -128.0f ? -128.0f : v;
    switch (act) {
    case DDL_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
    case DDL_ACT_GELU:
        return fma(v * 0.3989422804014327f,
                   __builtin_amdgcn_exp2f(v * v * (-0.5f * kLog2e)),
                   normal_cdf(v));
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

// What the epilogue reads for 8 results.
struct Fetched {
    u32x4 bias[1], residual[1], z_prev[1], old[1], old32[2];
};

template <class T, bool VEC>
__device__ __forceinline__ Fetched fetch8(const Epilogue &e, uint64_t m, uint64_t n) {
    using E = typename T::E;
    Fetched f;
    if (m >= e.m || n >= e.n)
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
// VEC: all 8 are inside C or none, and every array's rows start at 16-byte
// boundaries.
template <class T, bool VEC>
__device__ __forceinline__ void finish8(const Epilogue &e, uint64_t m, uint64_t n, float (&v)[8],
                                        const Fetched &f) {
    using E = typename T::E;
    if (m >= e.m || n >= e.n)
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
    // every 8 columns of the tile lie inside C or outside
    const bool whole = g.e.n % 8 == 0 || n0 + Core::BN <= g.e.n;
    auto nothing = [](uint32_t, uint32_t) { return 0; };
    if (g.splits > 1) {
        float *to = g.partial + ((uint64_t)s * g.e.m + m0) * g.e.n + n0;
        if (whole && g.e.n % 4 == 0)
            Core::each(acc, lds, nothing, [&](uint32_t mi, uint32_t ni, float (&v)[8], int) {
                if (m0 + mi < g.e.m && n0 + ni < g.e.n)
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

// 8 columns of linear_join.
template <class T>
__device__ __forceinline__ void join8(const Epilogue &e, const float *partial, uint32_t splits,
                                      uint64_t m, uint64_t n) {
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

// The sums of the parts (none: empty sums), in their order, and the epilogue.
// 8 columns a lane, and more than once only past kJoinLanes (empty sums of
// very large outputs).
constexpr uint64_t kJoinLanes = 1u << 31;  // a launch takes fewer than 2^32

template <class T>
__global__ __launch_bounds__(256) void linear_join(Epilogue e, const float *partial,
                                                   uint32_t splits) {
    const uint64_t groups = (e.n + 7) / 8;
    for (uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x; id < groups * e.m;
         id += kJoinLanes)
        join8<T>(e, partial, splits, id / groups, id % groups * 8);
}

// A few rows (a decoded token, or up to 16): the weights are read once and
// bound the time, so every lane loads them straight into the matrix
// instruction's registers, without LDS.  A workgroup of 8 waves takes 16
// columns, each wave an eighth of k; the waves' sums are added in their order.
constexpr int kSkinnyWaves = 8;
constexpr uint64_t kSkinnyRows = 16;

template <class T>
__global__ __launch_bounds__(kSkinnyWaves * 64) void skinny_kernel(Operand x, Operand w,
                                                                   Epilogue e) {
    __shared__ f32x4 sums[kSkinnyWaves][16][5];  // [wave][m][n / 4], a chunk of padding
    const uint32_t l = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = l & 15u, g = l >> 4;
    const uint32_t n0 = blockIdx.x * 16;
    const uint32_t steps = (uint32_t)((w.k + 31) / 32);
    const uint32_t s0 = steps * wave / kSkinnyWaves, s1 = steps * (wave + 1) / kSkinnyWaves;
    // rows past the end repeat the last one; their results are not stored
    const uint32_t rw = n0 + r < w.rows ? n0 + r : w.rows - 1, rx = r < x.rows ? r : x.rows - 1;
    const uint16_t *pw = w.plane[0] + (uint64_t)rw * w.ld + g * 8;
    const uint16_t *px = x.plane[0] + (uint64_t)rx * x.ld + g * 8;
    f32x4 acc = {0, 0, 0, 0};
    constexpr uint32_t U = 8;
    uint32_t s = s0;
    for (; s + U <= s1 && (uint64_t)(s + U) * 32 <= w.k; s += U) {
        gemm::s16x8 a[U], b[U];
#pragma unroll
        for (uint32_t i = 0; i < U; ++i) {
            b[i] = *(const gemm::s16x8 *)(pw + (uint64_t)(s + i) * 32);
            a[i] = *(const gemm::s16x8 *)(px + (uint64_t)(s + i) * 32);
        }
#pragma unroll
        for (uint32_t i = 0; i < U; ++i)
            acc = T::mfma(b[i], a[i], acc);
    }
    for (; s < s1; ++s) {
        gemm::s16x8 a = {}, b = {};
        if ((uint64_t)s * 32 + g * 8 < w.k) {  // k is a multiple of 8
            b = *(const gemm::s16x8 *)(pw + (uint64_t)s * 32);
            a = *(const gemm::s16x8 *)(px + (uint64_t)s * 32);
        }
        acc = T::mfma(b, a, acc);
    }
    sums[wave][r][g] = acc;
    __syncthreads();
    const uint32_t m = threadIdx.x >> 1, h = threadIdx.x & 1u;
    if (threadIdx.x >= 32 || m >= e.m || n0 + h * 8 >= e.n)
        return;
    const bool vec = e.vec && n0 + h * 8 + 8 <= e.n;
    const Fetched f = vec ? fetch8<T, true>(e, m, n0 + h * 8) : fetch8<T, false>(e, m, n0 + h * 8);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < kSkinnyWaves; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += sums[q][m][h * 2 + i / 4][i % 4];
    if (vec)
        finish8<T, true>(e, m, n0 + h * 8, v, f);
    else
        finish8<T, false>(e, m, n0 + h * 8, v, f);
}

// Column sums of dz[m, n]: workgroup (c, s) sums 64 columns over the rows of
// slice s, 8 lanes by 32 row groups.  One slice writes db itself, several
// leave their sums to column_join.
template <class T, class O>
__global__ __launch_bounds__(256) void column_sums(const typename T::E *dz, uint64_t ld,
                                                   uint64_t m, uint64_t n, uint32_t slices,
                                                   float *partial, O *db, int add) {
    using E = typename T::E;
    __shared__ float sum[32][65];
    const uint32_t lane = threadIdx.x & 7u, group = threadIdx.x >> 3;
    const uint64_t first = (uint64_t)blockIdx.x * 64, col = first + lane * 8;
    const uint64_t r0 = m * blockIdx.y / slices, r1 = m * (blockIdx.y + 1) / slices;
    const uint32_t have = col >= n ? 0 : n - col < 8 ? (uint32_t)(n - col) : 8;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (have == 8) {
#pragma unroll 8
        for (uint64_t r = r0 + group; r < r1; r += 32) {
            E h[8];
            __builtin_memcpy(h, dz + r * ld + col, 16);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += (float)h[i];
        }
    } else if (have) {
        for (uint64_t r = r0 + group; r < r1; r += 32)
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i)
                if (i < have)
                    v[i] += (float)dz[r * ld + col + i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sum[group][lane * 8 + i] = v[i];
    __syncthreads();
    const uint64_t at = first + threadIdx.x;
    if (threadIdx.x >= 64 || at >= n)
        return;
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q)
        t += sum[q][threadIdx.x];
    if (slices > 1)
        partial[(uint64_t)blockIdx.y * n + at] = t;
    else
        db[at] = (O)(add ? (float)db[at] + t : t);
}

template <class O>
__global__ __launch_bounds__(256) void column_join(const float *partial, uint32_t slices,
                                                   uint64_t n, O *db, int add) {
    const uint64_t c = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= n)
        return;
    float v = 0.0f;
#pragma unroll 8
    for (uint32_t s = 0; s < slices; ++s)
        v += partial[s * n + c];
    db[c] = (O)(add ? (float)db[c] + v : v);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

enum { kForward = DDL_LINEAR_FORWARD, kDgrad = DDL_LINEAR_DGRAD, kWgrad = DDL_LINEAR_WGRAD };
constexpr size_t kMaxRows = 1u << 30;

// Slices of db's sums, of 512 rows and more: from 1024 rows on several
// workgroups for 64 columns and a launch that joins them (the weight gradient
// of 1024 x 1024 x 1024: 22.3 us, with one workgroup 26.2; of 2048 x 4096 x
// 1024: 52.3 and 65.6 us).
uint32_t db_slices(uint64_t m) {
    return (uint32_t)std::min<uint64_t>(std::max<uint64_t>(m / 512, 1), 32);
}

// Forward products of so few rows that reading the weights is all the time,
// and of enough columns for every other compute unit.  By tiles and a joining
// launch instead, 1 x 2048 x 4096 takes 11.6 us against 7.7, 16 x 4096 x 4096
// 13.9 against 10.3, 16 x 16384 x 4096 31 against 33; short sums take the same
// (1 x 2048 x 256: 7.6 and 7.8).
bool skinny(uint64_t m, uint64_t n, uint64_t k) {
    return m <= kSkinnyRows && n >= 2048 && k >= 256;
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
    return partial_bytes(op, m, n, k) + (op == kWgrad && db_slices(m) > 1 ? db_slices(m) * n * 4 : 0);
}

bool sizes_ok(size_t m, size_t n, size_t k) {
    return m <= kMaxRows && n <= kMaxExtent && k <= kMaxExtent;
}

template <class T, bool TRA, bool TRB, bool STAGED>
int launch_tile(int tile, GemmArgs &g, uint64_t k, hipStream_t s) {
    auto go = [&](auto core) {
        using Core = decltype(core);
        g.kt = (uint32_t)((k + Core::BK - 1) / Core::BK);
        const int rc = allow_lds(linear_kernel<T, Core>, Core::LDS);
        return rc ? rc
                  : launch(linear_kernel<T, Core>, dim3(g.tm * g.tn, g.splits),
                           dim3(Core::THREADS), Core::LDS, s, g);
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
    const uint64_t lanes = std::min((e.n + 7) / 8 * e.m, kJoinLanes);
    return launch(linear_join<T>, dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, s, e,
                  g.partial, g.splits);
}

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
    if (skinny(m, n, k) && k % 8 == 0 && aligned16(a->x, a->ldx, 2) && aligned16(a->w, a->ldw, 2)) {
        const dim3 grid((uint32_t)((n + 15) / 16)), block(kSkinnyWaves * 64);
        return launch(a->dtype == DDL_F16 ? skinny_kernel<Half> : skinny_kernel<Bfloat>, grid,
                      block, 0, (hipStream_t)stream, x, w, e);
    }
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
        const dim3 sums((uint32_t)((n + 63) / 64), slices), join((uint32_t)((n + 255) / 256));
        auto go = [&](auto o) {
            using O = decltype(o);
            const int rc = launch(column_sums<T, O>, sums, dim3(256), 0, s, (const E *)a->dz,
                                  a->lddz, m, n, slices, partial, (O *)a->db, a->accumulate);
            return rc || slices == 1 ? rc
                                     : launch(column_join<O>, join, dim3(256), 0, s, partial,
                                              slices, n, (O *)a->db, a->accumulate);
        };
        const int rc = f32 ? go(float()) : go(E());
        if (rc)
            return rc;
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
