// cross_entropy_grad.hip -- the cross entropy's gradient (gfx950), from the
// forward pass's lse:
//
//     dz_ij = dloss_i scale (exp(z_ij - lse_i) - (1 - a) [j = target(i)] - a / n)
//     dx = dz w,   dw = dz^T x,   db = the column sums of dz
//
// The classes go through in pieces: a piece's logits are computed again, dz
// leaves the matrix instruction's registers in 16 bits, and two products take it
// from there.  So the memory held is a piece's dz, whatever the number of
// classes, and the price is one product more than with all logits kept.
//
// dz's rounding to 16 bits would be one that results see besides their own: 16-bit
// ones had 1.5 times the error of a result rounded once, and binary32 dw would lose
// half of its digits.  So dz is held more exactly:
//  - as a sum of two values of the operands' type (16 significant bits in bfloat16,
//    22 in binary16), whose products take two passes: 512 x 1000 x 2048 in binary16
//    42 us, with dz rounded 31.  bfloat16 with binary32 dw writes dz in two parts of
//    binary16 beside these, which dw takes with x as binary16 (below): 22 bits for
//    16, and 512 x 5000 x 2048 119 us for 110;
//  - with bfloat16 operands, where it is faster (widens), as binary16, against x
//    and w as binary16 too: their 8 bits fit it exactly down to 2^-31 of a column's
//    largest value, which a power of two takes to the top of its range, and smaller
//    ones to 2^-39 of it.  One pass then holds dz to 11 bits, and binary32 dw takes
//    two for 22.  8192 x 131072 x 4096 takes 21.6 ms, in two parts of bfloat16 35.4.
//    16-bit results so come out 0.5 to 1% further from the exact ones than binary32's
//    rounded once (0.00167 of their norm for 0.00166), and one in 30 to 50 is the neighbour
//    of that.
// db is summed from dz before it is rounded.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cross_entropy_internal.h"

namespace ddl {
namespace {

using gemm::Bfloat;
using gemm::f32x4;
using gemm::Half;

// ---------------------------------------------------------------------------
// dz of a piece
// ---------------------------------------------------------------------------

struct DzArgs {
    Rows rows;
    Operand x, w;           // w: the piece's rows
    const void *bias;       // T, the piece's, or null
    uint32_t tn, n;         // the piece's tiles, which cover ld, and columns
    uint32_t first;         // its first class
    float smooth, wanted;   // a / n, 1 - a
    uint16_t *dz[2];        // [up64(count)][ld]; the low parts: or null
    uint16_t *half[2];      // bfloat16: dz once more, in two parts of binary16; or null
    uint64_t ld;            // n rounded up to 64; rows past count and columns past n are 0
    float *db;              // [row tile][ld]: column sums, or null
};

// 8 values as V, to the second plane (or null) what that leaves of them.
template <class V>
__device__ __forceinline__ void put(uint16_t *const (&to)[2], uint64_t at, const float (&v)[8]) {
    store8<true>((V *)to[0] + at, 8, v);
    if (!to[1])
        return;
    float left[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        left[e] = v[e] - (float)(V)v[e];
    store8<true>((V *)to[1] + at, 8, left);
}

// D: the type that dz is held in.
template <class T, class D, class Core>
__global__ __launch_bounds__(Core::THREADS) void dz_kernel(DzArgs a) {
    using E = typename T::E;
    using H = typename D::E;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr uint32_t BM = Core::BM, BN = Core::BN;
    const uint32_t count = a.rows.head->count, tm = (count + BM - 1) / BM;
    if (blockIdx.x >= tm * a.tn)
        return;
    uint32_t ti, tj;
    tile_of(blockIdx.x, tm, a.tn, ti, tj);
    a.x.row0 = ti * BM;
    a.x.rows = count;
    a.w.row0 = tj * BN;
    const int exponent = a.rows.head->exponent;
    f32x4 acc[Core::FM][Core::FN] = {};
    // a tile of 32 columns may lie past the last class: its dz is 0
    if (a.x.k && a.w.row0 < a.n)
        Core::run(a.x, a.w, 0, (uint32_t)((a.x.k + Core::BK - 1) / Core::BK), 0, lds, acc);
    // dz in place of the logits.  A lane holds, of row l % 16 of each of its FM
    // fragments, 4 columns of each of the FN fragments.
    const uint32_t m0 = ti * BM, n0 = tj * BN, rows = (uint32_t)up64(count);
    const uint32_t wave = threadIdx.x >> 6, l = threadIdx.x & 63u;
    const uint32_t col = n0 + wave % Core::WC * (Core::FN * 16) + (l >> 4) * 4;
    const uint32_t row0 = m0 + wave / Core::WC * (Core::FM * 16) + (l & 15u);
    float lse[Core::FM], g[Core::FM];
    uint32_t want[Core::FM];
#pragma unroll
    for (int i = 0; i < Core::FM; ++i) {
        const uint32_t row = row0 + i * 16;
        const bool in = row < count;
        lse[i] = in ? a.rows.lse[row] : 0.0f;
        g[i] = in ? ldexpf(a.rows.g[row], exponent) : 0.0f;
        want[i] = (in ? (uint32_t)a.rows.target[row] : ~0u) - a.first - col;
    }
    if (a.bias)
#pragma unroll
        for (int j = 0; j < Core::FN; ++j) {
            const uint32_t c = col + j * 16;
            float b[4];
            load4((const E *)a.bias + c, c < a.n ? a.n - c : 0, b);
#pragma unroll
            for (int i = 0; i < Core::FM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] += b[e];
        }
#pragma unroll
    for (int i = 0; i < Core::FM; ++i) {
#pragma unroll
        for (int j = 0; j < Core::FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][j][e] =
                    (__builtin_amdgcn_exp2f((acc[i][j][e] - lse[i]) * kLog2e) - a.smooth) * g[i];
        // few rows have their target among the wave's columns
        if (__any(want[i] < Core::FN * 16))
#pragma unroll
            for (int j = 0; j < Core::FN; ++j)
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e)
                    if (want[i] == j * 16 + e)
                        acc[i][j][e] -= a.wanted * g[i];
    }
    if (m0 + BM > count || n0 + BN > a.n)
#pragma unroll
        for (int i = 0; i < Core::FM; ++i)
#pragma unroll
            for (int j = 0; j < Core::FN; ++j)
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e)
                    if (row0 + i * 16 >= count || col + j * 16 + e >= a.n)
                        acc[i][j][e] = 0.0f;
    float sums[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    Core::template each<false, 1>(
        acc, lds, [](uint32_t, uint32_t) { return 0; },
        [&](uint32_t mi, uint32_t ni, float (&v)[8], int) {
            const uint32_t m = m0 + mi, n = n0 + ni;
            if (m >= rows || n >= a.ld)
                return;
            const uint64_t at = m * a.ld + n;
            if (a.db)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sums[e] += v[e];
            if constexpr (std::is_same<D, Bfloat>::value)
                if (a.half[0])
                    put<_Float16>(a.half, at, v);
            put<H>(a.dz, at, v);
        });
    if (!a.db)
        return;
    // a lane holds the sums of 8 columns over its rows; the wave's other rows
    // of the same columns are in the lanes LANES apart
    constexpr uint32_t LANES = Core::FN * 2;
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (uint32_t d = LANES; d < 64; d *= 2)
            sums[e] += __shfl_xor(sums[e], d);
    __syncthreads();  // every wave is done with its part of LDS
    float *columns = (float *)lds;  // [WR][BN]
    if (l < LANES)
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
            columns[wave / Core::WC * BN + wave % Core::WC * (Core::FN * 16) + l * 8 + e] =
                sums[e];
    __syncthreads();
    if (threadIdx.x < BN && n0 + threadIdx.x < a.ld) {
        float s = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < Core::WR; ++w)
            s += columns[w * BN + threadIdx.x];
        a.db[ti * a.ld + n0 + threadIdx.x] = s;
    }
}

// db of a piece from its row tiles' sums.
struct DbArgs {
    const float *sums;  // [row tile][ld]
    uint64_t ld;
    uint32_t side, n;   // rows of a tile; the piece's classes
    void *db;           // of the piece, E or binary32; or null
    int f32, add;
};

template <class E>
__device__ __forceinline__ void db_of(const DbArgs &a, const RowsHead *head, uint32_t c) {
    if (c >= a.n)
        return;
    const uint32_t tm = (head->count + a.side - 1) / a.side;
    float v = 0.0f;
#pragma unroll 8
    for (uint32_t t = 0; t < tm; ++t)
        v += a.sums[t * a.ld + c];
    v = ldexpf(v, -head->exponent);
    if (a.f32) {
        float *to = (float *)a.db + c;
        *to = a.add ? *to + v : v;
    } else {
        E *to = (E *)a.db + c;
        *to = (E)(a.add ? (float)*to + v : v);
    }
}

template <class E>
__global__ __launch_bounds__(256) void db_kernel(const RowsHead *head, DbArgs a) {
    db_of<E>(a, head, blockIdx.x * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------
// bfloat16 as binary16
// ---------------------------------------------------------------------------

// Every column goes times a power of two of its own, which takes its largest value
// to [2^14, 2^15): a column of x or w is one of dw or dx, which takes the power back,
// so one that is small throughout loses nothing.
//
// Classes whose bias is -inf may hold anything: their dz is 0, without smoothing and
// unless one is wanted, so they do not count for the power and what passes binary16's
// range is held at its end (infinity would make 0 times it NaN).

// One of up to two matrices that a launch takes, x and a piece of w: two launches
// less for 4 us each.
struct Widened {
    const uint16_t *p;
    uint64_t ld, rows;
    const RowsHead *head;  // the rows are the packed ones; or null
    const uint16_t *bias;  // the rows are classes, some perhaps with a bias of -inf; or null
    uint32_t *tops;        // [ld_to]: the columns' largest, by their bits; 0 before
    uint32_t *next;        // [ld_to]: cleared for the next piece; or null
    uint16_t *to;
    uint32_t seek, groups; // workgroups of largest_kernel, by columns, and of convert_kernel
};
struct WidenArgs {
    Widened of[2];
    uint64_t cols, ld_to;
};

__device__ __forceinline__ bool never_wanted(const uint16_t *bias, uint64_t row) {
    return bias && bias[row] == 0xff80u;
}

// The exponent of a column whose largest value has the bits top.
__device__ __forceinline__ int column_exponent(uint32_t top) {
    return top ? 14 - ((int)(top >> 7) - 127) : 0;
}
// Those of 8 columns; tops: or null.
__device__ __forceinline__ void column_exponents(const uint32_t *tops, uint32_t n, int (&e)[8]) {
    u32x4 t[2] = {};
    if (tops) {
        t[0] = *(const u32x4 *)(tops + n);
        t[1] = *(const u32x4 *)(tops + n + 4);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e[i] = column_exponent(t[i / 4][i % 4]);
}

// The largest finite |v| of each column.  A workgroup takes 512 columns of every
// `seek`-th four rows: few rows by fewer workgroups, which meet at the same words at
// the end (1024 x 1000 x 2048, the whole gradient: 57 us with a workgroup for 16 rows,
// 64 with one for 4), many rows by no more than kTopGroups (1023 x 32003 x 1111 309 us,
// with 64 of them 329).
constexpr uint32_t kTopColumns = 512, kTopRows = 16, kTopGroups = 256;

__global__ __launch_bounds__(256) void largest_kernel(WidenArgs a) {
    __shared__ uint32_t top[kTopColumns];
    const Widened x = blockIdx.z ? a.of[1] : a.of[0];
    const uint16_t *p = x.p;
    const uint64_t ld = x.ld, cols = a.cols, rows = x.head ? x.head->count : x.rows;
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint64_t c0 = (uint64_t)blockIdx.y * kTopColumns, c = c0 + lane * 8;
    if (blockIdx.x >= x.seek)
        return;
    for (uint32_t i = threadIdx.x; i < kTopColumns; i += 256)
        top[i] = 0;
    __syncthreads();
    constexpr uint32_t U = 4;  // rows at a time
    const uint64_t step = (uint64_t)x.seek * 4;
    uint32_t most[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (c < cols)
        for (uint64_t r = blockIdx.x * 4 + wave; r < rows; r += U * step) {
            uint16_t v[U][8];
            const uint16_t *row[U];  // the last one again where there are no more
            uint32_t bits[U];
#pragma unroll
            for (uint32_t i = 0; i < U; ++i) {
                const uint64_t at = min(r + i * step, rows - 1);
                row[i] = p + at * ld + c;
                bits[i] = never_wanted(x.bias, at) ? 0u : 0x7fffu;
            }
            if (c + 8 <= cols) {
#pragma unroll
                for (uint32_t i = 0; i < U; ++i)
                    __builtin_memcpy(v[i], row[i], 16);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < U; ++i)
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        v[i][e] = c + e < cols ? row[i][e] : (uint16_t)0;
            }
#pragma unroll
            for (uint32_t i = 0; i < U; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t u = v[i][e] & bits[i];
                    most[e] = max(most[e], u < 0x7f80u ? u : 0u);
                }
        }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (most[e])
            atomicMax(&top[lane * 8 + e], most[e]);
    __syncthreads();
    // a maximum is the same in any order
    for (uint32_t i = threadIdx.x; i < kTopColumns; i += 256)
        if (top[i])
            atomicMax(&x.tops[c0 + i], top[i]);
}

// The matrix as binary16, rows of zeros behind it up to a multiple of 64.
constexpr uint32_t kConvertRows = 8;  // of a workgroup

__global__ __launch_bounds__(256) void convert_kernel(WidenArgs a) {
    const bool second = blockIdx.x >= a.of[0].groups;
    const Widened m = second ? a.of[1] : a.of[0];
    const uint32_t block = blockIdx.x - (second ? a.of[0].groups : 0u);
    const uint16_t *p = m.p;
    uint16_t *to = m.to;
    const uint64_t ld = m.ld, ld_to = a.ld_to, cols = a.cols;
    const uint64_t rows = m.head ? m.head->count : m.rows;
    const uint64_t r0 = (uint64_t)block * kConvertRows;
    if (m.next)
        for (uint64_t i = (uint64_t)block * 256 + threadIdx.x; i < ld_to;
             i += (uint64_t)m.groups * 256)
            m.next[i] = 0;
    if (r0 >= up64(rows))
        return;
    constexpr uint32_t U = 4;  // rows at a time
    for (uint64_t c = threadIdx.x * 8; c < ld_to; c += 256 * 8) {
        int e[8];
        column_exponents(m.tops, (uint32_t)c, e);
        for (uint64_t r = r0; r < r0 + kConvertRows; r += U) {
            uint16_t v[U][8];
            if (r + U <= rows && c + 8 <= cols) {
#pragma unroll
                for (uint32_t i = 0; i < U; ++i)
                    __builtin_memcpy(v[i], p + (r + i) * ld + c, 16);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < U; ++i)
#pragma unroll
                    for (uint32_t x = 0; x < 8; ++x)
                        v[i][x] = r + i < rows && c + x < cols ? p[(r + i) * ld + c + x]
                                                               : (uint16_t)0;
            }
#pragma unroll
            for (uint32_t i = 0; i < U; ++i) {
                const float most = r + i < rows && never_wanted(m.bias, r + i)
                                       ? 65504.0f
                                       : __builtin_huge_valf();
                _Float16 h[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float f =
                        ldexpf(__builtin_bit_cast(float, (uint32_t)v[i][x] << 16), e[x]);
                    h[x] = (_Float16)(fabsf(f) > most ? copysignf(most, f) : f);
                }
                __builtin_memcpy(to + (r + i) * ld_to + c, h, 16);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// the products that take dz
// ---------------------------------------------------------------------------

// C of a product: dx (of the packed rows; sums of the pieces so far are in
// `sum`) or dw (of the piece's classes).
struct Out {
    uint32_t m;       // rows: dw; dx: the rows with a target
    uint32_t n;       // columns
    void *c;          // dx: T, by the caller's rows; dw: T or binary32
    uint64_t ld;
    float *sum;       // dx: [count][sum_ld] of the pieces before, or null
    uint64_t sum_ld;
    const uint32_t *row;  // dx: the caller's
    int read, write;  // dx: whether sum is read, and written in c's place
    int f32, add;     // dw
    int vec;          // c's rows start on 16-byte boundaries, n is a multiple of 8
};

struct GradArgs {
    const RowsHead *head;
    const uint32_t *tops;  // b's columns', where it was converted; or null
    Operand a, b;
    uint32_t tn, splits;
    uint32_t tile_rows;  // tiles of m, of the caller's rows with dx
    float *partial;      // splits > 1: [splits][m][part_ld]
    uint64_t part_ld;    // n rounded up to 64
    Out o;
    DbArgs db;           // dw: taken by the workgroups of the first columns
};

struct Old {
    u32x4 v[2];
};

// As load8 and store8, in whole vectors wherever all 8 elements are there: global
// memory takes them at any element's address (dw of 32003 x 1111 in bfloat16, whose
// rows start anywhere: 107 us element by element).
template <bool VEC, class E>
__device__ __forceinline__ void read8(const E *p, uint32_t have, u32x4 (&out)[sizeof(E) / 2]) {
    if (VEC || have >= 8)
        __builtin_memcpy(out, p, 8 * sizeof(E));
    else
        load8<false>(p, have, out);
}
template <bool VEC, class E>
__device__ __forceinline__ void write8(E *p, uint32_t have, const float (&v)[8]) {
    if (VEC) {
        store8<true>(p, 8, v);
    } else if (have >= 8) {
        E t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = (E)v[i];
        __builtin_memcpy(p, t, sizeof(t));
    } else {
        store8<false>(p, have, v);
    }
}

template <class E, bool DX, bool VEC>
__device__ __forceinline__ Old old8(const Out &o, uint32_t m, uint32_t n) {
    Old f;
    if (m >= o.m || n >= o.n)
        return f;
    if (DX) {
        if (o.read)
            load8<true>(o.sum + m * o.sum_ld + n, 8, f.v);
    } else if (o.add) {
        const uint32_t have = o.n - n < 8 ? o.n - n : 8;
        if (o.f32) {
            read8<VEC>((const float *)o.c + m * o.ld + n, have, f.v);
        } else {
            u32x4 t[1];
            read8<VEC>((const E *)o.c + m * o.ld + n, have, t);
            f.v[0] = t[0];
        }
    }
    return f;
}

// The product is the gradient's times 2^exponent of each column.
template <class E, bool DX, bool VEC>
__device__ __forceinline__ void out8(const Out &o, const int (&exponent)[8], uint32_t m, uint32_t n,
                                     float (&v)[8], const Old &f) {
    if (m >= o.m || n >= o.n)
        return;
    const uint32_t have = o.n - n < 8 ? o.n - n : 8;
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = ldexpf(v[i], -exponent[i]);
    if (DX) {
        if (o.read) {
            widen8<float>(f.v, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += t[i];
        }
        if (o.write) {
            store8<true>(o.sum + m * o.sum_ld + n, 8, v);
            return;
        }
        write8<VEC>((E *)o.c + o.row[m] * o.ld + n, have, v);
        return;
    }
    if (o.add) {
        if (o.f32) {
            widen8<float>(f.v, t);
        } else {
            u32x4 h[1] = {f.v[0]};
            widen8<E>(h, t);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += t[i];
    }
    if (o.f32)
        write8<VEC>((float *)o.c + m * o.ld + n, have, v);
    else
        write8<VEC>((E *)o.c + m * o.ld + n, have, v);
}

// Of the product's columns n .. n + 7: dz's and b's.
__device__ __forceinline__ void exponents_of(const GradArgs &g, uint32_t n, int (&e)[8]) {
    column_exponents(n < g.o.n ? g.tops : nullptr, n, e);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e[i] += g.head->exponent;
}

// The parts of dx's sums: with fewer row tiles than were launched for, their
// workgroups take parts of k instead, which the same memory holds.
__device__ __forceinline__ uint32_t parts_of(const GradArgs &g, uint32_t tm, uint32_t kt) {
    if (g.splits == 1 || !tm)
        return g.splits;
    return min(g.splits * g.tile_rows / tm, max(kt / 4, g.splits));
}

// DX: C = dz w over the piece's classes.  Otherwise C = dz^T x over the packed
// rows.  PAIR: with dz in two parts, the low ones first.  E: the type of results in
// 16 bits.
// id: of the workgroup among the product's.
template <class E, class Core, bool DX, bool PAIR>
__device__ __forceinline__ void grad_tile(GradArgs &g, uint32_t id, uint8_t *lds) {
    const uint32_t count = g.head->count;
    if (DX) {
        g.a.rows = g.o.m = count;
    } else {
        g.a.k = g.b.k = up64(count);
    }
    const uint32_t tm = DX ? (count + Core::BM - 1) / Core::BM : g.tile_rows;
    const uint32_t kt = (uint32_t)((g.a.k + Core::BK - 1) / Core::BK);
    const uint32_t all = PAIR ? 2 * kt : kt;
    const uint32_t splits = DX ? parts_of(g, tm, kt) : g.splits;
    if (id >= tm * g.tn * splits)
        return;
    const uint32_t s = id / (tm * g.tn);
    uint32_t ti, tj;
    tile_of(id - s * tm * g.tn, tm, g.tn, ti, tj);
    g.a.row0 = ti * Core::BM;
    g.b.row0 = tj * Core::BN;
    const uint32_t t0 = (uint32_t)((uint64_t)all * s / splits);
    const uint32_t t1 = (uint32_t)((uint64_t)all * (s + 1) / splits);
    f32x4 acc[Core::FM][Core::FN] = {};
    // of the three passes over pairs, the two that take b's one part
    if (t0 < t1)
        Core::run(g.a, g.b, (PAIR ? kt : 0) + t0, (PAIR ? kt : 0) + t1, PAIR ? kt : 0, lds, acc);
    const uint32_t m0 = g.a.row0, n0 = g.b.row0;
    if (!DX && g.db.db && tj == 0 && s == 0)
        for (uint32_t c = threadIdx.x; c < Core::BM; c += Core::THREADS)
            db_of<E>(g.db, g.head, m0 + c);
    int exponent[8];
    if (g.splits == 1)
        exponents_of(g, n0 + Core::column(), exponent);
    if (g.splits > 1) {
        float *part = g.partial + (uint64_t)s * g.o.m * g.part_ld;
        Core::each(
            acc, lds, [](uint32_t, uint32_t) { return 0; },
            [&](uint32_t mi, uint32_t ni, float (&v)[8], int) {
                if (m0 + mi < g.o.m && n0 + ni < g.o.n)
                    store8<true>(part + (m0 + mi) * g.part_ld + n0 + ni, 8, v);
            });
    } else if (g.o.vec) {
        Core::each(
            acc, lds,
            [&](uint32_t mi, uint32_t ni) { return old8<E, DX, true>(g.o, m0 + mi, n0 + ni); },
            [&](uint32_t mi, uint32_t ni, float (&v)[8], const Old &f) {
                out8<E, DX, true>(g.o, exponent, m0 + mi, n0 + ni, v, f);
            });
    } else {
        Core::template each<false, 1>(
            acc, lds,
            [&](uint32_t mi, uint32_t ni) { return old8<E, DX, false>(g.o, m0 + mi, n0 + ni); },
            [&](uint32_t mi, uint32_t ni, float (&v)[8], const Old &f) {
                out8<E, DX, false>(g.o, exponent, m0 + mi, n0 + ni, v, f);
            });
    }
}

template <class E, class Core, bool DX, bool PAIR>
__global__ __launch_bounds__(Core::THREADS) void grad_kernel(GradArgs g) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    grad_tile<E, Core, DX, PAIR>(g, blockIdx.x, lds);
}

// Both products of a small piece in one launch, which leaves fewer compute units
// idle than one after the other (512 x 1000 x 2048 in binary16: 56 to 42 us for
// the whole gradient): the first `split` workgroups are dx's.
template <class E, class X, class W, bool PAIRX, bool PAIRW>
__global__ __launch_bounds__(X::THREADS) void both_kernel(GradArgs x, GradArgs w, uint32_t split) {
    static_assert(X::THREADS == W::THREADS, "one kind of workgroup");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    if (blockIdx.x < split)
        grad_tile<E, X, true, PAIRX>(x, blockIdx.x, lds);
    else
        grad_tile<E, W, false, PAIRW>(w, blockIdx.x - split, lds);
}

// The sums of the parts, in their order; 8 columns a lane.
template <class E, bool DX>
__global__ __launch_bounds__(256) void grad_join(GradArgs g, uint32_t side) {
    uint32_t splits = g.splits;
    if (DX) {
        g.o.m = g.head->count;
        splits = parts_of(g, (g.o.m + side - 1) / side, (uint32_t)((g.a.k + 63) / 64));
    }
    const uint32_t groups = (g.o.n + 7) / 8;
    const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= (uint64_t)groups * g.o.m)
        return;
    const uint32_t m = (uint32_t)(id / groups), n = (uint32_t)(id % groups) * 8;
    int exponent[8];
    exponents_of(g, n, exponent);
    const Old f = g.o.vec ? old8<E, DX, true>(g.o, m, n) : old8<E, DX, false>(g.o, m, n);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (uint32_t s = 0; s < splits; ++s) {
        const float *p = g.partial + ((uint64_t)s * g.o.m + m) * g.part_ld + n;
        const f32x4 x = *(const f32x4 *)p, y = *(const f32x4 *)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += x[i];
            v[4 + i] += y[i];
        }
    }
    if (g.o.vec)
        out8<E, DX, true>(g.o, exponent, m, n, v, f);
    else
        out8<E, DX, false>(g.o, exponent, m, n, v, f);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

bool packs(uint64_t k) { return k % 8; }

// bfloat16 operands go as binary16 where the passes that it saves, two or, with dw
// in binary32, one, cost more than two launches and the pass over w, 6 bytes of each
// of its elements.  In us, in parts and so, dw in 16 bits:
//   512 x 1000 x 2048 42, 44;  700 x 1000 x 2048 57, 53;  1024 x 1000 x 2048 65, 56;
//   256 x 65536 x 4096 787, 967;  512 x 65536 x 4096 1280, 1214;
//   64 x 131072 x 4096 1092, 1586;
// and in binary32:
//   1024 x 1000 x 1024 52, 51;  1024 x 1000 x 2048 75, 67;  4096 x 1000 x 300 87, 74;
//   512 x 65536 x 4096 1455, 1570;  1024 x 32000 x 4096 1268, 1185.
bool widens(uint64_t m, uint64_t n, uint64_t k, uint32_t passes) {
    return m * passes >= 1024 && (double)m * (double)n * (double)k >= 1.2e9;
}

// Classes of a piece: as many as dz and a packed w have room for, whole tiles, but
// all of them where they fit.
size_t piece_columns(size_t m, size_t n, size_t k) {
    const size_t rows = up64(m);  // of dz
    const size_t most = packs(k) || widens(m, n, k, 2) ? std::max<size_t>(rows, k) : rows;
    const size_t fit = std::max<size_t>(kPieceElements / most / 256, 1) * 256;
    return std::min<size_t>(fit, up64(n));
}

struct Buffers {
    Rows rows;
    uint16_t *dz[2], *half[2];
    uint16_t *w;         // packed
    uint16_t *x16, *w16; // bfloat16 as binary16
    uint32_t *tops;      // [3][ld]: of x, and of the even and the odd pieces of w
    float *sum;          // dx's over the pieces: [m][ld]
    float *db;
    float *partial;
};

// The largest of the products' parts, over whole pieces and the last one.
size_t partial_floats(size_t m, size_t n, size_t k, size_t piece) {
    const size_t kp = up64(k), last = n - (n - 1) / piece * piece;
    size_t most = 0;
    for (const size_t have : {std::min(piece, n), last}) {
        const Plan x = plan_product(m, k, have, false), w = plan_product(have, k, m, false);
        // whole tiles of rows: see parts_of
        const size_t rows = (m + kSideM[x.tile] - 1) / kSideM[x.tile] * kSideM[x.tile];
        most = std::max(most, x.splits > 1 ? x.splits * rows * kp : 0);
        most = std::max(most, w.splits > 1 ? w.splits * have * kp : 0);
    }
    return most;
}

Buffers carve_grad(Carve &c, size_t m, size_t n, size_t k) {
    Buffers b;
    b.rows = carve_rows(c, m, k);
    const size_t piece = piece_columns(m, n, k);
    b.dz[0] = c.take<uint16_t>(up64(m) * piece);
    b.dz[1] = c.take<uint16_t>(up64(m) * piece);
    b.w = c.take<uint16_t>(packs(k) ? piece * b.rows.ld : 0);
    const bool wide = widens(m, n, k, 2), always = widens(m, n, k, 1);
    for (uint16_t *&plane : b.half)
        plane = c.take<uint16_t>(always ? 0 : up64(m) * piece);
    b.x16 = c.take<uint16_t>(up64(m) * b.rows.ld);
    b.w16 = c.take<uint16_t>(wide ? up64(piece) * b.rows.ld : 0);
    b.rows.clear = c.take<uint32_t>(3 * b.rows.ld);
    b.rows.clear_count = 3 * b.rows.ld;
    b.tops = b.rows.clear;
    b.sum = c.take<float>(piece < n ? m * b.rows.ld : 0);
    b.db = c.take<float>((m + 63) / 64 * piece);
    b.partial = c.take<float>(partial_floats(m, n, k, piece));
    return b;
}

template <class T, class D, bool STAGED>
int launch_dz(DzArgs &a, const Plan &p, uint64_t m, hipStream_t s) {
    auto go = [&](auto core) {
        using Core = decltype(core);
        a.tn = (uint32_t)((a.ld + Core::BN - 1) / Core::BN);
        const int rc = allow_lds(dz_kernel<T, D, Core>, Core::LDS);
        return rc ? rc
                  : launch(dz_kernel<T, D, Core>,
                           dim3((uint32_t)((m + Core::BM - 1) / Core::BM) * a.tn),
                           dim3(Core::THREADS), Core::LDS, s, a);
    };
    if (p.tile == 0)
        return go(gemm::Core<T, 256, 256, 2, 4, 64, 2, false, false, STAGED, !STAGED>());
    if (p.tile == 1)
        return go(gemm::Core<T, 128, 128, 2, 2, 64, 2, false, false, STAGED>());
    if (p.tile == 2)
        return go(gemm::Core<T, 64, 64, 2, 2, 64, 3, false, false, STAGED>());
    return go(gemm::Core<T, 64, 32, 4, 1, 64, 3, false, false, STAGED>());
}

// The workgroups of a product of m rows by tiles of Core, into g.
template <class Core>
uint32_t lay_out(GradArgs &g, const Plan &c, uint64_t m) {
    g.tile_rows = (uint32_t)((m + Core::BM - 1) / Core::BM);
    g.tn = (g.o.n + Core::BN - 1) / Core::BN;
    g.splits = c.splits;
    return g.tile_rows * g.tn * g.splits;
}

template <class E, bool DX>
int launch_join(const GradArgs &g, uint64_t m, uint32_t side, hipStream_t s) {
    if (g.splits == 1)
        return DDL_OK;
    const uint64_t lanes = (uint64_t)(g.o.n + 7) / 8 * m;
    return launch(grad_join<E, DX>, dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, s, g,
                  side);
}

// T: the type of the operands, E: of results in 16 bits.
template <class T, class E, bool DX, bool PAIR, bool STAGED>
int launch_grad(GradArgs &g, const Plan &c, uint64_t m, hipStream_t s) {
    auto go = [&](auto core) {
        using Core = decltype(core);
        constexpr auto kernel = grad_kernel<E, Core, DX, PAIR>;
        const uint32_t groups = lay_out<Core>(g, c, m);
        int rc = allow_lds(kernel, Core::LDS);
        rc = rc ? rc : launch(kernel, dim3(groups), dim3(Core::THREADS), Core::LDS, s, g);
        return rc ? rc : launch_join<E, DX>(g, m, Core::BM, s);
    };
    if (c.tile == 0)
        return go(gemm::Core<T, 256, 256, 2, 4, 64, 2, !DX, true, STAGED, !STAGED>());
    if (c.tile == 1)
        return go(gemm::Core<T, 128, 128, 2, 2, 64, 2, !DX, true, STAGED>());
    return go(gemm::Core<T, 64, 64, 2, 2, 64, 3, !DX, true, STAGED>());
}

// dx by 64 x 64 tiles beside dw by 64 x 64 or 128 x 128, whole sums: the parts'
// memory is one product's.  Whole gradients in us, together and one after the other:
// 512 x 1000 x 2048 41, 56;  128 x 1000 x 2048 38, 45;  1024 x 1000 x 768 41, 59;
// 64 x 8000 x 512 27, 34;  300 x 520 x 2056 33, 43.
bool go_together(const Plan &x, const Plan &w) {
    return x.tile == 2 && w.tile >= 1 && w.splits == 1;
}

// TX, TW: the types of dx's and dw's operands.
template <class E, class TX, bool PAIRX, class TW, bool PAIRW>
int launch_both(GradArgs &x, GradArgs &w, const Plan &px, const Plan &pw, uint64_t m, uint64_t n,
                hipStream_t s) {
    using X = gemm::Core<TX, 64, 64, 2, 2, 64, 3, false, true, false>;
    auto go = [&](auto core) {
        using W = decltype(core);
        constexpr auto kernel = both_kernel<E, X, W, PAIRX, PAIRW>;
        constexpr int lds = X::LDS > W::LDS ? X::LDS : W::LDS;
        const uint32_t split = lay_out<X>(x, px, m), more = lay_out<W>(w, pw, n);
        int rc = allow_lds(kernel, lds);
        rc = rc ? rc : launch(kernel, dim3(split + more), dim3(X::THREADS), lds, s, x, w, split);
        return rc ? rc : launch_join<E, true>(x, m, X::BM, s);
    };
    return pw.tile == 1 ? go(gemm::Core<TW, 128, 128, 2, 2, 64, 2, true, true, false>())
                        : go(gemm::Core<TW, 64, 64, 2, 2, 64, 3, true, true, false>());
}

template <class T>
int gradient(const ddl_ce_grad_args *c, void *ws, hipStream_t s) {
    using E = typename T::E;
    const ddl_ce_args &l = c->layer;
    const size_t m = l.m, n = l.n, k = l.k;
    const bool f32 = c->dw_dtype == DDL_F32;
    Carve carve{(uint8_t *)ws};
    const Buffers b = carve_grad(carve, m, n, k);
    RowsArgs r = {};
    r.m = (uint32_t)m;
    r.n = n;
    r.k = k;
    r.x = l.x;
    r.ldx = l.ldx;
    r.target = l.target;
    r.lse = l.lse;
    r.dloss = c->dloss;
    r.scale = c->scale;
    r.dx = (uint16_t *)c->dx;
    r.lddx = c->lddx;
    int rc = pack_rows(r, b.rows, s);
    const size_t piece = piece_columns(m, n, k);
    // straight to LDS where w's rows start on 16 bytes, or a packed piece's do
    const bool pack = packs(k), direct = pack || (k % 8 == 0 && aligned16(l.w, l.ldw, 2));
    const size_t ldw = pack ? b.rows.ld : l.ldw, ld16 = b.rows.ld;
    const bool bf = std::is_same<T, Bfloat>::value, dw32 = c->dw && f32;
    const bool wide =
        bf && (c->dx ? widens(m, n, k, c->dw && !f32 ? 2 : 1) : dw32 || widens(m, n, k, 1));
    const bool twice = bf && !wide && dw32;  // in either type
    for (size_t first = 0; first < n && !rc; first += piece) {
        const size_t have = std::min(piece, n - first);
        const uint16_t *w = (const uint16_t *)l.w + first * l.ldw;
        if (pack) {
            rc = pack_matrix(w, l.ldw, have, k, b.w, s);
            if (rc)
                break;
            w = b.w;
        }
        WidenArgs v = {};
        v.cols = k;
        v.ld_to = ld16;
        uint32_t count = 0;
        auto widen = [&](const uint16_t *p, size_t ld, size_t rows, const RowsHead *head,
                         const uint16_t *bias, uint32_t *tops, uint32_t *next, uint16_t *to) {
            const uint32_t seek =
                (uint32_t)std::min<size_t>((rows + kTopRows - 1) / kTopRows, kTopGroups);
            v.of[count] = {p,    ld,   rows, head, bias,
                           tops, next, to,   seek, (uint32_t)(up64(rows) / kConvertRows)};
            ++count;
        };
        const size_t odd = first / piece % 2;
        uint32_t *now = b.tops + (1 + odd) * ld16, *next = b.tops + (2 - odd) * ld16;
        if ((wide || twice) && c->dw && k && first == 0)
            widen(b.rows.x, ld16, m, b.rows.head, nullptr, b.tops, nullptr, b.x16);
        if (wide && c->dx && k)
            widen(w, ldw, have, nullptr,
                  l.bias && l.smoothing == 0.0 ? (const uint16_t *)l.bias + first : nullptr,
                  now, next, b.w16);
        if (count && !rc) {
            const dim3 groups(std::max(v.of[0].seek, v.of[1].seek),
                              (uint32_t)((k + kTopColumns - 1) / kTopColumns), count);
            rc = launch(largest_kernel, groups, dim3(256), 0, s, v);
            rc = rc ? rc
                    : launch(convert_kernel, dim3(v.of[0].groups + v.of[1].groups), dim3(256), 0, s,
                             v);
        }
        if (rc)
            break;
        DzArgs d = {};
        d.rows = b.rows;
        // zeros past k on both sides of packed ones
        d.x = operand(b.rows.x, b.rows.ld, m, pack ? b.rows.ld : k);
        d.w = operand(w, ldw, have, pack ? ldw : k);
        d.bias = l.bias ? (const uint16_t *)l.bias + first : nullptr;
        d.n = (uint32_t)have;
        d.first = (uint32_t)first;
        d.smooth = (float)(l.smoothing / (double)n);
        d.wanted = (float)(1.0 - l.smoothing);
        d.dz[0] = b.dz[0];
        d.dz[1] = !wide || dw32 ? b.dz[1] : nullptr;
        if (twice)
            std::copy(b.half, b.half + 2, d.half);
        d.ld = (have + 63) / 64 * 64;
        d.db = c->db ? b.db : nullptr;
        const Plan p = plan_product(m, have, k, true);
        if (wide)
            rc = direct ? launch_dz<T, Half, false>(d, p, m, s)
                        : launch_dz<T, Half, true>(d, p, m, s);
        else
            rc = direct ? launch_dz<T, T, false>(d, p, m, s) : launch_dz<T, T, true>(d, p, m, s);
        const size_t esz = f32 ? 4 : 2;
        DbArgs db = {};
        if (c->db) {
            db.sums = b.db;
            db.ld = d.ld;
            db.side = kSideM[p.tile];
            db.n = d.n;
            db.db = (uint8_t *)c->db + first * esz;
            db.f32 = f32;
            db.add = c->accumulate;
            if (!rc && (!c->dw || !k))
                rc = launch(db_kernel<E>, dim3((uint32_t)((have + 255) / 256)), dim3(256), 0, s,
                            b.rows.head, db);
        }
        GradArgs x = {}, g = {};
        const Plan px = plan_product(m, k, have, false), pw = plan_product(have, k, m, false);
        if (c->dx && k) {
            x.head = b.rows.head;
            x.a = operand(b.dz[0], d.ld, m, have);
            x.a.plane[1] = b.dz[1];
            // a packed w's columns past k are zeros
            x.b = operand(w, ldw, pack ? ldw : k, have);
            if (wide) {  // so are its rows past the piece, and dz's columns
                x.tops = now;
                x.a.k = up64(have);
                x.b = operand(b.w16, ld16, ld16, up64(have));
            }
            x.partial = b.partial;
            x.part_ld = b.rows.ld;
            x.o.n = (uint32_t)k;
            x.o.c = c->dx;
            x.o.ld = c->lddx;
            x.o.sum = b.sum;
            x.o.sum_ld = b.rows.ld;
            x.o.row = b.rows.row;
            x.o.read = first > 0;
            x.o.write = first + have < n;
            x.o.vec = k % 8 == 0 && aligned16(c->dx, c->lddx, 2);
        }
        if (c->dw && k) {
            g.head = b.rows.head;
            g.db = db;
            g.a = operand(twice ? b.half[0] : b.dz[0], d.ld, d.ld, 0);
            g.a.plane[1] = twice ? b.half[1] : b.dz[1];
            g.tops = wide || twice ? b.tops : nullptr;
            g.b = operand(wide || twice ? b.x16 : b.rows.x, ld16, ld16, 0);
            g.partial = b.partial;
            g.part_ld = b.rows.ld;
            g.o.m = (uint32_t)have;
            g.o.n = (uint32_t)k;
            g.o.c = (uint8_t *)c->dw + first * c->lddw * esz;
            g.o.ld = c->lddw;
            g.o.f32 = f32;
            g.o.add = c->accumulate;
            g.o.vec = k % 8 == 0 && aligned16(g.o.c, c->lddw, esz);
        }
        if (rc || !k)
            continue;
        const bool both = c->dx && c->dw && go_together(px, pw);
        if constexpr (std::is_same<T, Bfloat>::value) {
            if (wide && both) {
                rc = f32 ? launch_both<E, Half, false, Half, true>(x, g, px, pw, m, have, s)
                         : launch_both<E, Half, false, Half, false>(x, g, px, pw, m, have, s);
                continue;
            }
            if (wide) {
                if (c->dx)
                    rc = launch_grad<Half, E, true, false, false>(x, px, m, s);
                if (!rc && c->dw)
                    rc = f32 ? launch_grad<Half, E, false, true, false>(g, pw, have, s)
                             : launch_grad<Half, E, false, false, false>(g, pw, have, s);
                continue;
            }
        }
        if (both && direct) {
            rc = twice ? launch_both<E, T, true, Half, true>(x, g, px, pw, m, have, s)
                       : launch_both<E, T, true, T, true>(x, g, px, pw, m, have, s);
            continue;
        }
        if (c->dx)
            rc = direct ? launch_grad<T, E, true, true, false>(x, px, m, s)
                        : launch_grad<T, E, true, true, true>(x, px, m, s);
        if (!rc && c->dw)
            rc = twice ? launch_grad<Half, E, false, true, false>(g, pw, have, s)
                       : launch_grad<T, E, false, true, false>(g, pw, have, s);
    }
    return rc;
}

// The gradients of no rows.
template <class V>
__global__ __launch_bounds__(256) void clear_kernel(V *p, uint64_t rows, uint64_t cols,
                                                    uint64_t ld) {
    for (uint64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (uint64_t c = threadIdx.x; c < cols; c += 256)
            p[r * ld + c] = 0;
}

template <class V>
int clear(const ddl_ce_grad_args *a, hipStream_t s) {
    const size_t n = a->layer.n, k = a->layer.k;
    const dim3 rows((uint32_t)std::min<size_t>(n, 65536));
    int rc = DDL_OK;
    if (a->dw && k)
        rc = launch(clear_kernel<V>, rows, dim3(256), 0, s, (V *)a->dw, n, k, a->lddw);
    if (a->db && !rc)
        rc = launch(clear_kernel<V>, dim3(1), dim3(256), 0, s, (V *)a->db, 1, n, n);
    return rc;
}

}  // namespace

size_t grad_workspace(size_t m, size_t n, size_t k) {
    if (!m)
        return 0;
    Carve c{nullptr};
    carve_grad(c, m, n, k);
    return c.used;
}

static bool sizes_ok(size_t m, size_t n, size_t k) {
    return m <= kMaxTargets && n >= 1 && n <= kMaxExtent && k <= kMaxExtent;
}

int check_cross_entropy(const ddl_ce_args *a, int op, const void *ws, size_t bytes) {
    const size_t m = a->m, n = a->n, k = a->k;
    if ((a->dtype != DDL_F16 && a->dtype != DDL_BF16) || !sizes_ok(m, n, k)
        || !(a->smoothing >= 0 && a->smoothing <= 1))
        return DDL_E_ARG;
    if (!m)
        return DDL_OK;
    if (!a->target || (k && (!a->x || !a->w)))
        return DDL_E_NULL;
    if (!row_ok(a->x, a->ldx, k, m) || !row_ok(a->w, a->ldw, k, n))
        return DDL_E_ARG;
    if (!element_ok(a->x, 2) || !element_ok(a->w, 2) || !element_ok(a->bias, 2)
        || !element_ok(a->target, 8) || !element_ok(a->lse, 4))
        return DDL_E_ALIGN;
    if (!ws)
        return DDL_E_NULL;
    if ((uintptr_t)ws % 16)
        return DDL_E_ALIGN;
    const size_t need =
        op == DDL_CE_FORWARD ? loss_workspace(m, n, k) : grad_workspace(m, n, k);
    return bytes < need ? DDL_E_SCRATCH : DDL_OK;
}

}  // namespace ddl

using namespace ddl;

extern "C" {

int ddl_cross_entropy_workspace(int op, size_t m, size_t n, size_t k, size_t *bytes) {
    if (!bytes)
        return DDL_E_NULL;
    if ((op != DDL_CE_FORWARD && op != DDL_CE_GRAD) || !sizes_ok(m, n, k))
        return DDL_E_ARG;
    *bytes = !m ? 0 : op == DDL_CE_FORWARD ? loss_workspace(m, n, k) : grad_workspace(m, n, k);
    return DDL_OK;
}

int ddl_cross_entropy_grad(const ddl_ce_grad_args *a, void *workspace, size_t workspace_bytes,
                           void *stream) {
    if (!a)
        return DDL_E_NULL;
    const ddl_ce_args &l = a->layer;
    int rc = check_cross_entropy(&l, DDL_CE_GRAD, workspace, workspace_bytes);
    if (rc)
        return rc;
    if ((a->dw_dtype != DDL_F32 && a->dw_dtype != l.dtype)
        || (a->accumulate != 0 && a->accumulate != 1) || !std::isfinite(a->scale)
        || !row_ok(a->dx, a->lddx, l.k, l.m) || !row_ok(a->dw, a->lddw, l.k, l.n))
        return DDL_E_ARG;
    if (l.k && !a->dx && !a->dw && !a->db)
        return DDL_E_NULL;
    const size_t esz = a->dw_dtype == DDL_F32 ? 4 : 2;
    if (!element_ok(a->dx, 2) || !element_ok(a->dw, esz) || !element_ok(a->db, esz)
        || !element_ok(a->dloss, 4))
        return DDL_E_ALIGN;
    if (!l.m)
        return a->accumulate ? DDL_OK
               : esz == 4    ? clear<uint32_t>(a, (hipStream_t)stream)
                             : clear<uint16_t>(a, (hipStream_t)stream);
    if (!l.lse)
        return DDL_E_NULL;
    return l.dtype == DDL_F16 ? gradient<Half>(a, workspace, (hipStream_t)stream)
                              : gradient<Bfloat>(a, workspace, (hipStream_t)stream);
}

}  // extern "C"
