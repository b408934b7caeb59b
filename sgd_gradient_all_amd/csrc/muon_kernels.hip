// muon_kernels.hip -- the Muon step (gfx950): momentum, the orthogonalisation
// of every matrix by five rounds of Newton-Schulz products, and the update.
//
//     X = U / (||U||_F + 1e-7),  s x l with s <= l (U^T where U is tall)
//     five times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// All matrices of a handle go through each product in one launch, whatever
// their shapes: a table names the matrix and the tile of every workgroup.
//
// Numbers.  The rounds amplify a rounding of X as they amplify its small
// singular values (3.4445 a round), so one 16-bit product is not enough: with
// binary16 operands alone X ends 0.2 to 0.4% off, more than bfloat16's own
// rounding.  X, A and B are held as sums of two binary16 values (22 bits), and
// a product takes three passes, high*high + high*low + low*high, which ends as
// close as binary32 products do, whatever the type of the result: fewer passes
// for bfloat16 (one for A, two for B X) were 0.11 to 0.15% off beside its
// rounding of 0.17%.  Values are kept times 2^14: no entry of X passes 1.3 and
// none of A or B 2.9 in magnitude (the spectral norms bound them), so nothing
// overflows binary16, and entries as small as 2^-28 are normal numbers.
//
// A and B are symmetric: tiles on and below the diagonal are computed and
// stored twice.  Workspaces are padded with zeros to whole tiles.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "../../include/ddl.h"
#include "device_common.h"
#include "gemm_core.h"
#include "optimizer_internal.h"

namespace ddl {
namespace {

using gemm::f32x4;
using gemm::Operand;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32v8 __attribute__((ext_vector_type(8)));

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int kRounds = 5;
constexpr double kNormEps = 1e-7;
constexpr float kScale = 16384.0f, kUnscale = 1.0f / 16384.0f;
constexpr uint32_t kNormChunk = 8192;

struct Mat {
    uint64_t at;         // of the flat buffers
    uint64_t x, a, b;    // of the workspace: 2 x 2 planes of X, 2 of A, 2 of B
    uint32_t rows, cols;
    uint32_t s, l, sp, lp;
    uint32_t tall;
    float scale;
    uint32_t chunk0, chunk1;  // its parts of the sum of squares
};

// A workgroup of a product: the tile, and its part of the k tiles.
struct Work {
    uint32_t mat;
    uint16_t ti, tj;
    uint16_t part, parts;
    uint32_t slot;   // of the first part's partial sums
    uint32_t ticket; // of the tile's count of finished parts
};

struct Update {
    const void *grad;
    float *momentum;  // null: no momentum, U = grad (orthogonalise)
    float mu;
    int nesterov;
    void *out;  // orthogonalise
    float keep, lr;
    void *copy;
    int copy_type;
    int vec;
};

struct StepArgs {
    const Mat *mats;
    const Work *work;
    uint32_t count;
    uint16_t *ws;
    float *partial;
    uint32_t *tickets;
    int from;  // which of X's two copies is read
    int last;
};

// The high part is rounded from the binary32 value that the low part completes:
// without the barrier the compiler may round the product behind v to binary16
// at once in one of its two uses, and the pair is then off by a binary16 step
// where the two roundings differ (one element in some thousands).
__device__ __forceinline__ void split(float v, _Float16 &h, _Float16 &l) {
    v = dev::opaque1(v);
    h = (_Float16)v;
    l = (_Float16)(v - (float)h);
}
__device__ __forceinline__ void store_pair(uint16_t *hi, uint16_t *lo, uint64_t at,
                                           const float (&v)[8]) {
    f16x8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        _Float16 a, b;
        split(v[e], a, b);
        h[e] = a;
        l[e] = b;
    }
    *(f16x8 *)(hi + at) = h;
    *(f16x8 *)(lo + at) = l;
}
// the momentum, and the sum of squares of U over each chunk
template <class G>
__global__ __launch_bounds__(256) void norm_kernel(const Chunk *chunks, Update u,
                                                   double *partial) {
    __shared__ double lds[4];
    const Chunk c = chunks[blockIdx.x];
    const G *g = (const G *)u.grad + c.at;
    float *m = u.momentum ? u.momentum + c.at : nullptr;
    typedef float V4 __attribute__((ext_vector_type(4)));
    typedef G G4 __attribute__((ext_vector_type(4)));
    double sum = 0.0;
    uint32_t done = 0;
    auto one = [&](float gv, float &mv) {
        mv = u.mu * mv + gv;
        return u.nesterov ? gv + u.mu * mv : mv;
    };
    if (u.vec && c.at % 8 == 0) {
        done = c.count & ~3u;
#pragma unroll 4
        for (uint32_t i = threadIdx.x * 4; i < done; i += 1024) {
            const G4 gv = *(const G4 *)(g + i);
            V4 x;
            if (m) {
                V4 mv = *(V4 *)(m + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float t = mv[e];
                    x[e] = one((float)gv[e], t);
                    mv[e] = t;
                }
                *(V4 *)(m + i) = mv;
            } else {
                x = __builtin_convertvector(gv, V4);
            }
            dev::add_squares(x, sum);
        }
    }
    for (uint32_t i = done + threadIdx.x; i < c.count; i += 256) {
        float x = (float)g[i];
        if (m) {
            float t = m[i];
            x = one(x, t);
            m[i] = t;
        }
        sum += (double)x * (double)x;
    }
    sum = dev::block_sum(sum, lds);
    if (threadIdx.x == 0)
        partial[blockIdx.x] = sum;
}

// X = U / norm, times kScale, as pairs, turned where tall and padded with
// zeros: a 64 x 64 block of X a workgroup.
template <class G>
__global__ __launch_bounds__(256) void normalise_kernel(const Mat *mats, const Work *work,
                                                        Update u, const double *partial,
                                                        uint16_t *ws) {
    __shared__ double lds[4];
    __shared__ float inv_lds;
    __shared__ float block[64][65];
    const Work w = work[blockIdx.x];
    const Mat t = mats[w.mat];
    double sum = 0.0;
    for (uint32_t i = t.chunk0 + threadIdx.x; i < t.chunk1; i += 256)
        sum += partial[i];
    sum = dev::block_sum(sum, lds);
    if (threadIdx.x == 0)
        inv_lds = (float)((double)kScale / (sqrt(sum) + kNormEps));
    const uint32_t s0 = w.ti * 64u, l0 = w.tj * 64u;
    // rows and columns of U from (r0, c0) on
    const uint32_t r0 = t.tall ? l0 : s0, c0 = t.tall ? s0 : l0;
    const uint32_t cc = threadIdx.x & 63u;
#pragma unroll 4
    for (uint32_t rr = threadIdx.x >> 6; rr < 64; rr += 4) {
        float x = 0.0f;
        if (r0 + rr < t.rows && c0 + cc < t.cols) {
            const uint64_t at = t.at + (uint64_t)(r0 + rr) * t.cols + c0 + cc;
            x = (float)((const G *)u.grad)[at];
            if (u.momentum)  // already this step's
                x = u.nesterov ? x + u.mu * u.momentum[at] : u.momentum[at];
        }
        block[rr][cc] = x;
    }
    __syncthreads();
    const float inv = inv_lds;
    uint16_t *hi = ws + t.x, *lo = hi + (uint64_t)t.sp * t.lp;
    const uint32_t k = (threadIdx.x & 7u) * 8;
#pragma unroll
    for (uint32_t q = threadIdx.x >> 3; q < 64; q += 32) {
        float v[8];
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
            v[e] = inv * (t.tall ? block[k + e][q] : block[q][k + e]);
        store_pair(hi, lo, (uint64_t)(s0 + q) * t.lp + l0 + k, v);
    }
}

enum { kGram, kPoly, kApply };
constexpr uint32_t kPasses = 3;  // over k in a product

// 8 results of the last round, from element `at` of the flat buffers on.
template <class G>
__device__ __forceinline__ void apply_update(const Update &u, const Replicas &r, uint64_t at,
                                             uint32_t have, float scale, const float (&v)[8]) {
    const bool vec = u.vec && have == 8 && at % 8 == 0;
    if (u.out) {
        G *o = (G *)u.out + at;
        typedef G G8 __attribute__((ext_vector_type(8)));
        G8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = (G)(v[e] * kUnscale);
        if (vec) {
            *(G8 *)o = x;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                if (e < have)
                    o[e] = x[e];
        }
        return;
    }
    const float *w0 = r.w[0] + at;
    f32v8 w = {};
    if (vec) {
        w = *(const f32v8 *)w0;
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
            if (e < have)
                w[e] = w0[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w[e] = u.keep * w[e] - scale * (v[e] * kUnscale);
    for (int k = 0; k < r.count; ++k) {
        float *o = r.w[k] + at;
        if (vec) {
            *(f32v8 *)o = w;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                if (e < have)
                    o[e] = w[e];
        }
    }
    if (u.copy) {
        uint16_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[e] = u.copy_type == DDL_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)w[e])
                                           : __builtin_bit_cast(uint16_t, (_Float16)w[e]);
        uint16_t *o = (uint16_t *)u.copy + at;
        if (vec) {
            __builtin_memcpy(__builtin_assume_aligned(o, 16), h, 16);
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                if (e < have)
                    o[e] = h[e];
        }
    }
}

// The sums of a tile whose k is dealt to several workgroups: each leaves its
// part in memory and takes a ticket; the last has all of them, added in their
// order.  False for the others.  The parts travel past the caches (agent-scope
// accesses, complete before the ticket is drawn), since a fence at that scope
// would write back and empty the die's L2 under the workgroups beside it.
template <class Core>
__device__ __forceinline__ bool join_parts(const StepArgs &p, const Work &w,
                                           f32x4 (&acc)[Core::FM][Core::FN], uint32_t &arrived) {
    constexpr uint32_t N = Core::FM * Core::FN;
    typedef unsigned long long U;
    U *slot = (U *)p.partial + (uint64_t)w.slot * N * 2 * Core::THREADS + threadIdx.x;
    U *mine = slot + (uint64_t)w.part * N * 2 * Core::THREADS;
    struct Two {
        U v[2];
    };
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) {
        const Two two = __builtin_bit_cast(Two, acc[i / Core::FN][i % Core::FN]);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h)
            __hip_atomic_store(mine + (i * 2 + h) * Core::THREADS, two.v[h], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        arrived = __hip_atomic_fetch_add(p.tickets + w.ticket, 1u, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrived != (uint32_t)w.parts - 1)
        return false;
    if (threadIdx.x == 0)  // for the next launch
        __hip_atomic_store(p.tickets + w.ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (uint32_t q = 0; q < w.parts; ++q) {
#pragma unroll
        for (uint32_t i = 0; i < N; ++i) {
            Two two;
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
                two.v[h] = __hip_atomic_load(slot + (i * 2 + h) * Core::THREADS,
                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            f32x4 &to = acc[i / Core::FN][i % Core::FN];
            const f32x4 from = __builtin_bit_cast(f32x4, two);
            to = q ? to + from : from;
        }
        slot += (uint64_t)N * 2 * Core::THREADS;
    }
    return true;
}

// One product over the tiles of every matrix.
template <class Core, int KIND, class G>
__global__ __launch_bounds__(Core::THREADS) void product_kernel(StepArgs p, Update u,
                                                                Replicas r) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ uint32_t arrived;
    // Workgroups go round the 8 dies; runs of 8 entries, which share operands,
    // stay on one.  The table has the longest sums first.
    uint32_t entry = blockIdx.x;
    if ((entry | 63u) < p.count)
        entry = (entry & ~63u) | (entry & 7u) << 3 | (entry >> 3 & 7u);
    const Work w = p.work[entry];
    const Mat t = p.mats[w.mat];
    const uint64_t nx = (uint64_t)t.sp * t.lp, na = (uint64_t)t.sp * t.sp;
    uint16_t *x = p.ws + t.x + p.from * 2 * nx, *y = p.ws + t.x + (p.from ^ 1) * 2 * nx;
    uint16_t *a = p.ws + t.a, *b = p.ws + t.b;
    Operand left, right;
    left.row0 = w.ti * Core::BM;
    right.row0 = w.tj * Core::BN;
    left.rows = t.sp;
    if (KIND == kGram) {
        left.plane[0] = right.plane[0] = x;
        left.plane[1] = right.plane[1] = x + nx;
        left.ld = left.k = t.lp;
        right.rows = t.sp;
    } else {
        left.plane[0] = KIND == kPoly ? a : b;
        left.plane[1] = left.plane[0] + na;
        left.ld = left.k = t.sp;
        right.plane[0] = KIND == kPoly ? a : x;
        right.plane[1] = KIND == kPoly ? a + na : x + nx;
        right.rows = KIND == kPoly ? t.sp : t.lp;
    }
    right.ld = KIND == kPoly ? t.sp : t.lp;
    right.k = left.k;
    const uint32_t kt = (uint32_t)(left.k / Core::BK), all = kt * kPasses;
    f32x4 acc[Core::FM][Core::FN] = {};
    Core::run(left, right, all * w.part / w.parts, all * (w.part + 1) / w.parts, kt, lds, acc);
    if (w.parts > 1 && !join_parts<Core>(p, w, acc, arrived))
        return;
    struct Pair {
        f16x8 h, l;
    };
    auto pair_at = [](const uint16_t *hi, uint64_t low, uint64_t at) {
        return Pair{*(const f16x8 *)(hi + at), *(const f16x8 *)(hi + low + at)};
    };
    const uint32_t m0 = left.row0, n0 = right.row0;
    if constexpr (KIND == kApply) {
        auto old = [&](uint32_t mi, uint32_t ni) {
            return pair_at(x, nx, (uint64_t)(m0 + mi) * t.lp + n0 + ni);
        };
        auto next = [&](float (&v)[8], const Pair &o) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = kA * ((float)o.h[e] + (float)o.l[e]) + v[e] * kUnscale;
        };
        if (!p.last) {
            Core::each(acc, lds, old, [&](uint32_t mi, uint32_t ni, float (&v)[8], const Pair &o) {
                next(v, o);
                store_pair(y, y + nx, (uint64_t)(m0 + mi) * t.lp + n0 + ni, v);
            });
        } else if (!t.tall) {
            Core::each(acc, lds, old, [&](uint32_t mi, uint32_t ni, float (&v)[8], const Pair &o) {
                const uint32_t m = m0 + mi, n = n0 + ni;
                if (m >= t.s || n >= t.l)
                    return;
                next(v, o);
                apply_update<G>(u, r, t.at + (uint64_t)m * t.cols + n,
                                t.l - n < 8 ? t.l - n : 8, u.lr * t.scale, v);
            });
        } else {
            Core::template each<true>(
                acc, lds,
                [&](uint32_t mi, uint32_t ni) {
                    const _Float16 *h = (const _Float16 *)x + (uint64_t)(m0 + mi) * t.lp + n0 + ni;
                    Pair o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        o.h[e] = h[(uint64_t)e * t.lp];
                        o.l[e] = h[nx + (uint64_t)e * t.lp];
                    }
                    return o;
                },
                [&](uint32_t mi, uint32_t ni, float (&v)[8], const Pair &o) {
                    const uint32_t m = m0 + mi, n = n0 + ni;
                    if (m >= t.s || n >= t.l)
                        return;
                    next(v, o);
                    apply_update<G>(u, r, t.at + (uint64_t)n * t.cols + m,
                                    t.s - m < 8 ? t.s - m : 8, u.lr * t.scale, v);
                });
        }
    } else {
        uint16_t *o = KIND == kGram ? a : b;
        // the results of row m (or, A being symmetric, of column m) at `at`
        auto fetch = [&](uint64_t at) { return KIND == kGram ? Pair{} : pair_at(a, na, at); };
        auto put = [&](uint64_t at, float (&v)[8], const Pair &q) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = KIND == kGram
                           ? v[e] * kUnscale
                           : kB * ((float)q.h[e] + (float)q.l[e]) + kC * (v[e] * kUnscale);
            store_pair(o, o + na, at, v);
        };
        auto row = [&](uint32_t mi, uint32_t ni) { return (uint64_t)(m0 + mi) * t.sp + n0 + ni; };
        auto column = [&](uint32_t mi, uint32_t ni) {
            return (uint64_t)(n0 + ni) * t.sp + m0 + mi;
        };
        Core::each(
            acc, lds, [&](uint32_t mi, uint32_t ni) { return fetch(row(mi, ni)); },
            [&](uint32_t mi, uint32_t ni, float (&v)[8], const Pair &q) {
                put(row(mi, ni), v, q);
            });
        if (w.ti != w.tj)  // the mirror image
            Core::template each<true>(
                acc, lds, [&](uint32_t mi, uint32_t ni) { return fetch(column(mi, ni)); },
                [&](uint32_t mi, uint32_t ni, float (&v)[8], const Pair &q) {
                    put(column(mi, ni), v, q);
                });
    }
}

// ---------------------------------------------------------------------------
// binary64 products, for orthogonalising binary32 matrices
//
// Pairs of binary16 values leave 1 to 2e-6 after the five rounds, some 20
// steps of a binary32 result; the form that returns binary32 therefore works
// in binary64 throughout, on v_mfma_f64_16x16x4.  A workgroup of 4 waves takes
// a 64 x 64 tile, 16 k at a time through LDS, the next 16 on their way to
// registers meanwhile; rows of LDS are 2 doubles longer than their contents,
// which spreads the banks.
// ---------------------------------------------------------------------------

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef double f64x2 __attribute__((ext_vector_type(2)));

template <int KIND>
__global__ __launch_bounds__(256) void product64_kernel(const Mat *mats, const Work *work,
                                                        double *ws, int from, int last,
                                                        float *out) {
    constexpr int K = 16;
    __shared__ __attribute__((aligned(16))) double la[64][K + 2];
    __shared__ __attribute__((aligned(16))) double lb[64][K + 2];  // [n][k]
    const Work w = work[blockIdx.x];
    const Mat t = mats[w.mat];
    const uint64_t nx = (uint64_t)t.sp * t.lp;
    // X twice, A and B, each half as many doubles as the pairs' halves
    double *x = ws + t.x / 2 + from * nx, *y = ws + t.x / 2 + (from ^ 1) * nx;
    double *a = ws + t.a / 2, *b = ws + t.b / 2;
    const double *left = KIND == kGram ? x : KIND == kPoly ? a : b;
    const double *right = KIND == kPoly ? a : x;
    const uint64_t ldl = KIND == kGram ? t.lp : t.sp, ldr = KIND == kPoly ? t.sp : t.lp;
    const uint32_t k = KIND == kGram ? t.lp : t.sp, m0 = w.ti * 64u, n0 = w.tj * 64u;
    const uint32_t l = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = l & 15u, g = l >> 4;
    const uint32_t mw = (wave >> 1) * 32, nw = (wave & 1u) * 32;
    // loads: 64 rows of 16 (two 8-lane pieces of a row), or 16 rows of 64
    const uint32_t row = threadIdx.x >> 2, piece = (threadIdx.x & 3u) * 4;
    const uint32_t krow = threadIdx.x >> 4, col = (threadIdx.x & 15u) * 4;
    f64x2 ra[2], rb[2];
    auto fetch = [&](uint32_t k0) {
        const double *p = left + (uint64_t)(m0 + row) * ldl + k0 + piece;
        ra[0] = *(const f64x2 *)p;
        ra[1] = *(const f64x2 *)(p + 2);
        p = KIND == kApply ? right + (uint64_t)(k0 + krow) * ldr + n0 + col
                           : right + (uint64_t)(n0 + row) * ldr + k0 + piece;
        rb[0] = *(const f64x2 *)p;
        rb[1] = *(const f64x2 *)(p + 2);
    };
    f64x4 acc[2][2] = {};
    fetch(0);
    for (uint32_t k0 = 0; k0 < k; k0 += K) {
        __syncthreads();
        *(f64x2 *)&la[row][piece] = ra[0];
        *(f64x2 *)&la[row][piece + 2] = ra[1];
        if (KIND == kApply) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                lb[col + e][krow] = rb[e / 2][e % 2];
        } else {
            *(f64x2 *)&lb[row][piece] = rb[0];
            *(f64x2 *)&lb[row][piece + 2] = rb[1];
        }
        __syncthreads();
        if (k0 + K < k)
            fetch(k0 + K);
#pragma unroll
        for (int kk = 0; kk < K; kk += 4) {
            double fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = la[mw + 16 * i + r][kk + g];
                fb[i] = lb[nw + 16 * i + r][kk + g];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(fa[i], fb[j], acc[i][j], 0,
                                                                     0, 0);
        }
    }
    // a lane's results: column r, rows 4 e + g of each 16 x 16
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m = m0 + mw + 16 * i + 4 * e + g, n = n0 + nw + 16 * j + r;
                const double v = acc[i][j][e];
                if (KIND == kApply) {
                    const uint64_t at = (uint64_t)m * t.lp + n;
                    const double q = 3.4445 * x[at] + v;
                    if (!last)
                        y[at] = q;
                    else if (m < t.s && n < t.l)
                        out[t.at + (t.tall ? (uint64_t)n * t.cols + m
                                           : (uint64_t)m * t.cols + n)] = (float)q;
                } else {
                    const uint64_t at = (uint64_t)m * t.sp + n;
                    const double q = KIND == kGram ? v : -4.7750 * a[at] + 2.0315 * v;
                    double *o = KIND == kGram ? a : b;
                    o[at] = q;
                    if (w.ti != w.tj)
                        o[(uint64_t)n * t.sp + m] = q;
                }
            }
}

// X = U / norm in binary64, as normalise_kernel does in pairs.
__global__ __launch_bounds__(256) void normalise64_kernel(const Mat *mats, const Work *work,
                                                          const float *u, const double *partial,
                                                          double *ws) {
    __shared__ double lds[4];
    __shared__ double norm_lds;
    __shared__ float block[64][65];
    const Work w = work[blockIdx.x];
    const Mat t = mats[w.mat];
    double sum = 0.0;
    for (uint32_t i = t.chunk0 + threadIdx.x; i < t.chunk1; i += 256)
        sum += partial[i];
    sum = dev::block_sum(sum, lds);
    if (threadIdx.x == 0)
        norm_lds = 1.0 / (sqrt(sum) + kNormEps);
    const uint32_t s0 = w.ti * 64u, l0 = w.tj * 64u;
    const uint32_t r0 = t.tall ? l0 : s0, c0 = t.tall ? s0 : l0;
    const uint32_t cc = threadIdx.x & 63u;
#pragma unroll 4
    for (uint32_t rr = threadIdx.x >> 6; rr < 64; rr += 4)
        block[rr][cc] = r0 + rr < t.rows && c0 + cc < t.cols
                            ? u[t.at + (uint64_t)(r0 + rr) * t.cols + c0 + cc]
                            : 0.0f;
    __syncthreads();
    const double inv = norm_lds;
    double *x = ws + t.x / 2;
    for (uint32_t q = threadIdx.x >> 6; q < 64; q += 4)
        x[(uint64_t)(s0 + q) * t.lp + l0 + cc] =
            inv * (double)(t.tall ? block[cc][q] : block[q][cc]);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr uint32_t kMaxSide = 65536;

uint32_t up(uint32_t v, uint32_t to) { return (v + to - 1) / to * to; }

}  // namespace
}  // namespace ddl

using namespace ddl;

struct ddl_muon_s {
    std::vector<Mat> mats;
    std::vector<Chunk> chunks;
    std::vector<Work> blocks;       // normalise
    std::vector<Work> gram, poly, apply;  // the products
    uint32_t tile = 64;
    uint64_t ws = 0;  // 16-bit elements of the workspace
    // binary64: the tables of 64 x 64 tiles, made by the first call
    std::vector<Work> tri64, all64;
    Work *d_tri64 = nullptr, *d_all64 = nullptr;
    double *d_ws64 = nullptr;
    uint64_t slots = 0;  // partial tiles
    uint32_t tickets = 0;
    std::vector<uint32_t> zeros;  // the tickets' start; made here: a step does not throw

    Handle dev;
    Mat *d_mats = nullptr;
    Chunk *d_chunks = nullptr;
    Work *d_blocks = nullptr, *d_gram = nullptr, *d_poly = nullptr, *d_apply = nullptr;
    uint16_t *d_ws = nullptr;
    float *d_partial = nullptr;
    uint32_t *d_tickets = nullptr;
    double *d_sums = nullptr;
};

namespace ddl {
namespace {

// Tiles of a product over all matrices, k cut into parts where the tiles
// alone do not fill the card.
void deal(ddl_muon_s &h, int kind, std::vector<Work> &out) {
    const uint32_t T = h.tile;
    uint64_t tiles = 0;
    auto count = [&](const Mat &m, auto &&then) {
        const uint32_t ni = m.sp / T, nj = kind == kApply ? m.lp / T : ni;
        for (uint32_t j = 0; j < nj; ++j)
            for (uint32_t i = kind == kApply ? 0 : j; i < ni; ++i)
                then(i, j);
    };
    uint64_t steps = 0;  // k tiles over all tiles
    auto depth = [&](const Mat &m) {
        return (uint64_t)(kind == kGram ? m.lp : m.sp) / 64 * kPasses;
    };
    for (const Mat &m : h.mats)
        count(m, [&](uint32_t, uint32_t) {
            ++tiles;
            steps += depth(m);
        });
    // parts of at most this many k tiles: the load of one of 512 equal shares
    // (ResNet-50's matrices: 1.32 ms, uncut 1.84, of 1024 shares 1.46; one 4096
    // x 1024 in 16 bits: 590 us, 886 and 649)
    const uint64_t share = std::max<uint64_t>((steps + 511) / 512, 16);
    uint64_t slots = 0;
    uint32_t tickets = 0;
    std::vector<uint32_t> order(h.mats.size());
    for (uint32_t i = 0; i < order.size(); ++i)
        order[i] = i;
    std::stable_sort(order.begin(), order.end(), [&](uint32_t x, uint32_t y) {
        return depth(h.mats[x]) > depth(h.mats[y]);
    });
    for (uint32_t i : order) {
        const uint64_t d = depth(h.mats[i]);
        const uint16_t parts =
            tiles >= 512 ? 1 : (uint16_t)std::max<uint64_t>(1, std::min<uint64_t>(d / share, 32));
        count(h.mats[i], [&](uint32_t ti, uint32_t tj) {
            for (uint16_t q = 0; q < parts; ++q)
                out.push_back({i, (uint16_t)ti, (uint16_t)tj, q, parts, (uint32_t)slots,
                               tickets});
            if (parts > 1) {
                slots += parts;
                ++tickets;
            }
        });
    }
    h.slots = std::max(h.slots, slots);
    h.tickets = std::max(h.tickets, tickets);
}

void lay_out(ddl_muon_s &h) {
    // The largest tile of which A's lower triangles give every compute unit
    // one (256) or every other (128): with fewer, too few workgroups hide each
    // other's waits, and the sums over k are cut into more parts to join
    // (ResNet-50's matrices: 2.2 ms with 256, 1.3 ms with 128; one 4096 x 1024
    // in bfloat16: 636 us with 128, 590 us with 64).  And of which the products
    // that are issued, padding and halves above the diagonal included, are not
    // more than what a larger tile's rate makes up for: 1.45 times those of 64
    // (1.43 times, 100 of 400 x 1600: 4.09 ms with 64, 3.87 with 128; 1.54
    // times, 100 of 300 x 900: 1.48 and 1.81 ms; 8 times, 300 of 64 x 64: 106
    // and 242 us, with 256 1095 us), 1.03 times those of 128 (1.03 times, 8 of
    // 2304 x 2304: 8.02 ms with 128, 7.53 with 256; 1.06 times, 26 of 1024 x
    // 1024: 2.76 and 3.03 ms).
    auto triangles = [&](uint32_t T) {
        uint64_t n = 0;
        for (const Mat &m : h.mats)
            n += (uint64_t)(up(m.s, T) / T) * (up(m.s, T) / T + 1) / 2;
        return n;
    };
    auto issued = [&](uint32_t T) {
        double n = 0;
        for (const Mat &m : h.mats) {
            const double s = up(m.s, T), l = up(m.l, T);
            n += s * (s + T) / 2 * (l + s) + s * s * l;
        }
        return n;
    };
    h.tile = 64;
    if (triangles(128) >= 128 && issued(128) <= 1.45 * issued(64)) {
        h.tile = 128;
        if (triangles(256) >= 256 && issued(256) <= 1.03 * issued(128))
            h.tile = 256;
    }
    for (uint32_t i = 0; i < h.mats.size(); ++i) {
        Mat &m = h.mats[i];
        m.sp = up(m.s, h.tile);
        m.lp = up(m.l, h.tile);
        m.x = h.ws;
        h.ws += 4ull * m.sp * m.lp;
        m.a = h.ws;
        h.ws += 2ull * m.sp * m.sp;
        m.b = h.ws;
        h.ws += 2ull * m.sp * m.sp;
        m.chunk0 = (uint32_t)h.chunks.size();
        cut_chunks({m.at, (uint64_t)m.rows * m.cols}, kNormChunk, h.chunks, i);
        m.chunk1 = (uint32_t)h.chunks.size();
        for (uint32_t a = 0; a < m.sp / 64; ++a)
            for (uint32_t b = 0; b < m.lp / 64; ++b)
                h.blocks.push_back({i, (uint16_t)a, (uint16_t)b, 0, 1, 0, 0});
        for (uint32_t b = 0; b < m.lp / 64; ++b)
            for (uint32_t a = 0; a < m.sp / 64; ++a) {
                h.all64.push_back({i, (uint16_t)a, (uint16_t)b, 0, 1, 0, 0});
                if (b <= a)
                    h.tri64.push_back(h.all64.back());
            }
    }
    deal(h, kGram, h.gram);
    deal(h, kPoly, h.poly);
    deal(h, kApply, h.apply);
    h.zeros.assign(h.tickets, 0);
}

int bind_muon(ddl_muon_s &h, hipStream_t s) {
    return h.dev.bind(s, [&]() -> int {
        int rc = upload(h.mats, &h.d_mats);
        rc = rc ? rc : upload(h.chunks, &h.d_chunks);
        rc = rc ? rc : upload(h.blocks, &h.d_blocks);
        rc = rc ? rc : upload(h.gram, &h.d_gram);
        rc = rc ? rc : upload(h.poly, &h.d_poly);
        rc = rc ? rc : upload(h.apply, &h.d_apply);
        rc = rc ? rc : upload(h.zeros, &h.d_tickets);
        rc = rc ? rc : device_memory(&h.d_ws, h.ws);
        rc = rc ? rc
                : device_memory(&h.d_partial,
                                std::max<uint64_t>(1, h.slots) * h.tile * h.tile);
        rc = rc ? rc : device_memory(&h.d_sums, h.chunks.size());
        if (rc) {  // nothing half made: the next call starts anew
            (void)hipFree(h.d_mats), (void)hipFree(h.d_chunks), (void)hipFree(h.d_blocks);
            (void)hipFree(h.d_tickets), (void)hipFree(h.d_ws), (void)hipFree(h.d_partial);
            (void)hipFree(h.d_sums), (void)hipFree(h.d_gram), (void)hipFree(h.d_poly);
            (void)hipFree(h.d_apply);
            h.d_mats = nullptr, h.d_chunks = nullptr, h.d_blocks = nullptr;
            h.d_tickets = nullptr, h.d_ws = nullptr, h.d_partial = nullptr, h.d_sums = nullptr;
            h.d_gram = h.d_poly = h.d_apply = nullptr;
        }
        return rc;
    });
}

template <class Core, int KIND, class G>
int launch_product(const StepArgs &p, const Update &u, const Replicas &r, hipStream_t s) {
    const int rc = allow_lds(product_kernel<Core, KIND, G>, Core::LDS);
    return rc ? rc
              : launch(product_kernel<Core, KIND, G>, dim3(p.count), dim3(Core::THREADS),
                       Core::LDS, s, p, u, r);
}

template <int T, class G>
int rounds(ddl_muon_s &h, const Update &u, const Replicas &r, hipStream_t s) {
    constexpr int WR = 2, WC = T == 256 ? 4 : 2;
    constexpr int BK = 64, S = T == 64 ? 3 : 2;
    using Rows = gemm::Core<gemm::Half, T, T, WR, WC, BK, S, false, false, false>;
    using Cols = gemm::Core<gemm::Half, T, T, WR, WC, BK, S, false, true, false>;
    StepArgs p;
    p.mats = h.d_mats;
    p.ws = h.d_ws;
    p.partial = h.d_partial;
    p.tickets = h.d_tickets;
    int rc = DDL_OK;
    for (int i = 0; i < kRounds && !rc; ++i) {
        p.from = i & 1;
        p.last = i == kRounds - 1;
        p.work = h.d_gram;
        p.count = (uint32_t)h.gram.size();
        rc = launch_product<Rows, kGram, float>(p, u, r, s);
        p.work = h.d_poly;
        p.count = (uint32_t)h.poly.size();
        rc = rc ? rc : launch_product<Rows, kPoly, float>(p, u, r, s);
        p.work = h.d_apply;
        p.count = (uint32_t)h.apply.size();
        rc = rc ? rc : launch_product<Cols, kApply, G>(p, u, r, s);
    }
    return rc;
}

// orthogonalise in binary32: the binary64 workspace (8 bytes for 4 of the
// pairs' planes) is allocated by the first such call.
int run64(ddl_muon_s &h, const Update &u, hipStream_t s) {
    if (!h.d_ws64) {
        int rc = Handle::not_capturing(s);
        rc = rc || h.d_tri64 ? rc : upload(h.tri64, &h.d_tri64);
        rc = rc || h.d_all64 ? rc : upload(h.all64, &h.d_all64);
        rc = rc ? rc : device_memory(&h.d_ws64, h.ws / 2);
        if (rc)
            return rc;
    }
    int rc = launch(norm_kernel<float>, dim3((uint32_t)h.chunks.size()), dim3(256), 0, s,
                    h.d_chunks, u, h.d_sums);
    rc = rc ? rc
            : launch(normalise64_kernel, dim3((uint32_t)h.blocks.size()), dim3(256), 0, s,
                     h.d_mats, h.d_blocks, (const float *)u.grad, h.d_sums, h.d_ws64);
    const dim3 tri((uint32_t)h.tri64.size()), all((uint32_t)h.all64.size());
    for (int i = 0; i < kRounds && !rc; ++i) {
        auto product = [&](auto kernel, dim3 grid, const Work *work) {
            rc = rc ? rc
                    : launch(kernel, grid, dim3(256), 0, s, h.d_mats, work, h.d_ws64, i & 1,
                             i == kRounds - 1, (float *)u.out);
        };
        product(product64_kernel<kGram>, tri, h.d_tri64);
        product(product64_kernel<kPoly>, tri, h.d_tri64);
        product(product64_kernel<kApply>, all, h.d_all64);
    }
    return rc;
}

template <class G>
int run_muon(ddl_muon_s &h, const Update &u, const Replicas &r, hipStream_t s) {
    int rc = launch(norm_kernel<G>, dim3((uint32_t)h.chunks.size()), dim3(256), 0, s, h.d_chunks,
                    u, h.d_sums);
    rc = rc ? rc
            : launch(normalise_kernel<G>, dim3((uint32_t)h.blocks.size()), dim3(256), 0, s,
                     h.d_mats, h.d_blocks, u, h.d_sums, h.d_ws);
    if (rc)
        return rc;
    return h.tile == 256   ? rounds<256, G>(h, u, r, s)
           : h.tile == 128 ? rounds<128, G>(h, u, r, s)
                           : rounds<64, G>(h, u, r, s);
}

int run_typed(ddl_muon_s &h, int type, const Update &u, const Replicas &r, void *stream) {
    hipStream_t s = (hipStream_t)stream;
    return type == DDL_F32   ? run_muon<float>(h, u, r, s)
           : type == DDL_F16 ? run_muon<_Float16>(h, u, r, s)
                             : run_muon<__bf16>(h, u, r, s);
}

}  // namespace
}  // namespace ddl

extern "C" {

int ddl_muon_create(ddl_muon *out, const ddl_muon_matrix *matrices, int nmatrices) {
    if (!out || (nmatrices > 0 && !matrices))
        return DDL_E_NULL;
    *out = nullptr;
    if (nmatrices < 0)
        return DDL_E_ARG;
    ddl_muon h = nullptr;
    int rc = DDL_OK;
    try {
        h = new ddl_muon_s;
        std::vector<Span> spans;
        for (int i = 0; i < nmatrices && !rc; ++i) {
            const ddl_muon_matrix &m = matrices[i];
            if (m.rows > kMaxSide || m.cols > kMaxSide || !std::isfinite(m.scale))
                rc = DDL_E_ARG;
            if (rc || !m.rows || !m.cols)
                continue;
            spans.push_back({m.offset, m.rows * m.cols});
            Mat t = {};
            t.at = m.offset;
            t.rows = (uint32_t)m.rows;
            t.cols = (uint32_t)m.cols;
            t.tall = m.rows > m.cols;
            t.s = std::min(t.rows, t.cols);
            t.l = std::max(t.rows, t.cols);
            t.scale = (float)m.scale;
            h->mats.push_back(t);
        }
        if (!rc && !disjoint(spans))
            rc = DDL_E_BUCKETS;
        if (!rc) {
            lay_out(*h);
            if (h->slots > UINT32_MAX || h->apply.size() > kMaxGrid
                || h->blocks.size() > kMaxGrid)
                rc = DDL_E_ARG;
        }
        if (!rc)
            register_handle(h);
    } catch (...) {
        rc = DDL_E_NOMEM;
    }
    if (rc) {
        delete h;
        return rc;
    }
    *out = h;
    return DDL_OK;
}

int ddl_muon_destroy(ddl_muon h) {
    if (!h)
        return DDL_E_NULL;
    if (!unregister_handle(h))
        return DDL_E_ARG;
    h->dev.release(h->d_mats, h->d_chunks, h->d_blocks, h->d_gram, h->d_poly, h->d_apply, h->d_ws,
                   h->d_partial, h->d_tickets, h->d_sums, h->d_tri64, h->d_all64, h->d_ws64);
    delete h;
    return DDL_OK;
}

int ddl_muon_orthogonalise(ddl_muon h, const void *grad, void *out, int dtype, void *stream) {
    if (!h)
        return DDL_E_NULL;
    std::unique_lock<std::mutex> lk;
    if (!hold_handle(h, lk) || !float_type(dtype))
        return DDL_E_ARG;
    if (h->mats.empty())
        return DDL_OK;
    if (!grad || !out)
        return DDL_E_NULL;
    if (!aligned_to(grad, dtype) || !aligned_to(out, dtype))
        return DDL_E_ALIGN;
    const int rc = bind_muon(*h, (hipStream_t)stream);
    if (rc)
        return rc;
    Update u = {};
    u.grad = grad;
    u.out = out;
    u.vec = !(((uintptr_t)grad | (uintptr_t)out) % 16);
    Replicas r = {};
    if (dtype == DDL_F32)
        return run64(*h, u, (hipStream_t)stream);
    return run_typed(*h, dtype, u, r, stream);
}

int ddl_muon_step(ddl_muon h, const void *grad, int grad_dtype, float *momentum,
                  float *const *weights, int nweights, void *copy, int copy_dtype, double lr,
                  double momentum_decay, int nesterov, double weight_decay, void *stream) {
    if (!h)
        return DDL_E_NULL;
    std::unique_lock<std::mutex> lk;
    if (!hold_handle(h, lk) || nweights < 1 || nweights > DDL_MAX_RANKS
        || !float_type(grad_dtype) || (copy && copy_dtype != DDL_F16 && copy_dtype != DDL_BF16)
        || (nesterov != 0 && nesterov != 1) || !std::isfinite(lr)
        || !std::isfinite(momentum_decay) || !std::isfinite(weight_decay))
        return DDL_E_ARG;
    if (h->mats.empty())
        return DDL_OK;
    Replicas r = {};
    int rc = take_replicas(weights, nweights, r);
    if (rc)
        return rc;
    if (!grad || !momentum)
        return DDL_E_NULL;
    if (!aligned_to(grad, grad_dtype) || !aligned_to(momentum, DDL_F32)
        || (copy && !aligned_to(copy, copy_dtype)))
        return DDL_E_ALIGN;
    rc = bind_muon(*h, (hipStream_t)stream);
    if (rc)
        return rc;
    Update u = {};
    u.grad = grad;
    u.momentum = momentum;
    u.mu = (float)momentum_decay;
    u.nesterov = nesterov;
    u.keep = (float)(1 - lr * weight_decay);
    u.lr = (float)lr;
    u.copy = copy;
    u.copy_type = copy_dtype;
    uintptr_t any = (uintptr_t)grad | (uintptr_t)momentum | (uintptr_t)copy;
    for (int i = 0; i < nweights; ++i)
        any |= (uintptr_t)weights[i];
    u.vec = any % 16 == 0;
    return run_typed(*h, grad_dtype, u, r, stream);
}

}  // extern "C"
