// cross_entropy_loss.hip -- softmax cross entropy of a projection (gfx950):
//
//     z = x w^T + bias,   lse_i = log sum_j exp z_ij
//     loss_i = lse_i - (1 - a) z_i,target(i) - a mean_j z_ij
//
// The logits stay in the matrix instruction's registers: every tile of the
// product leaves, for each of its rows, the largest logit and the sum of the
// exponentials under it (and the sum of the logits where a > 0), 8 bytes for 256
// logits, and a second kernel joins a row's tiles.  The product bounds it.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "cross_entropy_internal.h"

namespace ddl {
namespace {

using gemm::Bfloat;
using gemm::f32x4;
using gemm::Half;

constexpr float kNone = -__builtin_huge_valf();  // the largest of no logits

// exp(v - top), and 0 where all logits so far are -inf
__device__ __forceinline__ float part_of(float v, float top) {
    return __builtin_amdgcn_exp2f((v - (top == kNone ? 0.0f : top)) * kLog2e);
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

// The factor of row i's dz: rounded once, so that neither side's range is a limit.
__device__ __forceinline__ float factor_of(const RowsArgs &a, uint64_t i) {
    return (float)(a.dloss ? (double)a.dloss[i] * a.scale : a.scale);
}

__device__ __forceinline__ void write_row(const RowsArgs &a, const Rows &r, uint64_t at,
                                          uint32_t i, long long target) {
    const bool bad = (uint64_t)target >= a.n;
    r.row[at] = i;
    r.target[at] = bad ? kBadTarget : (int32_t)target;
    if (a.lse) {
        r.lse[at] = a.lse[i];
        r.g[at] = bad ? __builtin_nanf("") : factor_of(a, i);
    }
}

// |g| where it counts for the factor: an infinite one would take the others' digits.
__device__ __forceinline__ float size_of(float g) {
    return fabsf(g) < __builtin_huge_valf() ? fabsf(g) : 0.0f;
}

// Gradient: the exponent is that of the power of two that takes the largest
// |dloss scale| to [2^14, 2^15): from -113 to 163, which no binary32 factor holds.
// dz = 2^exponent dloss scale (p - wanted) is held in 16 bits, and |p - wanted| <= 1:
// so binary16 keeps 11 bits of every p down to 2^-29 of the largest row's, whatever
// the loss is scaled by.
__device__ __forceinline__ void write_head(const Rows &r, uint32_t count, float top) {
    int e = 0;
    if (top > 0.0f) {
        (void)frexpf(top, &e);  // top = f 2^e, f in [1/2, 1)
        e = 15 - e;
    }
    r.head->count = count;
    r.head->exponent = e;
}

// Packs the indices of the rows with a target, in their order: one workgroup,
// 4096 targets at a time (their counts by wave are then one wave's scan).
__global__ __launch_bounds__(1024) void rows_kernel(RowsArgs a, Rows r) {
    constexpr uint32_t U = 4, WAVES = 16;
    __shared__ uint32_t counts[U * WAVES], before[U * WAVES + 1];
    __shared__ float tops[WAVES];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    uint32_t base = 0;
    float top = 0.0f;
    for (uint32_t i0 = 0; i0 < a.m; i0 += U * 1024) {
        long long t[U];
        float g[U];
        uint64_t have[U];
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            const uint32_t i = i0 + j * 1024 + threadIdx.x;
            t[j] = i < a.m ? a.target[i] : -1;
            g[j] = i < a.m && a.lse ? factor_of(a, i) : 1.0f;
        }
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            t[j] = g[j] == 0.0f ? -1 : t[j];
            have[j] = __ballot(t[j] >= 0);
            if (lane == 0)
                counts[j * WAVES + wave] = (uint32_t)__popcll(have[j]);
        }
        __syncthreads();
        if (wave == 0) {
            uint32_t sum = counts[lane];
#pragma unroll
            for (uint32_t d = 1; d < 64; d *= 2) {
                const uint32_t left = __shfl_up(sum, d);
                sum += lane >= d ? left : 0;
            }
            before[lane + 1] = sum;
            if (lane == 0)
                before[0] = 0;
        }
        __syncthreads();
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            const uint32_t i = i0 + j * 1024 + threadIdx.x;
            if (t[j] >= 0) {
                const uint32_t at = base + before[j * WAVES + wave]
                                    + (uint32_t)__popcll(have[j] & ((1ull << lane) - 1));
                write_row(a, r, at, i, t[j]);
                if (a.lse)
                    top = fmaxf(top, size_of(g[j]));
            } else if (i < a.m && a.loss) {
                a.loss[i] = 0.0f;
                a.lse_out[i] = 0.0f;
            }
        }
        base += before[U * WAVES];
        __syncthreads();
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0)
        tops[wave] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t w = 1; w < WAVES; ++w)
            top = fmaxf(top, tops[w]);
        write_head(r, base, top);
    }
}

// One row of k elements by a workgroup, zeros up to ld.
__device__ __forceinline__ void copy_row(const uint16_t *from, uint64_t k, uint16_t *to,
                                         uint64_t ld) {
    for (uint64_t c = threadIdx.x * 8; c < ld; c += 256 * 8) {
        u32x4 v;
        if (c + 8 <= k) {
            __builtin_memcpy(&v, from + c, 16);
        } else {
            uint16_t e[8];
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i)
                e[i] = c + i < k ? from[c + i] : (uint16_t)0;
            __builtin_memcpy(&v, e, 16);
        }
        *(u32x4 *)(to + c) = v;
    }
}

__device__ __forceinline__ void zero_row(uint16_t *to, uint64_t ld) {
    for (uint64_t c = threadIdx.x * 8; c < ld; c += 256 * 8)
        *(u32x4 *)(to + c) = u32x4{0, 0, 0, 0};
}

__device__ __forceinline__ void clear_words(const Rows &r) {
    for (uint64_t i = blockIdx.x * 256 + threadIdx.x; i < r.clear_count;
         i += (uint64_t)gridDim.x * 256)
        r.clear[i] = 0;
}

__global__ __launch_bounds__(256) void matrix_kernel(const uint16_t *from, uint64_t ld, uint64_t k,
                                                     uint16_t *to, uint64_t ld_to) {
    copy_row(from + blockIdx.x * ld, k, to + blockIdx.x * ld_to, ld_to);
}

// Row blockIdx.x of the packed x, zeros up to its ld, and of dx, where the
// caller's row of that index is not packed.
__global__ __launch_bounds__(256) void pack_kernel(RowsArgs a, Rows r) {
    const uint64_t i = blockIdx.x, count = r.head->count;
    clear_words(r);
    if (i >= count && i < up64(count))
        zero_row(r.x + i * r.ld, r.ld);
    if (i < count) {
        const uint16_t *from = (const uint16_t *)a.x + (uint64_t)r.row[i] * a.ldx;
        uint16_t *to = r.x + i * r.ld;
        copy_row(from, a.k, to, r.ld);
    }
    if (a.dx && i < a.m && (a.target[i] < 0 || factor_of(a, i) == 0.0f))
        for (uint64_t c = threadIdx.x; c < a.k; c += 256)
            a.dx[i * a.lddx + c] = 0;
}

// Both at once for few rows, where a launch counts: workgroup i counts the targets
// before its own row.
constexpr uint32_t kPackFew = 1024;

__global__ __launch_bounds__(256) void pack_few_kernel(RowsArgs a, Rows r) {
    __shared__ uint32_t before[4], have[4];
    __shared__ float tops[4];
    const uint32_t i = blockIdx.x, lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    clear_words(r);
    auto target = [&](uint32_t at, float &g) {
        const bool in = at < a.m;
        const long long t = a.target[in ? at : 0];
        g = a.lse ? factor_of(a, in ? at : 0) : 1.0f;
        return in && g != 0.0f ? t : -1;
    };
    float own_g;
    const long long own = target(i, own_g);
    long long t[kPackFew / 256];
    float g[kPackFew / 256];
#pragma unroll
    for (uint32_t j = 0; j < kPackFew / 256; ++j) {
        t[j] = target(j * 256 + threadIdx.x, g[j]);
        g[j] = t[j] >= 0 ? size_of(g[j]) : 0.0f;
    }
    uint32_t b = 0, h = 0;
    float top = 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < kPackFew / 256; ++j) {
        h += (uint32_t)__popcll(__ballot(t[j] >= 0));
        b += (uint32_t)__popcll(__ballot(t[j] >= 0 && j * 256 + threadIdx.x < i));
        top = fmaxf(top, g[j]);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) {
        before[wave] = b;
        have[wave] = h;
        tops[wave] = top;
    }
    __syncthreads();
    const uint32_t at = before[0] + before[1] + before[2] + before[3];
    const uint32_t count = have[0] + have[1] + have[2] + have[3];
    if (i == 0 && threadIdx.x == 0)
        write_head(r, count, fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
    if (i >= count && i < up64(count))
        zero_row(r.x + i * r.ld, r.ld);
    if (i >= a.m)
        return;
    if (own >= 0) {
        if (threadIdx.x == 0)
            write_row(a, r, at, i, own);
        copy_row((const uint16_t *)a.x + i * a.ldx, a.k, r.x + at * r.ld, r.ld);
        return;
    }
    if (a.loss && threadIdx.x == 0) {
        a.loss[i] = 0.0f;
        a.lse_out[i] = 0.0f;
    }
    if (a.dx)
        for (uint64_t c = threadIdx.x; c < a.k; c += 256)
            a.dx[i * a.lddx + c] = 0;
}

}  // namespace

int pack_rows(const RowsArgs &a, const Rows &r, hipStream_t s) {
    if (a.m <= kPackFew)
        return launch(pack_few_kernel, dim3((uint32_t)up64(a.m)), dim3(256), 0, s, a, r);
    const int rc = launch(rows_kernel, dim3(1), dim3(1024), 0, s, a, r);
    return rc ? rc : launch(pack_kernel, dim3((uint32_t)up64(a.m)), dim3(256), 0, s, a, r);
}

int pack_matrix(const void *from, size_t ld, size_t rows, size_t k, uint16_t *to, hipStream_t s) {
    return launch(matrix_kernel, dim3((uint32_t)rows), dim3(256), 0, s, (const uint16_t *)from,
                  (uint64_t)ld, (uint64_t)k, to, (uint64_t)up64(k));
}

namespace {

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------

struct LossArgs {
    Rows rows;
    const long long *target;  // few rows, which are not packed: the caller's; or null
    Operand x, w;
    const void *bias;       // T or null
    uint64_t m, n;
    uint32_t first, tn;     // columns' tiles of this launch
    float *top, *sum, *all; // [part][m]; all: or null
};

// A tile's rows: largest logit and sum of exponentials.  A lane holds, of row
// l % 16 of each of its FM fragments, 4 columns of each of the FN fragments;
// the row's other columns of the wave are in the lanes 16, 32 and 48 on, and
// the waves' parts are joined through LDS.
template <class T, class Core>
__global__ __launch_bounds__(Core::THREADS) void loss_kernel(LossArgs a) {
    using E = typename T::E;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr uint32_t BM = Core::BM, BN = Core::BN;
    const uint32_t count = a.rows.head->count, tm = (count + BM - 1) / BM;
    if (blockIdx.x >= tm * a.tn)
        return;
    uint32_t ti, tj;
    tile_of(blockIdx.x, tm, a.tn, ti, tj);
    tj += a.first;
    a.x.row0 = ti * BM;
    a.x.rows = count;
    a.w.row0 = tj * BN;
    f32x4 acc[Core::FM][Core::FN] = {};
    if (a.x.k)
        Core::run(a.x, a.w, 0, (uint32_t)((a.x.k + Core::BK - 1) / Core::BK), 0, lds, acc);
    const uint32_t wave = threadIdx.x >> 6, l = threadIdx.x & 63u;
    const uint32_t m0 = (wave / Core::WC) * (Core::FM * 16) + (l & 15u);
    const uint32_t n0 = (wave % Core::WC) * (Core::FN * 16) + (l >> 4) * 4;
    const uint64_t col = (uint64_t)tj * BN + n0;
    if (a.bias)
#pragma unroll
        for (int j = 0; j < Core::FN; ++j) {
            const uint64_t c = col + j * 16;
            float b[4];
            load4((const E *)a.bias + c, c < a.n ? (uint32_t)(a.n - c) : 0u, b);
#pragma unroll
            for (int i = 0; i < Core::FM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] += b[e];
        }
    uint32_t want[Core::FM];  // the target, from the lane's first column on
#pragma unroll
    for (int i = 0; i < Core::FM; ++i) {
        const uint32_t row = ti * BM + m0 + i * 16;
        want[i] = (row < count ? (uint32_t)a.rows.target[row] : ~0u) - (uint32_t)col;
    }
    const bool whole = (uint64_t)(tj + 1) * BN <= a.n;
    gemm::wait_and_meet<0>();  // every wave is done with the tiles
    float *tops = (float *)lds, *sums = tops + Core::WC * BM, *alls = sums + Core::WC * BM;
    static_assert(3 * Core::WC * BM * 4 <= Core::LDS, "the rows' part of LDS");
#pragma unroll
    for (int i = 0; i < Core::FM; ++i) {
        const uint32_t in = m0 + i * 16, row = ti * BM + in;
        // few rows have their target among the wave's columns
        if (__any(want[i] < Core::FN * 16))
#pragma unroll
            for (int j = 0; j < Core::FN; ++j)
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e)
                    if (want[i] == j * 16 + e && col + j * 16 + e < a.n)
                        a.rows.at[row] = acc[i][j][e];
        float top = kNone, all = 0.0f;
        if (!whole)
#pragma unroll
            for (int j = 0; j < Core::FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = col + j * 16 + e < a.n ? acc[i][j][e] : kNone;
#pragma unroll
        for (int j = 0; j < Core::FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = fmaxf(top, acc[i][j][e]);
        if (a.all)
#pragma unroll
            for (int j = 0; j < Core::FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    all += whole || col + j * 16 + e < a.n ? acc[i][j][e] : 0.0f;
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        float sum = 0.0f;
        const float over = top == kNone ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < Core::FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum += __builtin_amdgcn_exp2f((acc[i][j][e] - over) * kLog2e);
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        all += __shfl_xor(all, 16);
        all += __shfl_xor(all, 32);
        if (l < 16) {
            const uint32_t at = (wave % Core::WC) * BM + in;
            tops[at] = top;
            sums[at] = sum;
            alls[at] = all;
        }
    }
    __syncthreads();
    const uint32_t row = ti * BM + threadIdx.x;
    if (threadIdx.x >= BM || row >= count)
        return;
    float top = kNone, sum = 0.0f, all = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < Core::WC; ++w)
        top = fmaxf(top, tops[w * BM + threadIdx.x]);
#pragma unroll
    for (uint32_t w = 0; w < Core::WC; ++w) {
        sum += sums[w * BM + threadIdx.x] * part_of(tops[w * BM + threadIdx.x], top);
        all += alls[w * BM + threadIdx.x];
    }
    const uint64_t at = (uint64_t)tj * a.m + row;
    a.top[at] = top;
    a.sum[at] = sum;
    if (a.all)
        a.all[at] = all;
}

// Few rows' kernels take x as it lies where its rows start on 16 bytes: what a row
// without a target gives is dropped at the end.
__device__ __forceinline__ uint32_t rows_of(const LossArgs &a) {
    return a.target ? (uint32_t)a.m : a.rows.head->count;
}
__device__ __forceinline__ uint32_t target_of(const LossArgs &a, uint32_t m) {
    if (!a.target)
        return (uint32_t)a.rows.target[m];
    const long long t = a.target[m];
    return t < 0 ? ~0u : (uint64_t)t >= a.n ? (uint32_t)kBadTarget : (uint32_t)t;
}

// Up to 64 rows of few classes (by_groups): the few steps of each sum bound the time.
// A workgroup takes 16 columns; its 8 waves take an eighth of k each, straight into the
// matrix instruction's registers, for R groups of 16 rows; then the lanes add the parts
// up, a row and column each, and join the rows' logits.
constexpr int kFewWaves = 8;
constexpr uint64_t kFewRows = 64;

template <class T, int R>
__global__ __launch_bounds__(kFewWaves * 64) void few_kernel(LossArgs a) {
    using E = typename T::E;
    __shared__ f32x4 parts[kFewWaves][R * 16][5];  // [wave][m][n / 4], a chunk of padding
    const uint32_t count = rows_of(a);
    const uint32_t l = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = l & 15u, g = l >> 4;
    if (!count)
        return;
    const uint32_t steps = (uint32_t)((a.x.k + 31) / 32);
    const uint32_t s0 = steps * wave / kFewWaves, s1 = steps * (wave + 1) / kFewWaves;
    const uint16_t *px[R];
#pragma unroll
    for (uint32_t i = 0; i < R; ++i) {
        const uint32_t row = i * 16 + r;
        px[i] = a.x.plane[0] + (uint64_t)(row < count ? row : count - 1) * a.x.ld + g * 8;
    }
    // the lane's rows and column where parts are added up
    constexpr uint32_t EACH = R < 2 ? 1 : R / 2;  // rows, 32 apart
    const uint32_t m0 = threadIdx.x >> 4, c = threadIdx.x & 15u;
    uint32_t want[EACH];
#pragma unroll
    for (uint32_t i = 0; i < EACH; ++i) {
        const uint32_t m = m0 + i * 32;
        want[i] = m < count ? target_of(a, m) : ~0u;
    }
    const uint64_t n0 = (uint64_t)blockIdx.x * 16;
    const uint64_t rw = n0 + r < a.n ? n0 + r : a.n - 1;
    const uint16_t *pw = a.w.plane[0] + rw * a.w.ld + g * 8;
    f32x4 acc[R] = {};
    constexpr uint32_t U = 8;
    uint32_t s = s0;
    for (; s + U <= s1 && (uint64_t)(s + U) * 32 <= a.x.k; s += U) {
        gemm::s16x8 w[U];
#pragma unroll
        for (uint32_t i = 0; i < U; ++i)
            w[i] = __builtin_nontemporal_load((const gemm::s16x8 *)(pw + (uint64_t)(s + i) * 32));
#pragma unroll
        for (int j = 0; j < R; ++j) {
            gemm::s16x8 x[U];
#pragma unroll
            for (uint32_t i = 0; i < U; ++i)
                x[i] = *(const gemm::s16x8 *)(px[j] + (uint64_t)(s + i) * 32);
#pragma unroll
            for (uint32_t i = 0; i < U; ++i)
                acc[j] = T::mfma(w[i], x[i], acc[j]);
        }
    }
    for (; s < s1; ++s) {
        const bool in = (uint64_t)s * 32 + g * 8 < a.x.k;  // k is a multiple of 8
        gemm::s16x8 w = {};
        if (in)
            w = *(const gemm::s16x8 *)(pw + (uint64_t)s * 32);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            gemm::s16x8 x = {};
            if (in)
                x = *(const gemm::s16x8 *)(px[j] + (uint64_t)s * 32);
            acc[j] = T::mfma(w, x, acc[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
        parts[wave][j * 16 + r][g] = acc[j];
    __syncthreads();
    const bool in = n0 + c < a.n;
    const float b = a.bias && in ? (float)((const E *)a.bias)[n0 + c] : 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < EACH; ++i) {
        const uint32_t m = m0 + i * 32;
        float z = kNone, all = 0.0f;
        if (m < count && in) {
            z = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w)
                z += parts[w][m][c / 4][c % 4];
            z += b;
            if (want[i] == (uint32_t)(n0 + c))
                a.rows.at[m] = z;
            all = z;
        }
        float top = z;  // a NaN is in the sum
#pragma unroll
        for (int d = 1; d < 16; d *= 2)
            top = fmaxf(top, __shfl_xor(top, d));
        float sum = part_of(z, top);
#pragma unroll
        for (int d = 1; d < 16; d *= 2) {
            sum += __shfl_xor(sum, d);
            all += __shfl_xor(all, d);
        }
        if (c == 0 && m < count) {
            const uint64_t at = (uint64_t)blockIdx.x * a.m + m;
            a.top[at] = top;
            a.sum[at] = sum;
            if (a.all)
                a.all[at] = all;
        }
    }
}

// A decoded token or a few: no matrix instruction, whose operand takes 64 bytes of
// a row at a time.  A wave reads four rows of w as they lie, 1 KB a time, against
// x in LDS, adds its lanes' sums up and keeps the largest logit and sum of its rows.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

template <class E>
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float s) {
    E x[8], y[8];
    __builtin_memcpy(x, &a, 16);
    __builtin_memcpy(y, &b, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s = __builtin_fmaf((float)x[e], (float)y[e], s);
    return s;
}

template <class T, int M>
__global__ __launch_bounds__(256) void vector_kernel(LossArgs a) {
    using E = typename T::E;
    constexpr uint32_t U = 4, WAVES = 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float tops[WAVES][M], sums[WAVES][M], alls[WAVES][M];
    const uint32_t count = rows_of(a), k = (uint32_t)a.x.k;  // a multiple of 8
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    if (!count)
        return;
    u32x4 *xs = (u32x4 *)lds;
    for (uint32_t c = threadIdx.x; c < M * k / 8; c += 256) {
        const uint32_t m = c / (k / 8);
        xs[c] = m < count ? ((const u32x4 *)(a.x.plane[0] + m * a.x.ld))[c - m * (k / 8)]
                          : u32x4{0, 0, 0, 0};
    }
    __syncthreads();
    float top[M], sum[M], all[M];
    uint32_t want[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        top[m] = kNone;
        sum[m] = all[m] = 0.0f;
        want[m] = (uint32_t)m < count ? target_of(a, m) : ~0u;
    }
    const uint64_t r0 = a.n * blockIdx.x / gridDim.x, r1 = a.n * (blockIdx.x + 1) / gridDim.x;
    for (uint64_t row = r0 + wave * U; row < r1; row += WAVES * U) {
        const u32x4 *w[U];
        float acc[U][M] = {};
#pragma unroll
        for (uint32_t u = 0; u < U; ++u)
            w[u] = (const u32x4 *)(a.w.plane[0] + (row + u < r1 ? row + u : r1 - 1) * a.w.ld);
        // all of a batch's loads before its products: 16 KB of w a wave in flight
        auto batch = [&](auto size, uint32_t c) {
            constexpr uint32_t P = decltype(size)::value;
            u32x4 v[P][U];
#pragma unroll
            for (uint32_t p = 0; p < P; ++p)
#pragma unroll
                for (uint32_t u = 0; u < U; ++u)
                    v[p][u] = __builtin_nontemporal_load(w[u] + c + p * 64);
            if (P > 1)
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t p = 0; p < P; ++p)
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const u32x4 x = xs[m * (k / 8) + c + p * 64];
#pragma unroll
                    for (uint32_t u = 0; u < U; ++u)
                        acc[u][m] = dot8<E>(v[p][u], x, acc[u][m]);
                }
        };
        uint32_t c0 = 0;
        for (; c0 + 256 <= k / 8; c0 += 256)
            batch(std::integral_constant<uint32_t, 4>(), c0 + lane);
        for (; c0 + lane < k / 8; c0 += 64)
            batch(std::integral_constant<uint32_t, 1>(), c0 + lane);
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint64_t n = row + u;
            if (n >= r1)
                break;
            const float b = a.bias ? (float)((const E *)a.bias)[n] : 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float z = wave_sum(acc[u][m]) + b;
                if (want[m] == (uint32_t)n && lane == 0)
                    a.rows.at[m] = z;
                all[m] += z;
                const float old = top[m];
                top[m] = fmaxf(old, z);
                sum[m] = sum[m] * part_of(old, top[m]) + part_of(z, top[m]);
            }
        }
    }
    if (lane == 0)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            tops[wave][m] = top[m];
            sums[wave][m] = sum[m];
            alls[wave][m] = all[m];
        }
    __syncthreads();
    const uint32_t m = threadIdx.x;
    if (m >= M || m >= count)
        return;
    float t = kNone, s = 0.0f, z = 0.0f;
#pragma unroll
    for (uint32_t v = 0; v < WAVES; ++v)
        t = fmaxf(t, tops[v][m]);
#pragma unroll
    for (uint32_t v = 0; v < WAVES; ++v) {
        s += sums[v][m] * part_of(tops[v][m], t);
        z += alls[v][m];
    }
    const uint64_t at = (uint64_t)blockIdx.x * a.m + m;
    a.top[at] = t;
    a.sum[at] = s;
    if (a.all)
        a.all[at] = z;
}

// A row's parts, joined: R rows by 256 / R lanes a workgroup.
template <int R>
__global__ __launch_bounds__(256) void join_kernel(LossArgs a, uint32_t parts, float smoothing,
                                                   float *loss, float *lse) {
    constexpr uint32_t LANES = 256 / R;
    __shared__ float tops[256], sums[256], alls[256];
    const uint32_t lane = threadIdx.x / R, in = threadIdx.x % R;
    const uint64_t row = (uint64_t)blockIdx.x * R + in;
    const uint32_t count = rows_of(a);
    if ((uint64_t)blockIdx.x * R >= count)
        return;
    float top = kNone, sum = 0.0f, all = 0.0f;
    if (row < count) {
#pragma unroll 8
        for (uint32_t p = lane; p < parts; p += LANES) {
            const uint64_t at = (uint64_t)p * a.m + row;
            const float t = a.top[at], s = a.sum[at], old = top;
            top = fmaxf(top, t);
            sum = sum * part_of(old, top) + s * part_of(t, top);
            if (a.all)
                all += a.all[at];
        }
    }
    tops[threadIdx.x] = top;
    sums[threadIdx.x] = sum;
    alls[threadIdx.x] = all;
    for (uint32_t half = LANES / 2; half; half /= 2) {
        __syncthreads();
        if (lane < half) {
            const uint32_t o = threadIdx.x + half * R;
            const float t = tops[o], old = top;
            top = fmaxf(top, t);
            sum = sum * part_of(old, top) + sums[o] * part_of(t, top);
            all += alls[o];
            tops[threadIdx.x] = top;
            sums[threadIdx.x] = sum;
            alls[threadIdx.x] = all;
        }
    }
    if (lane || row >= count)
        return;
    const uint32_t to = a.target ? (uint32_t)row : a.rows.row[row];
    const uint32_t t = target_of(a, (uint32_t)row);
    if (t == ~0u) {
        loss[to] = lse[to] = 0.0f;
        return;
    }
    const float l = top + logf(sum);
    float v = __builtin_nanf("");
    if (t != (uint32_t)kBadTarget) {
        v = l - (1.0f - smoothing) * a.rows.at[row];
        if (a.all)
            v -= smoothing * (all / (float)a.n);
    }
    loss[to] = v;
    lse[to] = l;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// Workgroups by vectors, as many as are there at the same time.  In us, 512, 1024 and
// 2048 of them: 1 x 131072 x 4096 166, 165, 173; 1 x 32000 x 4096 48, 46, 47;
// 4 x 131072 x 4096 179, 191, 188.
constexpr uint32_t kVectorGroups = 1024;

// vector_kernel: one row at any length that LDS holds; up to four where the sums over
// a wave, one for each row and class, are few beside the products.  In us, by vectors,
// by groups of 16 columns (few_kernel) and by tiles:
//   1 x 131072 x 4096 165, 203, 181;  1 x 32000 x 1024 16, 20, 19;
//   2 x 64000 x 4096 91, 112, 114;  2 x 16000 x 2048 19, 21, 24;
//   2 x 64000 x 1024 40, 31, 30;  4 x 64000 x 256 47, 16, 16;
//   4 x 64000 x 4096 103, 117, 114;  4 x 32000 x 4096 59, 62, 46;  4 x 4000 x 2048 14, 12, 20.
// More than 32 KB of x, by vectors and by the better of the others:
//   1 x 64000 x 24576 478, 549;  2 x 20000 x 12288 90, 113;  2 x 1000 x 12288 20, 22;
//   4 x 20000 x 5120 60, 44;  4 x 4000 x 6144 21, 16.
bool by_vectors(uint64_t m, uint64_t k) {
    if (!k || m > 4 || (m > 1 && k < 2048))
        return false;
    return m <= 2 ? m * k * 2 <= 49152 : 4 * k * 2 <= 32768;
}

// few_kernel: a workgroup that takes a second group of 16 columns waits for its loads
// again, which tiles copy ahead, and the more rows a group has the longer it holds up
// the next.  In us, by groups and by tiles:
//   64 x 4096 x 1024 13, 16;  64 x 5000 x 1024 18, 16;  64 x 4096 x 4096 29, 31;
//   64 x 5000 x 4096 48, 31;  32 x 8192 x 1024 14, 16;  32 x 8192 x 4096 34, 32;
//   32 x 12000 x 4096 47, 37;  16 x 12000 x 1024 14, 17;  16 x 12000 x 4096 34, 37;
//   16 x 16384 x 4096 43, 37;  64 x 131072 x 4096 671, 195.
bool by_groups(uint64_t m, uint64_t n) {
    const uint64_t groups = (n + 15) / 16;
    return m <= kFewRows && groups <= (m <= 16 ? 768u : m <= 32 ? 512u : 256u);
}

bool packs(uint64_t m, uint64_t k) { return k % 8 && m >= kPackLoss; }

struct LossCut {
    Plan plan;
    uint32_t parts;  // of a row
    size_t piece;    // columns whose w is packed at a time; 0: none are
};

LossCut loss_cut(uint64_t m, uint64_t n, uint64_t k) {
    LossCut c;
    c.plan = plan_product(m, n, k, true);
    c.parts = (uint32_t)((n + kSideN[c.plan.tile] - 1) / kSideN[c.plan.tile]);
    if (m <= kFewRows)  // at most 768 by groups, and by vectors
        c.parts = std::max(c.parts, kVectorGroups);
    // whole tiles
    c.piece = packs(m, k) ? std::min<size_t>(std::max<size_t>(kPieceElements / k / 256, 1) * 256,
                                             (n + 255) / 256 * 256)
                          : 0;
    return c;
}

struct LossBuffers {
    LossArgs a = {};
    uint16_t *w;
};

LossBuffers carve_loss(Carve &c, size_t m, size_t n, size_t k) {
    LossBuffers b;
    b.a.rows = carve_rows(c, m, k);
    const LossCut t = loss_cut(m, n, k);
    b.a.top = c.take<float>((size_t)t.parts * m);
    b.a.sum = c.take<float>((size_t)t.parts * m);
    b.a.all = c.take<float>((size_t)t.parts * m);
    b.w = c.take<uint16_t>(t.piece * b.a.rows.ld);
    return b;
}

// The tiles [first, last) of the columns.
template <class T, bool STAGED>
int launch_loss(LossArgs a, const Plan &p, uint32_t first, uint32_t last, hipStream_t s) {
    auto go = [&](auto core) {
        using Core = decltype(core);
        const uint64_t tm = (a.m + Core::BM - 1) / Core::BM;
        int rc = allow_lds(loss_kernel<T, Core>, Core::LDS);
        // a launch takes fewer than 2^32 lanes
        const uint32_t most = (uint32_t)((1ull << 31) / Core::THREADS / tm);
        for (a.first = first; !rc && a.first < last; a.first += a.tn) {
            a.tn = std::min(most, last - a.first);
            rc = launch(loss_kernel<T, Core>, dim3((uint32_t)tm * a.tn), dim3(Core::THREADS),
                        Core::LDS, s, a);
        }
        return rc;
    };
    if (p.tile == 0)
        return go(gemm::Core<T, 256, 256, 2, 4, 64, 2, false, false, STAGED, !STAGED>());
    if (p.tile == 1)
        return go(gemm::Core<T, 128, 128, 2, 2, 64, 2, false, false, STAGED>());
    if (p.tile == 2)
        return go(gemm::Core<T, 64, 64, 2, 2, 64, 3, false, false, STAGED>());
    return go(gemm::Core<T, 64, 32, 4, 1, 64, 3, false, false, STAGED>());
}

template <class T>
int loss(const ddl_ce_args *c, void *ws, hipStream_t s) {
    Carve carve{(uint8_t *)ws};
    LossBuffers buf = carve_loss(carve, c->m, c->n, c->k);
    LossArgs &a = buf.a;
    RowsArgs r = {};
    r.m = (uint32_t)c->m;
    r.n = c->n;
    r.k = c->k;
    r.x = c->x;
    r.ldx = c->ldx;
    r.target = c->target;
    r.loss = c->loss;
    r.lse_out = c->lse;
    // straight to LDS or registers where every row starts on 16 bytes
    const bool direct = c->k % 8 == 0 && aligned16(c->w, c->ldw, 2);
    const bool vectors = direct && by_vectors(c->m, c->k);
    const bool groups = direct && !vectors && by_groups(c->m, c->n);
    int rc = DDL_OK;
    if ((vectors || groups) && aligned16(c->x, c->ldx, 2)) {
        a.target = c->target;
        a.x = operand(c->x, c->ldx, c->m, c->k);
    } else {
        rc = pack_rows(r, a.rows, s);
        a.x = operand(a.rows.x, a.rows.ld, c->m, c->k);
    }
    if (rc)
        return rc;
    a.w = operand(c->w, c->ldw, c->n, c->k);
    a.bias = c->bias;
    a.m = c->m;
    a.n = c->n;
    if (c->smoothing == 0.0)
        a.all = nullptr;
    const LossCut t = loss_cut(c->m, c->n, c->k);
    const uint32_t side = kSideN[t.plan.tile];
    uint32_t parts = (uint32_t)((c->n + side - 1) / side);
    if (vectors) {
        const size_t m = c->m <= 2 ? c->m : 4;
        parts = (uint32_t)std::min<size_t>(kVectorGroups, (c->n + 15) / 16);
        rc = launch(m == 1   ? vector_kernel<T, 1>
                    : m == 2 ? vector_kernel<T, 2>
                             : vector_kernel<T, 4>,
                    dim3(parts), dim3(256), m * c->k * sizeof(uint16_t), s, a);
    } else if (groups) {
        parts = (uint32_t)((c->n + 15) / 16);
        rc = launch(c->m <= 16   ? few_kernel<T, 1>
                    : c->m <= 32 ? few_kernel<T, 2>
                                 : few_kernel<T, 4>,
                    dim3(parts), dim3(kFewWaves * 64), 0, s, a);
    } else if (t.piece) {
        a.x.k = a.rows.ld;  // zeros past k on both sides
        for (size_t first = 0; first < c->n && !rc; first += t.piece) {
            const size_t have = std::min(t.piece, c->n - first);
            rc = pack_matrix((const uint16_t *)c->w + first * c->ldw, c->ldw, have, c->k, buf.w, s);
            // tiles go by their columns' places in the whole of w
            a.w = operand(buf.w - first * a.rows.ld, a.rows.ld, c->n, a.rows.ld);
            if (!rc)
                rc = launch_loss<T, false>(a, t.plan, (uint32_t)(first / side),
                                           (uint32_t)((first + have + side - 1) / side), s);
        }
    } else {
        rc = direct ? launch_loss<T, false>(a, t.plan, 0, parts, s)
                    : launch_loss<T, true>(a, t.plan, 0, parts, s);
    }
    if (rc)
        return rc;
    const float smoothing = (float)c->smoothing;
    // few rows: a workgroup for each, so that a row's parts are read by many
    return c->m <= 256
               ? launch(join_kernel<1>, dim3((uint32_t)c->m), dim3(256), 0, s, a, parts, smoothing,
                        c->loss, c->lse)
               : launch(join_kernel<32>, dim3((uint32_t)((c->m + 31) / 32)), dim3(256), 0, s, a,
                        parts, smoothing, c->loss, c->lse);
}

}  // namespace

size_t loss_workspace(size_t m, size_t n, size_t k) {
    Carve c{nullptr};
    carve_loss(c, m, n, k);
    return c.used;
}

}  // namespace ddl

using namespace ddl;

extern "C" int ddl_cross_entropy(const ddl_ce_args *a, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    if (!a)
        return DDL_E_NULL;
    const int rc = check_cross_entropy(a, DDL_CE_FORWARD, workspace, workspace_bytes);
    if (rc || !a->m)
        return rc;
    if (!a->loss || !a->lse)
        return DDL_E_NULL;
    if (!element_ok(a->loss, 4) || !element_ok(a->lse, 4))
        return DDL_E_ALIGN;
    return a->dtype == DDL_F16 ? loss<Half>(a, workspace, (hipStream_t)stream)
                               : loss<Bfloat>(a, workspace, (hipStream_t)stream);
}
