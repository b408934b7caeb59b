// cross_entropy_internal.h -- what the cross entropy's loss and gradient share:
// the rows that have a target, packed together, and their workspace.
//
// Rows without a target (target < 0), and for the gradient those whose factor is
// 0, take no part in the products: the others are packed, x and all, so that a
// padded batch costs what its targets cost and whatever stands in a row without
// one, NaN included, reaches no sum.  How many rows that leaves is known on the
// device alone; launches are sized for all of them and workgroups past the last
// leave at once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ddl.h"
#include "gemm_core.h"
#include "hip_call.h"
#include "product_parts.h"

namespace ddl {

constexpr size_t kMaxTargets = 1u << 22;
constexpr int32_t kBadTarget = 0x7fffffff;  // a class that does not exist: its results are NaN
constexpr float kLog2e = 1.4426950408889634f;

// 4 consecutive values of 16 bits from anywhere; those past `have` are 0.
template <class E>
__device__ __forceinline__ void load4(const E *p, uint32_t have, float (&out)[4]) {
    E v[4];
    if (have >= 4) {
        __builtin_memcpy(v, p, 8);
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            v[e] = e < have ? p[e] : (E)0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        out[e] = (float)v[e];
}

// What the rows kernel counts.
struct RowsHead {
    uint32_t count;  // rows with a target
    int exponent;    // of the power of two that dz is held times (see write_head)
};

// The packed rows, on the device.
struct Rows {
    RowsHead *head;
    uint32_t *row;    // of the caller
    int32_t *target;
    float *lse;       // gradient: the caller's
    float *g;         // gradient: the factor of the row's dz
    float *at;        // loss: the target's logit
    uint16_t *x;      // [up64(count)][ld], zeros behind the k-th element and the last row
    uint64_t ld;      // k rounded up to 64: rows are whole lines of 128 bytes
    // cleared with the packing, for kernels that take maxima there
    uint32_t *clear;
    uint64_t clear_count;
};

// Sums over the packed rows run over whole k tiles: rows of zeros fill the last.
__host__ __device__ inline uint64_t up64(uint64_t n) { return (n + 63) / 64 * 64; }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Parts of one workspace, one after another on 256-byte boundaries.
struct Carve {
    uint8_t *base;
    size_t used = 0;
    template <class V>
    V *take(size_t count) {
        V *p = base ? (V *)(base + used) : nullptr;
        used += up256(count * sizeof(V));
        return p;
    }
};

inline Rows carve_rows(Carve &c, size_t m, size_t k) {
    Rows r;
    r.head = c.take<RowsHead>(1);
    r.row = c.take<uint32_t>(m);
    r.target = c.take<int32_t>(m);
    r.lse = c.take<float>(m);
    r.g = c.take<float>(m);
    r.at = c.take<float>(m);
    r.ld = up64(k);
    r.x = c.take<uint16_t>(up64(m) * r.ld);
    r.clear = nullptr;
    r.clear_count = 0;
    return r;
}

// The caller's side of the rows.  loss: loss and lse are set to 0 in rows
// without a target; gradient: dx (or NULL).
struct RowsArgs {
    uint32_t m;
    uint64_t n, k;
    const void *x;
    uint64_t ldx;
    const long long *target;
    float *loss, *lse_out;
    const float *lse, *dloss;
    double scale;
    uint16_t *dx;
    uint64_t lddx;
};

// Packs the rows (cross_entropy_loss.hip).
int pack_rows(const RowsArgs &a, const Rows &r, hipStream_t s);

// Rows of k elements that do not start on 16 bytes go through registers on their
// way to LDS, or a piece of w is packed first: for the gradient, whose three products
// take it, always (in us, through registers and packed: 20 x 1000 x 501 34, 22;
// 300 x 50001 x 2051 1022, 593; 4 x 20000 x 1001 72, 73); for the loss from this many
// rows of x on (768 x 20000 x 1001 51, 55; 1000 x 20000 x 1001 85, 80).
constexpr size_t kPackLoss = 1000;
// Elements of a packed or converted piece of w, and of each of dz's planes, that a call
// holds at a time.
constexpr size_t kPieceElements = 128u << 20;
// to: rows of up64(k) elements, whole lines of 128 bytes, zeros behind the k-th.
int pack_matrix(const void *from, size_t ld, size_t rows, size_t k, uint16_t *to, hipStream_t s);

// How a product is cut, by the time that it should take: rounds of workgroups over
// the chip, each of k tiles of 64 at what a tile was measured to take (us; with
// the chip full of its kind, 1.3, 1.0 and 0.65 PFLOP/s, and with one workgroup a
// compute unit, where copies to LDS set the pace), and where k is cut the parts'
// way through memory.  With every tile and number of parts measured on the twenty
// products of ten gradients, whole calls, the choice is within 2% of the best on fifteen
// of them, 8 to 12% behind on four and 23% on one, dx of 64 x 100000 x 4096 (526 us, in
// 16 parts by tiles of 128 429); with the logits' tiles on eight sizes, within 3%.
constexpr uint32_t kSideM[4] = {256, 128, 64, 64}, kSideN[4] = {256, 128, 64, 32};
struct Plan {
    int tile;  // of kSideM x kSideN; the last one with both operands by columns only
    uint32_t splits;
};

// whole: no parts of k, and both operands by columns (the logits).
inline Plan plan_product(uint64_t m, uint64_t n, uint64_t k, bool whole) {
    constexpr double kStep[4] = {1.65, 1.07, 0.62, 0.5}, kAlone[4] = {1.65, 0.95, 0.4, 0.3};
    constexpr double kStart[4] = {6, 4, 2.5, 2.5};
    constexpr uint64_t kSlots[4] = {256, 512, 768, 768};
    const uint64_t kt = std::max<uint64_t>((k + 63) / 64, 1);
    Plan best = {2, 1};
    double least = 1e300;
    for (int t = 0; t < (whole ? 4 : 3); ++t)
        for (const uint64_t p : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
            if (p > 1 && (whole || kt / p < 4))
                break;
            const uint64_t groups = ((m + kSideM[t] - 1) / kSideM[t])
                                    * ((n + kSideN[t] - 1) / kSideN[t]) * p;
            const double step = groups <= 256 ? kAlone[t] : kStep[t];
            double us = (double)((groups + kSlots[t] - 1) / kSlots[t])
                        * (kStart[t] + (double)((kt + p - 1) / p) * step);
            if (p > 1)
                us += 4 + (double)(p * m * n) * 8e-6 / 8;
            if (us < least) {
                least = us;
                best = {t, (uint32_t)p};
            }
        }
    return best;
}

// What both calls refuse (cross_entropy_grad.hip), and their workspaces.
int check_cross_entropy(const ddl_ce_args *a, int op, const void *ws, size_t bytes);
size_t loss_workspace(size_t m, size_t n, size_t k);
size_t grad_workspace(size_t m, size_t n, size_t k);

}  // namespace ddl
