// cross_entropy_internal.h -- what the cross entropy's loss and gradient share:
// the rows that have a target, packed together, and their workspace.
//
// Rows without a target (target < 0), and for the gradient those whose factor is
// 0, take no part in the products: the others are packed, x and all, so that a padded batch costs what its targets cost and
// whatever stands in a row without one, NaN included, reaches no sum.  How many
// rows that leaves is known on the device alone; launches are sized for all of
// them and workgroups past the last leave at once.
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

// What the rows kernel counts.
struct RowsHead {
    uint32_t count;  // rows with a target
    float factor;    // a power of two that dz is held times (see rows_kernel)
    float inverse;
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
    uint64_t ld;      // k rounded up to 8
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
    r.ld = (k + 7) / 8 * 8;
    r.x = c.take<uint16_t>(up64(m) * r.ld);
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
    float scale;
    uint16_t *dx;
    uint64_t lddx;
};

// Packs the rows (cross_entropy_loss.hip).
int pack_rows(const RowsArgs &a, const Rows &r, hipStream_t s);

// What both calls refuse (cross_entropy_grad.hip), and their workspaces.
int check_cross_entropy(const ddl_ce_args *a, int op, const void *ws, size_t bytes);
size_t loss_workspace(size_t m, size_t n, size_t k);
size_t grad_workspace(size_t m, size_t n, size_t k);

}  // namespace ddl
