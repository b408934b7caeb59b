// product_parts.h -- what the kernels around gemm_core.h's products share:
// vectors of 8 elements, the order of the tiles, and how a product is cut.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_core.h"

namespace ddl {

using gemm::Operand;
using gemm::u32x4;

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

constexpr size_t kMaxExtent = 1u << 22;   // columns and row strides (32-bit tile offsets)

// How a product is cut: tile size (0: 256 x 256, 1: 128 x 128, 2: 64 x 64)
// and parts of k.  A tile size needs 192 tiles, three for four compute units:
// with 182, 3328 x 3584 x 1024 takes 71 us in tiles of 256 and 41 in tiles of
// 128, 1664 x 1792 x 1024 23 in tiles of 128 and 15 in tiles of 64.  (With 196
// it depends on k: 1792 x 1792 x 1024 25 us in tiles of 128 and 21 of 64, x
// 4096 48 and 64; 3584 x 3584 x 1024 74 in tiles of 256 and 45 of 128, x 4096
// 157 and 133.)  With fewer tiles than compute units k is cut for 512
// workgroups: 512 x 1024 x 4096 17 us, uncut 30, cut for 256 21, for 1024 20.
// Padding is not weighed: 65536 x 64 x 1024 takes 44 us in tiles of 256, in
// tiles of 64 it would be 32.
struct Cut {
    int tile;
    uint32_t splits;
};
constexpr uint32_t kTile[3] = {256, 128, 64};

inline uint64_t tiles(uint64_t m, uint64_t n, int t) {
    return ((m + kTile[t] - 1) / kTile[t]) * ((n + kTile[t] - 1) / kTile[t]);
}

inline Cut cut(uint64_t m, uint64_t n, uint64_t k) {
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

inline bool aligned16(const void *p, size_t ld, size_t esz) {
    return ((uintptr_t)p | ld * esz) % 16 == 0;
}

// Even addresses: a 16-bit element does not straddle its own size.
inline bool element_ok(const void *p, size_t esz) { return (uintptr_t)p % esz == 0; }

// A matrix's distance from row to row.
inline bool row_ok(const void *p, size_t ld, size_t cols, size_t rows) {
    return !p || (ld <= kMaxExtent && (ld >= cols || rows <= 1));
}

inline Operand operand(const void *p, size_t ld, size_t rows, size_t k) {
    Operand o;
    o.plane[0] = o.plane[1] = (const uint16_t *)p;
    o.ld = ld;
    o.rows = (uint32_t)rows;
    o.row0 = 0;
    o.k = k;
    return o;
}

}  // namespace ddl
