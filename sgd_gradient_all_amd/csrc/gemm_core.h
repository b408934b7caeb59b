// gemm_core.h -- the tiled matrix product under the linear layer and Muon
// (gfx950).
//
//     C[m, n] = sum_k A(m, k) B(n, k)        16-bit operands, binary32 sums
//
// A workgroup of WR x WC waves computes a BM x BN tile of C.  Each operand
// lies in memory either with k contiguous (a row per m or n) or with its own
// index contiguous (a row per k, "TR"); tiles of 64 k go to LDS as they lie
// in memory, twice buffered, and the matrix instruction
// v_mfma_f32_16x16x32 gets its operands
//  - k contiguous: as one 16-byte LDS read per lane;
//  - TR: as two transposing 8-byte reads (ds_read_b64_tr_b16: the 16 lanes
//    of a quarter wave read 4 rows of 16 elements and each receives one
//    column of 4).
// The instruction is given (B, A), so that a lane ends with consecutive n of
// one m: B's rows are dealt to the fragments so that the 4 FN values of a
// lane are consecutive, and a tile's rows are stored 16 bytes at a time.
//
// Loads: with 16-byte aligned rows the tiles go from global memory straight
// to LDS (16 bytes a lane, no registers); otherwise (STAGED) through
// registers, element by element only at a row's end.  LDS is written in lane
// order, so the bank spread comes from permuting the 16-byte chunks of a row
// by an exclusive-or with a key of the row, on the global side of the copy
// and again at the read.
//
// Bounds: rows past the operand's extent repeat its last row (their results
// are not stored); chunks past the end of k come from a page of zeros, so no
// garbage, NaN included, enters a sum.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ddl {
namespace gemm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBK = 64;  // k of one tile

// An address in LDS, by its offset: kept apart from generic pointers, whose
// reads would go through the flat path and its counters.
template <class V>
__device__ __forceinline__ V lds_read(uint32_t at) {
    return *(const __attribute__((address_space(3))) V *)(uintptr_t)at;
}
template <class V>
__device__ __forceinline__ void lds_write(uint32_t at, V v) {
    *(__attribute__((address_space(3))) V *)(uintptr_t)at = v;
}

struct Half {
    using E = _Float16;
    __device__ static f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};
struct Bfloat {
    using E = __bf16;
    __device__ static f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};

// One operand.  rows: its extent in m (or n); row0: the tile's first.  k: its
// extent in k.  plane: its values; or the high and the low parts of values
// held as sums of two.
struct Operand {
    const uint16_t *plane[2];
    uint64_t ld;    // elements from row to row
    uint64_t k;
    uint32_t rows;
    uint32_t row0;
};

__device__ __attribute__((aligned(16))) uint32_t zero_page[4] = {0, 0, 0, 0};

// The row key that spreads LDS banks (see above).
template <bool TR, bool SECOND, int R, int F>
__device__ __forceinline__ uint32_t chunk_key(uint32_t row) {
    if (!TR)  // row = an m or n; the 8 lanes of a read group get 8 keys
        return SECOND ? (row & 3u) | (((row / (4u * F)) & 1u) << 2) : row & 7u;
    if (!SECOND)  // row = a k; 32 bytes of each of 4 rows
        return (row & 3u) << 1;
    if (R == 64)
        return ((row >> 1) & 1u) << 2;
    return (row & 1u) | ((row & 2u) << 2);  // 8 of every 32 bytes of 4 rows
}

// 16 bytes of every lane to LDS at `lds` + 16 lane, without registers between.
// Written in assembly because the compiler, which cannot tell the two buffers
// apart, would make every LDS read wait for the copy into the other one; the
// wait is wait_loads, before the barrier that opens the buffer.  The wait
// state between the write of m0 and its use is the s_nop.
__device__ __forceinline__ void load16_to_lds(const uint8_t *base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void load16_to_lds(const uint8_t *p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds), "v"(p)
                 : "memory");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <class T, int BM_, int BN_, int WR_, int WC_, bool TRA, bool TRB, bool STAGED>
struct Core {
    static constexpr int BM = BM_, BN = BN_, WR = WR_, WC = WC_;
    static constexpr int THREADS = WR * WC * 64;
    static constexpr int FM = BM / WR / 16, FN = BN / WC / 16;
    static constexpr int LA = BM * 8 / THREADS, LB = BN * 8 / THREADS;  // 16-byte loads a lane
    static constexpr int BYTES_A = BM * kBK * 2, BYTES_B = BN * kBK * 2;
    static constexpr int LDS = 2 * (BYTES_A + BYTES_B);
    static_assert(LA >= 1 && LB >= 1 && FN >= 2, "tile");

    // One side's loads of a tile: lane offsets from the tile's uniform base.
    template <bool TR, bool SECOND, int R, int F, int L>
    struct Side {
        uint32_t off[L];
        uint32_t kc[L];    // k of the load's first element, within the tile
        uint32_t have[L];  // TR and STAGED: elements of the chunk inside the row

        __device__ __forceinline__ void init(const Operand &o) {
            const uint32_t left = o.rows - o.row0;  // >= 1
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const uint32_t q = i * THREADS + threadIdx.x;
                if (!TR) {
                    const uint32_t row = q >> 3, c = (q & 7u) ^ chunk_key<TR, SECOND, R, F>(row);
                    const uint32_t r = row < left ? row : left - 1;
                    off[i] = r * (uint32_t)o.ld * 2u + c * 16u;
                    kc[i] = c * 8;
                } else {
                    const uint32_t row = q / (R / 8);
                    uint32_t c = (q % (R / 8)) ^ chunk_key<TR, SECOND, R, F>(row);
                    if (STAGED) {
                        have[i] = c * 8 >= left ? 0 : left - c * 8;
                        c = c * 8 >= left ? 0 : c;
                    } else {  // left is a multiple of 8
                        c = c * 8 < left ? c : left / 8 - 1;
                    }
                    off[i] = row * (uint32_t)o.ld * 2u + c * 16u;
                    kc[i] = row;
                }
            }
        }
        __device__ __forceinline__ static const uint8_t *base(const Operand &o, int plane,
                                                              uint64_t k0) {
            const uint64_t e = TR ? k0 * o.ld + o.row0 : (uint64_t)o.row0 * o.ld + k0;
            return (const uint8_t *)(o.plane[plane] + e);
        }
        // straight to LDS; left: k from this tile's first to the end
        __device__ __forceinline__ void issue(const uint8_t *b, uint64_t left,
                                              uint32_t lds) const {
            lds += __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
            if (left >= (uint64_t)kBK) {
#pragma unroll
                for (int i = 0; i < L; ++i)
                    load16_to_lds(b, off[i], lds + i * THREADS * 16);
            } else {
#pragma unroll
                for (int i = 0; i < L; ++i)
                    load16_to_lds(kc[i] < left ? b + off[i] : (const uint8_t *)zero_page,
                                  lds + i * THREADS * 16);
            }
        }
        __device__ __forceinline__ void fetch(const uint8_t *b, uint64_t left,
                                              u32x4 (&reg)[L]) const {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                uint32_t n = 8;
                if (TR)
                    n = kc[i] < left ? have[i] : 0;
                else if (left < (uint64_t)kBK)
                    n = kc[i] < left ? (uint32_t)left - kc[i] : 0;
                if (n >= 8) {
                    __builtin_memcpy(&reg[i], b + off[i], 16);
                } else {
                    uint32_t h[8];
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        h[e] = e < n ? ((const uint16_t *)(b + off[i]))[e] : 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        reg[i][e] = h[2 * e] | h[2 * e + 1] << 16;
                }
            }
        }
        __device__ __forceinline__ void put(const u32x4 (&reg)[L], uint32_t lds) const {
#pragma unroll
            for (int i = 0; i < L; ++i)
                lds_write(lds + (i * THREADS + threadIdx.x) * 16, reg[i]);
        }
    };

    // The fragment `i` (16 rows) of a side for the 32 k from kk * 32 on.
    // first: the wave's first row in the tile.
    template <bool TR, bool SECOND, int R, int F>
    __device__ __forceinline__ static s16x8 fragment(uint32_t lds, uint32_t first, int i,
                                                     int kk) {
        const uint32_t l = threadIdx.x & 63u, r = l & 15u, g = l >> 4;
        if (!TR) {
            const uint32_t row =
                first + (SECOND ? (r >> 2) * (4 * F) + 4 * i + (r & 3u) : 16 * i + r);
            const uint32_t c = (g + 4 * kk) ^ chunk_key<TR, SECOND, R, F>(row);
            return lds_read<s16x8>(lds + row * (kBK * 2) + c * 16);
        }
        const uint32_t col = first + (SECOND ? (r & 3u) * (4 * F) + 4 * i : 16 * i + (r & 3u) * 4);
        s16x4 h[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t k = kk * 32 + g * 8 + x * 4 + (r >> 2);
            const uint32_t c = (col >> 3) ^ chunk_key<TR, SECOND, R, F>(k);
            const uint32_t p = lds + k * (R * 2) + c * 16 + (col & 7u) * 2;
            h[x] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(uintptr_t)p);
        }
        return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }

    __device__ __forceinline__ static void multiply(uint32_t la, uint32_t lb, f32x4 (&acc)[FM][FN]) {
        const uint32_t wave = threadIdx.x >> 6;
        const uint32_t ma = (wave / WC) * (FM * 16), nb = (wave % WC) * (FN * 16);
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk) {
            s16x8 b[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[j] = fragment<TRB, true, BN, FN>(lb, nb, j, kk);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const s16x8 a = fragment<TRA, false, BM, FM>(la, ma, i, kk);
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = T::mfma(b[j], a, acc[i][j]);
            }
        }
    }

    // acc += the k tiles [t0, t1), t0 < t1.  Plain operands: pairs = 0.  Pairs
    // of high and low parts: pairs = the tiles of one pass over k; tiles go
    // through high * low, low * high, and high * high last, so that the sums
    // that all the large terms meet are rounded a third as often.
    __device__ __forceinline__ static void run(const Operand &a, const Operand &b, uint32_t t0,
                                               uint32_t t1, uint32_t pairs, uint8_t *lds,
                                               f32x4 (&acc)[FM][FN]) {
        Side<TRA, false, BM, FM, LA> sa;
        Side<TRB, true, BN, FN, LB> sb;
        sa.init(a);
        sb.init(b);
        constexpr int kBuf = BYTES_A + BYTES_B;
        u32x4 ra[STAGED ? LA : 1], rb[STAGED ? LB : 1];
        // the buffers' address in LDS, as the copies take it
        const uint32_t lds0 =
            (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
        auto load = [&](uint32_t t, uint32_t at) {
            const uint32_t pass = !pairs || t >= 2 * pairs ? 2 : t < pairs ? 0 : 1;
            const uint64_t k0 = (uint64_t)(t - pass * pairs) * kBK;
            const uint8_t *pa = sa.base(a, pass == 1, k0), *pb = sb.base(b, pass == 0, k0);
            if constexpr (STAGED) {
                sa.fetch(pa, a.k - k0, ra);
                sb.fetch(pb, b.k - k0, rb);
            } else {
                sa.issue(pa, a.k - k0, at);
                sb.issue(pb, b.k - k0, at + BYTES_A);
            }
        };
        load(t0, lds0);
        uint32_t cur = 0;
        if constexpr (STAGED) {
            sa.put(ra, lds0);
            sb.put(rb, lds0 + BYTES_A);
        }
        for (uint32_t t = t0; t < t1; ++t) {
            // tile t has landed, and every wave is done with the other buffer
            wait_loads();
            __syncthreads();
            const uint32_t now = lds0 + cur * kBuf, next = lds0 + (cur ^ 1) * kBuf;
            if (t + 1 < t1)
                load(t + 1, next);
            multiply(now, now + BYTES_A, acc);
            if constexpr (STAGED) {
                if (t + 1 < t1) {
                    sa.put(ra, next);
                    sb.put(rb, next + BYTES_A);
                }
            }
            cur ^= 1;
        }
    }

    // then(m, n, v) for every 8 consecutive n of a row m of the wave's results
    // (both within the tile); TURNED: for every 8 consecutive m of a column n.
    // They go through the wave's own part of LDS, so that 8 lanes (4 with
    // FN = 2) hold whole 128-byte pieces of a row or column and the epilogue
    // is a loop of small body rather than one of 128 registers.
    template <bool TURNED = false, class F>
    __device__ __forceinline__ static void each(const f32x4 (&acc)[FM][FN], uint8_t *lds,
                                                F &&then) {
        constexpr int G = FM < 4 ? FM : 4;         // fragments of rows at a time
        constexpr int C = 4 * FN;                  // 16-byte chunks of a row
        constexpr int PART = G * 16 * C * 16;      // bytes of a wave's part
        static_assert(PART * WR * WC <= LDS, "the results' part of LDS");
        const uint32_t wave = threadIdx.x >> 6, l = threadIdx.x & 63u;
        const uint32_t at =
            (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + wave * PART;
        const uint32_t m0 = (wave / WC) * (FM * 16), n0 = (wave % WC) * (FN * 16);
        __syncthreads();  // every wave is done with the tiles
#pragma unroll
        for (int i0 = 0; i0 < FM; i0 += G) {
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const uint32_t row = 16 * i + (l & 15u), c = (l >> 4) * FN + j;
                    lds_write(at + (row * C + (c ^ (row & (C - 1)))) * 16, acc[i0 + i][j]);
                }
            float v[8];
            if constexpr (TURNED) {
                constexpr int LANES = G * 2;  // of one column
#pragma unroll 1
                for (uint32_t n = l / LANES; n < 4 * C; n += 64 / LANES) {
                    const uint32_t r = (l % LANES) * 8;
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        v[e] = lds_read<float>(
                            at + ((r + e) * C + ((n >> 2) ^ ((r + e) & (C - 1)))) * 16
                            + (n & 3u) * 4);
                    then(m0 + i0 * 16 + r, n0 + n, v);
                }
            } else {
                constexpr int LANES = C / 2;  // of one row
#pragma unroll 1
                for (uint32_t r = l / LANES; r < G * 16; r += 64 / LANES) {
                    const uint32_t c = (l % LANES) * 2;
                    const f32x4 x = lds_read<f32x4>(at + (r * C + (c ^ (r & (C - 1)))) * 16);
                    const f32x4 y =
                        lds_read<f32x4>(at + (r * C + ((c + 1) ^ (r & (C - 1)))) * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = x[e];
                        v[4 + e] = y[e];
                    }
                    then(m0 + i0 * 16 + r, n0 + c * 4, v);
                }
            }
        }
    }
};

}  // namespace gemm
}  // namespace ddl
