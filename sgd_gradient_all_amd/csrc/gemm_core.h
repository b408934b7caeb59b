// gemm_core.h -- the tiled matrix product under the linear layer and Muon
// (gfx950).
//
//     C[m, n] = sum_k A(m, k) B(n, k)        16-bit operands, binary32 sums
//
// A workgroup of WR x WC waves computes a BM x BN tile of C.  Each operand
// lies in memory either with k contiguous (a row per m or n) or with its own
// index contiguous (a row per k, "TR"); tiles of BK k go to LDS as they lie
// in memory, several ahead of the one multiplied, and the matrix instruction
// v_mfma_f32_16x16x32 gets its operands
//  - k contiguous: as one 16-byte LDS read per lane;
//  - TR: as two transposing 8-byte reads (ds_read_b64_tr_b16: the 16 lanes
//    of a quarter wave read 4 rows of 16 elements and each receives one
//    column of 4).
// The instruction is given (B, A), so that a lane ends with 4 consecutive n of
// one m; results are dealt out again through LDS, 8 to a lane (see each).
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

#include <type_traits>

namespace ddl {
namespace gemm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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

// The row key that spreads LDS banks (see above).  R: the operand's extent of
// the tile.  LDS serves 256 bytes (32 lanes of 8 bytes, 16 of 16) at a time:
//  - k contiguous, rows of 128 bytes: 8 rows of one 16-byte chunk each;
//  - TR, rows of 2 R bytes: 32 bytes of 8 rows, k = 0 .. 3 and 8 .. 11 (or 4
//    on); rows of 128 bytes alternate between the halves by themselves.
template <bool TR, int R>
__device__ __forceinline__ uint32_t chunk_key(uint32_t row) {
    if (!TR)
        return row & 7u;
    if (R == 64)
        return ((row >> 1 & 1u) | (row >> 3 & 1u) << 1) << 1;
    return ((row & 3u) | (row >> 3 & 1u) << 2) << 1;
}

// 16 bytes of every lane to LDS at `lds` + 16 lane, without registers between.
// Written in assembly because the compiler, which cannot tell the two buffers
// apart, would make every LDS read wait for the copy into the other one; the
// wait is wait_and_meet, before the barrier that opens the buffer, and no copy
// passes one: what lies between two of them may be reordered around the copies,
// since they go to a buffer that is not read there.  The wait state between the
// write of m0 and its use is the s_nop.
// m0 is declared, since the compiler merges its own writes of it; that it is a
// reserved register, which the compiler warns of, is no harm: nothing of its
// own lives there.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load16_to_lds(const uint8_t *base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "m0");
}
__device__ __forceinline__ void load16_to_lds(const uint8_t *p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds), "v"(p)
                 : "m0");
}
#pragma clang diagnostic pop
// A base of copies, which the wave shares, in scalar registers: the compiler may
// have computed it in the others.
__device__ __forceinline__ const uint8_t *scalar(const uint8_t *p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint8_t *)((uint64_t)hi << 32 | lo);
}
// Waits until at most N of the wave's copies to LDS are in flight and its own
// LDS accesses are done, then for the workgroup's other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// SPREAD: copies are sent one by one between the products, from further ahead: see
// run_spread.
template <class T, int BM_, int BN_, int WR_, int WC_, int BK_, int STAGES, bool TRA, bool TRB,
          bool STAGED, bool SPREAD = false>
struct Core {
    static constexpr int BM = BM_, BN = BN_, WR = WR_, WC = WC_, BK = BK_;
    static constexpr int S = STAGED ? 2 : STAGES;  // tiles in LDS
    static constexpr int THREADS = WR * WC * 64;
    static constexpr int FM = BM / WR / 16, FN = BN / WC / 16;
    static constexpr int CH = BK / 8;  // 16-byte chunks of a row with k contiguous
    static constexpr int LA = BM * CH / THREADS, LB = BN * CH / THREADS;  // loads a lane
    static constexpr int BYTES_A = BM * BK * 2, BYTES_B = BN * BK * 2;
    static constexpr int LDS = S * (BYTES_A + BYTES_B) + (SPREAD ? BYTES_B : 0);
    static_assert(LA >= 1 && LB >= 1 && FN >= 2 && BK == 64 && S >= 2, "tile");
    static_assert(!SPREAD || (!STAGED && S == 2 && LDS <= 163840), "spread");

    // One side's loads of a tile: lane offsets from the tile's uniform base.
    template <bool TR, int R, int L>
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
                    const uint32_t row = q / CH;
                    const uint32_t c = (q % CH) ^ chunk_key<TR, R>(row);
                    const uint32_t r = row < left ? row : left - 1;
                    off[i] = r * (uint32_t)o.ld * 2u + c * 16u;
                    kc[i] = c * 8;
                } else {
                    const uint32_t row = q / (R / 8);
                    uint32_t c = (q % (R / 8)) ^ chunk_key<TR, R>(row);
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
        // load i straight to LDS; left: k from this tile's first to the end
        __device__ __forceinline__ void issue(int i, const uint8_t *b, uint64_t left,
                                              uint32_t lds) const {
            lds += __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024 + i * THREADS * 16;
            if (left >= (uint64_t)BK) {
                load16_to_lds(b, off[i], lds);
            } else {
                // the k of the load, anew: only the last tile asks for it
                const uint32_t q = i * THREADS + threadIdx.x;
                const uint32_t k =
                    TR ? q / (R / 8)
                       : ((q % CH) ^ chunk_key<TR, R>(q / CH)) * 8;
                load16_to_lds(k < left ? b + off[i] : (const uint8_t *)zero_page, lds);
            }
        }
        // WHOLE: left >= BK
        template <bool WHOLE>
        __device__ __forceinline__ void send(int i, const uint8_t *b, uint64_t left,
                                             uint32_t lds) const {
            issue(i, b, WHOLE ? (uint64_t)BK : left, lds);
        }
        __device__ __forceinline__ void fetch(const uint8_t *b, uint64_t left,
                                              u32x4 (&reg)[L]) const {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                uint32_t n = 8;
                if (TR)
                    n = kc[i] < left ? have[i] : 0;
                else if (left < (uint64_t)BK)
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
    template <bool TR, int R>
    __device__ __forceinline__ static s16x8 fragment(uint32_t lds, uint32_t first, int i,
                                                     uint32_t kk) {
        const uint32_t l = threadIdx.x & 63u, r = l & 15u, g = l >> 4;
        if (!TR) {
            const uint32_t row = first + 16 * i + r;
            const uint32_t c = (g + 4 * kk) ^ chunk_key<TR, R>(row);
            return lds_read<s16x8>(lds + row * (BK * 2) + c * 16);
        }
        const uint32_t col = first + 16 * i + (r & 3u) * 4;
        s16x4 h[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t k = kk * 32 + g * 8 + x * 4 + (r >> 2);
            const uint32_t c = (col >> 3) ^ chunk_key<TR, R>(k);
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
        for (uint32_t kk = 0; kk < BK / 32; ++kk) {
            s16x8 b[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[j] = fragment<TRB, BN>(lb, nb, j, kk);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const s16x8 a = fragment<TRA, BM>(la, ma, i, kk);
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = T::mfma(b[j], a, acc[i][j]);
            }
        }
    }

    // Two tiles of A and three of B in LDS.  A wave's copies are accepted at the rate
    // that the memory system serves all of the compute unit's, and a wave that
    // sends a whole tile of them at once stands still for it: so they go out one
    // at a time, every other fragment's products.  A's next tile first, which then
    // has half a tile's time to arrive, then B's next but one, which the wait
    // leaves in flight.  Fragments of A are read three steps before their products,
    // B's for the second half of k during the first.  8192 x 16384 x 4096: 1390
    // TFLOP/s, all of a tile's copies sent before its products 1180; with B by
    // rows 1360 and 1170, both by rows 1330 and 1120.
    __device__ __forceinline__ static void run_spread(const Operand &a, const Operand &b,
                                                      uint32_t t0, uint32_t t1, uint32_t pairs,
                                                      uint32_t lds0, f32x4 (&acc)[FM][FN]) {
        Side<TRA, BM, LA> sa;
        Side<TRB, BN, LB> sb;
        sa.init(a);
        sb.init(b);
        const uint32_t wave = threadIdx.x >> 6;
        const uint32_t ma = (wave / WC) * (FM * 16), nb = (wave % WC) * (FN * 16);
        struct Base {
            const uint8_t *p;
            uint64_t left;
        };
        auto base = [&](bool is_a, uint32_t t) {
            const uint32_t pass = !pairs || t >= 2 * pairs ? 2 : t < pairs ? 0 : 1;
            const uint64_t k0 = (uint64_t)(t - pass * pairs) * BK;
            return Base{scalar(is_a ? sa.base(a, pass == 1, k0) : sb.base(b, pass == 0, k0)),
                        a.k - k0};
        };
        uint32_t a_now = lds0, a_next = lds0 + BYTES_A;
        uint32_t b_now = lds0 + 2 * BYTES_A, b_next = b_now + BYTES_B, b_third = b_next + BYTES_B;
        auto send = [&](bool is_a, uint32_t t, uint32_t to) {
            const Base p = base(is_a, t);
            if (is_a) {
#pragma unroll
                for (int x = 0; x < LA; ++x)
                    sa.issue(x, p.p, p.left, to);
            } else {
#pragma unroll
                for (int x = 0; x < LB; ++x)
                    sb.issue(x, p.p, p.left, to);
            }
        };
        send(true, t0, a_now);
        send(false, t0, b_now);
        if (t0 + 1 < t1)
            send(false, t0 + 1, b_next);
        // PLAIN: both copies are there to send, of whole k tiles
        auto tile = [&](auto plain, uint32_t t) {
            constexpr bool PLAIN = decltype(plain)::value;
            constexpr int STEPS = BK / 32 * FM, AHEAD = 3;
            static_assert(2 * (LA + LB) <= STEPS && FM > FN, "a copy every other step");
            const bool more_a = PLAIN || t + 1 < t1, more_b = PLAIN || t + 2 < t1;
            Base p = {}, q = {};
            if (more_a)
                p = base(true, t + 1);
            if (more_b)
                q = base(false, t + 2);
            s16x8 fb[BK / 32][FN], fa[AHEAD + 1];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[0][j] = fragment<TRB, BN>(b_now, nb, j, 0);
#pragma unroll
            for (int d = 0; d < AHEAD; ++d)
                fa[d] = fragment<TRA, BM>(a_now, ma, d, 0);
#pragma unroll
            for (int step = 0; step < STEPS; ++step) {
                const int kk = step / FM, i = step % FM, ahead = step + AHEAD;
                if (ahead < STEPS)
                    fa[ahead % (AHEAD + 1)] =
                        fragment<TRA, BM>(a_now, ma, ahead % FM, ahead / FM);
                const int j1 = step - (FM - FN - 1);
                if (j1 >= 0 && j1 < FN)
                    fb[1][j1] = fragment<TRB, BN>(b_now, nb, j1, 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = T::mfma(fb[kk][j], fa[step % (AHEAD + 1)], acc[i][j]);
                const int x = step / 2;
                if (step % 2 == 0 && x < LA && more_a)
                    sa.template send<PLAIN>(x, p.p, p.left, a_next);
                if (step % 2 == 0 && x >= LA && x < LA + LB && more_b)
                    sb.template send<PLAIN>(x - LA, q.p, q.left, b_third);
                __builtin_amdgcn_sched_barrier(0);
            }
            const uint32_t x = a_now, y = b_now;
            a_now = a_next;
            a_next = x;
            b_now = b_next;
            b_next = b_third;
            b_third = y;
        };
        // whole tiles first: a check at every copy costs what their order gains
        const uint32_t whole =
            a.k % BK == 0 ? t1 : pairs ? t0 : (uint32_t)(a.k / BK) < t1 ? (uint32_t)(a.k / BK) : t1;
        uint32_t t = t0;
        for (; t + 2 < whole; ++t) {
            // tile t has landed, and every wave is done with the one before
            wait_and_meet<LB>();
            tile(std::true_type(), t);
        }
        for (; t < t1; ++t) {
            if (t + 1 < t1)
                wait_and_meet<LB>();
            else
                wait_and_meet<0>();
            tile(std::false_type(), t);
        }
    }

    // acc += the k tiles [t0, t1), t0 < t1.  Plain operands: pairs = 0.  Pairs
    // of high and low parts: pairs = the tiles of one pass over k; tiles go
    // through high * low, low * high, and high * high last, so that the sums
    // that all the large terms meet are rounded a third as often.
    __device__ __forceinline__ static void run(const Operand &a, const Operand &b, uint32_t t0,
                                               uint32_t t1, uint32_t pairs, uint8_t *lds,
                                               f32x4 (&acc)[FM][FN]) {
        Side<TRA, BM, LA> sa;
        Side<TRB, BN, LB> sb;
        sa.init(a);
        sb.init(b);
        constexpr int kBuf = BYTES_A + BYTES_B;
        // the buffers' address in LDS, as the copies take it
        const uint32_t lds0 =
            (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
        struct Bases {
            const uint8_t *a, *b;
            uint64_t left;
        };
        auto bases = [&](uint32_t t) {
            const uint32_t pass = !pairs || t >= 2 * pairs ? 2 : t < pairs ? 0 : 1;
            const uint64_t k0 = (uint64_t)(t - pass * pairs) * BK;
            return Bases{sa.base(a, pass == 1, k0), sb.base(b, pass == 0, k0), a.k - k0};
        };
        if constexpr (STAGED) {
            u32x4 ra[LA], rb[LB];
            auto load = [&](uint32_t t) {
                const Bases p = bases(t);
                sa.fetch(p.a, p.left, ra);
                sb.fetch(p.b, p.left, rb);
            };
            load(t0);
            sa.put(ra, lds0);
            sb.put(rb, lds0 + BYTES_A);
            uint32_t now = lds0, next = lds0 + kBuf;
            for (uint32_t t = t0; t < t1; ++t) {
                // tile t is there, and every wave is done with the other buffer
                wait_and_meet<0>();
                if (t + 1 < t1)
                    load(t + 1);
                multiply(now, now + BYTES_A, acc);
                if (t + 1 < t1) {
                    sa.put(ra, next);
                    sb.put(rb, next + BYTES_A);
                }
                const uint32_t x = now;
                now = next;
                next = x;
            }
        } else if constexpr (SPREAD) {
            run_spread(a, b, t0, t1, pairs, lds0, acc);
        } else {
            // S - 1 tiles are in flight ahead of the one multiplied, so that a
            // copy has that many tiles' time to arrive
            uint32_t in = lds0, now = lds0, t_in = t0;
            const uint32_t end = lds0 + S * kBuf;
            auto issue = [&]() {
                const Bases to = bases(t_in++);
#pragma unroll
                for (int x = 0; x < LA; ++x)
                    sa.issue(x, to.a, to.left, in);
#pragma unroll
                for (int x = 0; x < LB; ++x)
                    sb.issue(x, to.b, to.left, in + BYTES_A);
                in = in + kBuf == end ? lds0 : in + kBuf;
            };
#pragma unroll
            for (int i = 0; i < S - 1; ++i)
                if (t_in < t1)
                    issue();
            for (uint32_t t = t0; t < t1; ++t) {
                // tile t has landed, and every wave is done with the tile
                // whose place the next copy takes
                if (t + S - 2 < t1)
                    wait_and_meet<(S - 2) * (LA + LB)>();
                else
                    wait_and_meet<0>();
                if (t_in < t1)
                    issue();
                multiply(now, now + BYTES_A, acc);
                now = now + kBuf == end ? lds0 : now + kBuf;
            }
        }
    }

    // The n, within the tile, of all that `each` hands to this lane, not TURNED.
    __device__ __forceinline__ static uint32_t column() {
        const uint32_t wave = threadIdx.x >> 6, l = threadIdx.x & 63u;
        return (wave % WC) * (FN * 16) + l % (2 * FN) * 8;
    }

    // then(m, n, v, fetch(m, n)) for every 8 consecutive n of a row m of the
    // wave's results (both within the tile); TURNED: for every 8 consecutive m
    // of a column n.  They go through the wave's own part of LDS, so that 8
    // lanes (4 with FN = 2) hold whole 128-byte pieces of a row or column.
    // What the epilogue reads comes from fetch, AHEAD pieces before the stores
    // of the first, so that a piece need not wait for memory by itself: four
    // with waves of 64 rows (128 x 128 tiles); with 128 rows the registers
    // spill (8192 x 16384 x 4096 with GELU by tanh and z: 1036 us two ahead,
    // 1007 us one), with 32 there are two pieces.
    template <bool TURNED = false, int AHEAD = (BM_ / WR_ == 64 ? 4 : 1), class G, class F>
    __device__ __forceinline__ static void each(const f32x4 (&acc)[FM][FN], uint8_t *lds,
                                                G &&fetch, F &&then) {
        constexpr int H = FM < 4 ? FM : 4;         // fragments of rows at a time
        constexpr int C = 4 * FN;                  // 16-byte chunks of a row
        constexpr int PART = H * 16 * C * 16;      // bytes of a wave's part
        static_assert(PART * WR * WC <= LDS, "the results' part of LDS");
        const uint32_t wave = threadIdx.x >> 6, l = threadIdx.x & 63u;
        const uint32_t at =
            (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + wave * PART;
        const uint32_t m0 = (wave / WC) * (FM * 16), n0 = (wave % WC) * (FN * 16);
        constexpr int LANES = TURNED ? H * 2 : C / 2;          // of one row (or column)
        constexpr int STEP = 64 / LANES;
        constexpr int COUNT = (TURNED ? 4 * C : H * 16) / STEP;  // pieces of a lane
        constexpr int U = COUNT < AHEAD ? COUNT : AHEAD;
        wait_and_meet<0>();  // every wave is done with the tiles
        const uint32_t in = l % LANES, first = l / LANES;
        auto group = [&](auto from) {
            constexpr int i0 = decltype(from)::value;
#pragma unroll
            for (int i = 0; i < H; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const uint32_t row = 16 * i + (l & 15u), c = 4 * j + (l >> 4);
                    lds_write(at + (row * C + (c ^ (row & (C - 1)))) * 16, acc[i0 + i][j]);
                }
            auto m_of = [&](uint32_t p) { return m0 + i0 * 16 + (TURNED ? in * 8 : p); };
            auto n_of = [&](uint32_t p) { return n0 + (TURNED ? p : in * 8); };
#pragma unroll 1
            for (int q = 0; q < COUNT; q += U) {
                decltype(fetch(0u, 0u)) got[U];
#pragma unroll
                for (int x = 0; x < U; ++x) {
                    const uint32_t p = first + (q + x) * STEP;
                    got[x] = fetch(m_of(p), n_of(p));
                }
#pragma unroll
                for (int x = 0; x < U; ++x) {
                    const uint32_t p = first + (q + x) * STEP;
                    float v[8];
                    if constexpr (TURNED) {
#pragma unroll
                        for (uint32_t e = 0; e < 8; ++e) {
                            const uint32_t r = in * 8 + e;
                            v[e] = lds_read<float>(at + (r * C + ((p >> 2) ^ (r & (C - 1)))) * 16
                                                   + (p & 3u) * 4);
                        }
                    } else {
                        const f32x4 y =
                            lds_read<f32x4>(at + (p * C + ((in * 2) ^ (p & (C - 1)))) * 16);
                        const f32x4 z =
                            lds_read<f32x4>(at + (p * C + ((in * 2 + 1) ^ (p & (C - 1)))) * 16);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[e] = y[e];
                            v[4 + e] = z[e];
                        }
                    }
                    then(m_of(p), n_of(p), v, got[x]);
                }
            }
        };
        // by hand: the compiler does not unroll a loop with bodies this long,
        // and would keep acc in scratch memory
        static_assert(FM / H <= 2, "groups");
        group(std::integral_constant<int, 0>());
        if constexpr (FM > H)
            group(std::integral_constant<int, H>());
    }
};

}  // namespace gemm
}  // namespace ddl
