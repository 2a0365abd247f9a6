// linear_tiles.h -- device pieces of the tile kernels (linear.hip,
// orthogonalize.hip): the matrix instructions, the layout of operand tiles in
// shared memory and the copies into them.  Internal.
#ifndef ZERO_SHARD_LINEAR_TILES_H
#define ZERO_SHARD_LINEAR_TILES_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "linear_common.h"
#include "linear_plan.h"

namespace zero_linear_impl {

using zero_host::kWave;

using s16x4 = short __attribute__((ext_vector_type(4)));
using s16x8 = short __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// matrix instructions

template <class T>
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma<BF16>(s16x8 a, s16x8 b, f32x4 c) {
    using v = __bf16 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v, a),
                                                   __builtin_bit_cast(v, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma<FP16>(s16x8 a, s16x8 b, f32x4 c) {
    using v = _Float16 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v, a),
                                                  __builtin_bit_cast(v, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// tiles in shared memory, in 16-byte pieces of eight elements
//
// Which 16 rows of Q make a block is free, and is chosen for the outputs: row
// 4 g + r of blocks t = 2 p and 2 p + 1 is j = 32 p + 8 g + 4 (t & 1) + r, so
// that the two blocks leave a lane eight consecutive j of its i, and its four
// neighbours the 64 bytes that follow (Q = true below).  Blocks of P are 16
// consecutive rows.
//
// Rows of c: [ROWS][64], piece (row, s) at row * 8 + (s ^ twist(row)); a
// lane's operand is one piece, eight consecutive c of its row.  twist differs
// for any eight rows that are read at once, which spreads their pieces over
// all banks.
//
// Rows of lanes: [64][ROWS], in 32-byte units of 16 lanes.
// ds_read_b64_tr_b16 reads 4 x 4 quads, one of four rows c each, and hands
// every lane the four c of its own column; two of them make an operand.  The
// four rows must lie in different banks: unit u of row c is stored at
// u ^ flip(c), and tiles of 256 lanes, whose rows are two bank widths long,
// also skip 64 bytes after each 1024 (a wave's direct copy is 1024 bytes, so
// it is not cut).  flip touches few bits and depends on c mod 4 only, so that
// a lane's addresses are one or two registers plus constants.

template <bool Q>
__device__ __forceinline__ int twist(int row) {
    return Q ? (row & 3) | (row >> 1 & 4) : row & 7;
}
template <int ROWS>
constexpr int kFlipBits = ROWS == 256 ? 4 : ROWS == 128 ? 6 : 1;
template <int ROWS>
__device__ __forceinline__ int flip(int c) {
    return ROWS == 256 ? (c & 1) * 4 : ROWS == 128 ? (c & 3) * 2 : (c >> 1) & 1;
}
template <bool KC, int ROWS>
constexpr int kSkip = !KC && ROWS == 256 ? 32 : 0;  // elements after each 512
template <bool KC, int ROWS>
constexpr int kTile = ROWS * kBK + ROWS * kBK / 512 * kSkip<KC, ROWS>;

template <bool KC, int ROWS>
__device__ __forceinline__ int piece_row(int pos) {
    return KC ? pos >> 3 : pos / (ROWS / 8);
}
template <bool KC, int ROWS, bool Q>
__device__ __forceinline__ int piece_slot(int pos) {
    if (KC) return (pos & 7) ^ twist<Q>(pos >> 3);
    return (pos % (ROWS / 8)) ^ (2 * flip<ROWS>(pos / (ROWS / 8)));
}

// where piece pos lies in the tile
template <bool KC, int ROWS>
__device__ __forceinline__ int piece_at(int pos) {
    return pos * 8 + (pos >> 6) * kSkip<KC, ROWS>;
}

// A piece of the operand as eight elements, zeros past the row's or the
// contraction's end: one unaligned 16-byte load where all eight exist (global
// memory takes any alignment), element loads at the ends.
__device__ __forceinline__ u32x4 load_piece(const uint16_t *p, int64_t n) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (n >= 8) {
        __builtin_memcpy(&v, p, 16);
    } else if (n > 0) {
        uint16_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = e < n ? p[e] : 0;
        __builtin_memcpy(&v, h, 16);
    }
    return v;
}

template <bool KC, int ROWS, int THREADS, bool Q>
struct Stage {
    static constexpr int N = ROWS * kBK / 8 / THREADS;
    static_assert(N >= 1 && N * THREADS * 8 == ROWS * kBK, "whole pieces for every thread");
    u32x4 v[N];
    // rows [r0, rows), contraction [c0, c1)
    __device__ __forceinline__ void load(const uint16_t *p, int64_t ld, int64_t r0, int64_t rows,
                                         int64_t c0, int64_t c1) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int pos = n * THREADS + static_cast<int>(threadIdx.x);
            const int row = piece_row<KC, ROWS>(pos), s = piece_slot<KC, ROWS, Q>(pos);
            if (KC) {
                const int64_t r = r0 + row, c = c0 + s * 8;
                v[n] = load_piece(p + r * ld + c, r < rows ? c1 - c : 0);
            } else {
                const int64_t c = c0 + row, r = r0 + s * 8;
                v[n] = load_piece(p + c * ld + r, c < c1 ? rows - r : 0);
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t *tile) const {
#pragma unroll
        for (int n = 0; n < N; ++n)
            *reinterpret_cast<u32x4 *>(
                tile + piece_at<KC, ROWS>(n * THREADS + static_cast<int>(threadIdx.x))) = v[n];
    }
};

// Direct copies of whole steps from global memory into a tile: a wave's 64
// pieces of one instruction land at consecutive places, so the exclusive or
// is applied to where each lane reads instead.  Rows past the operand's last
// read that row again (their outputs are never stored).  The instruction is
// written out because the compiler makes every later read of shared memory
// wait for all copies it knows of; the kernel waits for the ones it needs.
// It has no output register, and its inputs are read when it issues.  The
// compiler writes m0 (the place in shared memory) but does not see that the
// statement holds a memory instruction: the five wait states before it are
// those after a vector write of the base's scalar registers (the way back of a
// spilled one), and cover the one after m0's.
template <bool KC, int ROWS, int THREADS, bool Q>
struct Direct {
    static constexpr int N = ROWS * kBK / 8 / THREADS;
    static constexpr int kRows = THREADS * 8 / ROWS;  // rows of lanes per copy
    static_assert(KC || kRows % 8 == 0, "a lane's unit has the same place in every copy");
    const char *base;       // of the next step
    int64_t stride;         // bytes from step to step
    int64_t apart;          // bytes from copy to copy (rows of lanes)
    uint32_t off[KC ? N : 1];
    // thread: of the THREADS that copy the tile
    __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int64_t r0, int64_t rows,
                                         int64_t c0, int thread) {
        base = reinterpret_cast<const char *>(KC ? p + r0 * ld + c0 : p + c0 * ld + r0);
        stride = (KC ? kBK : kBK * ld) * 2;
        apart = KC ? 0 : kRows * ld * 2;
        const int last = static_cast<int>(min(rows - r0, static_cast<int64_t>(ROWS))) - (KC ? 1 : 8);
#pragma unroll
        for (int n = 0; n < (KC ? N : 1); ++n) {
            const int pos = n * THREADS + thread;
            const int row = piece_row<KC, ROWS>(pos), s = piece_slot<KC, ROWS, Q>(pos);
            off[n] = KC ? static_cast<uint32_t>(min(row, last)) * static_cast<uint32_t>(ld * 2) + s * 16
                        : static_cast<uint32_t>(row) * static_cast<uint32_t>(ld * 2) +
                              min(s * 8, last) * 2;
        }
    }
    // copy n of a step; tile: its byte address in shared memory
    __device__ __forceinline__ void issue(int n, uint32_t tile, int wave) const {
        asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "{m0}"(tile + 2 * piece_at<KC, ROWS>(n * THREADS + wave * kWave)),
                       "v"(off[KC ? n : 0]), "s"(base + n * apart)
                     : "memory");
    }
    __device__ __forceinline__ void next() { base += stride; }
};

// a lane's operand of 16-row block f from row row0 on: its eight consecutive
// c of the 32 that start at kk * 32
template <bool KC, int ROWS, bool Q>
__device__ __forceinline__ s16x8 fragment(const uint16_t *tile, int row0, int f, int kk, int lane) {
    const int t = lane & 15, g = lane >> 4;
    if constexpr (KC) {
        const int r = Q ? (t >> 2) * 8 + (t & 3) : t;
        const int first = Q ? (f >> 1) * 32 + (f & 1) * 4 : f * 16;
        return *reinterpret_cast<const s16x8 *>(
            tile + (row0 + r) * kBK + (((kk * 4 + g) ^ twist<Q>(r)) * 8) + first * kBK);
    } else {
        const int c = g * 8 + (t >> 2);
        constexpr int F = kFlipBits<ROWS>;
        const int unit = Q ? (f >> 1) * 2 : f;      // of the block's first lane
        const int in = Q ? (t & 3) >> 1 : 0;        // units on
        const int at = c * ROWS + (c * ROWS >> 9) * kSkip<KC, ROWS> +
                       ((row0 / 16 + (unit & F) + in) ^ flip<ROWS>(c)) * 16 +
                       (Q ? (t & 1) * 8 + (f & 1) * 4 : (t & 3) * 4);
        using lds4 = __attribute__((address_space(3))) s16x4;
        s16x8 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            constexpr int per_row = ROWS + ROWS * kSkip<KC, ROWS> / 512;
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds4 *)(tile + at + (unit & ~F) * 16 + (kk * 32 + h * 4) * per_row));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h * 4 + e] = x[e];
        }
        return v;
    }
}

}  // namespace zero_linear_impl

#endif
