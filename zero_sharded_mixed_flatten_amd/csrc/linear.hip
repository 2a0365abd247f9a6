// linear.hip -- gfx950 kernels of the layer products on the flat buffers:
// zero_linear, zero_linear_dgrad, zero_linear_wgrad.
//
// All three are one contraction, out[i][j] = sum over c of P(i, c) Q(j, c),
// over operands stored with c contiguous ("rows of c") or with i or j
// contiguous ("rows of lanes"):
//   linear  i = m, j = n, c = k:  P = x  (rows of c),     Q = W (rows of c)
//   dgrad   i = m, j = k, c = n:  P = dy (rows of c),     Q = W (rows of lanes)
//   wgrad   i = n, j = k, c = m:  P = dy (rows of lanes), Q = x (rows of lanes)
//
// A workgroup computes a BI x BJ tile with v_mfma_f32_16x16x32.  Q is the
// instruction's row operand, so that a lane ends up with four consecutive j
// of one i: its outputs, residuals and biases are vectors.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "linear_common.h"
#include "linear_plan.h"

namespace {

using namespace zero_host;
using namespace zero_linear_impl;

using s16x4 = short __attribute__((ext_vector_type(4)));
using s16x8 = short __attribute__((ext_vector_type(8)));

struct Epilogue {
    const uint16_t *bias;
    const void *res;
    void *out;
    uint16_t *z;      // linear: written; dgrad: read
    void *db;         // wgrad
    int64_t ldr, ldo, ldz;
    int32_t act, out_f32, accumulate;
    Drop drop;
};

struct Args {
    const uint16_t *p, *q;
    int64_t ldp, ldq;
    int64_t ni, nj, nc;
    int64_t chunk;    // contraction elements of a part, a multiple of kBK
    int32_t parts;
    int32_t tiles_i, tiles_j;
    int32_t quarter;  // >= 0: the workgroups are quarters of the tiles from here on
    float *partial;   // [parts][ni][njp], then the column sums [parts][ni]
    Epilogue e;
};

__host__ __device__ inline int64_t padded4(int64_t n) { return (n + 3) & ~int64_t(3); }

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
// epilogue of four neighbouring outputs (i, j..j+3), n of them inside

template <int OP, class T>
__device__ __forceinline__ void emit(const Epilogue &e, int64_t i, int64_t j, int n, f32x4 v,
                                     u32x4 words, int half) {
    if constexpr (OP == WGRAD) {
        if (e.out_f32) {
            float *o = static_cast<float *>(e.out) + i * e.ldo + j;
            if (e.accumulate) v = load32(o, n) + v;
            store32(o, v, n);
        } else {
            uint16_t *o = static_cast<uint16_t *>(e.out) + i * e.ldo + j;
            if (e.accumulate) v = load16<T>(o, n) + v;
            store16<T>(o, v, n);
        }
        return;
    }
    if constexpr (OP == FWD) {
        if (e.bias != nullptr) v += load16<T>(e.bias + j, n);
        if (e.z != nullptr) store16<T>(e.z + i * e.ldz + j, v, n);
        if (e.act != ZERO_ACT_NONE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = act_value(v[k], e.act);
        }
    } else if (e.act != ZERO_ACT_NONE) {
        const f32x4 z = load16<T>(e.z + i * e.ldz + j, n);
        if (e.act == ZERO_ACT_RELU) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = z[k] > 0.0f ? v[k] : 0.0f;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] *= act_slope(z[k], e.act);
        }
    }
    if (e.drop.on) v = drop_apply(e.drop, words, half, v);
    if (e.out_f32) {
        if (e.res != nullptr)
            v = load32(static_cast<const float *>(e.res) + i * e.ldr + j, n) + v;
        store32(static_cast<float *>(e.out) + i * e.ldo + j, v, n);
    } else {
        if (e.res != nullptr)
            v = load16<T>(static_cast<const uint16_t *>(e.res) + i * e.ldr + j, n) + v;
        store16<T>(static_cast<uint16_t *>(e.out) + i * e.ldo + j, v, n);
    }
}

// the quads at j and j + 16 (j a multiple of 4 in the first half of its group
// of 32 columns), which share one draw of the mask
template <int OP, class T>
__device__ __forceinline__ void emit_pair(const Epilogue &e, int64_t i, int64_t j, int64_t nj,
                                          uint64_t stream, f32x4 v0, f32x4 v1) {
    if (j >= nj) return;
    u32x4 words = {0u, 0u, 0u, 0u};
    if (OP != WGRAD && e.drop.on)
        words = drop_words(e.drop, stream, static_cast<uint32_t>(i),
                           static_cast<uint32_t>((j >> 5) * 4 + ((j & 15) >> 2)));
    emit<OP, T>(e, i, j, static_cast<int>(nj - j < 4 ? nj - j : 4), v0, words, 0);
    const int64_t j1 = j + 16;
    if (j1 < nj) emit<OP, T>(e, i, j1, static_cast<int>(nj - j1 < 4 ? nj - j1 : 4), v1, words, 1);
}

// eight neighbouring outputs (i, j..j+7), n of them inside: the quads at j
// and j + 4, whose mask words are w0 and w1, the same half of both
template <int OP, class T>
__device__ __forceinline__ void emit8(const Epilogue &e, int64_t i, int64_t j, int n, f32x4 v0,
                                      f32x4 v1, u32x4 w0, u32x4 w1, int half) {
    if (n < 8) {
        emit<OP, T>(e, i, j, n < 4 ? n : 4, v0, w0, half);
        if (n > 4) emit<OP, T>(e, i, j + 4, n - 4, v1, w1, half);
        return;
    }
    f32x4 a, b;
    if constexpr (OP == WGRAD) {
        if (e.out_f32) {
            emit<OP, T>(e, i, j, 4, v0, w0, half);
            emit<OP, T>(e, i, j + 4, 4, v1, w1, half);
        } else {
            uint16_t *o = static_cast<uint16_t *>(e.out) + i * e.ldo + j;
            if (e.accumulate) {
                load16x8<T>(o, a, b);
                v0 = a + v0;
                v1 = b + v1;
            }
            stream16x8<T>(o, v0, v1);
        }
        return;
    }
    if constexpr (OP == FWD) {
        if (e.bias != nullptr) {
            load16x8<T>(e.bias + j, a, b);
            v0 += a;
            v1 += b;
        }
        if (e.z != nullptr) stream16x8<T>(e.z + i * e.ldz + j, v0, v1);
        if (e.act != ZERO_ACT_NONE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v0[k] = act_value(v0[k], e.act);
                v1[k] = act_value(v1[k], e.act);
            }
        }
    } else if (e.act != ZERO_ACT_NONE) {
        load16x8<T>(e.z + i * e.ldz + j, a, b);
        if (e.act == ZERO_ACT_RELU) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v0[k] = a[k] > 0.0f ? v0[k] : 0.0f;
                v1[k] = b[k] > 0.0f ? v1[k] : 0.0f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v0[k] *= act_slope(a[k], e.act);
                v1[k] *= act_slope(b[k], e.act);
            }
        }
    }
    if (e.drop.on) {
        v0 = drop_apply(e.drop, w0, half, v0);
        v1 = drop_apply(e.drop, w1, half, v1);
    }
    if (e.out_f32) {
        float *o = static_cast<float *>(e.out) + i * e.ldo + j;
        if (e.res != nullptr) {
            const float *r = static_cast<const float *>(e.res) + i * e.ldr + j;
            v0 = load32(r, 4) + v0;
            v1 = load32(r + 4, 4) + v1;
        }
        store32(o, v0, 4);
        store32(o + 4, v1, 4);
    } else {
        uint16_t *o = static_cast<uint16_t *>(e.out) + i * e.ldo + j;
        if (e.res != nullptr) {
            load16x8<T>(static_cast<const uint16_t *>(e.res) + i * e.ldr + j, a, b);
            v0 = a + v0;
            v1 = b + v1;
        }
        stream16x8<T>(o, v0, v1);
    }
}

// eight whole outputs without activation or with one of the two logistic ones
// (ACT), and with a mask (MASK: the words and half of emit8) or without
template <int OP, class T, bool ACT, bool MASK>
__device__ __forceinline__ void emit_light(const Epilogue &e, int64_t i, int64_t j, f32x4 v0,
                                           f32x4 v1, const Logistic &l, u32x4 w0, u32x4 w1,
                                           int half) {
    f32x4 a, b;
    if (OP == FWD && e.bias != nullptr) {
        load16x8<T>(e.bias + j, a, b);
        v0 += a;
        v1 += b;
    }
    if (OP == FWD && e.z != nullptr) stream16x8<T>(e.z + i * e.ldz + j, v0, v1);
    if (ACT && OP == DGRAD) load16x8<T>(e.z + i * e.ldz + j, a, b);
    if (ACT) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v0[k] = OP == FWD ? logistic_value(v0[k], l) : v0[k] * logistic_slope(a[k], l);
            v1[k] = OP == FWD ? logistic_value(v1[k], l) : v1[k] * logistic_slope(b[k], l);
        }
    }
    if (MASK) {
        v0 = drop_apply(e.drop, w0, half, v0);
        v1 = drop_apply(e.drop, w1, half, v1);
    }
    const bool add = OP == WGRAD ? e.accumulate != 0 : e.res != nullptr;
    const void *old = OP == WGRAD ? e.out : e.res;
    const int64_t at = i * (OP == WGRAD ? e.ldo : e.ldr) + j;
    if (e.out_f32) {
        if (add) {
            v0 = load32(static_cast<const float *>(old) + at, 4) + v0;
            v1 = load32(static_cast<const float *>(old) + at + 4, 4) + v1;
        }
        float *o = static_cast<float *>(e.out) + i * e.ldo + j;
        store32(o, v0, 4);
        store32(o + 4, v1, 4);
    } else {
        if (add) {
            load16x8<T>(static_cast<const uint16_t *>(old) + at, a, b);
            v0 = a + v0;
            v1 = b + v1;
        }
        stream16x8<T>(static_cast<uint16_t *>(e.out) + i * e.ldo + j, v0, v1);
    }
}

template <class T>
__device__ __forceinline__ void emit_db(const Epilogue &e, int64_t i, float v) {
    if (e.out_f32) {
        float *o = static_cast<float *>(e.db) + i;
        *o = e.accumulate ? *o + v : v;
    } else {
        uint16_t *o = static_cast<uint16_t *>(e.db) + i;
        *o = T::down(e.accumulate ? T::up(*o) + v : v);
    }
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
    __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int64_t r0, int64_t rows,
                                         int64_t c0) {
        base = reinterpret_cast<const char *>(KC ? p + r0 * ld + c0 : p + c0 * ld + r0);
        stride = (KC ? kBK : kBK * ld) * 2;
        apart = KC ? 0 : kRows * ld * 2;
        const int last = static_cast<int>(min(rows - r0, static_cast<int64_t>(ROWS))) - (KC ? 1 : 8);
#pragma unroll
        for (int n = 0; n < (KC ? N : 1); ++n) {
            const int pos = n * THREADS + static_cast<int>(threadIdx.x);
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

// The tile of this workgroup.  Workgroups go round the 8 XCDs in turn; each
// XCD is given one contiguous run of tiles, taken in bands of 8 rows of
// tiles, so that the tiles at work in one L2 share their operands.
__device__ __forceinline__ void tile_of(const Args &a, int b, int &ti, int &tj) {
    const int total = a.tiles_i * a.tiles_j;
    const int x = b & 7, q = total >> 3, r = total & 7;
    const int id = x * q + (x < r ? x : r) + (b >> 3);
    const int band = 8 * a.tiles_j, first = id / band * 8;
    const int high = min(8, a.tiles_i - first), in = id - first * a.tiles_j;
    ti = first + in % high;
    tj = in / high;
}

// The main loop goes by steps of 64 of the contraction, held in one of two
// buffers, each step in two halves of 32 with operands of their own registers:
//   first half:   multiply the first 32, reading the second 32 meanwhile;
//   wait for the reads and for the copies of the next step; barrier;
//   second half:  multiply the second 32, starting the copies of the step
//                 after next into this step's buffer, which nobody reads any
//                 more, and reading the first 32 of the next step.
// Reads, copies and products are dealt out one by one, so that the matrix
// unit has work from the same wave while a read is under way.  A wave of the
// largest tiles has a block of 128 x 64, two waves a SIMD (128 x 128 would
// read less but does not fit the registers).  Measured at 8192 x 4096 x 11008
// with mask and residual (555 us, 1.33 PFLOP/s): the matrix units are busy for
// 60 to 68 % of the cycles, waves wait for 36 to 38 % of theirs (3 % on shared
// memory), memory delivers 2 TB/s, and after some launches on end the clock
// inside this loop falls from 2.2 to 1.9 GHz.
template <int OP, class T, int BI, int BJ, int WI, int WJ, bool DIRECT, bool DB>
__global__ void __launch_bounds__(WI *WJ *kWave, 2) tile_kernel(Args a) {
    constexpr bool PKC = OP != WGRAD, QKC = OP == FWD;
    constexpr int THREADS = WI * WJ * kWave;
    constexpr int FI = BI / WI / 16, FJ = BJ / WJ / 16;
    constexpr int SLOT = kTile<PKC, BI> + kTile<QKC, BJ>;
    static_assert(FJ % 2 == 0, "mask draws pair two 16-column blocks");
    __shared__ __attribute__((aligned(1024))) uint16_t tiles[2 * SLOT];

    int ti, tj;
    if (BI == 128 && a.quarter >= 0) {
        tile_of(a, a.quarter + static_cast<int>(blockIdx.x >> 2), ti, tj);
        ti = 2 * ti + (blockIdx.x >> 1 & 1);
        tj = 2 * tj + (blockIdx.x & 1);
        if (static_cast<int64_t>(ti) * BI >= a.ni || static_cast<int64_t>(tj) * BJ >= a.nj) return;
    } else {
        tile_of(a, static_cast<int>(blockIdx.x), ti, tj);
    }
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int wi = wave / WJ * (BI / WI), wj = wave % WJ * (BJ / WJ);
    const int64_t i0 = static_cast<int64_t>(ti) * BI, j0 = static_cast<int64_t>(tj) * BJ;
    const int part = blockIdx.y;
    const int64_t c0 = part * a.chunk, c1 = min(a.nc, c0 + a.chunk);
    const int steps = c1 > c0 ? static_cast<int>((c1 - c0 + kBK - 1) / kBK) : 0;

    f32x4 acc[FI][FJ];
#pragma unroll
    for (int f = 0; f < FI; ++f)
#pragma unroll
        for (int t = 0; t < FJ; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // The column sums of dy are one more product of P's blocks, with a matrix
    // of ones.  The waves of a row of the tile share these blocks: each sums
    // SUMS of them, which it reads once more (its turn picks them, and
    // registers cannot be picked without branches).
    constexpr int SUMS = FI / WJ;
    static_assert(!DB || (FI % WJ == 0 && SUMS <= 2), "the waves share the blocks of P");
    f32x4 sums[DB ? SUMS : 1];
    s16x8 fs[2][DB ? SUMS : 1];
#pragma unroll
    for (int e = 0; e < (DB ? SUMS : 1); ++e) sums[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool with_db = DB && tj == 0;
    const int turn = wave % WJ;

    // whole steps go straight to shared memory (DIRECT); a last broken one is
    // staged through registers
    const int whole = DIRECT ? static_cast<int>((c1 - c0) / kBK) : 0;
    Stage<PKC, BI, THREADS, false> sp;
    Stage<QKC, BJ, THREADS, true> sq;
    Direct<PKC, BI, THREADS, false> dp;
    Direct<QKC, BJ, THREADS, true> dq;
    constexpr int NP = Direct<PKC, BI, THREADS, false>::N, NQ = Direct<QKC, BJ, THREADS, true>::N;
    if (DIRECT) {
        dp.init(a.p, a.ldp, i0, a.ni, c0);
        dq.init(a.q, a.ldq, j0, a.nj, c0);
    }
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint16_t *)tiles));
    auto slot_of = [&](int s) __attribute__((always_inline)) { return (s & 1) * SLOT; };
    auto load = [&](int s) __attribute__((always_inline)) {
        sp.load(a.p, a.ldp, i0, a.ni, c0 + static_cast<int64_t>(s) * kBK, c1);
        sq.load(a.q, a.ldq, j0, a.nj, c0 + static_cast<int64_t>(s) * kBK, c1);
    };
    auto put = [&](int s) __attribute__((always_inline)) {
        sp.store(tiles + slot_of(s));
        sq.store(tiles + slot_of(s) + kTile<PKC, BI>);
    };
    auto copy = [&](int n, int s) __attribute__((always_inline)) {
        if (n < NP)
            dp.issue(n, lds + 2 * slot_of(s), wave);
        else if (n < NP + NQ)
            dq.issue(n - NP, lds + 2 * (slot_of(s) + kTile<PKC, BI>), wave);
    };
    auto copied = [&]() __attribute__((always_inline)) {
        dp.next();
        dq.next();
    };
    s16x8 fp[2][FI], fq[2][FJ];
    auto read = [&](int n, int s, int kk) __attribute__((always_inline)) {
        const uint16_t *tp = tiles + slot_of(s), *tq = tp + kTile<PKC, BI>;
        if (n < FJ)
            fq[kk][n] = fragment<QKC, BJ, true>(tq, wj, n, kk, lane);
        else if (n < FJ + FI)
            fp[kk][n - FJ] = fragment<PKC, BI, false>(tp, wi, n - FJ, kk, lane);
    };
    // the products of half kk, with reads of half 1 - kk of step rs and (COPY)
    // copies of step cs between them
    auto half = [&](auto kk_, auto copy_, auto db_, int rs, int cs) __attribute__((always_inline)) {
        constexpr int kk = decltype(kk_)::value, READS = FI + FJ, N = FI * FJ;
        constexpr bool COPY = decltype(copy_)::value;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            // reads and copies are spread over the first three quarters
            constexpr int M = N * 3 / 4 > 0 ? N * 3 / 4 : 1;
            bool placed = false;
#pragma unroll
            for (int r = 0; r < READS; ++r)
                if (r * M / READS == n) {
                    read(r, rs, 1 - kk);
                    placed = true;
                }
            if (COPY) {
#pragma unroll
                for (int c = 0; c < NP + NQ; ++c)
                    if (c * M / (NP + NQ) == n) {
                        copy(c, cs);
                        placed = true;
                    }
            }
            if (decltype(db_)::value && kk == 0 && n == 0) {
#pragma unroll
                for (int e = 0; e < 2 * SUMS; ++e)
                    fs[e & 1][e / 2] = fragment<PKC, BI, false>(
                        tiles + slot_of(rs), wi + (turn * SUMS + e / 2) * 16, 0, e & 1, lane);
            }
            acc[n / FJ][n % FJ] = mfma<T>(fq[kk][n % FJ], fp[kk][n / FJ], acc[n / FJ][n % FJ]);
            if (decltype(db_)::value && kk == 0 && n == N - 1) {
                const short o = static_cast<short>(T::down(1.0f));
#pragma unroll
                for (int e = 0; e < 2 * SUMS; ++e)
                    sums[e / 2] = mfma<T>(s16x8{o, o, o, o, o, o, o, o}, fs[e & 1][e / 2],
                                          sums[e / 2]);
            }
            if (placed) __builtin_amdgcn_sched_barrier(0);
        }
    };
    using first = std::integral_constant<int, 0>;
    using second = std::integral_constant<int, 1>;
    // this wave's reads are done and what it copied or staged has landed
    auto arrive = [&]() __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    auto contract = [&](auto db) __attribute__((always_inline)) {
        if constexpr (DIRECT) {
            if (whole > 0) {
#pragma unroll
                for (int n = 0; n < NP + NQ; ++n) copy(n, 0);
                copied();
                arrive();
                if (whole > 1) {
#pragma unroll
                    for (int n = 0; n < NP + NQ; ++n) copy(n, 1);
                    copied();
                }
#pragma unroll
                for (int n = 0; n < FI + FJ; ++n) read(n, 0, 0);
                int s = 0;
#pragma unroll 1
                for (; s < whole - 2; ++s) {
                    half(first{}, std::false_type{}, db, s, 0);
                    arrive();
                    half(second{}, std::true_type{}, db, s + 1, s + 2);
                    copied();
                }
#pragma unroll 1
                for (; s < whole; ++s) {
                    half(first{}, std::false_type{}, db, s, 0);
                    arrive();
                    half(second{}, std::false_type{}, db, s + 1, 0);
                }
            }
            if (whole < steps) {  // the broken step, in the buffer nobody reads
                load(whole);
                put(whole);
                arrive();
#pragma unroll
                for (int n = 0; n < FI + FJ; ++n) read(n, whole, 0);
                half(first{}, std::false_type{}, db, whole, 0);
                half(second{}, std::false_type{}, db, whole, 0);
            }
        } else if (steps > 0) {
            load(0);
            put(0);
            arrive();
            if (steps > 1) load(1);
#pragma unroll
            for (int n = 0; n < FI + FJ; ++n) read(n, 0, 0);
#pragma unroll 1
            for (int s = 0; s < steps; ++s) {
                half(first{}, std::false_type{}, db, s, 0);
                if (s + 1 < steps) put(s + 1);
                arrive();
                if (s + 2 < steps) load(s + 2);
                half(second{}, std::false_type{}, db, s + 1, 0);
            }
        }
    };
    // two loops, so that the other tiles' has no branch of the sums' in it
    if (with_db)
        contract(std::integral_constant<bool, DB>{});
    else
        contract(std::false_type{});

    const int g = lane >> 4;
    const int64_t njp = padded4(a.nj);
    const uint64_t stream = OP != WGRAD && a.e.drop.on && a.parts == 1 ? drop_stream(a.e.drop) : 0;
    // values, not places: an array picked from by address would go to memory
    const float sum0 = sums[0][0], sum1 = sums[DB ? SUMS - 1 : 0][0];
    auto sum_of = [&](int f) __attribute__((always_inline)) {
        return SUMS == 2 && (f & 1) ? sum1 : sum0;
    };
    // A lane has quads 2 g and 2 g + 1 of each 32 columns; quad u takes the
    // mask block u % 4.  The four lanes of a row draw one block each and hand
    // them round, while all of them are there.
    auto draw = [&](int64_t i, int p, u32x4 &w0, u32x4 &w1) __attribute__((always_inline)) {
        const u32x4 w = drop_words(a.e.drop, stream, static_cast<uint32_t>(i),
                                   static_cast<uint32_t>((j0 + wj) / 8 + p * 4 + g));
        const int from = (lane & 15) + 16 * ((2 * g) & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w0[k] = static_cast<uint32_t>(__shfl(static_cast<int>(w[k]), from));
            w1[k] = static_cast<uint32_t>(__shfl(static_cast<int>(w[k]), from + 16));
        }
    };
    // The usual outputs are written by straight code, without a register to
    // move (8192 x 6400 x 1600: 205 -> 158 us); columns that are not eight
    // whole ones are left to the body below.  One such code for each kind,
    // and no more than the instruction cache holds: one for every activation
    // and mask together loses (with GELU and z 242 -> 252).
    const bool smooth = a.e.act == ZERO_ACT_GELU_TANH || a.e.act == ZERO_ACT_SILU;
    const bool masked = OP != WGRAD && a.e.drop.on;
    const bool light =
        a.parts == 1 && (a.e.act == ZERO_ACT_NONE || (smooth && !masked));
    if (light) {
        const Logistic l = logistic_of(a.e.act);
        auto write = [&](auto act, auto mask) __attribute__((always_inline)) {
            constexpr bool MASK = decltype(mask)::value;
#pragma unroll
            for (int f = 0; f < FI; ++f) {
                const int64_t i = i0 + wi + f * 16 + (lane & 15);
#pragma unroll
                for (int p = 0; p < FJ / 2; ++p) {
                    const int64_t j = j0 + wj + p * 32 + g * 8;
                    u32x4 w0 = {0u, 0u, 0u, 0u}, w1 = w0;
                    if (MASK) draw(i, p, w0, w1);
                    if (i < a.ni && j + 8 <= a.nj)
                        emit_light<OP, T, decltype(act)::value, MASK>(
                            a.e, i, j, acc[f][2 * p], acc[f][2 * p + 1], l, w0, w1, g >> 1);
                }
            }
        };
        using yes = std::integral_constant<bool, OP != WGRAD>;
        if (OP != WGRAD && smooth)
            write(yes{}, std::false_type{});
        else if (masked)
            write(std::false_type{}, yes{});
        else
            write(std::false_type{}, std::false_type{});
        const bool edge = (a.nj & 7) != 0 && j0 + BJ > a.nj;
        if (!edge && !with_db) return;
    }
    // one body for all rows of blocks: the block's registers are selected by
    // uniform branches
#pragma unroll 1
    for (int f = 0; f < FI; ++f) {
        f32x4 v[FJ];
#pragma unroll
        for (int s = 0; s < FI; ++s)
            if (s == f) {
#pragma unroll
                for (int t = 0; t < FJ; ++t) v[t] = acc[s][t];
            }
        const int64_t i = i0 + wi + f * 16 + (lane & 15);
        u32x4 w0[FJ / 2], w1[FJ / 2];
        if (OP != WGRAD && a.e.drop.on && a.parts == 1) {
#pragma unroll
            for (int p = 0; p < FJ / 2; ++p) draw(i, p, w0[p], w1[p]);
        }
        if (i >= a.ni) continue;
        if (a.parts > 1) {
            float *row = a.partial + (part * a.ni + i) * njp;
#pragma unroll
            for (int t = 0; t < FJ; ++t) {
                const int64_t j = j0 + wj + (t >> 1) * 32 + g * 8 + (t & 1) * 4;
                if (j < a.nj) *reinterpret_cast<f32x4 *>(row + j) = v[t];
            }
            if (DB && with_db && f / SUMS == turn && g == 0)
                a.partial[a.parts * a.ni * njp + part * a.ni + i] = sum_of(f);
            continue;
        }
#pragma unroll
        for (int p = 0; p < FJ / 2; ++p) {
            const int64_t j = j0 + wj + p * 32 + g * 8;
            if (j < a.nj && !(light && j + 8 <= a.nj))
                emit8<OP, T>(a.e, i, j, static_cast<int>(min(a.nj - j, int64_t(8))), v[2 * p],
                             v[2 * p + 1], w0[p], w1[p], g >> 1);
        }
        if (DB && with_db && f / SUMS == turn && g == 0) emit_db<T>(a.e, i, sum_of(f));
    }
}

// Few rows of x (decoding): the weight's bytes are all that counts.  A
// workgroup has 16 columns of the output: one for every CU from 4096 columns
// on, fewer below (100 at 1600, where the time is that of one workgroup's own
// contraction).  Its eight waves take chunks of 128 of the contraction in
// turn, straight from global memory into the operand registers (a lane's
// operand is 16 contiguous bytes of a row of W), the next chunk's loads under
// way while one is multiplied.  The waves' sums are added in their order in
// shared memory: one launch, no workspace.  Rows past the last repeat it;
// their outputs are not stored.  One row: 6400 x 1600 7.4 us (2.8 TB/s), 4096 x
// 6400 12.5 (4.2 TB/s), 1600 x 6400 10.2 (2.0 TB/s).
constexpr int kSkinnyWaves = 8, kSkinnyChunk = 128;

template <class T, int R>
__global__ void __launch_bounds__(kSkinnyWaves *kWave) skinny_kernel(Args a) {
    constexpr int U = kSkinnyChunk / 32;
    __shared__ f32x4 part[kSkinnyWaves][R][kWave];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * 16;
    const uint16_t *qp = a.q + min(j0 + r, a.nj - 1) * a.ldq + g * 8;
    const uint16_t *pp[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        pp[i] = a.p + min(static_cast<int64_t>(i * 16 + r), a.ni - 1) * a.ldp + g * 8;
    f32x4 acc[R];
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Chunk {
        u32x4 q[U], p[R][U];
    };
    auto load = [&](Chunk &c, int64_t at, auto whole) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t n = decltype(whole)::value ? 8 : a.nc - (at + u * 32 + g * 8);
            c.q[u] = load_piece(qp + at + u * 32, n);
#pragma unroll
            for (int i = 0; i < R; ++i) c.p[i][u] = load_piece(pp[i] + at + u * 32, n);
        }
    };
    auto multiply = [&](const Chunk &c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < R; ++i)
                acc[i] = mfma<T>(__builtin_bit_cast(s16x8, c.q[u]),
                                 __builtin_bit_cast(s16x8, c.p[i][u]), acc[i]);
    };
    const int64_t chunks = a.nc / kSkinnyChunk;
    int64_t c = wave;
    Chunk x, y;
    if (c < chunks) load(x, c * kSkinnyChunk, std::true_type{});
    while (c < chunks) {
        c += kSkinnyWaves;
        if (c < chunks) load(y, c * kSkinnyChunk, std::true_type{});
        multiply(x);
        if (c >= chunks) break;
        c += kSkinnyWaves;
        if (c < chunks) load(x, c * kSkinnyChunk, std::true_type{});
        multiply(y);
    }
    if (chunks * kSkinnyChunk < a.nc && wave == static_cast<int>(chunks % kSkinnyWaves)) {
        load(x, chunks * kSkinnyChunk, std::false_type{});
        multiply(x);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave >= R) return;
    const int64_t i = wave * 16 + r, j = j0 + g * 4;
    if (i >= a.ni || j >= a.nj) return;
    f32x4 v = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kSkinnyWaves; ++w) v += part[w][wave][lane];
    u32x4 words = {0u, 0u, 0u, 0u};
    if (a.e.drop.on)
        words = drop_words(a.e.drop, drop_stream(a.e.drop), static_cast<uint32_t>(i),
                           static_cast<uint32_t>((j >> 5) * 4 + ((j & 15) >> 2)));
    emit<FWD, T>(a.e, i, j, static_cast<int>(a.nj - j < 4 ? a.nj - j : 4), v, words,
                 static_cast<int>(j >> 4) & 1);
}

// Adds the parts of a divided contraction in their order and finishes the
// outputs; a thread has the two quads that share a draw of the mask.
template <int OP, class T>
__global__ void __launch_bounds__(256) join_kernel(Args a) {
    const int64_t quads = (a.nj + 31) / 32 * 4;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= a.ni * quads) return;
    const int64_t i = id / quads, u = id - i * quads;
    const int64_t j = u / 4 * 32 + u % 4 * 4;
    const int64_t njp = padded4(a.nj);
    const uint64_t stream = OP != WGRAD && a.e.drop.on ? drop_stream(a.e.drop) : 0;
    if (j < a.nj) {
        const bool second = j + 16 < a.nj;
        f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
        const float *row = a.partial + i * njp + j;
        for (int s = 0; s < a.parts; ++s, row += a.ni * njp) {
            v0 += *reinterpret_cast<const f32x4 *>(row);
            if (second) v1 += *reinterpret_cast<const f32x4 *>(row + 16);
        }
        emit_pair<OP, T>(a.e, i, j, a.nj, stream, v0, v1);
    }
    if (OP == WGRAD && a.e.db != nullptr && u == 0) {
        const float *col = a.partial + a.parts * a.ni * njp + i;
        float v = 0.0f;
        for (int s = 0; s < a.parts; ++s) v += col[s * a.ni];
        emit_db<T>(a.e, i, v);
    }
}

// ---------------------------------------------------------------------------
// host

constexpr int64_t kMaxTiles = int64_t(1) << 23;  // a launch has less than 2^32 threads

int64_t partial_bytes(const Plan &p, int64_t ni, int64_t nj) {
    return p.parts == 1 ? 0 : p.parts * ni * (padded4(nj) + 1) * 4 + 16;
}

template <int OP, class T, int BI, int BJ, int WI, int WJ, bool DIRECT>
void run_grid(const Args &a, int64_t groups, hipStream_t st) {
    const dim3 grid(static_cast<uint32_t>(groups), static_cast<uint32_t>(a.parts));
    // the bias gradient's sums take registers: only where they are asked for
    if (OP == WGRAD && a.e.db != nullptr)
        tile_kernel<OP, T, BI, BJ, WI, WJ, DIRECT, OP == WGRAD><<<grid, WI * WJ * kWave, 0, st>>>(a);
    else
        tile_kernel<OP, T, BI, BJ, WI, WJ, DIRECT, false><<<grid, WI * WJ * kWave, 0, st>>>(a);
}

template <int OP, class T, int BI, int BJ, int WI, int WJ, bool DIRECT>
zero_status run_tiles(Args &a, hipStream_t st) {
    a.tiles_i = static_cast<int32_t>(ceil_div(a.ni, BI));
    a.tiles_j = static_cast<int32_t>(ceil_div(a.nj, BJ));
    a.quarter = -1;
    const int64_t tiles = static_cast<int64_t>(a.tiles_i) * a.tiles_j;
    if (tiles >= kMaxTiles) return ZERO_EINVAL;
    const int64_t rest = BI == 256 ? quartered(tiles) : 0;
    if (rest > 0) {
        run_grid<OP, T, BI, BJ, WI, WJ, DIRECT>(a, tiles - rest, st);
        a.quarter = static_cast<int32_t>(tiles - rest);
        run_grid<OP, T, 128, 128, 2, 2, DIRECT>(a, 4 * rest, st);
    } else {
        run_grid<OP, T, BI, BJ, WI, WJ, DIRECT>(a, tiles, st);
    }
    return launch_status();
}

template <int OP, class T>
zero_status launch(Args a, void *stream) {
    const Plan p = plan_for(OP, a.ni, a.nj, a.nc);
    a.chunk = p.chunk;
    a.parts = p.parts;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (OP == FWD && p.bi <= 32) {
        const uint32_t groups = static_cast<uint32_t>(ceil_div(a.nj, 16));
        if (p.bi == 16)
            skinny_kernel<T, 1><<<groups, kSkinnyWaves * kWave, 0, st>>>(a);
        else
            skinny_kernel<T, 2><<<groups, kSkinnyWaves * kWave, 0, st>>>(a);
        return launch_status();
    }
    const bool d = direct_ok(a.p, a.ldp, OP == WGRAD ? a.ni : 0) &&
                   direct_ok(a.q, a.ldq, OP == FWD ? 0 : a.nj);
    zero_status status;
    if (p.bi == 64)
        status = d ? run_tiles<OP, T, 64, 128, 1, 4, true>(a, st)
                   : run_tiles<OP, T, 64, 128, 1, 4, false>(a, st);
    else if (!d)
        status = run_tiles<OP, T, 128, 128, 2, 2, false>(a, st);
    else if (p.bi == 128)
        status = run_tiles<OP, T, 128, 128, 2, 2, true>(a, st);
    else
        status = run_tiles<OP, T, 256, 256, 2, 4, true>(a, st);
    if (status != ZERO_OK) return status;
    if (a.parts > 1) {
        const int64_t threads = a.ni * (ceil_div(a.nj, 32) * 4);
        join_kernel<OP, T><<<static_cast<uint32_t>(ceil_div(threads, 256)), 256, 0, st>>>(a);
    }
    return launch_status();
}

template <int OP>
zero_status launch(const Args &a, zero_dtype dt, void *stream) {
    return dt == ZERO_BF16 ? launch<OP, BF16>(a, stream) : launch<OP, FP16>(a, stream);
}

bool workspace_ok(int64_t need, const void *ws, int64_t bytes) {
    return need == 0 || (ws != nullptr && aligned16(ws) && bytes >= need);
}

struct Shape {
    int64_t ni, nj, nc;
};

Shape shape_of(int op, int64_t m, int64_t n, int64_t k) {
    if (op == FWD) return {m, n, k};
    if (op == DGRAD) return {m, k, n};
    return {n, k, m};
}

// linear and dgrad after their own checks: out = residual + D(f(P Q))
template <int OP>
zero_status product(const Mat &p, const Mat &q, zero_dtype dt, const Shape &s, const Mat &bias,
                    zero_act act, const Mat &z, const zero_dropout_params *drop, const Mat &res,
                    const Mat &out, void *workspace, int64_t workspace_bytes, void *stream) {
    Args a{};
    if (static_cast<int>(act) < ZERO_ACT_NONE || static_cast<int>(act) > ZERO_ACT_SILU)
        return ZERO_EINVAL;
    if (!make_drop(drop, s.ni, &a.e.drop)) return ZERO_EINVAL;
    if (!p.ok() || !q.ok() || !out.ok() || (bias.p != nullptr && !bias.ok()) ||
        (res.p != nullptr && !res.ok()) || (z.p != nullptr && !z.ok()))
        return ZERO_EINVAL;
    if (OP == DGRAD && act != ZERO_ACT_NONE && z.p == nullptr && !out.empty()) return ZERO_EINVAL;
    if (out.empty()) return ZERO_OK;
    const int64_t need = partial_bytes(plan_for(OP, s.ni, s.nj, s.nc), s.ni, s.nj);
    if (!workspace_ok(need, workspace, workspace_bytes)) return ZERO_EINVAL;
    const bool z_out = OP == FWD;
    const Span sp = p.span(), sq = q.span(), sb = bias.span(), sr = res.span(), so = out.span(),
               sz = z.span(),
               sw = need ? span_of(workspace, need, 1) : Span{0, 0},
               st = a.e.drop.step ? span_of(a.e.drop.step, 8, 1) : Span{0, 0};
    for (const Span &r : {sp, sq, sb, st}) {
        if (overlap(so, r) || overlap(sw, r)) return ZERO_EALIAS;
        if (z_out && overlap(sz, r)) return ZERO_EALIAS;
    }
    if (overlap(so, sz) || overlap(so, sw) || overlap(sz, sw) || overlap(sr, sw) ||
        (z_out && overlap(sz, sr)))
        return ZERO_EALIAS;
    if (res.p != nullptr && overlap(so, sr) && !res.same_place(out)) return ZERO_EALIAS;
    a.p = static_cast<const uint16_t *>(p.p);
    a.q = static_cast<const uint16_t *>(q.p);
    a.ldp = p.ld;
    a.ldq = q.ld;
    a.ni = s.ni;
    a.nj = s.nj;
    a.nc = s.nc;
    a.partial = static_cast<float *>(workspace);
    a.e.bias = static_cast<const uint16_t *>(bias.p);
    a.e.res = res.p;
    a.e.ldr = res.ld;
    a.e.out = const_cast<void *>(out.p);
    a.e.ldo = out.ld;
    a.e.z = static_cast<uint16_t *>(const_cast<void *>(z.p));
    a.e.ldz = z.ld;
    a.e.act = act;
    a.e.out_f32 = out.elem == 4;
    return launch<OP>(a, dt, stream);
}

}  // namespace

extern "C" {

int64_t zero_linear_workspace_bytes(zero_linear_op op, int64_t m, int64_t n, int64_t k) {
    if (static_cast<int>(op) < FWD || static_cast<int>(op) > WGRAD || !dim_ok(m) || !dim_ok(n) ||
        !dim_ok(k))
        return -1;
    const Shape s = shape_of(op, m, n, k);
    if (s.ni == 0 || s.nj == 0) return 0;
    return partial_bytes(plan_for(op, s.ni, s.nj, s.nc), s.ni, s.nj);
}

zero_status zero_linear(const void *x, zero_dtype dt, int64_t ldx, const void *w, int64_t ldw,
                        const void *bias, int64_t m, int64_t n, int64_t k, zero_act act,
                        const zero_dropout_params *drop, const void *residual, int64_t ldr,
                        void *y, zero_dtype ydt, int64_t ldy, void *z, int64_t ldz,
                        void *workspace, int64_t workspace_bytes, void *stream) {
    if (!is16(dt) || !(ydt == dt || ydt == ZERO_FP32) || !dim_ok(m) || !dim_ok(n) || !dim_ok(k))
        return ZERO_EINVAL;
    const int64_t ye = size_of(ydt);
    return product<FWD>(Mat{x, m, k, ldx, 2}, Mat{w, n, k, ldw, 2}, dt, Shape{m, n, k},
                        Mat{bias, 1, n, n, 2}, act, Mat{z, m, n, ldz, 2}, drop,
                        Mat{residual, m, n, ldr, ye}, Mat{y, m, n, ldy, ye}, workspace,
                        workspace_bytes, stream);
}

zero_status zero_linear_dgrad(const void *dy, zero_dtype dt, int64_t lddy, const void *w,
                              int64_t ldw, int64_t m, int64_t n, int64_t k, zero_act act,
                              const void *z, int64_t ldz, const zero_dropout_params *drop,
                              const void *residual, int64_t ldr, void *dx, zero_dtype dxdt,
                              int64_t lddx, void *workspace, int64_t workspace_bytes,
                              void *stream) {
    if (!is16(dt) || !(dxdt == dt || dxdt == ZERO_FP32) || !dim_ok(m) || !dim_ok(n) || !dim_ok(k))
        return ZERO_EINVAL;
    const int64_t xe = size_of(dxdt);
    return product<DGRAD>(Mat{dy, m, n, lddy, 2}, Mat{w, n, k, ldw, 2}, dt, Shape{m, k, n},
                          Mat{nullptr, 1, k, k, 2}, act,
                          Mat{act == ZERO_ACT_NONE ? nullptr : z, m, k, ldz, 2}, drop,
                          Mat{residual, m, k, ldr, xe}, Mat{dx, m, k, lddx, xe}, workspace,
                          workspace_bytes, stream);
}

zero_status zero_linear_wgrad(const void *dy, zero_dtype dt, int64_t lddy, const void *x,
                              int64_t ldx, int64_t m, int64_t n, int64_t k, void *dw,
                              zero_dtype gdt, int64_t lddw, void *db, int32_t accumulate,
                              void *workspace, int64_t workspace_bytes, void *stream) {
    if (!is16(dt) || !(gdt == dt || gdt == ZERO_FP32) || !dim_ok(m) || !dim_ok(n) || !dim_ok(k))
        return ZERO_EINVAL;
    const int64_t ge = size_of(gdt);
    const Mat my{dy, m, n, lddy, 2}, mx{x, m, k, ldx, 2}, mw{dw, n, k, lddw, ge},
        mb{db, 1, n, n, ge};
    if (!my.ok() || !mx.ok() || !mw.ok() || (db != nullptr && !mb.ok())) return ZERO_EINVAL;
    if (n == 0 || k == 0) {
        // no column of dW: a bias gradient still has its sums
        if (n == 0 || db == nullptr) return ZERO_OK;
        return ZERO_EINVAL;
    }
    const Shape s = shape_of(WGRAD, m, n, k);
    const int64_t need = partial_bytes(plan_for(WGRAD, s.ni, s.nj, s.nc), s.ni, s.nj);
    if (!workspace_ok(need, workspace, workspace_bytes)) return ZERO_EINVAL;
    const Span sy = my.span(), sx = mx.span(), sd = mw.span(), sb = mb.span(),
               sw = need ? span_of(workspace, need, 1) : Span{0, 0};
    for (const Span &r : {sy, sx})
        if (overlap(sd, r) || overlap(sb, r) || overlap(sw, r)) return ZERO_EALIAS;
    if (overlap(sd, sb) || overlap(sd, sw) || overlap(sb, sw)) return ZERO_EALIAS;
    Args a{};
    a.p = static_cast<const uint16_t *>(dy);
    a.q = static_cast<const uint16_t *>(x);
    a.ldp = lddy;
    a.ldq = ldx;
    a.ni = s.ni;
    a.nj = s.nj;
    a.nc = s.nc;
    a.partial = static_cast<float *>(workspace);
    a.e.out = dw;
    a.e.ldo = lddw;
    a.e.out_f32 = gdt == ZERO_FP32;
    a.e.db = db;
    a.e.accumulate = accumulate != 0;
    return launch<WGRAD>(a, dt, stream);
}

}  // extern "C"
