// orthogonalize.hip -- gfx950 kernels of zero_orthogonalize.
//
// Each matrix is worked on with its shorter side first, X [r][c], r <= c, laid
// out in the workspace with both sides padded by zeros to multiples of 64, so
// that every operand of every product is copied straight to shared memory.  A
// round is three products on the matrix units:
//   gram    A = X X^T                    (symmetric)
//   square  P = a + b A + c A A          (symmetric)
//   apply   X = P X
// Rounding.  fp16 keeps 11 bits where bf16 keeps 8, at the same rate; every
// value here is scaled by 2^12, which leaves room up to 16 above and down to
// 2^-26 below at full precision.  X has that room by contract; A's and P's
// off-diagonals, up to half the square of X's largest singular value and half
// the spread of b s^2 + c s^4, are scaled by less where the coefficients could
// let them need more (rounds_of).  Rounding A, P or X as a whole would cost a
// few times 2^-11 of the result where singular values are alike, and all of
// its small singular directions where they are not, since those are what the
// rounds amplify.  So the diagonals, where the large part of A and P lies, are
// kept apart in fp32 and enter as row factors in fp32:
//   A = D + O:  A A = O O + (d_i + d_j) O_ij + (d_i^2 on the diagonal)
//   P = E + Q:  P X = e_i hi_ij + f_i lo_ij + Q hi
// with X itself held to 22 bits as hi + lo, and only O, Q and hi are fp16
// operands.
//
// f, lo's factor, makes up for Q lo, which is left out: twice the apply.
// Roundings that leave an error on one side of X's large directions only tilt
// these a little.  lo is noise on both sides, 2^-12 of X in every direction,
// and what the small directions get of it is multiplied with them, by the
// coefficient a in every later round (3.4445^4 = 141 after the first).  With
// f = a the error is (b A + c A A) lo, which the small directions, where b A +
// c A A vanishes, get nothing of; with f = e_i it is Q lo, less where A is
// mostly its diagonal, but noise in all directions where X has few and few rows
// carry them.  So f is a in the rounds whose error would still be multiplied by
// more than 4, and e_i in the others (of the usual five the last two), and in
// all where there is one row.  Against 64 bits, usual rounds, bf16 to fp16, the
// largest of 3 to 100 matrices a size and spectrum (flat, decaying, orthogonal,
// one to eight directions over noise), in parentheses the largest median :
// with e_i in all rounds:
//   64 x 64 to 2048 x 2048                      1.8e-3 (1.8e-3) : 8.2e-3 (3.5e-3)
//   16 x 16 to 32 x 32                          2.8e-3 (2.6e-3) : 2.1e-2 (1.1e-2)
//   one direction in 2 to 16 of 64 rows or more 2.1e-3 (1.4e-3) : 4.4e-2 (3.0e-2)
//   the same in as few of the columns           4.7e-3 (1.8e-3) : 5.4e-2 (2.2e-2)
//   5 x 9, 8 x 8                                4.4e-3 (1.9e-3) : 3.3e-2 (1.7e-2)
//   2 x 2 to 3 x 7                              8.8e-3 (1.9e-3) : 4.5e-2 (1.7e-2)
// where bf16's own rounding of the result is 1.7e-3.  Few rows' roundings do
// not average out, and the polynomial's slope multiplies them.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "linear_common.h"
#include "linear_plan.h"
#include "linear_tiles.h"
#include "orthogonalize_plan.h"
#include "zero_muon.h"

namespace {

using namespace zero_host;
using namespace zero_linear_impl;
using namespace zero_muon_impl;

constexpr float kScale = 4096.0f, kInv = 1.0f / 4096.0f, kInv2 = kInv * kInv;
struct Input {
    const void *u;
    int64_t ldu, su;
    int32_t rows, cols;  // as the caller has it
};

// element (i, j) of the caller's matrix
template <int DT>
__device__ __forceinline__ float element(const void *p, int64_t at) {
    if constexpr (DT == ZERO_FP32) return static_cast<const float *>(p)[at];
    const uint16_t h = static_cast<const uint16_t *>(p)[at];
    return DT == ZERO_BF16 ? BF16::up(h) : FP16::up(h);
}

template <int DT>
__device__ __forceinline__ void eight(const void *p, int64_t at, int n, float (&v)[8]) {
    if (n >= 8) {
        if constexpr (DT == ZERO_FP32) {
            const float *q = static_cast<const float *>(p) + at;
            const f32x4 a = load32(q, 4), b = load32(q + 4, 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = a[e];
                v[4 + e] = b[e];
            }
        } else {
            f32x4 a, b;
            const uint16_t *q = static_cast<const uint16_t *>(p) + at;
            if (DT == ZERO_BF16)
                load16x8<BF16>(q, a, b);
            else
                load16x8<FP16>(q, a, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = a[e];
                v[4 + e] = b[e];
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? element<DT>(p, at + e) : 0.0f;
    }
}

// eight elements as they lie in memory, to have the loads of several under way
template <int DT>
struct Raw {
    u16x8 h;
    __device__ __forceinline__ void clear() { h = u16x8{}; }
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        __builtin_memcpy(&h, static_cast<const uint16_t *>(p) + at, 16);
    }
    __device__ __forceinline__ float at(int e) const {
        return DT == ZERO_BF16 ? BF16::up(h[e]) : FP16::up(h[e]);
    }
};
template <>
struct Raw<ZERO_FP32> {
    f32x4 a, b;
    __device__ __forceinline__ void clear() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        __builtin_memcpy(&a, static_cast<const float *>(p) + at, 16);
        __builtin_memcpy(&b, static_cast<const float *>(p) + at + 4, 16);
    }
    __device__ __forceinline__ float at(int e) const { return e < 4 ? a[e & 3] : b[e & 3]; }
};

// ---------------------------------------------------------------------------
// |U|^2 in up to kParts fp64 parts a matrix: pieces of eight elements, in turn

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

template <int DT>
__global__ void __launch_bounds__(1024) squares_kernel(Input in, double *parts) {
    __shared__ double wave_part[16];
    const uint32_t a_row = static_cast<uint32_t>(in.cols + 7) / 8;
    const uint32_t total = a_row * static_cast<uint32_t>(in.rows);
    const int64_t base = static_cast<int64_t>(blockIdx.y) * in.su;
    double s = 0.0;
    for (uint32_t p = blockIdx.x * 1024u + threadIdx.x; p < total; p += gridDim.x * 1024u) {
        const uint32_t i = p / a_row, j = (p - i * a_row) * 8u;
        float v[8];
        eight<DT>(in.u, base + i * in.ldu + j, in.cols - static_cast<int>(j), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double d = static_cast<double>(v[e]);
            s = __builtin_fma(d, d, s);
        }
    }
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) wave_part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) s += wave_part[w];
        parts[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
    }
}

// ---------------------------------------------------------------------------
// X = U / (|U| + eps) (or its transpose), scaled, as hi and lo; zeros in the
// padding.  A workgroup has 64 x 64 of it.

__device__ __forceinline__ void split(float v, uint16_t &hi, uint16_t &lo) {
    hi = FP16::down(v);
    lo = FP16::down(v - FP16::up(hi));
}

// Eight fp16 values in four registers, pair by pair: elements of a 16-bit
// vector set one by one take a register each on the way.
using f32x2 = float __attribute__((ext_vector_type(2)));
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x2 pair(u32x4 h, int p) {
    const uint32_t w = h[p];  // a value: the bits of a vector's element are those of its first
    return __builtin_convertvector(__builtin_bit_cast(f16x2, w), f32x2);
}
__device__ __forceinline__ u32x4 pack(const float (&v)[8]) {
    u32x4 h;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        h[p] = __builtin_bit_cast(
            uint32_t, __builtin_convertvector(f32x2{v[2 * p], v[2 * p + 1]}, f16x2));
    return h;
}
// hi and what it leaves of v, in one instruction an element: a subtraction and
// the rounding of its exact result, which needs the factor kept from sight
__device__ __forceinline__ void split8(const float (&v)[8], u32x4 &hi, u32x4 &lo) {
    hi = pack(v);
    float minus = -1.0f;
    asm("" : "+s"(minus));
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const f32x2 h = pair(hi, p);
        lo[p] = __builtin_bit_cast(
            uint32_t, f16x2{static_cast<_Float16>(__builtin_fmaf(h[0], minus, v[2 * p])),
                            static_cast<_Float16>(__builtin_fmaf(h[1], minus, v[2 * p + 1]))});
    }
}

// kScale / (sqrt(s) + eps); NaN where a matrix has an Inf or a NaN, which is
// then NaN throughout
__device__ __forceinline__ double scale_of(double s, double eps) {
    const double norm = sqrt(s) + eps;
    return norm - norm == 0.0 ? static_cast<double>(kScale) / norm : norm - norm;
}

template <int DT, bool TALL>
__global__ void __launch_bounds__(256) spread_kernel(Input in, const double *parts, int32_t n_parts,
                                                     double eps,
                                                     uint16_t *hi, uint16_t *lo, int32_t rp,
                                                     int32_t cp) {
    __shared__ double wave_part[4];
    __shared__ float block[TALL ? 64 : 1][65];
    const int t = threadIdx.x;
    const int64_t m = blockIdx.z;
    double s = wave_sum(t < n_parts ? parts[m * n_parts + t] : 0.0);
    if ((t & 63) == 0) wave_part[t >> 6] = s;
    __syncthreads();
    s = ((wave_part[0] + wave_part[1]) + wave_part[2]) + wave_part[3];
    const double inv = scale_of(s, eps);
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    const int64_t base = m * in.su;
    if (TALL) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int y = (t >> 3) + 32 * h, x = (t & 7) * 8;  // u row j0 + y, columns i0 + x..
            float v[8];
            eight<DT>(in.u, base + (j0 + y) * in.ldu + i0 + x,
                      j0 + y < in.rows ? in.cols - (i0 + x) : 0, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) block[y][x + e] = v[e];
        }
        __syncthreads();
    }
    const int r = TALL ? in.cols : in.rows, c = TALL ? in.rows : in.cols;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int y = (t >> 3) + 32 * h, x = (t & 7) * 8, i = i0 + y, j = j0 + x;
        float v[8];
        if (TALL) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = block[x + e][y];
        } else {
            eight<DT>(in.u, base + i * in.ldu + j, i < r ? c - j : 0, v);
        }
        u16x8 a, b;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t p = 0, q = 0;
            if (i < r && j + e < c)
                split(static_cast<float>(static_cast<double>(v[e]) * inv), p, q);
            a[e] = p;
            b[e] = q;
        }
        const int64_t at = (m * rp + i) * cp + j;
        *reinterpret_cast<u16x8 *>(hi + at) = a;
        *reinterpret_cast<u16x8 *>(lo + at) = b;
    }
}

// ---------------------------------------------------------------------------
// the products

struct Args {
    const uint16_t *p, *q;      // the product's operands
    const uint16_t *hi, *lo;    // square: O in hi; apply: X
    uint16_t *out, *out_lo;     // the fp16 result; apply: the new X
    const float *diag;          // square: d of A; apply: e of P
    float *new_diag;            // gram: d; square: e
    void *o;                    // finish: the caller's result
    int64_t ldo, so;
    int32_t r, c;               // of X, without padding
    int32_t rp, cp;
    int32_t tiles, tiles_i, tiles_j, count;
    int32_t parts, part_steps;  // gram
    int32_t lo_diagonal;        // apply: lo's factor is e_i, else ca
    int32_t whole;   // tiles of 256 that the launch has, or
    int32_t quarter; // >= 0: the workgroups are quarters of those from here on
    f32x4 *partial;
    float ca, cb, cc;
    Scales scale;
    int32_t tall, bf16;
};

// Which tile of which matrix a workgroup has.  Workgroups go round the 8 XCDs
// in turn; each XCD is given one contiguous run of tiles.
__device__ __forceinline__ int run_of(int b, int total) {
    const int x = b & 7, q = total >> 3, r = total & 7;
    return x * q + (x < r ? x : r) + (b >> 3);
}

// the address in scalar registers, which the direct copies need it in
template <class P>
__device__ __forceinline__ P *uniform(P *p) {
    const uint64_t v = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32));
    return reinterpret_cast<P *>(static_cast<uintptr_t>(static_cast<uint64_t>(hi) << 32 | lo));
}

// KG > 1: that many groups of waves share a workgroup and its tile, each with
// buffers of its own and every KG-th step of the contraction, for products of
// few tiles; their sums are added in their order at the end.
// A gram product of few tiles and a long contraction is divided into a.parts
// of it (blockIdx.y), whose fp32 sums lie in the workspace as the lanes hold
// them; JOIN, a second launch, adds them in their order.
template <int KIND, int BT, int WI, int WJ, int KG, int ST, bool JOIN = false>
__global__ void __launch_bounds__(WI *WJ *KG *kWave, JOIN ? 1 : 2) product_kernel(Args a) {
    constexpr bool SYM = KIND == GRAM || KIND == SQUARE, QKC = SYM;
    constexpr int THREADS = WI * WJ * kWave;
    constexpr int FI = BT / WI / 16, FJ = BT / WJ / 16;
    constexpr int SLOT = kTile<true, BT> + kTile<QKC, BT>;
    __shared__ __attribute__((aligned(1024))) uint16_t all_tiles[KG * ST * SLOT];

    const bool quarters = BT == 128 && a.quarter >= 0;
    const int id = quarters ? a.quarter + static_cast<int>(blockIdx.x >> 2)
                            : run_of(static_cast<int>(blockIdx.x), a.whole);
    const int m = __builtin_amdgcn_readfirstlane(id / a.tiles), in = id - m * a.tiles;
    int ti, tj;
    if (SYM) {
        // The lower triangle: row by row, or (256) in bands of eight rows, each
        // column by column as below, so that the tiles at work in one L2 share
        // operands: four 4096 x 4096 matrices 5390 us for 5520.  Tiles of 128
        // lose by it: 3200 x 3200 892 for 861.
        const int rows = BT == 256 || quarters ? 8 : 1;
        // row k of a triangle starts at k (k + 1) / 2
        auto row_in = [](int at) __attribute__((always_inline)) {
            int k = static_cast<int>((sqrtf(8.0f * static_cast<float>(at) + 1.0f) - 1.0f) * 0.5f);
            while ((k + 1) * (k + 2) / 2 <= at) ++k;
            while (k * (k + 1) / 2 > at) --k;
            return k;
        };
        const int y = row_in(in), first = y - y % rows, high = min(rows, a.tiles_i - first);
        const int k = in - first * (first + 1) / 2, left = k - first * high;
        if (left < 0) {
            ti = first + k % high;
            tj = k / high;
        } else {
            const int z = row_in(left);
            ti = first + z;
            tj = first + left - z * (z + 1) / 2;
        }
    } else {
        const int band = 8 * a.tiles_j, first = in / band * 8;
        const int high = min(8, a.tiles_i - first), k = in - first * a.tiles_j;
        ti = first + k % high;
        tj = k / high;
    }
    if (quarters) {
        ti = 2 * ti + (blockIdx.x >> 1 & 1);
        tj = 2 * tj + (blockIdx.x & 1);
        if (ti * BT >= a.rp || tj * BT >= (SYM ? a.rp : a.cp) || (SYM && tj > ti)) return;
    }
    ti = __builtin_amdgcn_readfirstlane(ti);
    tj = __builtin_amdgcn_readfirstlane(tj);
    const int lane = threadIdx.x & 63;
    const int any_wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int kg = any_wave / (WI * WJ), wave = any_wave % (WI * WJ);
    const int wi = wave / WJ * (BT / WI), wj = wave % WJ * (BT / WJ);
    uint16_t *tiles = all_tiles + kg * ST * SLOT;
    const int i0 = ti * BT, j0 = tj * BT;
    const int nj = SYM ? a.rp : a.cp, nc = KIND == GRAM ? a.cp : a.rp;
    const int64_t px = static_cast<int64_t>(m) * a.rp * a.cp;
    const int64_t pa = static_cast<int64_t>(m) * a.rp * a.rp;
    const int64_t pd = static_cast<int64_t>(m) * a.rp;

    f32x4 acc[FI][FJ];
#pragma unroll
    for (int f = 0; f < FI; ++f)
#pragma unroll
        for (int t = 0; t < FJ; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int g = lane >> 4;
    auto sum_at = [&](int part, int f, int t) __attribute__((always_inline)) {
        const int64_t tile = (static_cast<int64_t>(part) * a.count + m) * a.tiles + in;
        return a.partial + tile * (BT * BT / 4) + ((f * FJ + t) * WI * WJ + wave) * kWave + lane;
    };
    if constexpr (JOIN) {
        for (int part = 0; part < a.parts; ++part)
#pragma unroll
            for (int f = 0; f < FI; ++f)
#pragma unroll
                for (int t = 0; t < FJ; ++t) acc[f][t] += *sum_at(part, f, t);
    } else {
    const int c0 = KIND == GRAM ? static_cast<int>(blockIdx.y) * a.part_steps * kBK : 0;
    Direct<true, BT, THREADS, false> dp;
    Direct<QKC, BT, THREADS, true> dq;
    constexpr int NP = Direct<true, BT, THREADS, false>::N;
    constexpr int NQ = Direct<QKC, BT, THREADS, true>::N;
    dp.init(a.p + (KIND == GRAM ? px : pa), nc, i0, a.rp, c0 + kg * kBK,
            wave * kWave + lane);
    dq.init(a.q + (KIND == SQUARE ? pa : px), SYM ? nc : nj, j0, nj,
            c0 + kg * kBK, wave * kWave + lane);
    dp.base = uniform(dp.base);
    dq.base = uniform(dq.base);
    dp.stride *= KG;
    dq.stride *= KG;
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint16_t *)tiles));
    auto slot_of = [&](int s) __attribute__((always_inline)) {
        return (s & (ST - 1)) * SLOT;
    };
    auto copy = [&](int n, int s) __attribute__((always_inline)) {
        if (n < NP)
            dp.issue(n, lds + 2 * slot_of(s), wave);
        else if (n < NP + NQ)
            dq.issue(n - NP, lds + 2 * (slot_of(s) + kTile<true, BT>), wave);
    };
    auto copied = [&]() __attribute__((always_inline)) {
        dp.next();
        dq.next();
    };
    s16x8 fp[2][FI], fq[2][FJ];
    auto read = [&](int n, int s, int kk) __attribute__((always_inline)) {
        const uint16_t *tp = tiles + slot_of(s), *tq = tp + kTile<true, BT>;
        if (n < FJ)
            fq[kk][n] = fragment<QKC, BT, true>(tq, wj, n, kk, lane);
        else if (n < FJ + FI)
            fp[kk][n - FJ] = fragment<true, BT, false>(tp, wi, n - FJ, kk, lane);
    };
    // The main loop of the layer products: steps of 64 of the contraction in
    // two buffers, each in two halves of 32 whose products, reads of the other
    // half and (second half) copies of the step after next are dealt out one
    // by one; one barrier a step.
    auto half = [&](auto kk_, auto copy_, int rs, int cs) __attribute__((always_inline)) {
        constexpr int kk = decltype(kk_)::value, READS = FI + FJ, N = FI * FJ;
        constexpr int M = N * 3 / 4 > 0 ? N * 3 / 4 : 1;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            bool placed = false;
#pragma unroll
            for (int r = 0; r < READS; ++r)
                if (r * M / READS == n) {
                    read(r, rs, 1 - kk);
                    placed = true;
                }
            if (decltype(copy_)::value) {
#pragma unroll
                for (int c = 0; c < NP + NQ; ++c)
                    if (c * M / (NP + NQ) == n) {
                        copy(c, cs);
                        placed = true;
                    }
            }
            acc[n / FJ][n % FJ] =
                mfma<FP16>(fq[kk][n % FJ], fp[kk][n / FJ], acc[n / FJ][n % FJ]);
            if (placed) __builtin_amdgcn_sched_barrier(0);
        }
    };
    using first_half = std::integral_constant<int, 0>;
    using second_half = std::integral_constant<int, 1>;
    // this wave's reads are done and all but the last `flying` of its copies
    // have landed
    auto arrive = [&](auto flying) __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(flying)::value) : "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    using none = std::integral_constant<int, 0>;
    constexpr int EACH_STEP = NP + NQ;
    // this group's steps; the groups meet at every barrier, also those that
    // have none left
    const int total = KIND == GRAM ? min(a.part_steps, nc / kBK - c0 / kBK) : nc / kBK;
    const int most = (total + KG - 1) / KG;
    const int steps = KG == 1 ? total : (total - kg + KG - 1) / KG;
#pragma unroll
    for (int t = 0; t < ST; ++t)
        if (t < steps) {
#pragma unroll
            for (int n = 0; n < EACH_STEP; ++n) copy(n, t);
            copied();
        }
    if (steps >= ST)
        arrive(std::integral_constant<int, (ST - 1) * EACH_STEP>{});
    else
        arrive(none{});
#pragma unroll
    for (int n = 0; n < FI + FJ; ++n) read(n, 0, 0);
    int s = 0;
#pragma unroll 1
    for (; s < steps - ST; ++s) {
        half(first_half{}, std::false_type{}, s, 0);
        arrive(std::integral_constant<int, (ST - 2) * EACH_STEP>{});
        half(second_half{}, std::true_type{}, s + 1, s + ST);
        copied();
    }
#pragma unroll 1
    for (; s < steps; ++s) {
        half(first_half{}, std::false_type{}, s, 0);
        arrive(none{});
        half(second_half{}, std::false_type{}, s + 1, 0);
    }
    if constexpr (KG > 1) {
        if (steps < most) arrive(none{});  // one step fewer, at most
        // each group has a share of the units to finish: the others' sums of
        // these come through the buffers, which nobody reads any more
        static_assert(FI % KG == 0 && (KG - 1) * 2 * BT * BT <= KG * ST * SLOT, "the sums fit");
        f32x4 *sums = reinterpret_cast<f32x4 *>(all_tiles);
        constexpr int EACH = FI / KG * FJ * WI * WJ * kWave;  // of one group's share
        arrive(none{});
#pragma unroll
        for (int f = 0; f < FI; ++f) {
            const int to = f / (FI / KG);
            if (to == kg) continue;
            const int slot = to * (KG - 1) + (kg < to ? kg : kg - 1);
#pragma unroll
            for (int t = 0; t < FJ; ++t)
                sums[slot * EACH + ((f % (FI / KG) * FJ + t) * WI * WJ + wave) * kWave + lane] =
                    acc[f][t];
        }
        arrive(none{});
#pragma unroll
        for (int f = 0; f < FI; ++f) {
            if (f / (FI / KG) != kg) continue;
#pragma unroll
            for (int t = 0; t < FJ; ++t) {
                f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KG; ++k) {
                    const int slot = kg * (KG - 1) + (k < kg ? k : k - 1);
                    const f32x4 w =
                        k == kg ? acc[f][t]
                                : sums[slot * EACH +
                                       ((f % (FI / KG) * FJ + t) * WI * WJ + wave) * kWave + lane];
                    v = k == 0 ? w : v + w;
                }
                acc[f][t] = v;
            }
        }
    }

    if (KIND == GRAM && a.parts > 1) {
#pragma unroll
        for (int f = 0; f < FI; ++f) {
            if (KG > 1 && f / (FI / KG) != kg) continue;
#pragma unroll
            for (int t = 0; t < FJ; ++t) *sum_at(blockIdx.y, f, t) = acc[f][t];
        }
        return;
    }
    }

    // Eight neighbouring results (i, j..j+7) a lane and unit.  The loads of X
    // (or O) run a group of units ahead of the stores, since a load behind a
    // store waits for it: four 4096 x 4096 matrices 505 us; one unit after the
    // other 538, all loads before all stores 541.
    constexpr int UNITS = FI * FJ / 2, GROUP = UNITS < 4 ? UNITS : 4, GROUPS = UNITS / GROUP;
    // places in the tile, whose own place is in scalar registers
    const int in_i = wi + (lane & 15), in_j = wj + g * 8;
    const int rows = a.rp - i0, columns = nj - j0, ld = SYM ? a.rp : a.cp;
    const int64_t corner = (SYM ? pa : px) + static_cast<int64_t>(i0) * ld + j0;
    auto row_of = [&](int u) __attribute__((always_inline)) { return in_i + u / (FJ / 2) * 16; };
    auto column_of = [&](int u) __attribute__((always_inline)) {
        return in_j + u % (FJ / 2) * 32;
    };
    auto offset = [&](int i, int j) __attribute__((always_inline)) {
        return static_cast<uint32_t>(i * ld + j);
    };
    uint16_t *tile = KIND == FINISH ? nullptr : uniform(a.out + corner);
    uint16_t *tile_lo = KIND == APPLY ? uniform(a.out_lo + corner) : nullptr;
    auto store = [&](int u) __attribute__((always_inline)) {
        const int i = row_of(u), j = column_of(u), f = u / (FJ / 2), p = u % (FJ / 2);
        if (i >= rows || j >= columns) return;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[f][2 * p + e / 4][e & 3];
        if constexpr (SYM) {
            // the diagonal in fp32 (gram: d; square: e), zero in the fp16 matrix
            u16x8 h;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool diagonal = ti == tj && i == j + e;
                if (diagonal) a.new_diag[pd + i0 + i] = KIND == GRAM ? v[e] * kInv2 : v[e];
                h[e] = diagonal ? 0 : FP16::down(KIND == GRAM ? v[e] * a.scale.to_a : v[e]);
            }
            *reinterpret_cast<u16x8 *>(tile + offset(i, j)) = h;
            if (ti != tj) {
                uint16_t *o = a.out + pa + static_cast<int64_t>(j0 + j) * a.rp + i0 + i;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e * a.rp] = h[e];
            }
        } else if constexpr (KIND == APPLY) {
            u16x8 nh, nl;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint16_t x, y;
                split(v[e], x, y);
                nh[e] = x;
                nl[e] = y;
            }
            *reinterpret_cast<u16x8 *>(tile + offset(i, j)) = nh;
            *reinterpret_cast<u16x8 *>(tile_lo + offset(i, j)) = nl;
        } else if (i0 + i < a.r) {
            uint16_t *o = static_cast<uint16_t *>(a.o) + m * a.so;
            const int64_t gi = i0 + i, gj = j0 + j;
            u16x8 h;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e] = a.bf16 ? BF16::down(v[e] * kInv) : FP16::down(v[e] * kInv);
            if (!a.tall && gj + 8 <= a.c) {
                __builtin_memcpy(o + gi * a.ldo + gj, &h, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (gj + e < a.c)
                        o[a.tall ? (gj + e) * a.ldo + gi : gi * a.ldo + gj + e] = h[e];
            }
        }
    };
    auto mine = [&](int u) __attribute__((always_inline)) {
        return KG == 1 || u / (UNITS / KG) == kg;
    };
    if constexpr (KIND == GRAM) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
            if (mine(u)) store(u);
    }
    if constexpr (KIND != GRAM) {
        u16x8 xh[2][GROUP], xl[2][KIND == SQUARE ? 1 : GROUP];
        float ei[2][GROUP];
        f32x4 dj[FJ];  // square: d of this lane's columns
        if (KIND == SQUARE) {
#pragma unroll
            for (int t = 0; t < FJ; ++t) {
                const int j = min(column_of(t / 2), columns - 8) + (t & 1) * 4;
                dj[t] = *reinterpret_cast<const f32x4 *>(a.diag + pd + j0 + j);
            }
        }
        const uint16_t *hi_tile = uniform(a.hi + corner);
        const uint16_t *lo_tile = KIND == SQUARE ? nullptr : uniform(a.lo + corner);
        const float *diag_tile = uniform(a.diag + pd + i0);
        auto fetch = [&](int group) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < GROUP; ++k) {
                const int u = group * GROUP + k;
                if (!mine(u)) continue;
                const uint32_t i = min(row_of(u), rows - 1);
                const uint32_t at = offset(i, min(column_of(u), columns - 8));
                xh[group & 1][k] = *reinterpret_cast<const u16x8 *>(hi_tile + at);
                if (KIND != SQUARE)
                    xl[group & 1][k] = *reinterpret_cast<const u16x8 *>(lo_tile + at);
                ei[group & 1][k] = diag_tile[i];
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        fetch(0);
#pragma unroll
        for (int group = 0; group < GROUPS; ++group) {
            if (group + 1 < GROUPS) fetch(group + 1);
#pragma unroll
            for (int k = 0; k < GROUP; ++k) {
                const int u = group * GROUP + k, f = u / (FJ / 2), p = u % (FJ / 2);
                if (!mine(u)) continue;
                const u16x8 hi = xh[group & 1][k];
                const float ri = ei[group & 1][k], fi = a.lo_diagonal ? ri : a.ca;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = acc[f][2 * p + e / 4][e & 3];
                    if constexpr (KIND == SQUARE) {
                        const float oo = v * a.scale.from_aa,
                                    oij = FP16::up(hi[e]) * a.scale.from_a;
                        const float sq = __builtin_fmaf(ri + dj[2 * p + e / 4][e & 3], oij, oo);
                        const bool diagonal = ti == tj && row_of(u) == column_of(u) + e;
                        v = diagonal ? a.ca + a.cb * ri + a.cc * (oo + ri * ri)
                                     : __builtin_fmaf(a.cc, sq, a.cb * oij) * a.scale.to_p;
                    } else {
                        const u16x8 lo = xl[group & 1][k];
                        const float rest =
                            __builtin_fmaf(fi, FP16::up(lo[e]), v * a.scale.from_p);
                        v = __builtin_fmaf(ri, FP16::up(hi[e]), rest);
                    }
                    acc[f][2 * p + e / 4][e & 3] = v;
                }
                store(u);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// ---------------------------------------------------------------------------
// Small matrices: one workgroup does all rounds of a matrix, with X (hi), A
// and P in shared memory; only lo goes through the workspace.  The products'
// launches, seventeen for five rounds, take at least 4 us each.  A call by one
// workgroup a matrix : by launches, us: 64 x 64 14 : 60, 64 x 512 32 : 73,
// 64 x 1024 56 : 84 (its transpose 62 : 85), 128 x 128 34 : 70, 128 x 384
// 61 : 71, 128 x 448 71 : 74, 48 of 64 x 1024 58 : 125, 300 of 128 x 448
// 152 : 357, 1000 of 64 x 64 53 : 596.  A CU's vector units (hi and lo of every
// element, each round) and its reads of shared memory bound it; longer rows,
// which shared memory does not hold, are left to the products.
//
// X and A lie row by row in 16-byte pieces, piece s of row i at s ^ tw(i): tw
// differs for any eight rows in turn, and among four of them in the units of
// 32 bytes that the transposing reads take.

__device__ __forceinline__ int tw(int row) { return (row & 3) * 2 | (row >> 2 & 1); }
__device__ __forceinline__ int piece_of(int row, int ld, int s) {
    return row * ld + (s ^ tw(row)) * 8;
}

// a lane's operand, its eight consecutive c of the 32 from c0 on: of 16 rows
// from row0 on, or (Q) of block f of the rows from row0 on, in the order that
// leaves a lane eight neighbouring results of two blocks
template <bool Q>
__device__ __forceinline__ s16x8 rows_at(const uint16_t *m, int ld, int row0, int f, int c0,
                                         int lane) {
    const int t = lane & 15, g = lane >> 4;
    const int row = row0 + (Q ? (f >> 1) * 32 + (t >> 2) * 8 + (f & 1) * 4 + (t & 3) : f * 16 + t);
    return *reinterpret_cast<const s16x8 *>(m + piece_of(row, ld, c0 / 8 + g));
}
// the same of 16 columns, block f of those from column j0 on, in that order:
// the rows c0 .. c0 + 31 are the contraction
__device__ __forceinline__ s16x8 columns_at(const uint16_t *m, int ld, int j0, int f, int c0,
                                            int lane) {
    const int t = lane & 15, g = lane >> 4;
    const int s = j0 / 8 + (f >> 1) * 4 + (t & 3);
    using lds4 = __attribute__((address_space(3))) s16x4;
    s16x8 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = c0 + g * 8 + h * 4 + (t >> 2);
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4 *)(m + piece_of(row, ld, s) + (f & 1) * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h * 4 + e] = x[e];
    }
    return v;
}

constexpr int kSmallWaves = 8;

// What eight waves hold of A, [R][R], and make of it: a wave has R / WI rows
// of 32 columns, a lane eight neighbouring elements (i, j..j+7) of FI rows.
template <int R>
struct Square {
    static constexpr int WJ = R / 32, WI = kSmallWaves / WJ, FI = R / WI / 16;
    f32x4 acc[FI][2];
    u32x4 own[FI];
    int lane, wi, wj, j;
    __device__ __forceinline__ Square(int wave, int lane_)
        : lane(lane_), wi(wave / WJ * (R / WI)), wj(wave % WJ * 32), j(wj + (lane_ >> 4) * 8) {}
    __device__ __forceinline__ int row(int f) const { return wi + f * 16 + (lane & 15); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int f = 0; f < FI; ++f) acc[f][0] = acc[f][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // adds the products of m's rows over 64 of the contraction, from k on; the
    // loads of all first
    __device__ __forceinline__ void multiply(const uint16_t *m, int ld, int k) {
        s16x8 q[2][2], p[2][FI];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < 2; ++b) q[h][b] = rows_at<true>(m, ld, wj, b, k + 32 * h, lane);
#pragma unroll
            for (int f = 0; f < FI; ++f)
                p[h][f] = rows_at<false>(m, ld, wi, f, k + 32 * h, lane);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < FI; ++f)
#pragma unroll
                for (int b = 0; b < 2; ++b) acc[f][b] = mfma<FP16>(q[h][b], p[h][f], acc[f][b]);
    }
    // acc is X X^T: its diagonal to diag, the rest to A in shared memory
    __device__ __forceinline__ void put(uint16_t *A, float *diag, float to_a) {
#pragma unroll
        for (int f = 0; f < FI; ++f) {
            const int i = row(f);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = acc[f][e / 4][e & 3];
                if (i == j + e) diag[i] = v[e] * kInv2;
                v[e] = i == j + e ? 0.0f : v[e] * to_a;
            }
            own[f] = pack(v);
            *reinterpret_cast<u32x4 *>(A + piece_of(i, R, j / 8)) = own[f];
        }
    }
    // A and its diagonal become P = a + b A + c A A and its diagonal; all waves
    // see A before, and P after it
    __device__ __forceinline__ void polynomial(uint16_t *A, float *diag, float ca, float cb,
                                               float cc, const Scales scale) {
        clear();
#pragma unroll
        for (int k = 0; k < R; k += 64) multiply(A, R, k);
        float di[FI], dj[8];
#pragma unroll
        for (int f = 0; f < FI; ++f) di[f] = diag[row(f)];
#pragma unroll
        for (int e = 0; e < 8; ++e) dj[e] = diag[j + e];
        __syncthreads();  // nobody reads A and its diagonal any more
#pragma unroll
        for (int f = 0; f < FI; ++f) {
            const int i = row(f);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float oo = acc[f][e / 4][e & 3] * scale.from_aa;
                const float oij = pair(own[f], e / 2)[e & 1] * scale.from_a;
                const float sq = __builtin_fmaf(di[f] + dj[e], oij, oo);
                if (i == j + e) diag[i] = ca + cb * di[f] + cc * (oo + di[f] * di[f]);
                v[e] = i == j + e ? 0.0f : __builtin_fmaf(cc, sq, cb * oij) * scale.to_p;
            }
            *reinterpret_cast<u32x4 *>(A + piece_of(i, R, j / 8)) = pack(v);
        }
        __syncthreads();
    }
};

struct SmallArgs {
    Input in;
    uint16_t *lo;
    void *o;
    int64_t ldo, so;
    double eps;
    int32_t cp, steps, tall, bf16;
    Round rounds[ZERO_NS_MAX_STEPS];
};

// Where row i's eight lo from column j on lie.  Of 64 rows as the waves have
// them when they make X = P X, lane by lane, 16 rows of 32 columns at a time:
// row by row, 16 rows of 1024 fell on two channels of the L2 (13.8 -> 10.3
// thousand cycles a round).  Of 128 shorter rows row by row (11.3; 12.3).
template <int R>
__device__ __forceinline__ int lo_of(int i, int j, int C) {
    return R == 64 ? ((j / 32 * (R / 16) + i / 16) * kWave + j / 8 % 4 * 16 + i % 16) * 8
                   : i * C + j;
}

constexpr int kAhead = 4;  // pieces a lane has under way

template <int DT, int R>
__global__ void __launch_bounds__(kSmallWaves *kWave) small_kernel(SmallArgs a) {
    constexpr int THREADS = kSmallWaves * kWave;
    __shared__ __attribute__((aligned(128))) uint16_t X[R * kSmallColumns<R>];
    __shared__ __attribute__((aligned(128))) uint16_t A[R * R];
    __shared__ float diag[R];
    // From shared memory, not the arguments: the compiler has no scalar register
    // left for them (3 x 77 x 333 66 us for 60.5, and so with a choice of lo's
    // factor in the loops, which it makes two copies of).
    __shared__ Round rounds[ZERO_NS_MAX_STEPS];
    __shared__ double wave_part[kSmallWaves];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m = blockIdx.x, base = m * a.in.su;
    const int C = a.cp;
    const int r = a.tall ? a.in.cols : a.in.rows, c = a.tall ? a.in.rows : a.in.cols;
    uint16_t *lo = a.lo + m * R * C;
    if (tid < a.steps) rounds[tid] = a.rounds[tid];

    // |U|^2: whole pieces, kAhead of them under way, then the rows' ends
    double s = 0.0;
    {
        const int a_row = a.in.cols / 8, total = a_row * a.in.rows, rest = a.in.cols % 8;
        for (int p0 = tid; p0 < total; p0 += kAhead * THREADS) {
            Raw<DT> u[kAhead];
#pragma unroll
            for (int b = 0; b < kAhead; ++b) {
                const int p = p0 + b * THREADS, i = p / a_row;
                u[b].clear();
                if (p < total) u[b].load(a.in.u, base + i * a.in.ldu + (p - i * a_row) * 8);
            }
#pragma unroll
            for (int b = 0; b < kAhead; ++b)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double d = static_cast<double>(u[b].at(e));
                    s = __builtin_fma(d, d, s);
                }
        }
        for (int p = tid; p < rest * a.in.rows; p += THREADS) {
            const int i = p / rest;
            const double d = static_cast<double>(
                element<DT>(a.in.u, base + i * a.in.ldu + a_row * 8 + p - i * rest));
            s = __builtin_fma(d, d, s);
        }
    }
    s = wave_sum(s);
    if (lane == 0) wave_part[wave] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) s += wave_part[w];
    const double inv = scale_of(s, a.eps);
    // X
    const auto set = [&](int i, int j, float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = static_cast<float>(static_cast<double>(v[e]) * inv);
        u32x4 h, l;
        split8(v, h, l);
        *reinterpret_cast<u32x4 *>(X + piece_of(i, C, j / 8)) = h;
        *reinterpret_cast<u32x4 *>(lo + lo_of<R>(i, j, C)) = l;
    };
    const int a_row = C / 8;
    if (a.tall) {  // a column's elements; neighbouring lanes have neighbouring columns
        constexpr int B = kAhead / 2;
        for (int p0 = tid; p0 < R * a_row; p0 += B * THREADS) {
            float v[B][8];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int p = min(p0 + b * THREADS, R * a_row - 1);
                const int64_t at = base + min(p % R, r - 1);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[b][e] = element<DT>(a.in.u, at + min(p / R * 8 + e, c - 1) * a.in.ldu);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int p = p0 + b * THREADS, i = p % R, j = p / R * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[b][e] = i < r && j + e < c ? v[b][e] : 0.0f;
                if (p < R * a_row) set(i, j, v[b]);
            }
        }
    } else {
        for (int p0 = tid; p0 < R * a_row; p0 += kAhead * THREADS) {
            Raw<DT> u[kAhead];
#pragma unroll
            for (int b = 0; b < kAhead; ++b) {
                const int p = p0 + b * THREADS, i = p / a_row, j = (p - i * a_row) * 8;
                u[b].clear();
                if (i < r && j + 8 <= c) u[b].load(a.in.u, base + i * a.in.ldu + j);
            }
#pragma unroll
            for (int b = 0; b < kAhead; ++b) {
                const int p = p0 + b * THREADS, i = p / a_row, j = (p - i * a_row) * 8;
                if (i >= R || (i < r && j < c && j + 8 > c)) continue;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = u[b].at(e);
                set(i, j, v);
            }
        }
        if (c % 8 != 0 && tid < r) {  // the rows' ends
            const int j = c & ~7;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = element<DT>(a.in.u, base + tid * a.in.ldu + min(j + e, c - 1));
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = j + e < c ? v[e] : 0.0f;
            set(tid, j, v);
        }
    }
    __syncthreads();

    // X = P X: a wave has all rows of 32 columns at a time, and is the only
    // one to read and to write them.  The last time it is the result; a copy of
    // the code of its own, or its conversions are made every time.
    uint16_t *const out = static_cast<uint16_t *>(a.o) + m * a.so;
    const auto apply = [&](auto last, float share, float rest,
                           float from_p) __attribute__((always_inline)) {
#pragma unroll 1
        for (int j0 = wave * 32; j0 < C; j0 += kSmallWaves * 32) {
            const int j = j0 + g * 8;
            u32x4 l[R / 16];
#pragma unroll
            for (int f = 0; f < R / 16; ++f)
                l[f] = *reinterpret_cast<const u32x4 *>(lo + lo_of<R>(f * 16 + (lane & 15), j, C));
            __builtin_amdgcn_sched_barrier(0);
            f32x4 x[R / 16][2];
#pragma unroll
            for (int f = 0; f < R / 16; ++f) x[f][0] = x[f][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int k = 0; k < R; k += 64) {
                s16x8 q[2][2], p[2][R / 16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        q[h][b] = columns_at(X, C, j0, b, k + 32 * h, lane);
#pragma unroll
                    for (int f = 0; f < R / 16; ++f)
                        p[h][f] = rows_at<false>(A, R, 0, f, k + 32 * h, lane);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int f = 0; f < R / 16; ++f)
#pragma unroll
                        for (int b = 0; b < 2; ++b) x[f][b] = mfma<FP16>(q[h][b], p[h][f], x[f][b]);
            }
            constexpr int G = R == 64 ? 4 : 1;  // rows of hi read ahead, as registers allow
            u32x4 xh[G];
            float d[G];
#pragma unroll
            for (int f = 0; f < R / 16; ++f) {
                const int i = f * 16 + (lane & 15);
                if (f % G == 0) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int q = 0; q < G; ++q) {
                        xh[q] = *reinterpret_cast<const u32x4 *>(
                            X + piece_of(i + 16 * q, C, j / 8));
                        d[q] = diag[i + 16 * q];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                uint16_t *xp = X + piece_of(i, C, j / 8);
                const u32x4 h = xh[f % G];
                const float e_i = d[f % G], f_i = __builtin_fmaf(share, e_i, rest);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = __builtin_fmaf(pair(h, e / 2)[e & 1], e_i,
                                          __builtin_fmaf(pair(l[f], e / 2)[e & 1], f_i,
                                                         x[f][e / 4][e & 3] * from_p));
                if constexpr (!decltype(last)::value) {
                    u32x4 nh, nl;
                    split8(v, nh, nl);
                    *reinterpret_cast<u32x4 *>(xp) = nh;
                    *reinterpret_cast<u32x4 *>(lo + lo_of<R>(i, j, C)) = nl;
                } else if (i < r) {
                    u32x4 y;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float v0 = v[2 * p] * kInv, v1 = v[2 * p + 1] * kInv;
                        const uint16_t y0 = a.bf16 ? BF16::down(v0) : FP16::down(v0),
                                       y1 = a.bf16 ? BF16::down(v1) : FP16::down(v1);
                        y[p] = y0 | static_cast<uint32_t>(y1) << 16;
                    }
                    uint16_t *o = out + (a.tall ? j * a.ldo + i : i * a.ldo + j);
                    if (!a.tall && j + 8 <= c) {
                        __builtin_memcpy(o, &y, 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e, o += a.tall ? a.ldo : 1)
                            if (j + e < c) *o = static_cast<uint16_t>(y[e / 2] >> (e & 1) * 16);
                    }
                }
            }
        }
    };
    Square<R> square(wave, lane);
#pragma unroll 1
    for (int step = 0; step < a.steps; ++step) {
        square.clear();
#pragma unroll 1
        for (int k = 0; k < C; k += 64) square.multiply(X, C, k);
        // each constant is read where it is used, and in either branch: held any
        // longer, the registers it takes make the compiler of 128 rows read one
        // operand at a time (3 x 77 x 333 65 us for 60.5)
        square.put(A, diag, rounds[step].scale.to_a);
        __syncthreads();
        square.polynomial(A, diag, a.rounds[step].a, a.rounds[step].b, a.rounds[step].c,
                          rounds[step].scale);
        if (step + 1 == a.steps) {
            apply(std::true_type{}, rounds[step].lo_share, rounds[step].lo_rest,
                  rounds[step].scale.from_p);
            return;
        }
        apply(std::false_type{}, rounds[step].lo_share, rounds[step].lo_rest,
              rounds[step].scale.from_p);
        __syncthreads();
    }
}

// Up to 128 rows, too long for that: A and P by one workgroup a matrix in one
// launch, from X itself in chunks that pass through shared memory, or (JOIN)
// from the gram product's parts.  A launch less a round: 64 x 2048 82 -> 66
// us, 77 x 333 (before one workgroup did all of it) 79 -> 71.
constexpr int kChunk = 192;

template <int R, bool JOIN>
__global__ void __launch_bounds__(kSmallWaves *kWave) narrow_kernel(Args a) {
    constexpr int THREADS = kSmallWaves * kWave;
    constexpr int PIECES = kChunk / 8, N = R * PIECES / THREADS;
    __shared__ __attribute__((aligned(128))) uint16_t X[JOIN ? 8 : R * kChunk];
    __shared__ __attribute__((aligned(128))) uint16_t A[R * R];
    __shared__ float diag[R];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m = blockIdx.x;
    Square<R> square(wave, lane);
    if constexpr (JOIN) {
        // chunks of the lanes' sums as tiles of 64 hold them: two by two waves
        // of 32 x 32, two by two blocks of 16 x 16 each
        for (int at = wave; at < a.tiles * 4; at += kSmallWaves) {
            const int tile = at >> 2, w = at & 3;
            const int ti = tile == 0 ? 0 : 1, tj = tile == 2 ? 1 : 0;
            f32x4 sum[2][2];
#pragma unroll
            for (int f = 0; f < 2; ++f) sum[f][0] = sum[f][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            const f32x4 *p = a.partial + (m * a.tiles + tile) * 1024 + w * kWave + lane;
#pragma unroll 4
            for (int part = 0; part < a.parts; ++part) {
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int t = 0; t < 2; ++t) sum[f][t] += p[(f * 2 + t) * 4 * kWave];
                p += static_cast<int64_t>(a.count) * a.tiles * 1024;
            }
            const int j = tj * 64 + (w & 1) * 32 + (lane >> 4) * 8;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int i = ti * 64 + (w >> 1) * 32 + f * 16 + (lane & 15);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] = sum[f][e / 4][e & 3];
                    if (i == j + e) diag[i] = v[e] * kInv2;
                    v[e] = i == j + e ? 0.0f : v[e] * a.scale.to_a;
                }
                *reinterpret_cast<u32x4 *>(A + piece_of(i, R, j / 8)) = pack(v);
                if (ti != tj) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        A[piece_of(j + e, R, i / 8) + (i & 7)] = FP16::down(v[e]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int f = 0; f < Square<R>::FI; ++f)
            square.own[f] = *reinterpret_cast<const u32x4 *>(A + piece_of(square.row(f), R,
                                                                          square.j / 8));
    } else {
        const uint16_t *x = a.p + m * R * a.cp;
        u32x4 next[N];
        auto load = [&](int c0) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int p = n * THREADS + tid, i = p / PIECES, c = c0 + p % PIECES * 8;
                // past the row's end its first piece, which is not multiplied
                next[n] = *reinterpret_cast<const u32x4 *>(x + i * a.cp + (c < a.cp ? c : 0));
            }
        };
        load(0);
        square.clear();
#pragma unroll 1
        for (int c0 = 0; c0 < a.cp; c0 += kChunk) {
            __syncthreads();
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int p = n * THREADS + tid;
                *reinterpret_cast<u32x4 *>(X + piece_of(p / PIECES, kChunk, p % PIECES)) = next[n];
            }
            if (c0 + kChunk < a.cp) load(c0 + kChunk);
            __syncthreads();
            const int left = a.cp - c0;
#pragma unroll
            for (int k = 0; k < kChunk; k += 64)
                if (k < left) square.multiply(X, kChunk, k);
        }
        square.put(A, diag, a.scale.to_a);
        __syncthreads();
    }
    square.polynomial(A, diag, a.ca, a.cb, a.cc, a.scale);
    uint16_t *out = a.out + m * R * R;
    for (int p = tid; p < R * R / 8; p += THREADS) {
        const int i = p / (R / 8), s = p % (R / 8);
        *reinterpret_cast<u32x4 *>(out + p * 8) =
            *reinterpret_cast<const u32x4 *>(A + piece_of(i, R, s));
    }
    if (tid < R) a.new_diag[m * R + tid] = diag[tid];
}

// ---------------------------------------------------------------------------
// host

template <int KIND>
zero_status run(Args a, const Work &w, hipStream_t st) {
    const Way p = way_of(KIND, w, a.count);
    const int64_t tiles = tiles_of(KIND, w, p.side), groups = tiles * a.count;
    a.tiles = static_cast<int32_t>(tiles);
    a.tiles_i = static_cast<int32_t>(ceil_div(w.rp, p.side));
    a.tiles_j = static_cast<int32_t>(ceil_div(w.cp, p.side));
    a.parts = p.parts;
    a.part_steps = static_cast<int32_t>(p.steps);
    const int64_t rest = rest_of(KIND, w, a.count);
    a.whole = static_cast<int32_t>(groups - rest);
    a.quarter = -1;
    const uint32_t n = static_cast<uint32_t>(groups - rest);
    const dim3 grid(n, static_cast<uint32_t>(p.parts));
    if (p.side == 256) {
        product_kernel<KIND, 256, 2, 4, 1, 2><<<grid, 512, 0, st>>>(a);
        a.quarter = static_cast<int32_t>(groups - rest);
        if (rest > 64)
            product_kernel<KIND, 128, 2, 2, 1, 2>
                <<<static_cast<uint32_t>(4 * rest), 256, 0, st>>>(a);
        else if (rest > 0)
            product_kernel<KIND, 128, 2, 2, 2, 2>
                <<<static_cast<uint32_t>(4 * rest), 512, 0, st>>>(a);
    } else if (p.side == 128 && p.groups == 1) {
        product_kernel<KIND, 128, 2, 2, 1, 2><<<grid, 256, 0, st>>>(a);
    } else if (p.side == 128) {
        product_kernel<KIND, 128, 2, 2, 2, 2><<<grid, 512, 0, st>>>(a);
    } else if (p.buffers == 2) {
        product_kernel<KIND, 64, 2, 2, 1, 2><<<grid, 256, 0, st>>>(a);
    } else {
        product_kernel<KIND, 64, 2, 2, 1, 4><<<grid, 256, 0, st>>>(a);
    }
    if constexpr (KIND == GRAM) {
        // up to 128 rows the parts are added by the kernel that squares
        if (p.parts > 1 && w.rp > 128)
            product_kernel<GRAM, 64, 2, 2, 1, 2, true><<<n, 256, 0, st>>>(a);
    }
    return launch_status();
}

template <int DT>
void spread(const Input &in, const Work &w, int64_t count, double eps, char *ws, bool tall,
            hipStream_t st) {
    auto *parts = reinterpret_cast<double *>(ws + w.parts);
    auto *hi = reinterpret_cast<uint16_t *>(ws + w.hi0);
    auto *lo = reinterpret_cast<uint16_t *>(ws + w.lo);
    const uint32_t n = static_cast<uint32_t>(count);
    // a piece a thread, more in large matrices
    const int64_t pieces = in.rows * ceil_div(in.cols, 8);
    const int32_t n_parts =
        static_cast<int32_t>(std::min<int64_t>(kParts, ceil_div(pieces, 1024)));
    squares_kernel<DT><<<dim3(static_cast<uint32_t>(n_parts), n), 1024, 0, st>>>(in, parts);
    const dim3 grid(static_cast<uint32_t>(w.cp / 64), static_cast<uint32_t>(w.rp / 64), n);
    const int32_t rp = static_cast<int32_t>(w.rp), cp = static_cast<int32_t>(w.cp);
    if (tall)
        spread_kernel<DT, true><<<grid, 256, 0, st>>>(in, parts, n_parts, eps, hi, lo, rp, cp);
    else
        spread_kernel<DT, false><<<grid, 256, 0, st>>>(in, parts, n_parts, eps, hi, lo, rp, cp);
}

void run_narrow(const Args &a, bool join, hipStream_t st) {
    const uint32_t n = static_cast<uint32_t>(a.count);
    if (a.rp == 64)
        join ? narrow_kernel<64, true><<<n, kSmallWaves * kWave, 0, st>>>(a)
             : narrow_kernel<64, false><<<n, kSmallWaves * kWave, 0, st>>>(a);
    else
        join ? narrow_kernel<128, true><<<n, kSmallWaves * kWave, 0, st>>>(a)
             : narrow_kernel<128, false><<<n, kSmallWaves * kWave, 0, st>>>(a);
}

template <int DT>
void run_small(const SmallArgs &a, int64_t rp, int64_t count, hipStream_t st) {
    const uint32_t n = static_cast<uint32_t>(count);
    if (rp == 64)
        small_kernel<DT, 64><<<n, kSmallWaves * kWave, 0, st>>>(a);
    else
        small_kernel<DT, 128><<<n, kSmallWaves * kWave, 0, st>>>(a);
}

// a stack of count matrices: the span of all, and whether its strides hold
bool stack_ok(const Mat &one, int64_t count, int64_t stride, Span *all) {
    if (!one.ok()) return false;
    if (count > 1 && (stride < one.extent() || stride > (kMaxSpan - one.extent()) / (count - 1)))
        return false;
    *all = span_of(one.p, (count - 1) * (count > 1 ? stride : 0) + one.extent(), one.elem);
    return true;
}

}  // namespace

extern "C" {

int64_t zero_orthogonalize_workspace_bytes(int64_t count, int64_t rows, int64_t cols) {
    if (!sides_ok(count, rows, cols)) return -1;
    if (count == 0 || rows == 0 || cols == 0) return 0;
    return work_of(count, rows, cols).bytes;
}

zero_status zero_orthogonalize(const void *u, zero_dtype udt, int64_t ldu, int64_t su,
                               int64_t count, int64_t rows, int64_t cols,
                               const zero_ns_params *ns, void *o, zero_dtype odt, int64_t ldo,
                               int64_t so, void *workspace, int64_t workspace_bytes,
                               void *stream) {
    const zero_ns_params usual{5, 0, 1e-7, nullptr};
    const zero_ns_params &k = ns != nullptr ? *ns : usual;
    if ((!is16(udt) && udt != ZERO_FP32) || !is16(odt) || !sides_ok(count, rows, cols))
        return ZERO_EINVAL;
    if (k.steps < 1 || k.steps > ZERO_NS_MAX_STEPS || k.reserved != 0 ||
        !(std::isfinite(k.eps) && k.eps >= 0.0))
        return ZERO_EINVAL;
    for (int i = 0; k.coeffs != nullptr && i < 3 * k.steps; ++i)
        if (!std::isfinite(static_cast<float>(k.coeffs[i]))) return ZERO_EINVAL;
    if (count == 0 || rows == 0 || cols == 0) return ZERO_OK;
    Span si, sr;
    if (!stack_ok(Mat{u, rows, cols, ldu, size_of(udt)}, count, su, &si) ||
        !stack_ok(Mat{o, rows, cols, ldo, 2}, count, so, &sr))
        return ZERO_EINVAL;
    const Work w = work_of(count, rows, cols);
    // a launch has less than 2^32 threads
    for (int kind : {GRAM, SQUARE, APPLY}) {
        const Way p = way_of(kind, w, count);
        if (count * tiles_of(kind, w, p.side) * p.parts >= kMaxTiles) return ZERO_EINVAL;
    }
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < w.bytes)
        return ZERO_EINVAL;
    const Span sw = span_of(workspace, w.bytes, 1);
    if (overlap(sr, si) || overlap(sr, sw) || overlap(si, sw)) return ZERO_EALIAS;

    const hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const bool tall = rows > cols;
    const Input in{u, ldu, su, static_cast<int32_t>(rows), static_cast<int32_t>(cols)};
    if (is_small(w)) {
        SmallArgs a{in, reinterpret_cast<uint16_t *>(ws + w.lo), o, ldo, so, k.eps,
                    static_cast<int32_t>(w.cp), k.steps, tall, odt == ZERO_BF16, {}};
        rounds_of(k, w.r, a.rounds);
        if (udt == ZERO_BF16)
            run_small<ZERO_BF16>(a, w.rp, count, st);
        else if (udt == ZERO_FP16)
            run_small<ZERO_FP16>(a, w.rp, count, st);
        else
            run_small<ZERO_FP32>(a, w.rp, count, st);
        return launch_status();
    }
    if (udt == ZERO_BF16)
        spread<ZERO_BF16>(in, w, count, k.eps, ws, tall, st);
    else if (udt == ZERO_FP16)
        spread<ZERO_FP16>(in, w, count, k.eps, ws, tall, st);
    else
        spread<ZERO_FP32>(in, w, count, k.eps, ws, tall, st);

    uint16_t *hi[2] = {reinterpret_cast<uint16_t *>(ws + w.hi0),
                       reinterpret_cast<uint16_t *>(ws + w.hi1)};
    uint16_t *lo = reinterpret_cast<uint16_t *>(ws + w.lo);
    uint16_t *A = reinterpret_cast<uint16_t *>(ws + w.a);
    uint16_t *Q = reinterpret_cast<uint16_t *>(ws + w.q);
    float *d = reinterpret_cast<float *>(ws + w.d), *e = reinterpret_cast<float *>(ws + w.e);
    Args base{};
    base.r = static_cast<int32_t>(w.r);
    base.c = static_cast<int32_t>(w.c);
    base.rp = static_cast<int32_t>(w.rp);
    base.cp = static_cast<int32_t>(w.cp);
    base.count = static_cast<int32_t>(count);
    base.o = o;
    base.ldo = ldo;
    base.so = so;
    base.tall = tall;
    base.bf16 = odt == ZERO_BF16;
    base.partial = reinterpret_cast<f32x4 *>(ws + w.partial);
    const Way gram = way_of(GRAM, w, count);
    Round rounds[ZERO_NS_MAX_STEPS];
    rounds_of(k, w.r, rounds);
    zero_status status = launch_status();
    for (int i = 0; i < k.steps && status == ZERO_OK; ++i) {
        const Round &round = rounds[i];
        const uint16_t *x = hi[i & 1];
        base.ca = round.a;
        base.cb = round.b;
        base.cc = round.c;
        base.scale = round.scale;
        Args g = base;
        g.p = g.q = x;
        g.out = A;
        g.new_diag = d;
        Args s = base;
        s.p = s.q = s.hi = A;
        s.out = Q;
        s.diag = d;
        s.new_diag = e;
        const bool divided = gram.parts > 1;
        if (w.rp > 128 || divided) status = run<GRAM>(g, w, st);
        if (status != ZERO_OK) break;
        if (w.rp > 128) {
            status = run<SQUARE>(s, w, st);
        } else {
            s.p = x;
            s.tiles = static_cast<int32_t>(tiles_of(GRAM, w, 64));
            s.parts = gram.parts;
            run_narrow(s, divided, st);
            status = launch_status();
        }
        if (status != ZERO_OK) break;
        Args p = base;
        p.p = Q;
        p.q = p.hi = x;
        p.lo = lo;
        p.out = hi[(i + 1) & 1];
        p.out_lo = lo;
        p.diag = e;
        p.lo_diagonal = round.lo_share != 0.0f;
        status = i + 1 < k.steps ? run<APPLY>(p, w, st) : run<FINISH>(p, w, st);
    }
    return status;
}

}  // extern "C"
