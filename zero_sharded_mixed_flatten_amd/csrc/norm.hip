// norm.hip -- gfx950 kernels of the layer norm on the flat buffers:
// zero_layernorm, zero_layernorm_backward.
//
// Both read each row once and hold it in registers: W waves share a row, a
// lane has K pieces of eight consecutive elements, and the row's sums are
// wave sums joined through shared memory.  What bounds them is HBM.  Rows too
// long for that are read more than once (the *_loop kernels).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "linear_common.h"
#include "linear_plan.h"
#include "zero_norm.h"

namespace {

using namespace zero_host;
using namespace zero_linear_impl;

// ---------------------------------------------------------------------------
// eight consecutive elements, 16-bit or fp32, as they lie in memory

template <class T, bool F32>
struct Oct;

template <class T>
struct Oct<T, false> {
    u16x8 h;
    // n of them (zeros past the end); whole ones by one access, whatever their
    // alignment, which global memory takes
    __device__ __forceinline__ void load(const void *base, int64_t at, int64_t n) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if (n >= 8) {
            __builtin_memcpy(&h, p, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = e < n ? p[e] : 0;
        }
    }
    __device__ __forceinline__ void whole(const void *base, int64_t at) {
        __builtin_memcpy(&h, static_cast<const uint16_t *>(base) + at, 16);
    }
    __device__ __forceinline__ float at(int e) const { return T::up(h[e]); }
    static __device__ __forceinline__ void put(void *base, int64_t at, float v) {
        static_cast<uint16_t *>(base)[at] = T::down(v);
    }
    static __device__ __forceinline__ void store(void *base, int64_t at, int64_t n,
                                                 const float (&v)[8]) {
        uint16_t *p = static_cast<uint16_t *>(base) + at;
        u16x8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = T::down(v[e]);
        if (n >= 8) {
            __builtin_memcpy(p, &o, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) p[e] = o[e];
        }
    }
};

template <class T>
struct Oct<T, true> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const void *base, int64_t at, int64_t n) {
        const float *p = static_cast<const float *>(base) + at;
        if (n >= 8) {
            __builtin_memcpy(&a, p, 16);
            __builtin_memcpy(&b, p + 4, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = e < n ? p[e] : 0.0f;
                b[e] = e + 4 < n ? p[e + 4] : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void whole(const void *base, int64_t at) {
        const float *p = static_cast<const float *>(base) + at;
        __builtin_memcpy(&a, p, 16);
        __builtin_memcpy(&b, p + 4, 16);
    }
    __device__ __forceinline__ float at(int e) const { return e < 4 ? a[e & 3] : b[e & 3]; }
    static __device__ __forceinline__ void put(void *base, int64_t at, float v) {
        static_cast<float *>(base)[at] = v;
    }
    static __device__ __forceinline__ void store(void *base, int64_t at, int64_t n,
                                                 const float (&v)[8]) {
        float *p = static_cast<float *>(base) + at;
        if (n >= 8) {
            const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
            __builtin_memcpy(p, &a, 16);
            __builtin_memcpy(p + 4, &b, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) p[e] = v[e];
        }
    }
};

// a 16-bit weight's eight elements, or ones (zeros) where there is none
template <class T>
__device__ __forceinline__ Oct<T, false> affine(const uint16_t *w, int64_t at, int64_t n,
                                                float none) {
    Oct<T, false> o;
    if (w != nullptr) {
        o.load(w, at, n);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o.h[e] = T::down(none);
    }
    return o;
}

// A lane's piece of a row of n >= 8: elements first .. first + 7, of which
// the first `skip` belong to another lane's piece.  Only the last piece of a
// row whose length is no multiple of eight skips some, and pieces past the
// row's end skip all: every lane loads eight elements of the row and no load
// waits for a branch (pieces cut off by branches had taken 8192 x 6400's
// backward pass 140 us, where 8192 x 8192 took 99).
struct Piece {
    int first, skip;
};
__device__ __forceinline__ Piece piece_of(int at, int n) {
    const int first = min(at, n - 8);
    return Piece{first, min(at - first, 8)};
}
template <class O>
__device__ __forceinline__ void store_piece(void *base, int64_t row, const Piece &p,
                                            const float (&v)[8]) {
    if (p.skip == 0) {
        O::store(base, row + p.first, 8, v);
    } else {
#pragma unroll
        for (int e = 1; e < 8; ++e)
            if (e >= p.skip) O::put(base, row + p.first + e, v[e]);
    }
}

// ---------------------------------------------------------------------------
// sums

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                         0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
}

// The sum over each group of L lanes, the same in all of them: within rows of
// 16 lanes by quad permutes and rotations, two rows by a swap, the wave's row
// by row into the last lane and from there through a scalar register.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
    v += dpp<0xB1, 0xF>(v);   // the neighbour of each pair
    v += dpp<0x4E, 0xF>(v);   // the other pair of each quad
    v += dpp<0x124, 0xF>(v);  // rotated by 4
    v += dpp<0x128, 0xF>(v);  // rotated by 8
    if (L == 32) v += __shfl_xor(v, 16);
    if (L == 64) {
        v += dpp<0x142, 0xA>(v);  // rows 0 and 2 into rows 1 and 3
        v += dpp<0x143, 0xC>(v);  // row 1 into rows 2 and 3
        v = __builtin_bit_cast(float,
                               __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    }
    return v;
}
__device__ __forceinline__ float wave_sum(float v) { return lane_sum<64>(v); }

// sums of two values over the waves first .. first + count - 1 of the
// workgroup, through part (two floats a wave); all waves of it call this
__device__ __forceinline__ void join_waves(float &a, float &b, float (*part)[2], int wave,
                                           int first, int count) {
    part[wave][0] = a;  // every lane the same value
    part[wave][1] = b;
    __syncthreads();
    a = part[first][0];
    b = part[first][1];
    for (int w = 1; w < count; ++w) {
        a += part[first + w][0];
        b += part[first + w][1];
    }
}

// ---------------------------------------------------------------------------
// forward

struct NormArgs {
    const void *x;
    const uint16_t *w, *b;
    void *y;
    float *mean, *rstd;
    int64_t ldx, ldy, m, n;
    float eps;
    int32_t waves_a_row;
};

constexpr int kLimit = 16384;  // elements of a row held in registers, at most
inline bool in_registers(int64_t n) { return n >= 8 && n <= kLimit; }

// mean and 1 / sqrt(var + eps) of a row of n from the sums s1, s2 of its
// differences d from mean0 and of their squares.  mean0 is the row's mean up
// to the rounding of its sum; what it lacks, s1 / n, is known from the
// differences to their own precision, however far the mean is from 0.
__device__ __forceinline__ float finish_row(float s1, float s2, float n, float eps, float &rest) {
    rest = s1 / n;
    const float var = fmaxf(s2 / n - rest * rest, 0.0f);
    // fmaxf drops a NaN: s2 is one where the row holds an Inf or a NaN, and Inf
    // less Inf is one where only the squares pass fp32's range
    if (s2 != s2) return s2;
    return s2 == __builtin_inff() ? 0.0f : 1.0f / sqrtf(var + eps);
}

// W waves of a workgroup share a row, or (W = 1, K = 1) a wave has 64 / L
// rows.  Workgroups stay and take rows in turn: the weight and the bias are
// read once, and the next row's loads are under way while the current one is
// summed.
template <class T, bool XF, bool YF, int K, int L, bool MULTI>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a) {
    __shared__ float part[2][MULTI ? 8 : 1][2];
    const int lane = threadIdx.x & (L - 1);
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int W = a.waves_a_row, R = MULTI ? (static_cast<int>(blockDim.x) >> 6) / W : 0;
    const int rg = MULTI ? wave / W : 0, wl = MULTI ? wave - rg * W : 0;
    const int at_once = MULTI ? R : static_cast<int>(blockDim.x) / L;
    const int mine = MULTI ? rg : static_cast<int>(threadIdx.x) / L;
    const int64_t step = static_cast<int64_t>(gridDim.x) * at_once;
    const float n = static_cast<float>(a.n);
    Piece p[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        p[k] = piece_of(((k * W + wl) * L + lane) * 8, static_cast<int>(a.n));
    Oct<T, XF> x[K], next[K];
    Oct<T, false> w[K], b[K];
    auto load = [&](Oct<T, XF> (&q)[K], int64_t row) __attribute__((always_inline)) {
        row = min(row, a.m - 1);
#pragma unroll
        for (int k = 0; k < K; ++k) q[k].whole(a.x, row * a.ldx + p[k].first);
    };
    const int64_t first = static_cast<int64_t>(blockIdx.x) * at_once;
    load(next, first + mine);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        w[k] = affine<T>(a.w, p[k].first, 8, 1.0f);
        b[k] = affine<T>(a.b, p[k].first, 8, 0.0f);
    }
    for (int64_t base = first; base < a.m; base += step) {
        const int64_t row = base + mine;
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = next[k];
        load(next, row + step);
        float s = 0.0f, zero = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += e < p[k].skip ? 0.0f : x[k].at(e);
        s = lane_sum<L>(s);
        if (MULTI) join_waves(s, zero, part[0], wave, rg * W, W);
        const float mean0 = s / n;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < p[k].skip ? 0.0f : x[k].at(e) - mean0;
                s1 += d;
                s2 = __builtin_fmaf(d, d, s2);
            }
        s1 = lane_sum<L>(s1);
        s2 = lane_sum<L>(s2);
        if (MULTI) join_waves(s1, s2, part[1], wave, rg * W, W);
        float rest;
        const float rstd = finish_row(s1, s2, n, a.eps, rest);
        if (row >= a.m) continue;
        if (lane == 0 && wl == 0) {
            if (a.mean != nullptr) a.mean[row] = rest == rest ? mean0 + rest : mean0;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf((x[k].at(e) - mean0 - rest) * rstd, w[k].at(e), b[k].at(e));
            store_piece<Oct<T, YF>>(a.y, row * a.ldy, p[k], v);
        }
    }
}

// rows of more than kLimit elements or fewer than eight: a workgroup reads the
// row three times
template <class T, bool XF, bool YF>
__global__ void __launch_bounds__(1024) norm_loop_kernel(NormArgs a) {
    __shared__ float part[2][16][2];
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const float n = static_cast<float>(a.n);
    const int64_t c0 = static_cast<int64_t>(threadIdx.x) * 8;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        float s = 0.0f, zero = 0.0f;
        for (int64_t c = c0; c < a.n; c += 8192) {
            Oct<T, XF> x;
            x.load(a.x, row * a.ldx + c, a.n - c);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t += x.at(e);
            s += t;
        }
        s = wave_sum(s);
        join_waves(s, zero, part[0], wave, 0, 16);
        const float mean0 = s / n;
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = c0; c < a.n; c += 8192) {
            Oct<T, XF> x;
            x.load(a.x, row * a.ldx + c, a.n - c);
            float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = c + e < a.n ? x.at(e) - mean0 : 0.0f;
                t1 += d;
                t2 = __builtin_fmaf(d, d, t2);
            }
            s1 += t1;
            s2 += t2;
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        join_waves(s1, s2, part[1], wave, 0, 16);
        float rest;
        const float rstd = finish_row(s1, s2, n, a.eps, rest);
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = rest == rest ? mean0 + rest : mean0;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
        for (int64_t c = c0; c < a.n; c += 8192) {
            Oct<T, XF> x;
            x.load(a.x, row * a.ldx + c, a.n - c);
            const Oct<T, false> w = affine<T>(a.w, c, a.n - c, 1.0f),
                                b = affine<T>(a.b, c, a.n - c, 0.0f);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf((x.at(e) - mean0 - rest) * rstd, w.at(e), b.at(e));
            Oct<T, YF>::store(a.y, row * a.ldy + c, a.n - c, v);
        }
    }
}

// ---------------------------------------------------------------------------
// backward

struct BackArgs {
    const void *dy, *x, *res;
    const uint16_t *w;
    const float *mean, *rstd;
    void *dx, *dw, *db;
    float *partial;  // [groups][16][pieces]: of a piece's columns dw (8), then db (8)
    int64_t lddy, ldx, ldr, lddx, m, n, pieces;
    int32_t waves_a_row, groups, grads_f32, accumulate;
};

constexpr int kBackWaves = 8;
constexpr int kRowWaves = 16;  // of a row, one piece a lane
constexpr int kGroups = 512;   // workgroups that keep column sums
constexpr int kFewRows = 512;  // whose column sums are other workgroups'

// where a piece's eight columns start
__device__ __forceinline__ int64_t first_of(int64_t at, int64_t n) {
    return n >= 8 ? min(at, n - 8) : 0;
}

// a column's sum over all rows, t, to its place: value e (dw 0..7, db 8..15)
// of a piece
template <class T>
__device__ __forceinline__ void put_column(const BackArgs &a, int e, int64_t piece, float t) {
    const int64_t at = piece * 8, c = first_of(at, a.n) + (e & 7);
    void *out = e < 8 ? a.dw : a.db;
    if (out == nullptr || c < at || c >= a.n) return;
    if (a.grads_f32) {
        float *p = static_cast<float *>(out) + c;
        *p = a.accumulate ? *p + t : t;
    } else {
        uint16_t *p = static_cast<uint16_t *>(out) + c;
        *p = T::down(a.accumulate ? T::up(*p) + t : t);
    }
}

// The column sums of few rows, by workgroups behind those of dx: dw and db
// need mean and rstd only, not the rows' sums.  A workgroup has the columns of
// 16 pieces, 16 lanes of it take every so manyth row.
constexpr int kFewPieces = 16;

template <class T, bool XF, bool DF, int WAVES>
__device__ __forceinline__ void few_columns(const BackArgs &a, int64_t block) {
    __shared__ float sums[WAVES * kWave / kFewPieces][16][kFewPieces];
    const int at_once = static_cast<int>(blockDim.x) / kFewPieces;
    const int l = threadIdx.x % kFewPieces, mine = threadIdx.x / kFewPieces;
    const int64_t c = first_of(min(block * kFewPieces + l, a.pieces - 1) * 8, a.n);
    float dw[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
#pragma unroll 4
    for (int64_t row = mine; row < a.m; row += at_once) {
        Oct<T, XF> x;
        Oct<T, DF> dy;
        x.whole(a.x, row * a.ldx + c);
        dy.whole(a.dy, row * a.lddy + c);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[e] = __builtin_fmaf(dy.at(e), (x.at(e) - mean) * rstd, dw[e]);
            db[e] += dy.at(e);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sums[mine][e][l] = dw[e];
        sums[mine][8 + e][l] = db[e];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * kFewPieces; o += static_cast<int>(blockDim.x)) {
        const int e = o / kFewPieces, v = o % kFewPieces;
        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r = 0; r < at_once; r += 4)
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] += sums[r + k][e][v];
        const int64_t piece = block * kFewPieces + v;
        if (piece < a.pieces) put_column<T>(a, e, piece, (t[0] + t[1]) + (t[2] + t[3]));
    }
}

// A workgroup takes rows in turn, R at a time: as many as eight waves hold, or
// one of more waves.
// A lane has the same columns of all of them, so the sums of dw and db stay
// in its registers until the end, where they are joined over the rows in
// shared memory and stored once a workgroup.  The next rows are loaded before
// the current ones' sums are joined (PF, where the registers hold both).  Of
// few rows (FEW) the sums are other workgroups' of the launch.
enum Grads { NONE, SUMS, FEW };

template <class T, bool XF, bool DF, int K, Grads HOW, bool PF>
__global__ void __launch_bounds__((K == 1 ? kRowWaves : kBackWaves) * kWave)
back_kernel(BackArgs a) {
    constexpr bool GRADS = HOW == SUMS;
    if constexpr (HOW == FEW) {
        if (blockIdx.x >= static_cast<uint32_t>(a.groups))
            return few_columns<T, XF, DF, K == 1 ? kRowWaves : kBackWaves>(a, blockIdx.x - a.groups);
    }
    __shared__ float part[2][K == 1 ? kRowWaves : kBackWaves][2];
    __shared__ float cols[GRADS ? kBackWaves : 1][16][kWave];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int W = a.waves_a_row, R = (static_cast<int>(blockDim.x) >> 6) / W;
    const int rg = wave / W, wl = wave - rg * W;
    const float n = static_cast<float>(a.n);
    const int64_t step = static_cast<int64_t>(a.groups) * R;
    struct Row {
        Oct<T, XF> x[K], r[K];
        Oct<T, DF> dy[K];
        float mean, rstd;
    };
    Piece p[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        p[k] = piece_of(((k * W + wl) * 64 + lane) * 8, static_cast<int>(a.n));
    auto load = [&](Row &q, int64_t row) __attribute__((always_inline)) {
        row = min(row, a.m - 1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            q.dy[k].whole(a.dy, row * a.lddy + p[k].first);
            q.x[k].whole(a.x, row * a.ldx + p[k].first);
            if (PF && a.res != nullptr) q.r[k].whole(a.res, row * a.ldr + p[k].first);
        }
        q.mean = a.mean[row];
        q.rstd = a.rstd[row];
    };
    Oct<T, false> w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = affine<T>(a.w, p[k].first, 8, 1.0f);
    float dw[K][8], db[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[k][e] = db[k][e] = 0.0f;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * R;
    Row q, next;
    if (PF) load(next, first + rg);
    int turn = 0;
    for (int64_t base = first; base < a.m; base += step, turn ^= 1) {
        const int64_t row = base + rg;
        if (PF) {
            q = next;
            load(next, row + step);
        } else {
            load(q, row);
        }
        float s1 = 0.0f, s2 = 0.0f;
        if (row < a.m) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float dy = e < p[k].skip ? 0.0f : q.dy[k].at(e);
                    // selected, not multiplied away: x may be anything there
                    const float h = e < p[k].skip ? 0.0f : (q.x[k].at(e) - q.mean) * q.rstd;
                    const float g = e < p[k].skip ? 0.0f : dy * w[k].at(e);
                    s1 += g;
                    s2 = __builtin_fmaf(g, h, s2);
                    if (GRADS) {
                        dw[k][e] = __builtin_fmaf(dy, h, dw[k][e]);
                        db[k][e] += dy;
                    }
                }
        }
        if (!PF && a.res != nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                q.r[k].whole(a.res, min(row, a.m - 1) * a.ldr + p[k].first);
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if (W > 1) join_waves(s1, s2, part[turn], wave, rg * W, W);
        const float c1 = s1 / n, c2 = s2 / n;
        if (row >= a.m) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = (q.x[k].at(e) - q.mean) * q.rstd;
                const float g = q.dy[k].at(e) * w[k].at(e);
                v[e] = q.rstd * __builtin_fmaf(-h, c2, g - c1);
            }
            if (a.res != nullptr) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += q.r[k].at(e);
            }
            store_piece<Oct<T, XF>>(a.dx, row * a.lddx, p[k], v);
        }
    }
    if constexpr (GRADS) {
        float *sums = a.partial + static_cast<int64_t>(blockIdx.x) * 16 * a.pieces;
        if (R == 1) {  // each column is one lane's
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int piece = (k * W + wl) * 64 + lane;
                if (piece >= a.pieces) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sums[e * a.pieces + piece] = dw[k][e];
                    sums[(8 + e) * a.pieces + piece] = db[k][e];
                }
            }
            return;
        }
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
            __syncthreads();
#pragma unroll
            for (int s = 0; s < K; ++s)
                if (s == k) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        cols[wave][e][lane] = dw[s][e];
                        cols[wave][8 + e][lane] = db[s][e];
                    }
                }
            __syncthreads();
            for (int o = threadIdx.x; o < W * 1024; o += static_cast<int>(blockDim.x)) {
                const int l = o & 63, e = o >> 6 & 15, v = o >> 10;
                float t = cols[v][e][l];
                for (int r = 1; r < R; ++r) t += cols[r * W + v][e][l];
                const int piece = (k * W + v) * 64 + l;
                if (piece < a.pieces) sums[e * a.pieces + piece] = t;
            }
        }
    }
}

// such rows: a workgroup reads the row twice
template <class T, bool XF, bool DF>
__global__ void __launch_bounds__(1024) back_loop_kernel(BackArgs a) {
    __shared__ float part[2][16][2];
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const float n = static_cast<float>(a.n);
    const int64_t c0 = static_cast<int64_t>(threadIdx.x) * 8;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x, turn ^= 1) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = c0; c < a.n; c += 8192) {
            Oct<T, XF> x;
            Oct<T, DF> dy;
            x.load(a.x, row * a.ldx + c, a.n - c);
            dy.load(a.dy, row * a.lddy + c, a.n - c);
            const Oct<T, false> w = affine<T>(a.w, c, a.n - c, 1.0f);
            float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = dy.at(e) * w.at(e);
                const float h = c + e < a.n ? (x.at(e) - mean) * rstd : 0.0f;
                t1 += g;
                t2 = __builtin_fmaf(g, h, t2);
            }
            s1 += t1;
            s2 += t2;
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        join_waves(s1, s2, part[turn], wave, 0, 16);
        const float c1 = s1 / n, c2 = s2 / n;
        for (int64_t c = c0; c < a.n; c += 8192) {
            Oct<T, XF> x, r;
            Oct<T, DF> dy;
            x.load(a.x, row * a.ldx + c, a.n - c);
            dy.load(a.dy, row * a.lddy + c, a.n - c);
            const Oct<T, false> w = affine<T>(a.w, c, a.n - c, 1.0f);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = (x.at(e) - mean) * rstd;
                v[e] = rstd * __builtin_fmaf(-h, c2, dy.at(e) * w.at(e) - c1);
            }
            if (a.res != nullptr) {
                r.load(a.res, row * a.ldr + c, a.n - c);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += r.at(e);
            }
            Oct<T, XF>::store(a.dx, row * a.lddx + c, a.n - c, v);
        }
    }
}

// the column sums of such rows, before dx may be written over dy: a lane has
// a piece, the eight waves of a workgroup and the workgroups along y take
// rows in turn
template <class T, bool XF, bool DF>
__global__ void __launch_bounds__(kBackWaves *kWave) back_columns_kernel(BackArgs a) {
    __shared__ float cols[kBackWaves][16][kWave];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 64 + lane) * 8;
    const int64_t c = first_of(at, a.n);
    float dw[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * kBackWaves + wave; row < a.m;
         row += static_cast<int64_t>(a.groups) * kBackWaves) {
        Oct<T, XF> x;
        Oct<T, DF> dy;
        x.load(a.x, row * a.ldx + c, a.n - c);
        dy.load(a.dy, row * a.lddy + c, a.n - c);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[e] = __builtin_fmaf(dy.at(e), (x.at(e) - mean) * rstd, dw[e]);
            db[e] += dy.at(e);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cols[wave][e][lane] = dw[e];
        cols[wave][8 + e][lane] = db[e];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < 1024; o += kBackWaves * kWave) {
        const int l = o & 63, e = o >> 6;
        float t = cols[0][e][l];
        for (int r = 1; r < kBackWaves; ++r) t += cols[r][e][l];
        const int64_t p = static_cast<int64_t>(blockIdx.x) * 64 + l;
        if (p < a.pieces)
            a.partial[(static_cast<int64_t>(blockIdx.y) * 16 + e) * a.pieces + p] = t;
    }
}

// Adds the workgroups' column sums in their order and writes dw and db: a
// workgroup has 64 columns, 16 waves a sixteenth of the sums each.
template <class T>
__global__ void __launch_bounds__(1024) columns_kernel(BackArgs a) {
    __shared__ float cols[16][kWave];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int64_t total = 16 * a.pieces;
    const int each = (a.groups + 15) / 16;
    for (int64_t o0 = static_cast<int64_t>(blockIdx.x) * 64; o0 < total;
         o0 += static_cast<int64_t>(gridDim.x) * 64) {
        const int64_t o = o0 + lane;
        float t = 0.0f;
        if (o < total) {
            const int g1 = min(a.groups, (wave + 1) * each);
#pragma unroll 16
            for (int g = wave * each; g < g1; ++g) t += a.partial[g * total + o];
        }
        cols[wave][lane] = t;
        __syncthreads();
        if (wave == 0 && o < total) {
            for (int v = 1; v < 16; ++v) t += cols[v][lane];
            const int64_t e = o / a.pieces;
            put_column<T>(a, static_cast<int>(e), o - e * a.pieces, t);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// host

constexpr int64_t kMaxGroups = int64_t(1) << 21;  // a launch has less than 2^32 threads

template <class T, bool XF, bool YF, int K>
void run_norm(const NormArgs &a, hipStream_t st) {
    // As many workgroups as stay on the card at once, for their registers;
    // from fp32 to fp32, twice the bytes under way, fewer waves in larger
    // workgroups with two pieces a lane keep HBM busiest (16384 x 4096
    // 102 -> 95 us; to 16-bit 74 -> 72, but rows of 3500 67 -> 76).
    constexpr bool kBulk = XF && YF && K > 1;
    const int W = a.waves_a_row, R = std::max(1, (kBulk ? 8 : 4) / W);
    const int a_cu = std::max(1, (kBulk || K == 4 ? 12 : 16) / (W * R));
    const uint32_t g =
        static_cast<uint32_t>(std::min<int64_t>(ceil_div(a.m, R), kCUs * a_cu));
    if (W > 1)
        norm_kernel<T, XF, YF, K, 64, true><<<g, W * R * kWave, 0, st>>>(a);
    else
        norm_kernel<T, XF, YF, K, 64, false><<<g, R * kWave, 0, st>>>(a);
}

template <class T, bool XF, bool YF>
zero_status launch_norm(NormArgs a, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (!in_registers(a.n)) {
        norm_loop_kernel<T, XF, YF>
            <<<static_cast<uint32_t>(std::min(a.m, kMaxGroups)), 1024, 0, st>>>(a);
        return launch_status();
    }
    a.waves_a_row = 1;
    if (a.n <= 128) {
        norm_kernel<T, XF, YF, 1, 16, false>
            <<<static_cast<uint32_t>(std::min<int64_t>(ceil_div(a.m, 16), kCUs * 8)), 256, 0, st>>>(a);
        return launch_status();
    }
    if (a.n <= 256) {
        norm_kernel<T, XF, YF, 1, 32, false>
            <<<static_cast<uint32_t>(std::min<int64_t>(ceil_div(a.m, 8), kCUs * 8)), 256, 0, st>>>(a);
        return launch_status();
    }
    const int64_t waves = ceil_div(a.n, 512);  // of one piece a lane
    // Few rows are spread over waves.  Otherwise four pieces a lane (fp32 to
    // fp32 two), three beyond 8192 elements, where eight waves are enough for
    // those.
    const int pieces = a.m <= 512 ? 1 : waves > 16 ? 3 : XF && YF ? 2 : 4;
    a.waves_a_row = static_cast<int32_t>(std::min<int64_t>(8, ceil_div(waves, pieces)));
    switch (ceil_div(waves, a.waves_a_row)) {
        case 1: run_norm<T, XF, YF, 1>(a, st); break;
        case 2: run_norm<T, XF, YF, 2>(a, st); break;
        case 3: run_norm<T, XF, YF, 3>(a, st); break;
        default: run_norm<T, XF, YF, 4>(a, st); break;
    }
    return launch_status();
}

template <class T>
zero_status launch_norm(const NormArgs &a, bool xf, bool yf, void *stream) {
    if (xf) return yf ? launch_norm<T, true, true>(a, stream) : launch_norm<T, true, false>(a, stream);
    return yf ? launch_norm<T, false, true>(a, stream) : launch_norm<T, false, false>(a, stream);
}

template <class T, bool XF, bool DF, int K>
void run_back(const BackArgs &a, int threads, Grads how, hipStream_t st) {
    constexpr bool PF = K <= (XF || DF ? 1 : 3);  // what the registers hold
    if (how == SUMS) {
        back_kernel<T, XF, DF, K, SUMS, PF><<<a.groups, threads, 0, st>>>(a);
    } else if (how == FEW) {
        const uint32_t g = a.groups + static_cast<uint32_t>(ceil_div(a.pieces, kFewPieces));
        back_kernel<T, XF, DF, K, FEW, false><<<g, threads, 0, st>>>(a);
    } else {
        back_kernel<T, XF, DF, K, NONE, false><<<a.groups, threads, 0, st>>>(a);
    }
}

template <class T, bool XF, bool DF>
zero_status launch_back(BackArgs a, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool grads = a.dw != nullptr || a.db != nullptr;
    const int64_t waves = ceil_div(a.n, 512);
    Grads how = grads ? SUMS : NONE;
    if (a.m > 0 && in_registers(a.n)) {
        // One piece a lane up to 8192 elements, three or four beyond; two of
        // 16-bit rows that take eight waves, where there are many (16384 rows
        // of 3592 103 us for 121, of 3840 101 for 121, of 4096 106 for 120;
        // 8192 of them 59 for 66, 58 for 66, 61 for 65, 4096 of 4096 37 for
        // 36).  One workgroup on a CU keeps the column sums that go through
        // memory few (16384 x 1600 fp32 82 us for two's 88, 4096 x 4500 42 for
        // 47).  Two pay where x is 16-bit, each has rows enough, and one is
        // short of eight waves (16384 x 2304 107 -> 70, with dy fp32 111 ->
        // 81; 2048 x 3008 fp32 22 -> 24) or, with dy 16-bit too, has shorter
        // rows (16384 x 1600 58 -> 51; with dy fp32 59 -> 60).
        const bool twos = !XF && !DF && waves == kBackWaves && a.m >= 8192;
        const int most = waves <= kRowWaves ? kRowWaves : kBackWaves;
        const int W = static_cast<int>(twos ? kBackWaves / 2 : std::min<int64_t>(most, waves));
        const int R = std::max(1, kBackWaves / W);
        a.waves_a_row = W;
        const int64_t turns = ceil_div(a.m, R);
        const bool two = !XF && !twos && turns >= 4 * kGroups &&
                         (W * R < kBackWaves || (!DF && W < kBackWaves));
        a.groups =
            static_cast<int32_t>(std::min<int64_t>(two ? kGroups : kGroups / 2, turns));
        const int threads = W * R * kWave;
        // One launch for two, which read x and dy twice: a row of 1600 7.3 ->
        // 3.0 us, 256 rows 10.7 -> 4.7, 512 10.7 -> 10.1, 1023 11.7 -> 17.8;
        // 256 of 11008 18.9 -> 9.6, 512 of 600 9.7 -> 6.5 (replayed from a
        // graph).  Of 13 widths from 64 to 16384 all gain at 256 rows, 11 to
        // 58 %; at 512 up to 35 %, but 2304 loses (11.5 -> 14.6) and, with x
        // and dy fp32, 2304 and 6401 do (12.5 -> 15.6, 19.9 -> 22.4); at 768
        // as many lose as gain.  Not in place: nobody may write dy before the
        // columns' workgroups have read it.
        if (grads && a.m <= kFewRows && a.dx != a.dy) how = FEW;
        switch (ceil_div(waves, W)) {
            case 1: run_back<T, XF, DF, 1>(a, threads, how, st); break;
            case 2:
                if constexpr (!XF && !DF) run_back<T, XF, DF, 2>(a, threads, how, st);
                break;
            case 3: run_back<T, XF, DF, 3>(a, threads, how, st); break;
            default: run_back<T, XF, DF, 4>(a, threads, how, st); break;
        }
    } else if (a.m > 0) {
        a.groups = static_cast<int32_t>(std::min<int64_t>(16, ceil_div(a.m, kBackWaves)));
        if (grads)
            back_columns_kernel<T, XF, DF>
                <<<dim3(static_cast<uint32_t>(ceil_div(a.pieces, 64)),
                        static_cast<uint32_t>(a.groups)),
                   kBackWaves * kWave, 0, st>>>(a);
        back_loop_kernel<T, XF, DF>
            <<<static_cast<uint32_t>(std::min(a.m, kMaxGroups)), 1024, 0, st>>>(a);
    } else {
        a.groups = 0;
    }
    if (how == SUMS)
        columns_kernel<T>
            <<<static_cast<uint32_t>(std::min(ceil_div(16 * a.pieces, 64), kMaxGroups)), 1024, 0,
               st>>>(a);
    return launch_status();
}

template <class T>
zero_status launch_back(const BackArgs &a, bool xf, bool df, void *stream) {
    if (xf) return df ? launch_back<T, true, true>(a, stream) : launch_back<T, true, false>(a, stream);
    return df ? launch_back<T, false, true>(a, stream) : launch_back<T, false, false>(a, stream);
}

bool type_ok(zero_dtype t, zero_dtype wdt) { return t == wdt || t == ZERO_FP32; }

int64_t partial_bytes(int64_t m, int64_t n) {
    const int64_t groups = in_registers(n) ? std::min<int64_t>(kGroups, m)
                                           : std::min<int64_t>(16, ceil_div(m, kBackWaves));
    return groups * ceil_div(n, 8) * 64;
}

}  // namespace

extern "C" {

zero_status zero_layernorm(const void *x, zero_dtype xdt, int64_t ldx, const void *w,
                           const void *b, zero_dtype wdt, int64_t m, int64_t n, double eps,
                           void *y, zero_dtype ydt, int64_t ldy, float *mean, float *rstd,
                           void *stream) {
    if (!is16(wdt) || !type_ok(xdt, wdt) || !type_ok(ydt, wdt) || !dim_ok(m) || !dim_ok(n))
        return ZERO_EINVAL;
    const float eps32 = static_cast<float>(eps);
    if (!(std::isfinite(eps32) && eps32 > 0.0f)) return ZERO_EINVAL;
    const Mat mx{x, m, n, ldx, size_of(xdt)}, my{y, m, n, ldy, size_of(ydt)}, mw{w, 1, n, n, 2},
        mb{b, 1, n, n, 2}, ms{mean, 1, m, m, 4}, mr{rstd, 1, m, m, 4};
    if (!mx.ok() || !my.ok()) return ZERO_EINVAL;
    for (const Mat *v : {&mw, &mb, &ms, &mr})
        if (v->p != nullptr && !v->ok()) return ZERO_EINVAL;
    if (n == 0 && m > 0 && (mean != nullptr || rstd != nullptr)) return ZERO_EINVAL;
    if (m == 0 || n == 0) return ZERO_OK;
    const Span so = my.span(), sm = ms.span(), sr = mr.span(), sx = mx.span();
    for (const Span &r : {mw.span(), mb.span()})
        if (overlap(so, r) || overlap(sm, r) || overlap(sr, r)) return ZERO_EALIAS;
    if (overlap(sx, sm) || overlap(sx, sr) || overlap(so, sm) || overlap(so, sr) ||
        overlap(sm, sr) || (overlap(sx, so) && !mx.same_place(my)))
        return ZERO_EALIAS;
    NormArgs a{x, static_cast<const uint16_t *>(w), static_cast<const uint16_t *>(b), y, mean,
               rstd, ldx, ldy, m, n, eps32, 1};
    const bool xf = xdt == ZERO_FP32, yf = ydt == ZERO_FP32;
    return wdt == ZERO_BF16 ? launch_norm<BF16>(a, xf, yf, stream)
                            : launch_norm<FP16>(a, xf, yf, stream);
}

int64_t zero_layernorm_workspace_bytes(int64_t m, int64_t n) {
    if (!dim_ok(m) || !dim_ok(n)) return -1;
    return partial_bytes(m, n);
}

zero_status zero_layernorm_backward(const void *dy, zero_dtype dydt, int64_t lddy, const void *x,
                                    zero_dtype xdt, int64_t ldx, const void *w, zero_dtype wdt,
                                    const float *mean, const float *rstd, int64_t m, int64_t n,
                                    const void *residual, int64_t ldr, void *dx, int64_t lddx,
                                    void *dw, void *db, zero_dtype gdt, int32_t accumulate,
                                    void *workspace, int64_t workspace_bytes, void *stream) {
    if (!is16(wdt) || !type_ok(xdt, wdt) || !type_ok(dydt, wdt) || !type_ok(gdt, wdt) ||
        !dim_ok(m) || !dim_ok(n))
        return ZERO_EINVAL;
    const int64_t ge = size_of(gdt), xe = size_of(xdt);
    const Mat my{dy, m, n, lddy, size_of(dydt)}, mx{x, m, n, ldx, xe}, mr{residual, m, n, ldr, xe},
        md{dx, m, n, lddx, xe}, mw{w, 1, n, n, 2}, mm{mean, 1, m, m, 4}, mt{rstd, 1, m, m, 4},
        ga{dw, 1, n, n, ge}, gb{db, 1, n, n, ge};
    if (!my.ok() || !mx.ok() || !md.ok()) return ZERO_EINVAL;
    if (n > 0 && (!mm.ok() || !mt.ok())) return ZERO_EINVAL;
    for (const Mat *v : {&mr, &mw, &ga, &gb})
        if (v->p != nullptr && !v->ok()) return ZERO_EINVAL;
    if (n == 0 || (m == 0 && dw == nullptr && db == nullptr)) return ZERO_OK;
    const bool grads = dw != nullptr || db != nullptr;
    const int64_t need = grads ? partial_bytes(m, n) : 0;
    if (need > 0 && (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need))
        return ZERO_EINVAL;
    const Span sd = md.span(), sa = ga.span(), sb = gb.span(), sr = mr.span(), sy = my.span(),
               sw = need ? span_of(workspace, need, 1) : Span{0, 0};
    for (const Span &r : {mx.span(), mw.span(), mm.span(), mt.span()})
        if (overlap(sd, r) || overlap(sa, r) || overlap(sb, r) || overlap(sw, r))
            return ZERO_EALIAS;
    for (const Span &r : {sr, sy})
        if (overlap(sa, r) || overlap(sb, r) || overlap(sw, r)) return ZERO_EALIAS;
    if (overlap(sd, sa) || overlap(sd, sb) || overlap(sd, sw) || overlap(sa, sb) ||
        overlap(sa, sw) || overlap(sb, sw))
        return ZERO_EALIAS;
    if (overlap(sd, sr) && !mr.same_place(md)) return ZERO_EALIAS;
    if (overlap(sd, sy) && !my.same_place(md)) return ZERO_EALIAS;
    BackArgs a{};
    a.dy = dy;
    a.x = x;
    a.res = residual;
    a.w = static_cast<const uint16_t *>(w);
    a.mean = mean;
    a.rstd = rstd;
    a.dx = dx;
    a.dw = dw;
    a.db = db;
    a.partial = static_cast<float *>(workspace);
    a.lddy = lddy;
    a.ldx = ldx;
    a.ldr = ldr;
    a.lddx = lddx;
    a.m = m;
    a.n = n;
    a.pieces = ceil_div(n, 8);
    a.grads_f32 = gdt == ZERO_FP32;
    a.accumulate = accumulate != 0;
    const bool xf = xdt == ZERO_FP32, df = dydt == ZERO_FP32;
    return wdt == ZERO_BF16 ? launch_back<BF16>(a, xf, df, stream)
                            : launch_back<FP16>(a, xf, df, stream);
}

}  // extern "C"
