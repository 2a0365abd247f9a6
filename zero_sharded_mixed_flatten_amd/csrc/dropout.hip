// dropout.hip -- gfx950 kernel of zero_dropout: y = residual + D(x) with the
// counter-based mask of zero_linear.h, stored nowhere.
//
// One pass, eight elements and one Philox call a lane.  fp32: the two quads
// that share a draw (columns 4b.. and 16 + 4b.. of a group of 32), two
// 16-byte accesses each 64 bytes contiguous over four lanes.  16-bit types:
// eight neighbouring columns, one 16-byte access; the four lanes of a group
// draw one block each and pass the words on by DPP.  (With the fp32 layout,
// 8-byte accesses, 16384 x 4096 bf16 with a residual took 81 us, 4.97 TB/s.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "linear_common.h"

namespace {

using namespace zero_host;
using namespace zero_linear_impl;

constexpr int64_t kLaunchGroups = int64_t(1) << 22;

struct Args {
    const void *x, *res;
    void *y;
    int64_t ldx, ldr, ldy;
    int64_t rows, cols;
    int64_t group0;  // the launch's first workgroup
    Drop drop;
};

// This thread's row and lane of the row.  A workgroup is 256 consecutive
// (row, lane) pairs; the one division is of its first pair, in scalar
// registers, and rows shorter than a workgroup take a 32-bit one more.
__device__ __forceinline__ bool place(const Args &a, int64_t &i, uint32_t &u) {
    const int64_t lanes = (a.cols + 31) / 32 * 4, first = (a.group0 + blockIdx.x) * 256;
    const int64_t i0 = first / lanes;
    const uint32_t n = static_cast<uint32_t>(lanes);
    const uint32_t at = static_cast<uint32_t>(first - i0 * lanes) + threadIdx.x;
    const uint32_t rows = n >= 256 ? (at >= n ? 1u : 0u) : at / n;
    i = i0 + rows;
    u = at - rows * n;
    return i < a.rows;
}

template <int CTRL>
__device__ __forceinline__ u32x4 from_lane(u32x4 w) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = static_cast<uint32_t>(
            __builtin_amdgcn_update_dpp(0, static_cast<int>(w[e]), CTRL, 0xF, 0xF, false));
    return w;
}

template <class T>
__global__ void __launch_bounds__(256) dropout16_kernel(Args a) {
    int64_t i;
    uint32_t u;
    if (!place(a, i, u)) return;  // whole groups of four lanes
    const int64_t j = static_cast<int64_t>(u) * 8;
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + i * a.ldx + j;
    const uint16_t *r = static_cast<const uint16_t *>(a.res) + i * a.ldr + j;
    const bool whole = j + 8 <= a.cols, res = a.res != nullptr;
    const int n0 = static_cast<int>(j >= a.cols ? 0 : a.cols - j < 4 ? a.cols - j : 4);
    const int n1 = static_cast<int>(j + 4 >= a.cols ? 0 : a.cols - j - 4);
    f32x4 v0, v1, r0 = {0.f, 0.f, 0.f, 0.f}, r1 = r0;
    if (whole) {
        load16x8<T>(x, v0, v1);
        if (res) load16x8<T>(r, r0, r1);
    } else {
        v0 = load16<T>(x, n0);
        v1 = load16<T>(x + 4, n1);
        if (res) {
            r0 = load16<T>(r, n0);
            r1 = load16<T>(r + 4, n1);
        }
    }
    if (a.drop.on) {
        const u32x4 w = drop_words(a.drop, drop_stream(a.drop), static_cast<uint32_t>(i), u);
        // quads 2 q and 2 q + 1 of the group: blocks 0, 2, 0, 2 and 1, 3, 1, 3
        const int half = static_cast<int>(u >> 1) & 1;
        v0 = drop_apply(a.drop, from_lane<0x88>(w), half, v0);
        v1 = drop_apply(a.drop, from_lane<0xDD>(w), half, v1);
    }
    if (res) {
        v0 = r0 + v0;
        v1 = r1 + v1;
    }
    uint16_t *y = static_cast<uint16_t *>(a.y) + i * a.ldy + j;
    if (whole) {
        store16x8<T>(y, v0, v1);
    } else {
        store16<T>(y, v0, n0);
        store16<T>(y + 4, v1, n1);
    }
}

__global__ void __launch_bounds__(256) dropout32_kernel(Args a) {
    const float *x = static_cast<const float *>(a.x), *res = static_cast<const float *>(a.res);
    float *y = static_cast<float *>(a.y);
    int64_t i;
    uint32_t u;
    if (!place(a, i, u)) return;
    const int64_t j = static_cast<int64_t>(u / 4) * 32 + u % 4 * 4;
    if (j >= a.cols) return;
    const int n0 = static_cast<int>(a.cols - j < 4 ? a.cols - j : 4);
    const int64_t left = a.cols - j - 16;
    const int n1 = static_cast<int>(left < 0 ? 0 : left < 4 ? left : 4);
    f32x4 v0 = load32(x + i * a.ldx + j, n0);
    f32x4 v1 = load32(x + i * a.ldx + j + 16, n1);
    f32x4 r0 = {0.f, 0.f, 0.f, 0.f}, r1 = r0;
    if (res != nullptr) {
        r0 = load32(res + i * a.ldr + j, n0);
        r1 = load32(res + i * a.ldr + j + 16, n1);
    }
    if (a.drop.on) {
        const u32x4 w = drop_words(a.drop, drop_stream(a.drop), static_cast<uint32_t>(i), u);
        v0 = drop_apply(a.drop, w, 0, v0);
        v1 = drop_apply(a.drop, w, 1, v1);
    }
    if (res != nullptr) {
        v0 = r0 + v0;
        v1 = r1 + v1;
    }
    store32(y + i * a.ldy + j, v0, n0);
    store32(y + i * a.ldy + j + 16, v1, n1);
}

}  // namespace

extern "C" zero_status zero_dropout(const void *x, zero_dtype dt, int64_t ldx, int64_t rows,
                                    int64_t cols, const zero_dropout_params *drop,
                                    const void *residual, int64_t ldr, void *y, int64_t ldy,
                                    void *stream) {
    if (!(is16(dt) || dt == ZERO_FP32) || !dim_ok(rows) || !dim_ok(cols) || drop == nullptr)
        return ZERO_EINVAL;
    const int64_t e = size_of(dt);
    const Mat mx{x, rows, cols, ldx, e}, mr{residual, rows, cols, ldr, e},
        my{y, rows, cols, ldy, e};
    Args a{};
    if (!make_drop(drop, rows, &a.drop) || !mx.ok() || !my.ok() ||
        (residual != nullptr && !mr.ok()))
        return ZERO_EINVAL;
    if (my.empty()) return ZERO_OK;
    if (overlap(my.span(), mx.span()) && !my.same_place(mx)) return ZERO_EALIAS;
    if (residual != nullptr && overlap(my.span(), mr.span()) && !my.same_place(mr))
        return ZERO_EALIAS;
    if (a.drop.step != nullptr && overlap(my.span(), span_of(a.drop.step, 8, 1)))
        return ZERO_EALIAS;
    a.x = x;
    a.res = residual;
    a.y = y;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldy = ldy;
    a.rows = rows;
    a.cols = cols;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t quads = (cols + 31) / 32 * 4;
    const int64_t groups = (rows * quads + 255) / 256;
    // a launch has less than 2^32 threads: longer ranges go out as several
    for (a.group0 = 0; a.group0 < groups; a.group0 += kLaunchGroups) {
        const uint32_t n = static_cast<uint32_t>(std::min(kLaunchGroups, groups - a.group0));
        if (dt == ZERO_BF16)
            dropout16_kernel<BF16><<<n, 256, 0, st>>>(a);
        else if (dt == ZERO_FP16)
            dropout16_kernel<FP16><<<n, 256, 0, st>>>(a);
        else
            dropout32_kernel<<<n, 256, 0, st>>>(a);
    }
    return launch_status();
}
