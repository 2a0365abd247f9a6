// dropout.hip -- gfx950 kernel of zero_dropout: y = residual + D(x) with the
// counter-based mask of zero_linear.h, stored nowhere.
//
// One pass: a lane takes the two quads of a row that share a draw of the
// mask (columns 4b.. and 16 + 4b.. of a group of 32), so eight elements cost
// one Philox call, about 120 integer cycles of a SIMD against 32 bytes of
// traffic (bf16); the pass is bound by HBM.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "linear_common.h"

namespace {

using namespace zero_host;
using namespace zero_linear_impl;

struct Args {
    const void *x, *res;
    void *y;
    int64_t ldx, ldr, ldy;
    int64_t rows, cols;
    Drop drop;
};

struct FP32 {};

template <class T>
struct Access {
    static __device__ __forceinline__ f32x4 load(const void *p, int64_t at, int n) {
        return load16<T>(static_cast<const uint16_t *>(p) + at, n);
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, f32x4 v, int n) {
        store16<T>(static_cast<uint16_t *>(p) + at, v, n);
    }
};
template <>
struct Access<FP32> {
    static __device__ __forceinline__ f32x4 load(const void *p, int64_t at, int n) {
        return load32(static_cast<const float *>(p) + at, n);
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, f32x4 v, int n) {
        store32(static_cast<float *>(p) + at, v, n);
    }
};

template <class T>
__global__ void __launch_bounds__(256) dropout_kernel(Args a) {
    using A = Access<T>;
    const int64_t quads = (a.cols + 31) / 32 * 4;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= a.rows * quads) return;
    const int64_t i = id / quads, u = id - i * quads;
    const int64_t j = u / 4 * 32 + u % 4 * 4;
    if (j >= a.cols) return;
    const int n0 = static_cast<int>(a.cols - j < 4 ? a.cols - j : 4);
    const int64_t left = a.cols - j - 16;
    const int n1 = static_cast<int>(left < 0 ? 0 : left < 4 ? left : 4);
    f32x4 v0 = A::load(a.x, i * a.ldx + j, n0);
    f32x4 v1 = A::load(a.x, i * a.ldx + j + 16, n1);
    f32x4 r0 = {0.f, 0.f, 0.f, 0.f}, r1 = r0;
    if (a.res != nullptr) {
        r0 = A::load(a.res, i * a.ldr + j, n0);
        r1 = A::load(a.res, i * a.ldr + j + 16, n1);
    }
    if (a.drop.on) {
        const u32x4 w = drop_words(a.drop, drop_stream(a.drop), static_cast<uint32_t>(i),
                                   static_cast<uint32_t>(u));
        v0 = drop_apply(a.drop, w, 0, v0);
        v1 = drop_apply(a.drop, w, 1, v1);
    }
    if (a.res != nullptr) {
        v0 = r0 + v0;
        v1 = r1 + v1;
    }
    A::store(a.y, i * a.ldy + j, v0, n0);
    A::store(a.y, i * a.ldy + j + 16, v1, n1);
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
    const int64_t blocks = (rows * quads + 255) / 256;
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    if (dt == ZERO_BF16)
        dropout_kernel<BF16><<<static_cast<uint32_t>(blocks), 256, 0, st>>>(a);
    else if (dt == ZERO_FP16)
        dropout_kernel<FP16><<<static_cast<uint32_t>(blocks), 256, 0, st>>>(a);
    else
        dropout_kernel<FP32><<<static_cast<uint32_t>(blocks), 256, 0, st>>>(a);
    return launch_status();
}
