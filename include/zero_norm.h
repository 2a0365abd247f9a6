/*
 * zero_norm.h -- C ABI of the layer norm on the flat 16-bit buffers, in the
 * same library as zero_shard.h.
 *
 *   zero_layernorm           y = (x - mean) rstd w + b, row by row
 *   zero_layernorm_backward  dx, and dw (+)=, db (+)= into the gradient row
 * The weight and the bias are read where the all-gather left them, in the
 * flat weight buffer, and their gradients are written where the
 * reduce-scatter takes them: both start at whatever element the flat layout
 * gives them.
 *
 * The conventions of zero_shard.h hold (device pointers of the caller's, work
 * enqueued on `stream`, arguments checked on the host before anything is
 * launched, nothing allocated, no global state), and of zero_linear.h those
 * on matrices: a first element and a row stride ld in elements, rows of
 * contiguous elements, nothing between a row's end and the next row's start
 * read or written, dimensions 0 <= m, n <= 2^31 - 1024, a span of at most
 * 2^60 elements; an empty output is a no-op.  All arithmetic is fp32, each
 * output is rounded once, to nearest even, and the same call gives the same
 * bits on every run.
 */
#ifndef ZERO_NORM_H
#define ZERO_NORM_H

#include "zero_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

/* For each of the m rows of n elements:
 *   mean = sum(x) / n, var = sum((x - mean)^2) / n,
 *   rstd = 1 / sqrt(var + eps), y = (x - mean) * rstd * w + b.
 * The variance is centred: the row is held while its mean is formed, and its
 * differences are what is squared.  A row with an Inf or a NaN gives NaN
 * throughout; no other row is affected.  In a row of finite values so large
 * that the sum of the squared differences passes fp32's range rstd is 0 and y
 * is b; one whose sum or differences do is NaN.
 *   x:    type xdt: wdt or FP32 (an fp32 residual stream).
 *   w, b: n elements of type wdt (BF16 or FP16); NULL for ones, and zeros.
 *   y:    type ydt: wdt or FP32.  It may be x itself (the same address, type
 *         and row stride).
 *   mean, rstd: fp32[m] each, for the backward pass, or NULL.
 * EINVAL: a bad type, a dimension out of range, a row stride below its row, a
 * NULL pointer to something read or written, a pointer not aligned to its
 * element, an eps that is not finite and > 0 as an fp32 value, or mean or rstd where n is 0
 * and m is not.  EALIAS: y, mean or rstd overlaps anything else (y == x
 * excepted). */
ZERO_API zero_status zero_layernorm(const void *x, zero_dtype xdt, int64_t ldx, const void *w,
                                    const void *b, zero_dtype wdt, int64_t m, int64_t n,
                                    double eps, void *y, zero_dtype ydt, int64_t ldy, float *mean,
                                    float *rstd, void *stream);

/* Bytes of device workspace that the backward pass of m rows of n needs when
 * dw or db is asked for: each workgroup's column sums lie there in fp32 and
 * are added in a fixed order by a second kernel.  16-byte aligned scratch
 * that overlaps no other argument; calls that share one must not run at the
 * same time.  0 where none is needed, -1 for dimensions out of range. */
ZERO_API int64_t zero_layernorm_workspace_bytes(int64_t m, int64_t n);

/* With h = (x - mean) rstd and g = dy * w, for each row:
 *   dx = residual + rstd * (g - sum(g) / n - h * sum(g h) / n)
 * and over the rows dw = sum(dy h), db = sum(dy), or dw + that and db + that
 * with accumulate != 0 (a later micro-batch).
 *   dy:   type dydt: wdt or FP32.
 *   x:    type xdt: wdt or FP32, as the forward call read it.
 *   mean, rstd: fp32[m], as the forward call wrote them.
 *   w:    n elements of type wdt, or NULL for ones.
 *   residual: type xdt, or NULL: a gradient that reaches x another way.  It
 *         may be dx itself.
 *   dx:   type xdt.  It may be dy (the same address, type and row stride),
 *         but not x.
 *   dw, db: n elements each of type gdt: wdt or FP32, or NULL.  Accumulation
 *         adds the fp32 sum to the widened old value and rounds once.  Without
 *         rows the sums are zero.  Equal calls give equal bits; the order of a
 *         sum, and so its rounding, goes by sizes, types and whether dx is dy.
 * EINVAL as for zero_layernorm; also for a missing, unaligned or short
 * workspace when dw or db is given.  EALIAS: dx, dw, db or the workspace
 * overlaps anything else (dx == residual and dx == dy excepted). */
ZERO_API zero_status zero_layernorm_backward(
    const void *dy, zero_dtype dydt, int64_t lddy, const void *x, zero_dtype xdt, int64_t ldx,
    const void *w, zero_dtype wdt, const float *mean, const float *rstd, int64_t m, int64_t n,
    const void *residual, int64_t ldr, void *dx, int64_t lddx, void *dw, void *db, zero_dtype gdt,
    int32_t accumulate, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_NORM_H */
