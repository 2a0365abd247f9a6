/*
 * zero_linear.h -- C ABI of the layer products on the flat 16-bit buffers and
 * of the counter-based dropout, in the same library as zero_shard.h.
 *
 * Between two sharded steps a rank runs layers on the full weight buffer that
 * the all-gather filled and writes gradients into the flat row that the next
 * reduce-scatter takes.  These entry points are the products of that part, on
 * those buffers in place:
 *   zero_linear        y  = R + D(act(z)),  z = x W^T + b
 *   zero_linear_dgrad  dx = R + D(act'(z) * (dy W))
 *   zero_linear_wgrad  dW (+)= dy^T x,      db (+)= the column sums of dy
 *   zero_dropout       y  = R + D(x)
 * A parameter starts at whatever element the flat layout gives it, so every
 * matrix may have any element alignment and any row stride.
 *
 * The conventions of zero_shard.h hold (device pointers of the caller's, work
 * enqueued on `stream`, arguments checked on the host before anything is
 * launched, nothing allocated, no global state), and:
 *  - A matrix argument is its first element and a row stride ld in elements;
 *    elements of a row are contiguous.  Nothing between a row's end and the
 *    next row's start is read or written.
 *  - A matrix occupies its span, from its first element to one past its last:
 *    two matrices that interleave (column ranges of one buffer) overlap.
 *  - Dimensions are 0 <= m, n, k <= 2^31 - 1024, a matrix spans at most 2^60
 *    elements, and a product has less than 2^23 output tiles of 64 x 128.  An
 *    empty output is a no-op; an empty contraction gives sums of zero.
 *  - Products of 16-bit elements are exact in fp32 and are summed in fp32 by
 *    the matrix instructions; bias, activation, dropout and residual are
 *    fp32, and each output is rounded once, to nearest even.  The order of a
 *    sum depends on the sizes, the alignment of the operands and nothing
 *    else: the same call gives the same bits on every run.
 *  - A dropped element and a pre-activation that ReLU's derivative masks are
 *    selected away, never multiplied: they give 0 where the value is Inf or
 *    NaN too.
 */
#ifndef ZERO_LINEAR_H
#define ZERO_LINEAR_H

#include "zero_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations.  GELU is 0.5 v (1 + erf(v / sqrt 2)); GELU_TANH is
 * 0.5 v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))); SILU is v / (1 + e^-v).
 * RELU keeps a NaN; its derivative is 1 for v > 0 and 0 elsewhere. */
typedef enum zero_act {
    ZERO_ACT_NONE = 0,
    ZERO_ACT_RELU = 1,
    ZERO_ACT_GELU = 2,
    ZERO_ACT_GELU_TANH = 3,
    ZERO_ACT_SILU = 4
} zero_act;

/* Dropout D with a mask that is a function of (seed, stream, row, column) and
 * is stored nowhere: the backward pass draws it again.
 *   T = min(65535, rint(65536 p)); an element whose 16 random bits are below
 *   T becomes 0, any other is multiplied by fl32(65536 / (65536 - T)).
 * The bits are Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random
 * numbers: as easy as 1, 2, 3", 2011) of the counter (block, row0 + row,
 * stream low, stream high) under the key (seed low, seed high).  Column c
 * lies in block (c / 32) * 4 + (c % 16) / 4 and takes that block's word c % 4:
 * its low 16 bits when c % 32 < 16, its high 16 bits otherwise.
 * stream = offset + *step when step is given (mod 2^64), else offset.  step
 * is a device int64 read when the kernel runs, for instance the counter that
 * zero_step_counter_advance moves, so that a captured graph draws a new mask
 * at every replay.  row0 places a call's rows in a longer batch: a batch
 * split over calls by rows draws the mask of one call.
 * Under one seed, two calls whose streams (offset + *step) are equal draw the
 * same mask: a layer and its backward pass on purpose, but a layer at offset 1
 * in step 5 also that of a layer at offset 0 in step 6.  Calls that should
 * draw independent masks take different seeds, or offsets that the step
 * counter never bridges: multiples of 2^32 serve 2^32 steps. */
typedef struct zero_dropout_params {
    double p;            /* in [0, 1) */
    uint64_t seed;
    uint64_t offset;
    int64_t row0;        /* >= 0; row0 + rows <= 2^32 */
    const int64_t *step; /* device, 8-byte aligned, or NULL */
} zero_dropout_params;

/* The products, for zero_linear_workspace_bytes. */
typedef enum zero_linear_op {
    ZERO_LINEAR = 0,
    ZERO_LINEAR_DGRAD = 1,
    ZERO_LINEAR_WGRAD = 2
} zero_linear_op;

/* Bytes of device workspace that a product of these dimensions needs (0 for
 * many): few output tiles with a long contraction are computed in parts over
 * the contraction, whose fp32 partial sums lie in the workspace and are added
 * in a fixed order by a second kernel.  16-byte aligned scratch that overlaps
 * no other argument; calls that share one must not run at the same time.
 * Returns -1 for a bad op or dimensions out of range. */
ZERO_API int64_t zero_linear_workspace_bytes(zero_linear_op op, int64_t m, int64_t n, int64_t k);

/* y[m][n] = residual + D(act(z)), z = x[m][k] W[n][k]^T + bias[n].
 *   dt:       BF16 or FP16, the type of x, w, bias and z.
 *   bias:     n elements of type dt, or NULL.
 *   drop:     host struct, or NULL for none (p = 0 is none too).
 *   residual: type ydt, or NULL.  It may be y itself (the same address and
 *             row stride).
 *   y:        type ydt: dt or FP32.
 *   z:        the pre-activation rounded to dt, for the backward pass, or
 *             NULL; act is applied to the unrounded sum.
 * EINVAL: a bad dt, ydt or act, a dimension out of range, a row stride below
 * its row, a NULL pointer to something read or written, a pointer not
 * aligned to its element, dropout parameters out of their domain, or a
 * missing, unaligned or short workspace.  EALIAS: y, z or the workspace
 * overlaps anything else (residual == y with the same stride excepted). */
ZERO_API zero_status zero_linear(const void *x, zero_dtype dt, int64_t ldx, const void *w,
                                 int64_t ldw, const void *bias, int64_t m, int64_t n, int64_t k,
                                 zero_act act, const zero_dropout_params *drop,
                                 const void *residual, int64_t ldr, void *y, zero_dtype ydt,
                                 int64_t ldy, void *z, int64_t ldz, void *workspace,
                                 int64_t workspace_bytes, void *stream);

/* dx[m][k] = residual + D(act'(z) * (dy[m][n] W[n][k])): the gradient of the
 * layer's input, carried on through the activation and dropout that made this
 * input.  For x = D(act(z)), act, z ([m][k], type dt, as zero_linear wrote
 * it; NULL with ZERO_ACT_NONE) and drop are those of the call that wrote x;
 * residual (type dxdt, or NULL; it may be dx itself) is a gradient that
 * reaches the same tensor another way.
 * Types and errors as for zero_linear; EINVAL also for an act without z. */
ZERO_API zero_status zero_linear_dgrad(const void *dy, zero_dtype dt, int64_t lddy, const void *w,
                                       int64_t ldw, int64_t m, int64_t n, int64_t k, zero_act act,
                                       const void *z, int64_t ldz,
                                       const zero_dropout_params *drop, const void *residual,
                                       int64_t ldr, void *dx, zero_dtype dxdt, int64_t lddx,
                                       void *workspace, int64_t workspace_bytes, void *stream);

/* dw[n][k] = dy[m][n]^T x[m][k], or dw + that with accumulate != 0 (a later
 * micro-batch); db[n] likewise from the column sums of dy, or NULL.
 *   dw, db: type gdt: dt, or FP32 (an fp32 gradient row).  Accumulation adds
 *           the fp32 sum to the widened old value and rounds once.
 * Errors as for zero_linear; EINVAL also for a db where k is 0. */
ZERO_API zero_status zero_linear_wgrad(const void *dy, zero_dtype dt, int64_t lddy, const void *x,
                                       int64_t ldx, int64_t m, int64_t n, int64_t k, void *dw,
                                       zero_dtype gdt, int64_t lddw, void *db, int32_t accumulate,
                                       void *workspace, int64_t workspace_bytes, void *stream);

/* y[rows][cols] = residual + D(x), and with the same drop its own backward
 * pass (dx = D(dy)).
 *   dt: BF16, FP16 or FP32, the type of x, residual (or NULL) and y.  y may
 *       be x or residual (the same address and row stride).
 * EINVAL and EALIAS as for zero_linear; EINVAL also for a NULL drop. */
ZERO_API zero_status zero_dropout(const void *x, zero_dtype dt, int64_t ldx, int64_t rows,
                                  int64_t cols, const zero_dropout_params *drop,
                                  const void *residual, int64_t ldr, void *y, int64_t ldy,
                                  void *stream);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_LINEAR_H */
