/*
 * zero_muon.h -- C ABI of the Muon step of a shard, in the same library as
 * zero_shard.h.
 *
 * Muon steps the matrices of a model by their momentum, orthogonalised with a
 * few Newton-Schulz products; vectors (norms, biases) and the embedding stay
 * with AdamW.  On the flat buffers a step is:
 *   zero_muon_momentum   the ranks' rows reduced, the momentum of this rank's
 *                        shard updated, what is to be orthogonalised written
 *                        into the shard's place of a full buffer;
 *   (an all-gather of that buffer, where a matrix spans more than one shard)
 *   zero_orthogonalize   whole matrices, one or a stack at a stride, read
 *                        from and written to flat buffers;
 *   zero_muon_update     the shard's part of the result applied to its fp32
 *                        master, and the 16-bit cast into the weight slot.
 *
 * The conventions of zero_shard.h hold.  zero_muon_momentum and
 * zero_muon_update keep its arithmetic: every operation below is one fp32
 * operation, in the order written, rounded to nearest even, and any range can
 * be split over calls.
 */
#ifndef ZERO_MUON_H
#define ZERO_MUON_H

#include "zero_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

/* For j in [0, len), with a_j = G_0[j] + ... + G_{n_rows-1}[j] summed left to
 * right as in zero_shard_reduce:
 *   g = a_j * s, mom[j] = b1 * mom[j] + g,
 *   u[j] = nesterov ? g + b1 * mom[j] : mom[j]   (mom as updated)
 * with b1 = fl(beta1), the momentum, and s = fl(grad_scale) of hp (see
 * zero_adamw_hparams; its lr, beta2, eps and weight_decay are checked and
 * take no part), or s from the loss scale and g times the clip coefficient as
 * for zero_shard_adamw_ex when ctl (nullable) says so; ctl->skip set: nothing
 * is written.
 *   grads: device, type gdt (BF16, FP16 or FP32), n_rows rows ld elements
 *          apart: the ranks' rows, or one fp32 row, the accumulator of
 *          zero_shard_reduce.
 *   mom:   device fp32[len].
 *   u:     device, len elements of type udt (BF16, FP16 or FP32), rounded to
 *          it once.
 * EINVAL: as for zero_shard_reduce and zero_shard_adamw_ex (n_rows < 1, len
 * < 0, ld < len, a bad type, hyperparameters or control out of their domain,
 * a NULL required pointer or one not aligned to its element).  EALIAS: mom or
 * u overlaps anything else.  len == 0 is a no-op. */
ZERO_API zero_status zero_muon_momentum(const void *grads, zero_dtype gdt, int32_t n_rows,
                                        int64_t ld, int64_t len, float *mom, void *u,
                                        zero_dtype udt, int32_t nesterov,
                                        const zero_adamw_hparams *hp,
                                        const zero_step_control *ctl, void *stream);

/* The same with its constants read from consts (device; b1, s and grad_scale
 * are used) when the kernel runs, as for zero_shard_adamw_dc: a step whose
 * constants have a NaN s is held. */
ZERO_API zero_status zero_muon_momentum_dc(const void *grads, zero_dtype gdt, int32_t n_rows,
                                           int64_t ld, int64_t len, float *mom, void *u,
                                           zero_dtype udt, int32_t nesterov,
                                           const zero_step_consts *consts,
                                           const zero_step_control *ctl, void *stream);

/* Newton-Schulz rounds of zero_orthogonalize: steps of them, round i with the
 * coefficients coeffs[3 i .. 3 i + 2] (host memory, read during the call), or
 * (3.4445, -4.7750, 2.0315) in every round where coeffs is NULL. */
#define ZERO_NS_MAX_STEPS 32
typedef struct zero_ns_params {
    int32_t steps;        /* 1 <= steps <= ZERO_NS_MAX_STEPS */
    int32_t reserved;     /* zero */
    double eps;           /* finite, >= 0 */
    const double *coeffs; /* finite as fp32 values, or NULL */
} zero_ns_params;

/* Bytes of device workspace that zero_orthogonalize needs for count matrices
 * of rows x cols: 16-byte aligned scratch that overlaps no other argument;
 * calls that share one must not run at the same time.  -1 for dimensions out
 * of range. */
ZERO_API int64_t zero_orthogonalize_workspace_bytes(int64_t count, int64_t rows, int64_t cols);

/* For each of count matrices U of rows x cols:
 *   X = U / (|U| + eps), |U| the Frobenius norm; then steps times
 *   A = X X^T, X = a X + (b A + c A A) X; O = X
 * (with X^T X in place of X X^T, on the other side, where rows > cols: the
 * same result).  Singular vectors stay, singular values go through the
 * polynomial a s + b s^3 + c s^5.
 *   u: type udt (BF16, FP16 or FP32); matrix i starts at element i * su, its
 *      rows are ldu elements apart, elements of a row are contiguous.
 *   o: type odt (BF16 or FP16), at i * so and ldo likewise.
 *   ns: host struct, or NULL for five rounds with eps 1e-7.
 * The norm is summed in fp64.  X is held to 22 bits as a pair of fp16 values,
 * the diagonals of A and of the polynomial in fp32; the products take the
 * first fp16 value of X and the rest of A and of the polynomial in fp16,
 * and sum in fp32.  With the default rounds the result is off the definition,
 * of its norm and before its own rounding (bf16's is 1.7e-3), by 1e-3 as a rule
 * and 1.8e-3 at most (as measured, over full-rank, decaying and low-rank
 * spectra) where 64 rows and columns or more carry the matrix, 2.8e-3 where 16
 * do, 5e-3 where four do and 9e-3 where two do.
 * Singular values must stay below 16 in every round (with the default
 * coefficients they stay below 1.3).  Coefficients that could lift a singular
 * value of up to 1 above 4, or whose b s^2 + c s^4 could spread over more than
 * 16, leave the small elements of A or of the polynomial fewer bits.  Inf or
 * NaN in a matrix makes all of that matrix NaN, and no other; a matrix of zeros
 * stays zero where eps > 0 and is NaN where eps is 0.
 * 0 <= count <= 65535, 0 <= rows, cols <= 65536, a stack spans at most 2^60
 * elements, and a call has less than 2^23 tiles (of 64 x 64 to 256 x 256).  A
 * matrix occupies its span, from its first element to one past its last, and
 * su and so are at least that where count > 1; nothing between a row's end and
 * the next row's start is read or written.  An empty call or matrix is a
 * no-op.
 * EINVAL: a bad type, a dimension or parameter out of range, a stride below
 * what it spans, a NULL or unaligned pointer, a missing, unaligned or short
 * workspace.  EALIAS: o or the workspace overlaps anything else. */
ZERO_API zero_status zero_orthogonalize(const void *u, zero_dtype udt, int64_t ldu, int64_t su,
                                        int64_t count, int64_t rows, int64_t cols,
                                        const zero_ns_params *ns, void *o, zero_dtype odt,
                                        int64_t ldo, int64_t so, void *workspace,
                                        int64_t workspace_bytes, void *stream);

/* For j in [0, len): w = master[j] * d - lr * (k * o[j]), k = fl(update_scale)
 * (for instance 0.2 sqrt(max(rows, cols)), or sqrt(max(1, rows / cols))), lr
 * and d as for zero_adamw_hparams; master[j] = w, and w rounded to wdt into
 * weight_full[rank * shard + shard_off + j].
 *   o:     device, len elements of type odt (BF16 or FP16): the range's part
 *          of zero_orthogonalize's result.
 *   Everything else as for zero_shard_adamw, update_scale finite as
 *   an fp32 value. */
ZERO_API zero_status zero_muon_update(const void *o, zero_dtype odt, float *master,
                                      void *weight_full, zero_dtype wdt,
                                      const zero_layout *layout, int32_t rank, int64_t shard_off,
                                      int64_t len, const zero_adamw_hparams *hp,
                                      double update_scale, const uint32_t *skip, void *stream);

/* The same with lr and d read from consts (device) when the kernel runs; a
 * step whose constants have a NaN s is held. */
ZERO_API zero_status zero_muon_update_dc(const void *o, zero_dtype odt, float *master,
                                         void *weight_full, zero_dtype wdt,
                                         const zero_layout *layout, int32_t rank,
                                         int64_t shard_off, int64_t len,
                                         const zero_step_consts *consts, double update_scale,
                                         const uint32_t *skip, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* ZERO_MUON_H */
