/*
 * fsdp_norm.h -- C ABI of librank_step.so: the norm in front of a linear layer
 * and its gradients, on an AMD Instinct MI355X (gfx950).
 *
 *   fsdp_norm_forward    y = (x - mean) rstd w + b, row by row
 *   fsdp_norm_backward   its gradients to x, w and b
 * w and b are read from the copy that the all-gather delivers (or from fp32
 * parameters), and dw and db are gradient slices of the next step, as in
 * fsdp_linear.h, whose conventions hold: status codes and fsdp_last_error, all
 * arguments checked on the host before any work is queued, work queued on the
 * caller's stream without host synchronisation or allocation, results that are
 * the same run to run (no atomics), every call capturable into a HIP graph;
 * matrices row-major with a row stride in elements, rows that may start at any
 * element, nothing written between a row's end and the next row's start; a
 * written buffer overlaps no other buffer of the call but where it says so.
 * Sizes are at most 2^30.  Arithmetic and sums are fp32, and each output is
 * rounded once, to nearest even.  A NaN makes its row's outputs NaN; so does an
 * infinity (FSDP_NORM_RMS: its own output NaN and the row's others b).
 */
#ifndef FSDP_NORM_H
#define FSDP_NORM_H

#include "fsdp_step.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FSDP_NORM_LAYER = 0, /* mean and variance of the row */
    FSDP_NORM_RMS = 1    /* mean 0, the row's mean square for the variance */
} fsdp_norm_kind;

/* With x a row of n elements:
 *   mean = sum(x) / n (FSDP_NORM_RMS: 0),  var = sum((x - mean)^2) / n,
 *   rstd = 1 / sqrt(var + eps),            y = (x - mean) rstd w + b
 *   y, x      [m, n] of dtype (FSDP_DT_F32 or FSDP_DT_BF16); y may be x itself
 *   mean      fp32 [m], written, or NULL; must be NULL for FSDP_NORM_RMS
 *   rstd      fp32 [m], written, or NULL: what the backward call takes
 *   weight    w_dtype [n], or NULL for ones
 *   bias      w_dtype [n], or NULL for zeros
 *   eps       at least 0, finite in fp32.  With 0 a row without variance gives NaN.
 * The variance is summed about the mean, so a mean that is large against the
 * row's spread costs no more than the mean's own rounding to fp32.  A row whose
 * sum, or sum of squares, is past fp32's range, or whose var + eps is under
 * 2^-100, is summed in 64 bits (8192 rows of 4096 bf16: 0.13 ms, for 0.03), so y
 * holds for all finite x.  For n = 0 nothing is written. */
int32_t fsdp_norm_forward(void* y, int64_t ldy, float* mean, float* rstd, const void* x, int64_t ldx,
                          int32_t dtype, int32_t kind, const void* weight, const void* bias,
                          int32_t w_dtype, double eps, int64_t m, int64_t n, hipStream_t stream);

/* With xhat = (x - mean) rstd (FSDP_NORM_RMS: x rstd) and g = dy w:
 *   dx = rstd (g - sum(g) / n - xhat sum(g xhat) / n) + residual
 *        (FSDP_NORM_RMS: without the term sum(g) / n)
 *   dw = column sums of dy xhat,  db = column sums of dy
 *   dx        [m, n] of dtype, written (NULL: not wanted)
 *   dw, db    dw_dtype [n] (FSDP_DT_F32 or FSDP_DT_BF16), written, or added to
 *             what they hold if accumulate is 1 (one fp32 add, then the
 *             rounding); NULL: not wanted
 *   dy, x     [m, n] of dtype; x as the forward call read it
 *   weight    w_dtype [n], or NULL for ones
 *   mean      fp32 [m] as the forward call stored it; NULL for FSDP_NORM_RMS
 *   rstd      fp32 [m] as the forward call stored it.  It has fp32's digits for
 *             rows with a spread from 2^-127 to 2^126, and x - mean must not
 *             exceed fp32's range.
 *   residual  [m, n] of dtype, or NULL: the gradient that reaches x past the
 *             norm; may be dx itself
 *   workspace, workspace_bytes  as in fsdp_linear.h: device memory the call may
 *             use, 16-byte aligned, or NULL and 0; at most
 *             FSDP_NORM_WORKSPACE_BYTES of it is used.  Column sums over many
 *             rows are split over the rows when the parts fit there, and joined
 *             in a fixed order: speed only, but for the order of the sums.
 *             8 n bytes are a part; 8192 rows of 4096 take 0.06 ms with room
 *             for 512 of them, 1.5 ms with none.
 * A column's rows are added in fp32 by at most 64 one after the other, and those
 * sums joined in 64 bits: the error of a sum, at most 143 * 2^-24 of the sum
 * of their terms' magnitudes, does not grow with m. */
#define FSDP_NORM_WORKSPACE_BYTES ((int64_t)64 << 20)

int32_t fsdp_norm_backward(void* dx, int64_t lddx, void* dw, void* db, int32_t dw_dtype,
                           int32_t accumulate, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           int32_t dtype, int32_t kind, const void* weight, int32_t w_dtype,
                           const float* mean, const float* rstd, const void* residual, int64_t ldr,
                           int64_t m, int64_t n, void* workspace, int64_t workspace_bytes,
                           hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FSDP_NORM_H */
