/*
 * fsdp_linear.h -- C ABI of librank_step.so: the linear layer on either side
 * of a rank's optimizer step, on an AMD Instinct MI355X (gfx950).
 *
 * fsdp_step.h's calls read N gradient slices of every parameter and write the
 * bf16 or fp8 copy that the next forward's all-gather delivers.  The calls
 * here read that copy and produce those gradients:
 *   fsdp_linear_forward            z = x W^T + b;  y = D(act(z)) + r
 *   fsdp_linear_epilogue_backward  dz = D(dy) act'(z), db = its column sums
 *   fsdp_linear_grad_input         dx = dz W
 *   fsdp_linear_grad_weight        dW = dz^T x, stored or accumulated
 *   fsdp_dropout                   y = D(x) + r; its gradient is D(dy)
 * D is dropout with a mask drawn from a counter-based generator and never
 * stored.  A layer's backward pass is the middle three in that order, with
 * the forward call's dropout record given to the second.  Without activation
 * and dropout dz is dy itself, and the second is needed for db only.
 *
 * The conventions of fsdp_step.h hold: status codes and fsdp_last_error, all
 * arguments checked on the host before any work is queued, device pointers on
 * the current device, work queued on the caller's stream without host
 * synchronisation or allocation, results that are the same run to run (no
 * atomics).  Every call can be captured into a HIP graph.  In addition:
 *   - Matrices are row-major with a row stride (ld*) in elements, at least the
 *     row's length; rows may start at any element.  Elements between a row's
 *     end and the next row's start are not written, and nothing depends on
 *     them; reads stay within the aligned 4-byte words of a row's elements.
 *   - A size of 0 is allowed; a buffer without elements may be NULL.  m, n
 *     and k are at most 2^30, and a launch holds at most 2^22 - 1 workgroups,
 *     each of which takes up to 256 x 256 outputs (else FSDP_E_CAPACITY).  A
 *     product over no terms is 0.
 *   - A written matrix must not overlap another buffer of the call
 *     (FSDP_E_ALIAS), except where a call says that it may be the same matrix
 *     (same address and stride).  Matrices of one row stride that take
 *     different columns of it (the parts of a packed projection) do not
 *     overlap.
 *   - Products accumulate in fp32 over bf16 operands (E4M3 codes widen to
 *     bf16 exactly); everything after the product is fp32, and each output is
 *     rounded once, to nearest even.  NaN gives NaN.  The division by an E4M3
 *     weight's scale is a product with the scale's reciprocal rounded to fp32,
 *     which has to be a normal number: it is for every scale 448 / max(amax,
 *     1e-12) of a finite amax.
 *   - workspace, workspace_bytes: device memory the call may use, 16-byte
 *     aligned, or NULL and 0.  A long product over few output tiles is split
 *     over its length when the partial sums fit there, and column sums over
 *     many rows are split over the rows; joined in a fixed order.
 *     FSDP_LINEAR_WORKSPACE_BYTES is the most any call uses.  Speed only, but
 *     for the order of the fp32 sums.  A call owns its workspace until its
 *     work has finished: calls that may run at the same time (two streams,
 *     two graphs replayed side by side) need one each; calls in stream order
 *     can share one.
 *   - Speed, not correctness: products take their fastest loads when rows
 *     start on 16-byte boundaries and row lengths are multiples of 8.
 */
#ifndef FSDP_LINEAR_H
#define FSDP_LINEAR_H

#include "fsdp_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A weight matrix's element type besides FSDP_DT_BF16: the OCP E4M3 codes
 * that fsdp_mt_cast_fp8 and fsdp_mt_step_fp8 write, with their scale. */
enum { FSDP_DT_E4M3 = 2 };

/* Activations: z; max(z, 0); z Phi(z) with the normal distribution function
 * (the "erf" form); z / (1 + exp(-z)). */
typedef enum {
    FSDP_ACT_NONE = 0,
    FSDP_ACT_RELU = 1,
    FSDP_ACT_GELU = 2,
    FSDP_ACT_SILU = 3
} fsdp_activation;

#define FSDP_LINEAR_WORKSPACE_BYTES ((int64_t)64 << 20)

/* A dropout mask.  Element (i, j) of an [m, n] matrix takes 16 random bits:
 * those of the Philox-4x32-10 block (Salmon, Moraes, Dror and Shaw, "Parallel
 * random numbers: as easy as 1, 2, 3", 2011) with
 *   counter = (B mod 2^32, B / 2^32, o mod 2^32, o / 2^32),
 *             B = i * ceil(n / 8) + j / 8,  o = offset + *offset_dev (mod 2^64)
 *   key     = (seed mod 2^32, seed / 2^32)
 * word (j mod 8) / 2 of the block's four, its low half for even j and its
 * high half for odd j.  With T = rint(65536 p) the element is kept where its
 * bits are at least T and multiplied by 65536 / (65536 - T); others become +0
 * whatever they held.  T = 0 keeps everything, T = 65536 nothing.  So p acts
 * in steps of 2^-16, and the expectation is exact for the p in effect.
 * The mask is a function of the record and the element's place alone, so the
 * backward pass draws the forward's again from the same record, whatever the
 * row strides and whether fused or alone.  Different offsets give independent
 * masks: use one per layer and step.
 *   offset_dev  NULL, or a device int64 [1] read in stream order when the
 *               kernel runs (8-byte aligned): a graph's replays draw new masks
 *               when it names a counter that advances between them, such as
 *               the step_dev of the _capturable step calls.  The backward
 *               launch must read the value that the forward launch read. */
typedef struct {
    double p; /* probability of dropping, 0 <= p <= 1 */
    uint64_t seed, offset;
    const int64_t* offset_dev;
} fsdp_dropout_mask;

/* The forward product.  z = x W^T (divided by the scale for E4M3 weights)
 * + bias, y = D(act(z)) + residual.
 *   x         bf16 [m, k]
 *   w         [n, k] of w_dtype (FSDP_DT_BF16 or FSDP_DT_E4M3): a parameter as
 *             the all-gather delivers it
 *   w_scale   E4M3: device fp32 [1], the tensor's scale (weight = code /
 *             scale; an entry of scale_out of fsdp_mt_cast_fp8); bf16: NULL
 *   bias      bf16 [n], or NULL
 *   residual  [m, n] of y_dtype, or NULL; may be y itself
 *   y         [m, n] of y_dtype (FSDP_DT_BF16 or FSDP_DT_F32), written
 *   z         bf16 [m, n], written, or NULL: the pre-activation that the
 *             backward pass needs
 *   dropout   NULL for none */
typedef struct {
    int64_t m, n, k;
    const uint16_t* x;
    int64_t ldx;
    const void* w;
    int64_t ldw;
    const float* w_scale;
    const uint16_t* bias;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
    uint16_t* z;
    int64_t ldz;
    const fsdp_dropout_mask* dropout;
    void* workspace;
    int64_t workspace_bytes;
    int32_t w_dtype, y_dtype, act;
    int32_t reserved; /* must be 0 */
} fsdp_linear;

int32_t fsdp_linear_forward(const fsdp_linear* a, hipStream_t stream);

/* The gradient of the forward call's epilogue.
 *   dz = D(dy) * act'(z)   bf16 [m, n], written (NULL: not stored; may be dy
 *                          or z itself)
 *   db = column sums of D(dy) * act'(z), taken before dz is rounded, of
 *        db_dtype [n]; added to what db holds if accumulate is 1 (NULL: none)
 * dy: bf16 [m, n].  z: bf16 [m, n] as the forward call stored it; may be NULL
 * when act is FSDP_ACT_NONE.  At z = 0 relu's slope is 0.  Both select: where
 * an element is dropped dz is 0 whatever dy and z hold, and where relu has
 * z <= 0 whatever dy holds.  Where z is NaN and the element is kept dz is NaN,
 * relu's too (but with FSDP_ACT_NONE z is not read).  The residual's gradient
 * is dy.  dy is bf16 also where y was fp32 (rounded by the caller). */
int32_t fsdp_linear_epilogue_backward(uint16_t* dz, int64_t lddz, void* db, int32_t db_dtype,
                                      int32_t accumulate, const uint16_t* dy, int64_t lddy,
                                      const uint16_t* z, int64_t ldz, int32_t act,
                                      const fsdp_dropout_mask* dropout, int64_t m, int64_t n,
                                      void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* dx = dz W (divided by the scale for E4M3 weights): bf16 [m, k], written.
 * dz: bf16 [m, n]; w, w_scale, w_dtype as in fsdp_linear. */
int32_t fsdp_linear_grad_input(uint16_t* dx, int64_t lddx, const uint16_t* dz, int64_t lddz,
                               const void* w, int64_t ldw, int32_t w_dtype, const float* w_scale,
                               int64_t m, int64_t n, int64_t k, void* workspace,
                               int64_t workspace_bytes, hipStream_t stream);

/* dW = dz^T x: [n, k] of dw_dtype (FSDP_DT_BF16 or FSDP_DT_F32), written, or
 * added to what dw holds if accumulate is 1 (one fp32 add, then the
 * rounding).  Rows [r ceil(n/N), (r+1) ceil(n/N)) of a packed dw are the
 * gradient slice that rank r of N receives in the Shard(0) layout.
 * dz: bf16 [m, n]; x: bf16 [m, k]. */
int32_t fsdp_linear_grad_weight(void* dw, int64_t lddw, int32_t dw_dtype, int32_t accumulate,
                                const uint16_t* dz, int64_t lddz, const uint16_t* x, int64_t ldx,
                                int64_t m, int64_t n, int64_t k, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream);

/* y = D(x) + residual on [rows, cols] matrices of one dtype (FSDP_DT_F32 or
 * FSDP_DT_BF16); residual may be NULL; x or the residual may be y itself.
 * With dy for x and no residual it is the gradient. */
int32_t fsdp_dropout(void* y, int64_t ldy, const void* x, int64_t ldx, const void* residual,
                     int64_t ldr, int32_t dtype, int64_t rows, int64_t cols,
                     const fsdp_dropout_mask* mask, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FSDP_LINEAR_H */
