/*
 * fsdp_mx4.h -- C ABI of librank_step.so: matrices in microscaled 4-bit
 * floating point, and their products, on an AMD Instinct MI355X (gfx950).
 *
 *   fsdp_mx4_quantize     a matrix, and its transpose, to 4-bit copies
 *   fsdp_mx4_dequantize   the values that a copy stands for
 *   fsdp_mx4_product      y = D(act(A B^T + bias)) + residual of two copies
 * A third all-gather copy beside fsdp_step.h's bf16 and fp8 ones: a rank
 * quantises its rows of a weight, the gathered bytes are the whole weight's
 * copy, and the product takes them at up to four times bf16's rate.  That holds
 * for W, whose blocks lie along rows.  The blocks of its transpose lie across the
 * ranks' rows, and each rank's piece [k, rows of a rank] has blocks and padding of
 * its own, so gathered pieces are not one operand: the input gradient is either
 * the product with a transpose that is quantised from the whole weight (the
 * gathered bf16 copy, say), or one product a piece, with the columns of dz that
 * are that rank's rows quantised by themselves, added in place (residual = y).
 * A layer
 * y = x W^T in 4 bits is
 *   forward       product of x and W                    (blocks along the input features)
 *   input grad    product of dz and W's transpose       (along the output features)
 *   weight grad   product of dz's and x's transposes    (along the tokens)
 * with the conventions of fsdp_linear.h: status codes and fsdp_last_error, all
 * arguments checked on the host before any work is queued, work queued on the
 * caller's stream without host synchronisation or allocation, results that are
 * the same run to run, every call capturable into a HIP graph; a written buffer
 * overlaps no other buffer of the call but where it says so; a size of 0 is
 * allowed, and a buffer without elements may be NULL.
 *
 * The format (the OCP microscaling format MXFP4).  32 neighbours of a row are
 * a block; a row's last block may be shorter.  A block is 16 bytes of codes,
 * element 2i in the low half of byte i and 2i + 1 in the high half, and one
 * scale byte.  A code is a sign (bit 3) and one of the magnitudes
 *   0, 0.5, 1, 1.5, 2, 3, 4, 6   (bits 2..0, in this order);
 * it stands for that times 2^(scale - 127).  Scale 255 makes the whole block
 * NaN.  In memory a matrix [rows, cols] is
 *   codes   rows of FSDP_MX4_CODE_BYTES(cols): whole blocks, zeros behind the
 *           row's end
 *   scales  rows of FSDP_MX4_SCALE_BYTES(cols): one byte a block, rounded up
 *           to a multiple of 16 by zeros
 * Rows start on 16-byte boundaries: addresses and row strides (ld*, in bytes)
 * are multiples of 16 (else FSDP_E_ALIGN); a stride is at least the row's bytes.
 * fsdp_mx4_quantize writes the zeros; the other calls rely on them.
 */
#ifndef FSDP_MX4_H
#define FSDP_MX4_H

#include "fsdp_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FSDP_MX4_BLOCK 32
#define FSDP_MX4_CODE_BYTES(cols) (((cols) + 31) / 32 * 16)
#define FSDP_MX4_SCALE_BYTES(cols) (((cols) + 511) / 512 * 16)

/* The copy of x, with blocks along its rows, and of its transpose, with blocks
 * along its columns; x is read once for both.
 *   codes, scales      [rows, cols] as above, written, or both NULL
 *   codes_t, scales_t  [cols, rows] as above, written, or both NULL
 *   x                  [rows, cols] of x_dtype (FSDP_DT_F32 or FSDP_DT_BF16),
 *                      row stride ldx in elements; rows may start at any element
 * A block whose largest magnitude is a has scale 127 + max(floor(log2 a) - 2,
 * -127) (0 for a block of zeros); each element becomes the nearest code, ties to
 * the even one, and what is above 6 times the scale becomes 6 times it.  A
 * block with a NaN or an infinity has scale 255 and codes 0.  rows and cols are
 * at most 2^30, and with codes_t a launch holds 2^22 - 1 tiles of 256 x 128
 * elements, rows and (with codes) cols rounded up to 512, and refuses more with
 * FSDP_E_CAPACITY (up to 512 columns, more than 2^28 - 512 rows). */
int32_t fsdp_mx4_quantize(uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, uint8_t* codes_t,
                          int64_t ldct, uint8_t* scales_t, int64_t ldst, const void* x, int64_t ldx,
                          int32_t x_dtype, int64_t rows, int64_t cols, hipStream_t stream);

/* The values of a copy: y [rows, cols] of y_dtype (FSDP_DT_F32 or FSDP_DT_BF16,
 * both of which hold them exactly; magnitudes from 2^128 on become infinite),
 * row stride ldy in elements, rows from any element. */
int32_t fsdp_mx4_dequantize(void* y, int64_t ldy, int32_t y_dtype, const uint8_t* codes, int64_t ldc,
                            const uint8_t* scales, int64_t lds, int64_t rows, int64_t cols,
                            hipStream_t stream);

/* z = A B^T + bias, y = D(act(z)) + residual.
 *   a, a_scales  [m, k] as above
 *   b, b_scales  [n, k] as above
 *   bias         bf16 [n], or NULL
 *   residual     [m, n] of y_dtype, or NULL; may be y itself (so a gradient is
 *                accumulated in place)
 *   y            [m, n] of y_dtype (FSDP_DT_BF16 or FSDP_DT_F32), written
 *   z            bf16 [m, n], written, or NULL
 *   dropout      NULL for none; act, dropout and residual as in fsdp_linear
 * Row strides: of a, a_scales, b and b_scales in bytes, at most 2^22 (else
 * FSDP_E_CAPACITY); of the others in elements, their rows from any element.
 * m and n are at most 2^30, k at most 2^23 (whose row of codes is 2^22 bytes),
 * and a launch holds at most 2^22 - 1 workgroups: else FSDP_E_CAPACITY.
 * The products of two elements are exact and are added in fp32 by the matrix
 * instructions; what follows is fp32, and each output is rounded once.  A NaN
 * block of A makes its row NaN, one of B its column.
 *   workspace, workspace_bytes  as in fsdp_linear.h, at most
 *                FSDP_MX4_WORKSPACE_BYTES of it is used: a long product over
 *                few output tiles is split over its length when the partial sums
 *                fit there.  Speed only, but for the order of the sums. */
#define FSDP_MX4_WORKSPACE_BYTES ((int64_t)64 << 20)

typedef struct {
    int64_t m, n, k;
    const uint8_t* a;
    int64_t lda;
    const uint8_t* a_scales;
    int64_t ldas;
    const uint8_t* b;
    int64_t ldb;
    const uint8_t* b_scales;
    int64_t ldbs;
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
    int32_t y_dtype, act;
} fsdp_mx4_operands;

int32_t fsdp_mx4_product(const fsdp_mx4_operands* a, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FSDP_MX4_H */
