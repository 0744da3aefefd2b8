/*
 * lpgemm: the operators of a quantised mixture-of-experts feed-forward layer
 * around the GEMMs of lpgemm.h, for one AMD Instinct MI355X (gfx950).
 *
 *   lpgemm_add_rmsnorm_quantize   residual addition, RMSNorm, int8 rows
 *   lpgemm_silu_mul_quantize      silu(gate) * up, int8 rows
 *   lpgemm_*_grouped              rows sorted by expert times that expert's
 *                                 weights (int8 with scales, binary16, MXFP4)
 *   lpgemm_quantize_mxfp4, lpgemm_dequantize_mxfp4, lpgemm_mxfp4
 *                                 microscaled 4-bit floating point
 *
 * The conventions of lpgemm.h hold: device pointers owned by the caller, work
 * enqueued on `stream` without synchronising, nothing allocated, no state
 * kept between calls, the same status codes checked on the host in the same
 * order (sizes, shape rules, empty problem, NULL pointers, alignment, then
 * the device and the launch).  Weights are K-contiguous (N rows of K).
 * Outputs must not overlap inputs except where a function says so.
 *
 * Sixteen-bit tensors are binary16 or bfloat16 (lpgemm_type); a product's C
 * is binary32 or one of the two, rounded once, to nearest even, from the
 * binary32 result (a value beyond the type's range becomes an infinity).
 */
#ifndef LPGEMM_MOE_H
#define LPGEMM_MOE_H

#include "lpgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lpgemm_type {
    LPGEMM_F32 = 0,
    LPGEMM_F16 = 1,
    LPGEMM_BF16 = 2
} lpgemm_type;

/* Residual addition, root-mean-square norm and int8 rows in one pass, the
 * step in front of lpgemm_i8_dequant or lpgemm_i8_dequant_grouped:
 *   h   = X + R, the sum rounded to `type` (R NULL: h = X);  H = h if H is
 *         not NULL (the residual stream for the next addition);
 *   z_k = h_k * weight_k in binary32, a = max_k |z_k|;
 *   Q_k = the nearest-even integer to z_k * (127 * (1 / a)), each operation
 *         rounded to binary32;
 *   row_scale = (a / 127) / sqrt(mean_k h_k^2 + eps), in binary32,
 * so that Q_k * row_scale is the normalised, weighted row.  The norm's own
 * factor cancels out of the codes, which therefore depend on no sum.
 * A row with a below 2^-100 (an all-zero row) gets scale 0 and codes 0.  A
 * row with an infinity or a NaN among its h or z, or whose sum of squares
 * is above the binary32 range, gets scale NaN and codes 0.  Squares that are
 * too small for binary32 count all the same: eps may be 0.
 * X, R, H: M rows of K values of `type` (LPGEMM_F16 or LPGEMM_BF16), row
 * strides in elements, at least K and multiples of 8 (a stride of an absent
 * R or H is not read); weight: K values of `type`; Q: M x K int8;
 * row_scale: M floats.  K a multiple of 8, at most LPGEMM_MAX_K_QUANT.
 * H may be X or R (same pointer and stride).  eps >= 0.  Pointers 16-byte
 * aligned, row_scale 4-byte.  M = 0 is a no-op; K = 0 sets row_scale to 0. */
lpgemm_status lpgemm_add_rmsnorm_quantize(int64_t M, int64_t K, lpgemm_type type, const void *X,
                                          int64_t x_stride, const void *R, int64_t r_stride,
                                          const void *weight, float eps, void *H, int64_t h_stride,
                                          int8_t *Q, float *row_scale, hipStream_t stream);

/* The gated activation between an expert's two products, with int8 rows for
 * the second: z_k = g_k / (1 + exp(-g_k)) * u_k in binary32, where a row of X
 * holds the K gate values g and then the K values u (the layout the product
 * with gate and up weights stacked along N writes); a, Q and the zero and
 * non-finite rows as for lpgemm_add_rmsnorm_quantize, row_scale = a / 127.
 * z_k is within 8 units of 2^-24 of its exact value, relative (12 for g_k below
 * -86), so a code may be the neighbour of the correctly rounded one where
 * z_k * 127 / a lies that near to halfway between two.  Below g_k = -88.72
 * exp(-g_k) leaves binary32 and z_k is a zero.
 * X: M rows of 2K values of `type`, x_stride >= 2K in elements, a multiple of
 * 8; Q: M x K int8; row_scale: M floats.  K a multiple of 8, at most
 * LPGEMM_MAX_K_QUANT.  Pointers 16-byte aligned, row_scale 4-byte.  M = 0 is
 * a no-op; K = 0 sets row_scale to 0. */
lpgemm_status lpgemm_silu_mul_quantize(int64_t M, int64_t K, lpgemm_type type, const void *X,
                                       int64_t x_stride, int8_t *Q, float *row_scale, hipStream_t stream);

/* MXFP4: blocks of 32 values along k share one power-of-two scale 2^(b-127)
 * (b the block's E8M0 byte, 255 = NaN); a value is a 4-bit E2M1 number
 * (sign, magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 as codes 0..7) times that
 * scale.  Codes: rows of K/2 bytes, the even k in the low nibble.  Scales:
 * rows of LPGEMM_MXFP4_SCALE_STRIDE(K) bytes, of which the first K/32 are
 * the row's blocks in order (the rest is padding, never read as a scale).
 * K is a multiple of 32, at most LPGEMM_MAX_K_MXFP4. */
#define LPGEMM_MXFP4_SCALE_STRIDE(K) ((((K) / 32) + 15) / 16 * 16)
#define LPGEMM_MAX_K_MXFP4 1048576

/* rows x K values of `type` (LPGEMM_F16 or LPGEMM_BF16) to MXFP4.  With a the
 * block's largest magnitude, b = clamp(floor(log2 a) - 2 + 127, 0, 254) (0
 * for a block of zeros); each value over 2^(b-127) is rounded to the nearest
 * E2M1 number (halfway: to the even code), magnitudes above 6 to 6.  A block
 * that holds an infinity or a NaN gets b = 255 and codes 0.  Padding bytes of
 * `scales` are set to 0.  x_stride in elements, at least K, a multiple of 8.
 * Pointers 16-byte aligned.  rows = 0 or K = 0 is a no-op. */
lpgemm_status lpgemm_quantize_mxfp4(int64_t rows, int64_t K, lpgemm_type type, const void *X,
                                    int64_t x_stride, uint8_t *codes, uint8_t *scales, hipStream_t stream);

/* The values MXFP4 rows stand for: Y = rows x K of `type` (any of the three),
 * each rounded once to it (exact in binary32 and bfloat16 unless the value
 * leaves the type's range); blocks with scale byte 255 give NaN. */
lpgemm_status lpgemm_dequantize_mxfp4(int64_t rows, int64_t K, const uint8_t *codes, const uint8_t *scales,
                                      lpgemm_type type, void *Y, hipStream_t stream);

/* C = A . B for two MXFP4 operands (A: M x K, B: N x K, each with its
 * scales), summed in binary32 by the chip's scaled matrix instructions;
 * C: M x N of `type`.  The order of the sum depends on the sizes only.
 * M and N at most 2^31 - 257, and below 2^24 tiles of C (UNSUPPORTED_SHAPE
 * otherwise).  Pointers 16-byte aligned.  M = 0 or N = 0 is a no-op; K = 0
 * sets C to 0. */
lpgemm_status lpgemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t *A, const uint8_t *A_scale,
                           const uint8_t *B, const uint8_t *B_scale, lpgemm_type type, void *C,
                           hipStream_t stream);

/* Products grouped by expert.  C has `rows` rows, sorted by expert: rows
 * offsets[g] .. offsets[g+1]-1 belong to group g, and row i is
 *   C[i] = A[row_index[i]] . B_g   (row_index NULL: A[i], and a_rows = rows;
 *                                   INVALID_VALUE otherwise)
 * with B_g the g-th of `groups` N x K weight matrices stored one after the
 * other.  offsets (groups + 1 int32) and row_index (rows int32) are read on
 * the device, so no host synchronisation is needed to build them; groups may
 * be empty or hold every row.  Offsets outside 0..rows are clamped to it and
 * a group whose end is not above its start is empty; rows that belong to no
 * group are left as they were; where groups overlap, what C holds is
 * undefined.  A row_index outside 0..a_rows-1 gives a row of zeros.
 * With a row_index the tokens A must stay below 2 GiB (UNSUPPORTED_SHAPE).
 * groups = 0, rows = 0 or N = 0 is a no-op; K = 0 leaves empty sums, grouped
 * rows of 0 (int8: 0 times the scales);
 * a_rows = 0 with rows > 0 needs a row_index and gives rows of zeros.
 * groups is at most LPGEMM_MAX_GROUPS, rows and N at most 2^31 - 257, and the
 * tiles of C must fit one launch (below 2^24 workgroups; UNSUPPORTED_SHAPE
 * otherwise).  A, B and C 16-byte aligned, offsets,
 * row_index and fp32 scales 4-byte.
 *
 * lpgemm_i8_dequant_grouped: A a_rows x K int8, row_scale a_rows floats (one
 * per row of A), B groups x N x K int8, col_scale groups x N floats,
 *   C[i][j] = ((float)sum * row_scale) * col_scale, as lpgemm_i8_dequant.
 * lpgemm_f16_grouped: binary16 A and B, sums in binary32.
 * lpgemm_mxfp4_grouped: MXFP4 A and B, each with its scales (B_scale: groups
 * x N rows).  K rules as for lpgemm_i8, lpgemm_f16 and lpgemm_mxfp4. */
#define LPGEMM_MAX_GROUPS 65536
lpgemm_status lpgemm_i8_dequant_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows,
                                        const int8_t *A, const int8_t *B, const int32_t *offsets,
                                        const int32_t *row_index, const float *row_scale,
                                        const float *col_scale, lpgemm_type type, void *C,
                                        hipStream_t stream);
lpgemm_status lpgemm_f16_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows,
                                 const void *A, const void *B, const int32_t *offsets,
                                 const int32_t *row_index, lpgemm_type type, void *C, hipStream_t stream);
lpgemm_status lpgemm_mxfp4_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows,
                                   const uint8_t *A, const uint8_t *A_scale, const uint8_t *B,
                                   const uint8_t *B_scale, const int32_t *offsets,
                                   const int32_t *row_index, lpgemm_type type, void *C,
                                   hipStream_t stream);

/* Ablation hook, as lpgemm_force_config: the grouped and MXFP4 products have
 * lpgemm_grouped_config_count() kernels, of which every call takes one by its
 * sizes.  lpgemm_force_grouped_config(c) pins kernel c for every later call in
 * the process, or restores the choice for any other value (-1), and returns
 * the previous setting (-1 = by size).  Every kernel computes every size; the
 * integer results do not depend on it, the order of the others' sums does.
 * lpgemm_grouped_auto_config tells the choice for a device with `cu_count`
 * compute units: kind 2 lpgemm_f16_grouped, 3 lpgemm_i8_dequant_grouped, 6
 * MXFP4 (groups = 1: also lpgemm_mxfp4); -1 for other kinds, empty sizes or
 * sizes out of range.  Host arithmetic only. */
int lpgemm_grouped_config_count(void);
int lpgemm_force_grouped_config(int config);
int lpgemm_grouped_auto_config(int kind, int64_t rows, int64_t groups, int64_t N, int64_t K, int cu_count);

#ifdef __cplusplus
}
#endif

#endif /* LPGEMM_MOE_H */
