/*
 * lapsum_experts8.h -- C ABI of the experts' products in 8 bits: rows and
 * weights as 8-bit floating point with a power-of-two scale for each block of
 * 128, for serving.
 *
 * Rows in 8 bits are two arrays, both contiguous:
 *   values : e4m3 (finite, "fn") bytes [rows, blocks * 128], blocks =
 *            ceil(width / 128); zeros past the width.
 *   scales : e8m0 bytes [rows, blocks]: the byte s stands for 2^(s - 127), 255
 *            for NaN.
 * An element stands for its value times its block's scale.
 *
 * The conventions are those of lapsum_experts.h.
 */
#ifndef LAPSUM_EXPERTS8_H_
#define LAPSUM_EXPERTS8_H_

#include "lapsum_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LAPSUM_BLOCK8 128
#define LAPSUM_MAX_WIDTH8 0x100000 /* of rows that are multiplied */
#define LAPSUM_MAX_TILES8 0xFFFC00 /* (rows / 256 + experts + 1) * ceil(out / 256), at most */

/*
 * Rows to 8 bits: a block's scale is the least power of two 2^e (e >= -127;
 * 1 for a block of zeros) with which its largest finite magnitude is at most
 * 448, and a value is x / 2^e to the nearest e4m3, ties to even.  Infinities and NaN
 * become NaN and do not count for the scale.
 *   x : dtype[rows, width].  values 16-byte aligned.
 * 0 <= rows <= LAPSUM_MAX_PAIRS, 0 <= width <= LAPSUM_MAX_PAIRS.
 */
lapsum_status_t lapsum_expert_quantize(const void* x, lapsum_dtype_t dtype, int64_t rows, int64_t width, void* values,
                                       void* scales, lapsum_stream_t stream);

/* What rows in 8 bits stand for, rounded to dtype (in fp16 a value past 65504
 * is infinite). */
lapsum_status_t lapsum_expert_dequantize(const void* values, const void* scales, lapsum_dtype_t dtype, int64_t rows,
                                         int64_t width, void* x, lapsum_stream_t stream);

/*
 * Every expert's product over its rows, as lapsum_expert_linear: ys = act(z), z
 * = xs W_e^T + b_e.  For fp32 results the products are exact (of operands down to
 * 2^-126) and their sums fp32.  For 16-bit results the 8-bit matrix instruction
 * adds the products of eight neighbours along the sum first, and drops from each
 * what is below 2^-13 of the largest one's power of two: of a group whose largest
 * product is m, less than 7 * 2^-13 m is lost (random rows: 1.5e-5 of the result
 * in the 2-norm).  Groups are summed in fp32.
 *   xs, weight  : rows in 8 bits, [rows, width] and [experts, out, width],
 *                 values 16-byte aligned.
 *   bias        : dtype[experts, out] or NULL.   ys: dtype[rows, out], zeros
 *                 past offsets[experts].
 * rows, out <= LAPSUM_MAX_PAIRS, width <= LAPSUM_MAX_WIDTH8, and the product in
 * tiles as LAPSUM_MAX_TILES8 says.
 */
lapsum_status_t lapsum_expert_linear_fp8(const void* xs, const void* xs_scales, const void* weight,
                                         const void* weight_scales, const void* bias, lapsum_dtype_t dtype,
                                         int64_t rows, int64_t width, int64_t out, int64_t experts,
                                         const int32_t* offsets, lapsum_act_t act, void* ys, lapsum_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAPSUM_EXPERTS8_H_ */
