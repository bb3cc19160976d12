/*
 * s6_q4.h -- C ABI of libs6 for a layer's projections in few bits: products
 * with 4-bit weights and group scales, and the norm before a block with an
 * 8-bit output, which those products read.  AMD MI355X (gfx950).
 *
 * The status codes, types, the stream argument and the rules for workspaces and
 * pointers are those of s6.h: every call only enqueues work, checks its
 * arguments before any HIP call, allocates nothing and keeps no state.  Values
 * are not checked: NaN and infinities propagate.
 *
 * 4-bit weights.  A matrix (outer, inner) as codes, two in a byte with the
 * lower index in the lower half, rows of inner / 2 bytes, and one bf16 scale
 * per `group` consecutive columns of a row, (outer, inner / group); group is
 * 32, 64 or 128 and divides inner, which is at most 2^20.  A weight is value(code) * scale; the
 * values of codes 0 to 7 are 0, 0.5, 1, 1.5, 2, 3, 4, 6 and those of 8 to 15
 * the same with a minus (the 4-bit float with two exponent bits and one
 * mantissa bit).
 */
#ifndef S6_Q4_H_
#define S6_Q4_H_

#include "s6.h"

#ifdef __cplusplus
extern "C" {
#endif

#define S6_E4M3 2 /* 8-bit floats, largest value 448 (x of s6_q4_linear only) */

/* codes and scales of w (outer rows of w_stride elements, in_dtype): per group,
 * scale = max|w| / 6 rounded to bf16, codes the values nearest to w / scale
 * (ties to the even code), 0 where the scale is 0.  A group that holds a NaN
 * or an infinity has a scale that is not finite. */
int s6_q4_pack(int64_t outer, int64_t inner, int64_t group, int in_dtype, const void* w, int64_t w_stride,
               void* codes, void* scales, void* stream);

/* y = x W^T: x (rows of x_stride elements, inner wide) in x_dtype S6_F32,
 * S6_BF16, or S6_E4M3 with one fp32 factor per row in x_scale (NULL: 1; only
 * with S6_E4M3); y (rows, outer) contiguous, in y_dtype S6_F32 or S6_BF16.
 * Products are exact, sums fp32, scales fp32; an fp32 x enters in full (three
 * bf16 parts; below 2^-109 up to 2^-134).  The sum of a group of finite values is
 * finite: what overflows is the result, or a sum of scaled groups past 2^138 (8-bit
 * x: 2^128).  Any number of rows; made for the few rows of single tokens.  codes
 * are 16-byte aligned, x_stride is at most 2^20.  workspace:
 * s6_q4_linear_workspace_size bytes, 0 up to 16 rows (of fp32: 6).  Repeated calls
 * give identical bits. */
int s6_q4_linear(int64_t rows, int64_t inner, int64_t outer, int64_t group, int x_dtype, int y_dtype, const void* x,
                 int64_t x_stride, const float* x_scale, const void* codes, const void* scales, void* y,
                 void* workspace, size_t workspace_bytes, void* stream);
int s6_q4_linear_workspace_size(int64_t rows, int64_t inner, int64_t outer, int64_t group, int x_dtype,
                                size_t* bytes);

/* s6_add_norm_fwd (s6_block.h) with its output in 8 bits: per row,
 *   r' = r + scale * gamma o x,  o = r' / sqrt(mean(r'^2) + eps) o weight,
 *   out_scale = max|o| / 448,  out = o / out_scale rounded to e4m3.
 * out: (rows, dim) bytes; out_scale: (rows) fp32.  o, out_scale and the quotient
 * are fp32, the quotient is rounded to e4m3 once; the mean is formed without
 * overflow and without loss of small squares.  A row whose largest |o| is below
 * 2^-100 is stored as zeros with out_scale 0; one that holds a value that is not
 * finite as NaN with out_scale NaN. */
int s6_add_norm_q8_fwd(int64_t rows, int64_t dim, int in_dtype, int res_dtype, const void* x, int64_t x_stride,
                       const void* residual, const float* weight, const float* gamma, float scale, float eps, void* out,
                       float* out_scale, void* residual_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* S6_Q4_H_ */
