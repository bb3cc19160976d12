/*
 * s6_block.h -- C ABI of libs6 for a selective state-space block with heads:
 * the multi-head selective scan (linear attention with a decay for each
 * head), its gradients and its single-token step, and the norms before and
 * after it.  AMD MI355X (gfx950).
 *
 * The status codes, in_dtype values, S6_DELTA_SOFTPLUS, the stream argument
 * and the rules for workspaces and pointers are those of s6.h: every call
 * only enqueues work, checks its arguments before any HIP call, allocates
 * nothing and keeps no state.  Values are not checked: NaN and infinities
 * propagate.
 *
 * The scan.  Heads h of P = headdim channels share one decay each; B and C are
 * shared by the heads of a group (head h belongs to group h / (heads/groups)).
 * Per sequence and head, with the state S (P x N, N = dstate) and the step
 *   s_t = delta_t + delta_bias, through softplus with S6_DELTA_SOFTPLUS
 *         (1 where delta is NULL):
 *   S_t = e^{s_t A} S_{t-1} + w_t x_t B_t^T,   w_t = s_t, or 1 with S6_UNIT_INPUT
 *   y_t = S_t C_t + D x_t
 * This is the recurrence of s6_scan_fwd with A[d, n] = A[head], many states
 * and the heads' B and C in groups; S6_UNIT_INPUT makes s_t A a plain log
 * decay of linear attention (keys B, queries C, values x), and a NULL delta
 * a fixed decay per head.  A sequence packed after another starts from an
 * empty state where s_t A = -infinity (or below about -104; such a decay is 0
 * and has no gradient).  Steps that large go with S6_UNIT_INPUT, since
 * otherwise they scale the sequence's first input as well.
 *
 * Layout: token-major, last index fastest.
 *   x, y, dy, dx : (batch, seqlen, heads, headdim)   delta : (batch, seqlen, heads)
 *   Bm, Cm : (batch, seqlen, groups, dstate)
 *   A, D, delta_bias : (heads) fp32     h0, h_last, h : (batch, heads, headdim, dstate) fp32
 * x, delta, Bm and Cm may be slices of wider rows: their batch and token
 * strides (elements) are given, the rows themselves are contiguous.  Every
 * other tensor is contiguous.  in_dtype is that of x, delta, Bm, Cm, y, dy and
 * the gradients dx, ddelta, dBm, dCm; parameters, states and their gradients
 * are fp32.
 * Sizes: heads a multiple of groups, 1 <= dstate <= 128, headdim >= 1; batch,
 * seqlen and heads may be 0 (no work; h_last is then h0 or zeros).
 *
 * Arithmetic: sums, states, decays and steps in fp32.  fp32 inputs: fp32
 * products.  bf16 inputs: bf16 matrix products with fp32 accumulation; the
 * products of inputs are exact; an fp32 factor enters in full in the states
 * (three bf16 parts) and in the gradients of steps and parameters, and as two bf16
 * parts (within 2^-17) in y, dx, dBm and dCm.  So all of these and ddelta meet one
 * rounding to bf16, that of the result.
 * A decay e^{c_t - c_s} between two tokens of a chunk is taken from running sums
 * held in two floats each: its relative error is about 2^-24 times its own
 * exponent, whatever decays lie before it (sequences packed closely one after
 * another lose nothing).  Repeated calls give identical bits.
 * An x that is not finite leaves its channel not finite from its token on; other
 * channels and earlier tokens keep their values.  In the backward such a value
 * may also reach the other tokens of its block of 128 (fp32: 64).
 */
#ifndef S6_BLOCK_H_
#define S6_BLOCK_H_

#include "s6.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flag of the heads entry points beside S6_DELTA_SOFTPLUS: the input term is
 * x B^T instead of s x B^T. */
#define S6_UNIT_INPUT 4

typedef struct {
  int64_t batch, seqlen, heads, headdim, groups, dstate;
  /* strides in elements; a row is heads*headdim (x), heads (delta) or
   * groups*dstate (Bm, Cm) contiguous elements */
  int64_t x_batch, x_token;
  int64_t delta_batch, delta_token;
  int64_t b_batch, b_token;
  int64_t c_batch, c_token;
} s6_heads_dims;

/* The scan of whole sequences.  delta, delta_bias, D, h0 and h_last are
 * nullable (delta_bias needs delta).  workspace:
 * s6_heads_scan_fwd_workspace_size bytes, 0 where the batch x heads fill the
 * GPU; few long rows are cut into segments. */
int s6_heads_scan_fwd(const s6_heads_dims* dims, int in_dtype, int flags, const void* x, const void* delta,
                      const float* delta_bias, const float* A, const void* Bm, const void* Cm, const float* D,
                      const float* h0, void* y, float* h_last, void* workspace, size_t workspace_bytes, void* stream);
int s6_heads_scan_fwd_workspace_size(const s6_heads_dims* dims, int in_dtype, size_t* bytes);

/* Gradients of <dy, y> + <dh_last, h_last> for s6_heads_scan_fwd with the
 * same inputs.  Required: dy, dx, dBm, dCm, dA, and ddelta where delta is
 * given.  Nullable: dh_last (zero), dD, dh0, ddelta_bias.  The states
 * entering each block of tokens and their adjoints are recomputed into the
 * workspace (s6_heads_scan_bwd_workspace_size bytes).  Sums over heads,
 * sequences and tokens are taken in a fixed order. */
int s6_heads_scan_bwd(const s6_heads_dims* dims, int in_dtype, int flags, const void* x, const void* delta,
                      const float* delta_bias, const float* A, const void* Bm, const void* Cm, const float* D,
                      const float* h0, const void* dy, const float* dh_last, void* dx, void* ddelta, float* dA,
                      void* dBm, void* dCm, float* dD, float* dh0, float* ddelta_bias, void* workspace,
                      size_t workspace_bytes, void* stream);
int s6_heads_scan_bwd_workspace_size(const s6_heads_dims* dims, int in_dtype, size_t* bytes);

/* One token for every sequence: h is advanced in place.  seqlen and the
 * token strides of dims are not read; x, y : (batch, heads, headdim), delta :
 * (batch, heads), Bm, Cm : (batch, groups, dstate), with the batch strides of
 * dims (y contiguous). */
int s6_heads_state_update(const s6_heads_dims* dims, int in_dtype, int flags, float* h, const void* x,
                          const void* delta, const float* delta_bias, const float* A, const void* Bm,
                          const void* Cm, const float* D, void* y, void* stream);

/* The norm before a block, with the residual add and scale of the block
 * before it: per row of dim elements,
 *   r' = r + scale * gamma o x        (r absent where residual is NULL, gamma = 1 where NULL)
 *   out = r' / sqrt(mean(r'^2) + eps) o weight
 * x: rows of x_stride elements; residual, out, residual_out contiguous.
 * in_dtype: x, out, dout, dx.  res_dtype: residual, residual_out and their
 * gradients; S6_F32, or in_dtype.  weight, gamma: (dim) fp32.  out is taken
 * from r' before its rounding to res_dtype.  residual_out may be the
 * residual's own buffer. */
int s6_add_norm_fwd(int64_t rows, int64_t dim, int in_dtype, int res_dtype, const void* x, int64_t x_stride,
                    const void* residual, const float* weight, const float* gamma, float scale, float eps, void* out,
                    void* residual_out, void* stream);

/* Gradients of <dout, out> + <dresidual_out, residual_out>, from the stored
 * residual_out: dresidual = dresidual_out (0 where NULL) + the norm's part;
 * dx = scale * gamma o dresidual; dweight; dgamma = scale * sum over rows of
 * x o dresidual (needs x; required where gamma is given).  dx, dresidual and
 * dweight are nullable (not all three).  workspace:
 * s6_add_norm_bwd_workspace_size bytes (the column sums' parts). */
int s6_add_norm_bwd(int64_t rows, int64_t dim, int in_dtype, int res_dtype, const void* dout,
                    const void* dresidual_out, const void* residual_out, const void* x, int64_t x_stride,
                    const float* weight, const float* gamma, float scale, float eps, void* dx, void* dresidual,
                    float* dweight, float* dgamma, void* workspace, size_t workspace_bytes, void* stream);
int s6_add_norm_bwd_workspace_size(int64_t rows, int64_t dim, size_t* bytes);

/* The norm after the scan, with its gate: per row and group of dim/groups
 * elements,
 *   out = rms(y o SiLU(z)) o weight,  or  rms(y) o weight o SiLU(z) with S6_GATE_AFTER,
 * rms(u) = u / sqrt(mean(u^2) + eps).  y, z: rows of y_stride, z_stride
 * elements; z is nullable (no gate).  weight: (dim) fp32. */
#define S6_GATE_AFTER 8
int s6_gated_norm_fwd(int64_t rows, int64_t dim, int64_t groups, int in_dtype, int flags, const void* y,
                      int64_t y_stride, const void* z, int64_t z_stride, const float* weight, float eps, void* out,
                      void* stream);

/* Its gradients: dy and (where z is given) dz, contiguous and required;
 * dweight nullable.  workspace: s6_gated_norm_bwd_workspace_size bytes. */
int s6_gated_norm_bwd(int64_t rows, int64_t dim, int64_t groups, int in_dtype, int flags, const void* dout,
                      const void* y, int64_t y_stride, const void* z, int64_t z_stride, const float* weight, float eps,
                      void* dy, void* dz, float* dweight, void* workspace, size_t workspace_bytes, void* stream);
int s6_gated_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* S6_BLOCK_H_ */
