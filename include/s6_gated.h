/*
 * s6_gated.h -- C ABI of libs6 for a gated linear recurrence: one state per
 * channel whose decay and input are gated anew at every token, its gradients
 * and its single-token step.  AMD MI355X (gfx950).
 *
 * The status codes, in_dtype values, the stream argument and the rules for
 * workspaces and pointers are those of s6.h: every call only enqueues work,
 * checks its arguments before any HIP call, allocates nothing and keeps no
 * state.  Values are not checked: NaN and infinities propagate.
 *
 * Per sequence, channel and token t, with
 *   r_t = sigmoid(gate_a_t + bias_a),  i_t = sigmoid(gate_x_t + bias_x)  (1 where gate_x is NULL):
 *   a_t = e^{A r_t},  b_t = sqrt(1 - a_t^2), or 1 with S6_UNIT_INPUT
 *   h_t = a_t h_{t-1} + b_t i_t x_t,   y_t = h_t
 * A is at most 0 and finite.  A token whose byte in starts is not 0 begins a
 * sequence of its own: there a_t = 0 and b_t = 1, whatever the state before it
 * and gate_a hold, and nothing flows back over it.
 *
 * Layout: token-major, last index fastest.
 *   x, gate_a, gate_x, y, dy, dx, dgate_a, dgate_x : (batch, seqlen, dim)
 *   starts : (batch, seqlen) bytes       A, bias_a, bias_x : (dim) fp32
 *   h0, h_last, h : (batch, dim) fp32    states : (batch, ceil(seqlen / 128), dim) fp32
 * x, gate_a and gate_x may be slices of wider rows: their batch and token
 * strides (elements) are given, the rows themselves are contiguous.  Every
 * other tensor is contiguous.  in_dtype is that of x, the gates, y, dy and the
 * gradients of x and the gates; all else is fp32.
 * batch, seqlen and dim may be 0 (no work; h_last is then h0 or zeros).  dim
 * and the token strides are at most 2^24, and there are fewer than about 2^31
 * tiles of 128 tokens by 64 channels.
 *
 * Arithmetic: gates, decays, states, adjoints and sums in fp32; y and the
 * gradients in in_dtype meet one rounding, that of the result.  1 - a^2 keeps
 * its relative accuracy as a approaches 1, until r or 1 - a^2 itself is below
 * 2^-126 (a gate below about -87): there b may be 0 (off by at most 2^-63
 * sqrt(1 + 2 |A|)), and where it is, its share of the gradients of the gate
 * and of A is 0.
 * 1 - r and 1 - i, factors of the gates' gradients, keep theirs as r and i
 * approach 1, until they are below 2^-126 (a gate above about 87) and may be 0.
 * Repeated calls give identical bits.
 */
#ifndef S6_GATED_H_
#define S6_GATED_H_

#include "s6.h"

#ifdef __cplusplus
extern "C" {
#endif

#ifndef S6_UNIT_INPUT
#define S6_UNIT_INPUT 4 /* as in s6_block.h: no factor on the input term */
#endif

#define S6_GATED_TOKENS 128 /* tokens from one of `states` to the next */

typedef struct {
  int64_t batch, seqlen, dim;
  /* strides in elements; a row is dim contiguous elements */
  int64_t x_batch, x_token;
  int64_t a_batch, a_token; /* gate_a */
  int64_t g_batch, g_token; /* gate_x */
} s6_gated_dims;

/* The recurrence over whole sequences.  gate_x, bias_a, bias_x (needs
 * gate_x), starts, h0, h_last and states are nullable.  states receives the
 * state entering every S6_GATED_TOKENS tokens, which the backward can take.
 * workspace: s6_gated_scan_fwd_workspace_size bytes (0 for sequences of at
 * most S6_GATED_TOKENS). */
int s6_gated_scan_fwd(const s6_gated_dims* dims, int in_dtype, int flags, const void* x, const void* gate_a,
                      const float* bias_a, const void* gate_x, const float* bias_x, const float* A,
                      const uint8_t* starts, const float* h0, void* y, float* h_last, float* states, void* workspace,
                      size_t workspace_bytes, void* stream);
int s6_gated_scan_fwd_workspace_size(const s6_gated_dims* dims, size_t* bytes);

/* Gradients of <dy, y> + <dh_last, h_last> for s6_gated_scan_fwd with the
 * same inputs.  states: those of the forward, or NULL (then formed again in
 * the workspace).  Required: dy, dx, dgate_a, and dgate_x where gate_x is
 * given.  Nullable: dh_last (zero), dA, dbias_a, dbias_x (needs gate_x), dh0.
 * Sums over sequences and tokens are taken in a fixed order.  workspace:
 * s6_gated_scan_bwd_workspace_size bytes; has_states: whether states will be
 * given. */
int s6_gated_scan_bwd(const s6_gated_dims* dims, int in_dtype, int flags, const void* x, const void* gate_a,
                      const float* bias_a, const void* gate_x, const float* bias_x, const float* A,
                      const uint8_t* starts, const float* h0, const float* states, const void* dy,
                      const float* dh_last, void* dx, void* dgate_a, void* dgate_x, float* dA, float* dbias_a,
                      float* dbias_x, float* dh0, void* workspace, size_t workspace_bytes, void* stream);
int s6_gated_scan_bwd_workspace_size(const s6_gated_dims* dims, int has_states, size_t* bytes);

/* One token for every sequence: h is advanced in place.  seqlen and the token
 * strides of dims are not read; x, gate_a, gate_x, y : (batch, dim), with the
 * batch strides of dims (y contiguous). */
int s6_gated_state_update(const s6_gated_dims* dims, int in_dtype, int flags, float* h, const void* x,
                          const void* gate_a, const float* bias_a, const void* gate_x, const float* bias_x,
                          const float* A, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* S6_GATED_H_ */
