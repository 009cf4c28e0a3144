/*
 * recurrent.h -- C ABI of the recurrent-layer operators next to retention: the
 * selective state space scan, its short causal convolution and the products with
 * 4-bit weights.  Part of the same library as retention.h, whose status codes,
 * dtypes, error reporting (retention_last_error) and stream rules hold here too.
 *
 * Where retention decays its state by one constant per head, the selective scan
 * decays every state by its own rate times a time step that the token chooses:
 *   dt_t  = softplus(delta_t + delta_bias)            (or without softplus)
 *   h_t   = exp(dt_t A) h_{t-1} + dt_t u_t B_t        (per channel d, state n)
 *   y_t   = C_t . h_t + D u_t,     out_t = y_t silu(z_t),   silu(x) = x / (1 + e^-x)
 *
 * Conventions beside those of retention.h:
 *   - Activations are token-major, [B, L, ...].  Where a call takes a row stride
 *     `ld` (elements between a token and the next), the sequence b starts at
 *     element b * L * ld, so that slices of one projection's rows are read in
 *     place.  Tensors without one are dense.
 *   - Pointers need the alignment of their elements (4 bytes for fp32, 2 for
 *     bf16); aligned, 4-divisible rows are read with wider loads.
 *   - lengths: DEVICE int32 [B] or NULL.  Sequence b ends after
 *     min(max(lengths[b], 0), L) tokens: later rows are neither read nor (in a
 *     forward call) written, gradients there are zero, and the final state is the
 *     one after the last token.
 *   - Accumulators and states are fp32; results are rounded once to out_dtype.
 *   - L == 0: nothing to compute; a final state is the initial one (or zero).
 *   - A workspace query's size serves every call of at most that L with the same
 *     other sizes (not of other B: more sequences can need less).
 *   - Outputs must not overlap inputs, the workspace or each other, except where
 *     a call says so.  Calls sharing a workspace must not overlap in time; two
 *     captured graphs that may run at once need two workspaces.
 */
#ifndef RECURRENT_H_
#define RECURRENT_H_

#include "retention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Library limits (UNSUPPORTED beyond them). */
#define RECURRENT_MAX_STATE 64             /* N of the scan */
#define RECURRENT_MAX_TAPS 8               /* K of the convolution */
#define RECURRENT_MAX_TOKENS (1LL << 28)   /* B * L of one call */
#define RECURRENT_MAX_ELEMENTS (1LL << 37) /* B * L * D, B * L * G * N of one call */
#define RECURRENT_MAX_CHANNELS (1LL << 20) /* D */
#define RECURRENT_MAX_STATES (1LL << 31)   /* B * D * N, B * D * K of one call */
/* Beside them, B * G * ceil(D / G / 16) of a scan is below 2^24, and N and K of
 * linear_w4 at most 2^26. */

/*
 * The scan over L tokens.
 *   u, delta, z : [B, L, D] in_dtype (z NULL: no gate)  row strides u_ld, delta_ld, z_ld
 *   Bm, Cm      : [B, L, G, N] in_dtype, row strides b_ld, c_ld; channel d reads group
 *                 d / (D / G); G divides D
 *   A           : [D, N] fp32, meant to be at most 0 (where it is not, the products of
 *                 exp(dt A) along the call have to stay finite); -inf decays at once
 *   D_skip, delta_bias : [D] fp32 or NULL
 *   out         : [B, L, D] out_dtype, dense
 *   state_in    : [B, D, N] fp32 state before token 0, or NULL for zeros
 *   state_out   : [B, D, N] fp32 state after the last token, or NULL; may be state_in
 *   workspace   : selective_scan_workspace_bytes() bytes (NULL where that is 0)
 */
size_t selective_scan_workspace_bytes(int B, int L, int D, int N, int G);
ret_status_t selective_scan(const void *u, const void *delta, const float *A, const void *Bm,
                            const void *Cm, const float *D_skip, const void *z,
                            const float *delta_bias, void *out, const int *lengths,
                            const float *state_in, float *state_out, int B, int L, int D, int N,
                            int G, long long u_ld, long long delta_ld, long long z_ld,
                            long long b_ld, long long c_ld, int delta_softplus,
                            ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *workspace,
                            size_t workspace_bytes, void *hip_stream);

/*
 * Gradients of the scan for the output gradient d_o ([B, L, D] in_dtype, dense) and
 * the final state's gradient d_state_out ([B, D, N] fp32, or NULL for zero).  With
 * dy = d_o silu(z) and g_t = C_t dy_t + exp(dt_{t+1} A) g_{t+1} (d_state_out behind
 * the last token):
 *   dB_t = sum_d g_t dt_t u_t          dC_t = sum_d dy_t h_t      (over the group's channels)
 *   ddt_t = sum_n g_t (A exp(dt_t A) h_{t-1} + u_t B_t),  ddelta = ddt softplus'
 *   du_t = dt_t sum_n g_t B_t + D dy_t       dz_t = d_o y_t silu'(z_t)
 *   dA = sum_t g_t dt_t exp(dt_t A) h_{t-1}   dD = sum_t dy_t u_t   ddelta_bias = sum_t ddelta_t
 *   d_state_in = exp(dt_0 A) g_0
 * The states are computed again from the inputs; nothing of the forward call is kept.
 * The workspace holds a state every 16 tokens (N <= 16), 8 (N <= 32) or 4: some 4 B L D N / 16,
 * / 8 or / 4 bytes, 9.9 GB at B 8, L 4096, D 4096, N 64.  A token whose time step softplus
 * makes 0 has ddelta 0, whatever the rates.
 *   du, ddelta, dz : [B, L, D] out_dtype, dense (dz NULL exactly where z is)
 *   dB, dC : [B, L, G, N] out_dtype, dense
 *   dA : [D, N] fp32    dD, ddelta_bias : [D] fp32, or NULL where not wanted
 *   d_state_in : [B, D, N] fp32, or NULL
 * Sums run in a fixed order: the same inputs give the same bits.
 */
size_t selective_scan_bwd_workspace_bytes(int B, int L, int D, int N, int G);
ret_status_t selective_scan_bwd(const void *u, const void *delta, const float *A, const void *Bm,
                                const void *Cm, const float *D_skip, const void *z,
                                const float *delta_bias, const void *d_o, const int *lengths,
                                const float *state_in, const float *d_state_out, void *du,
                                void *ddelta, float *dA, void *dB, void *dC, float *dD, void *dz,
                                float *ddelta_bias, float *d_state_in, int B, int L, int D, int N,
                                int G, long long u_ld, long long delta_ld, long long z_ld,
                                long long b_ld, long long c_ld, int delta_softplus,
                                ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *workspace,
                                size_t workspace_bytes, void *hip_stream);

/*
 * One token of the scan for B sequences; state [B, D, N] fp32 is updated in place.
 *   u, delta, z : [B, D]   Bm, Cm : [B, G, N]   (row strides as above, a row a sequence)
 *   out : [B, D] out_dtype, dense
 */
ret_status_t selective_scan_step(const void *u, const void *delta, const float *A, const void *Bm,
                                 const void *Cm, const float *D_skip, const void *z,
                                 const float *delta_bias, void *out, float *state, int B, int D,
                                 int N, int G, long long u_ld, long long delta_ld, long long z_ld,
                                 long long b_ld, long long c_ld, int delta_softplus,
                                 ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *hip_stream);

/*
 * Short causal depthwise convolution, the one in front of the scan:
 *   c_t = act(bias + sum_j w_j x_{t-K+1+j}),   act = silu or the identity
 *   x : [B, L, D] (row stride x_ld)   w : [D, K], 2 <= K <= RECURRENT_MAX_TAPS
 *   bias : [D] or NULL       out : [B, L, D] dense         (all of `dtype`)
 *   state_in  : [B, K-1, D] dtype, the inputs before token 0, oldest first; NULL: zeros
 *   state_out : [B, K-1, D] dtype, the last K-1 inputs, or NULL; not state_in
 */
ret_status_t causal_conv1d(const void *x, const void *w, const void *bias, void *out,
                           const int *lengths, const void *state_in, void *state_out, int B, int L,
                           int D, int K, long long x_ld, int silu, ret_dtype_t dtype,
                           void *hip_stream);

/*
 * Its gradients for d_o [B, L, D] (dense) and d_state_out [B, K-1, D] (or NULL), all
 * of `dtype`: dx [B, L, D] dtype, dw [D, K] fp32, dbias [D] fp32 or NULL, d_state_in
 * [B, K-1, D] dtype or NULL.  Sums run in a fixed order.
 */
size_t causal_conv1d_bwd_workspace_bytes(int B, int L, int D, int K);
ret_status_t causal_conv1d_bwd(const void *x, const void *w, const void *bias, const void *d_o,
                               const int *lengths, const void *state_in, const void *d_state_out,
                               void *dx, float *dw, float *dbias, void *d_state_in, int B, int L,
                               int D, int K, long long x_ld, int silu, ret_dtype_t dtype,
                               void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * One token of the convolution for B sequences: x [B, D] (row stride x_ld), out [B, D];
 * state [B, K-1, D] is shifted by one token in place.
 */
ret_status_t causal_conv1d_step(const void *x, const void *w, const void *bias, void *out,
                                void *state, int B, int D, int K, long long x_ld, int silu,
                                ret_dtype_t dtype, void *hip_stream);

/*
 * Products with 4-bit weights for few tokens: out = x W^T,
 *   W[n, k] = (q[n, k] - zero[n, k / group]) scale[n, k / group]
 *   x : [M, K] bf16 (row stride x_ld)        out : [M, N] bf16 or fp32, dense
 *   q : [N, K / 2] bytes, element 2 i in the low half of byte i, 2 i + 1 in the high one
 *   scale : [N, K / group] bf16     zero : [N, K / group] bytes in 0..15, or NULL for 8
 * group is 32, 64 or a multiple of 128 and divides K; q is 16-byte aligned.  The products
 * are exact (integers against bf16), sums fp32, each group's sum scaled in fp32.  The
 * zero points are taken out of sums of x (16 + q), so x has to be finite and below 2^118
 * in magnitude: an infinity gives NaN.  Made for few tokens; any M is computed.
 */
ret_status_t linear_w4(const void *x, const void *q, const void *scale, const void *zero, void *out,
                       int M, int N, int K, int group, long long x_ld, ret_dtype_t out_dtype,
                       void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RECURRENT_H_ */
