/*
 * language.h -- C ABI of the operators around the layers of a language model: the
 * scaled embedding, the GroupNorm with its gate, products with bias, activation and
 * residual, the selection of beams and the reordering of their states.  Part of the
 * same library as retention.h, whose status codes, dtypes, error reporting
 * (retention_last_error) and stream rules hold here too.
 *
 * Conventions beside those of retention.h:
 *   - Activations are token-major unless a call says otherwise.  A row stride `ld`
 *     counts elements between a row and the next.  Tensors without one are dense.
 *   - Pointers need the alignment of their elements (4 bytes for fp32 and int32, 2
 *     for bf16); workspaces 16 bytes.
 *   - Accumulators and statistics are fp32 or wider; results are rounded once to
 *     out_dtype.  Sums run in a fixed order: the same inputs give the same bits.
 *   - Outputs must not overlap inputs, the workspace or each other, except where
 *     a call says so.  Calls sharing a workspace must not overlap in time; two
 *     captured graphs that may run at once need two workspaces.
 *   - A workspace query's size is for the sizes it was asked for, whatever the call's other
 *     arguments are.  It does not grow with every size: a caller with calls of several sizes
 *     takes the largest of their answers (a product of fewer rows may be cut into more parts).
 *   - A call without rows (n, M, B or L of 0 where the call allows it) launches
 *     nothing, or writes the zeros that an empty sum is.
 */
#ifndef LANGUAGE_H_
#define LANGUAGE_H_

#include "retention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Library limits (UNSUPPORTED beyond them). */
#define LANGUAGE_MAX_TOKENS (1LL << 28)   /* n of the embedding, B * L of the norm, M of linear */
#define LANGUAGE_MAX_VOCAB (1 << 24)      /* V */
#define LANGUAGE_MAX_CHANNELS (1 << 20)   /* D of the embedding, H * W of the norm */
#define LANGUAGE_MAX_ELEMENTS (1LL << 37) /* n * D, V * D, B * L * H * W of one call */
#define LANGUAGE_MAX_NORM_WIDTH RETENTION_MAX_DV /* W of the norm */
#define LANGUAGE_MAX_FEATURES (1 << 22)   /* N and K of linear */
#define LANGUAGE_MAX_BEAMS 64             /* W and K of beam_select, W of beam_reorder */
#define LANGUAGE_MAX_BEAM_ROWS (1 << 23)  /* B * W of beam_select */
#define LANGUAGE_MAX_BEAM_LISTS 2048      /* W * ceil(V / 2048) of beam_select */
#define LANGUAGE_MAX_REORDERED 64         /* tensors of one beam_reorder */
#define LANGUAGE_MAX_REORDER_BATCH 65535  /* B of beam_reorder */

/*
 * Scaled lookup: out[t] = scale table[ids[t]], and zero where ids[t] is outside 0..V-1
 * (padding, by convention -1).
 *   ids   : DEVICE int32 [n]
 *   table : [V, D] in_dtype        out : [n, D] out_dtype
 */
ret_status_t embedding(const int *ids, const void *table, void *out, long long n, int V, int D,
                       float scale, ret_dtype_t in_dtype, ret_dtype_t out_dtype, void *hip_stream);

/*
 * Its gradient: dtable[v] = scale sum_{t : ids[t] = v} d_o[t], the tokens in their order, for
 * every v (zero for one that no token names).  Ids outside 0..V-1 have none.
 *   d_o : [n, D] in_dtype, row stride o_ld        dtable : [V, D] out_dtype
 */
size_t embedding_bwd_workspace_bytes(long long n, int V, int D);
ret_status_t embedding_bwd(const int *ids, const void *d_o, void *dtable, long long n, int V, int D,
                           long long o_ld, float scale, ret_dtype_t in_dtype, ret_dtype_t out_dtype,
                           void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * GroupNorm of every token and head with a gate, the end of a gated retention
 * ("Retentive Network" paper summary, Sec. 2.2):
 *   xh = (x - mean) / sqrt(var + eps)   over the head's W channels, biased variance
 *   n  = weight xh + bias               (weight NULL: 1; bias NULL: 0)
 *   out = n act(gate), act = silu or the identity; without a gate act(n)
 *   x    : in_dtype, element (b, h, t, c) at b x_sb + h x_sh + t x_sl + c: a retention's
 *          [B, H, L, W], or the heads of a token-major row
 *   gate : [B, L, H W] in_dtype, row stride gate_ld (sequence b from b L gate_ld), or NULL
 *   weight, bias : [H W] fp32 or NULL
 *   out  : [B, L, H W] out_dtype
 *   lengths : DEVICE int32 [B] or NULL.  Sequence b ends after min(max(lengths[b], 0), L)
 *             tokens: later rows are neither read nor written.
 * eps is finite and above 0.
 */
ret_status_t group_norm_gate(const void *x, const void *gate, const float *weight,
                             const float *bias, void *out, const int *lengths, int B, int H, int L,
                             int W, long long x_sb, long long x_sh, long long x_sl,
                             long long gate_ld, int silu, float eps, ret_dtype_t in_dtype,
                             ret_dtype_t out_dtype, void *hip_stream);

/*
 * Its gradients for d_o ([B, L, H W] in_dtype, dense).  The statistics are computed again
 * from x.  With dn the gradient of n, r = 1 / sqrt(var + eps):
 *   dx = r (weight dn - mean(weight dn) - xh mean(weight dn xh))    dgate = d_o n act'(gate)
 *   dweight = sum dn xh      dbias = sum dn        (over all tokens)
 *   dx : [B, H, L, W] out_dtype, dense      dgate : [B, L, H W] out_dtype, dense (NULL
 *   exactly where gate is)      dweight, dbias : [H W] fp32, or NULL where not wanted
 * Rows behind a sequence's end have zero gradients.
 */
size_t group_norm_gate_bwd_workspace_bytes(int B, int H, int L, int W);
ret_status_t group_norm_gate_bwd(const void *x, const void *gate, const float *weight,
                                 const float *bias, const void *d_o, const int *lengths, void *dx,
                                 void *dgate, float *dweight, float *dbias, int B, int H, int L,
                                 int W, long long x_sb, long long x_sh, long long x_sl,
                                 long long gate_ld, int silu, float eps, ret_dtype_t in_dtype,
                                 ret_dtype_t out_dtype, void *workspace, size_t workspace_bytes,
                                 void *hip_stream);

/*
 * Products with bias, activation and residual, bf16 operands:
 *   z = x w^T + bias,    out = act(z) + residual
 *   x : [M, K] bf16, row stride x_ld      w : [N, K] bf16      bias : [N] bf16 or NULL
 *   residual : [M, N] residual_dtype, dense, or NULL; out may be residual (one dtype)
 *   out : [M, N] out_dtype                pre : [M, N] bf16 or NULL: z, for the gradients
 *   act : LINEAR_ACT_*; gelu(z) = z Phi(z), silu(z) = z / (1 + e^-z).  Before out's rounding they
 *         are good to (10 + 2 z^2) and (8 + 2 |z|) 2^-24 of their value, gelu for a bf16 out to
 *         5.7e-6 (z >= -6; behind that it goes to zero and is off by less than 1e-13)
 *   workspace : linear_workspace_bytes() bytes (NULL where that is 0)
 */
enum { LINEAR_ACT_NONE = 0, LINEAR_ACT_GELU = 1, LINEAR_ACT_SILU = 2 };
size_t linear_workspace_bytes(long long M, int N, int K);
ret_status_t linear(const void *x, const void *w, const void *bias, const void *residual, void *out,
                    void *pre, long long M, int N, int K, long long x_ld, int act,
                    ret_dtype_t residual_dtype, ret_dtype_t out_dtype, void *workspace,
                    size_t workspace_bytes, void *hip_stream);

/*
 * Its gradients for d_o ([M, N] bf16, dense) and the forward call's pre:
 *   dz = d_o act'(pre)     dx = dz w     dw = dz^T x     dbias = sum_m dz
 * (the residual's gradient is d_o; gelu' is good to 3.2e-8, absolute).  dz is rounded to bf16
 * for the two products, as their operands are bf16; dbias sums it unrounded.
 *   pre : [M, N] bf16 (not read without an activation)
 *   dx : [M, K], dw : [N, K] out_dtype      dbias : [N] fp32     each NULL where not wanted
 */
size_t linear_bwd_workspace_bytes(long long M, int N, int K);
ret_status_t linear_bwd(const void *x, const void *w, const void *d_o, const void *pre, void *dx,
                        void *dw, float *dbias, long long M, int N, int K, long long x_ld, int act,
                        ret_dtype_t out_dtype, void *workspace, size_t workspace_bytes,
                        void *hip_stream);

/*
 * One step of a beam search: of the W V continuations of a request the K best by
 *   scores[b, w] + log_softmax(logits[b, w])[v]
 * in descending order, ties to the lowest w V + v (within a beam by logit, then by v).
 *   logits : [B, W, V] dtype, row stride logits_ld (beam w of request b at row b W + w)
 *   scores : [B, W] fp32      ended : bytes [B, W] or NULL: a beam with a byte other than
 *            zero offers token eos at its own score and nothing else
 *   tokens, parents : int32 [B, K]     out_scores : fp32 [B, K]
 *   workspace : beam_select_workspace_bytes() bytes (NULL where that is 0)
 * Scores, score + (logit - s), are compared in 64 bits.  s is the row's largest logit +
 * log(1 + sum of e^-d) over the others, each d below it; an exponential in this sum is good to
 * (16 + 3 d) 2^-24 of itself, the logarithm and what follows are in 64 bits.
 * A continuation without a finite score (a logit of -inf, the other tokens of an ended beam;
 * all of a beam whose score is not finite, or whose logits hold a NaN or +inf or nothing above
 * -inf) counts as -inf: it is taken after all others, by index.  K is at most W V.
 */
size_t beam_select_workspace_bytes(int B, int W, int V, int K);
ret_status_t beam_select(const void *logits, const float *scores, const unsigned char *ended,
                         int *tokens, int *parents, float *out_scores, int B, int W, int V, int K,
                         long long logits_ld, int eos, ret_dtype_t dtype, void *workspace,
                         size_t workspace_bytes, void *hip_stream);

/*
 * State of a search following its beams, in place: states[i][b, w] <- states[i][b, parents[b, w]]
 * for `count` tensors of [B, W] beams of bytes[i] bytes each (any type, dense).
 *   states, bytes : HOST arrays of `count` DEVICE pointers and sizes
 *   parents : DEVICE int32 [B, W]; a beam whose parent is outside 0..W-1 keeps its own
 * The tensors must not overlap each other or parents.
 */
ret_status_t beam_reorder(void *const *states, const long long *bytes, int count,
                          const int *parents, int B, int W, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* LANGUAGE_H_ */
