/*
 * liger_layer.h -- C-ABI of libliger.so, third part: the operators of a decoder
 * layer with layer norms and biased projections, and of scoring a head's logits,
 * beside those of liger.h and liger_train.h, whose conventions (status codes,
 * dtypes, alignment, ownership of buffers, streams, threads) hold here too.
 *
 *   - layer norm, forward and backward;
 *   - the projection with bias, activation and residual sum in its epilogue,
 *     forward and backward;
 *   - rotary positions on the first part of each head, with frequencies scaled
 *     for long contexts, forward and backward;
 *   - log-probabilities of given tokens from logits, with the entropy, the top
 *     alternatives and the gradient of the logits.
 *
 * Every call queues work only, waits for nothing on the host, allocates
 * nothing, and can be captured in a CUDA graph after a first call on the device.
 * Results are the same from run to run on one device (sums in a fixed order,
 * no atomics).  A bounded wait that expires in a kernel (see liger.h) leaves
 * NaN in the outputs that it did not finish; the layer norm's is recorded with
 * RMSNorm's, the projection's with FusedLinearSwiGLU's and the rotation's with
 * RoPE's, and liger_device_status names both.
 */
#ifndef LIGER_LAYER_H
#define LIGER_LAYER_H

#include "liger.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------- layer norm
 * Forward, per row t of x [rows, cols]:
 *     mean = sum_j x[t,j] / cols
 *     rstd = 1 / sqrt(sum_j (x[t,j] - mean)^2 / cols + eps)
 *     y[t,j] = (x[t,j] - mean) rstd w[j] + b[j]
 *   w, b [cols], each may be NULL (1, 0).  mean, rstd: float [rows], each may
 *   be NULL (not stored).  The variance is the mean of squared differences
 *   (not E x^2 - mean^2), all in fp32; y is rounded once.
 *   x, w, b, y 16-byte aligned; y may be x; no other overlap.  eps >= 0.
 *   A row that holds an infinity or NaN is NaN. */
int liger_layernorm_fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd, int64_t rows,
                        int64_t cols, float eps, int dtype, void* stream);

/* Bytes of workspace liger_layernorm_bwd needs (fp32 partial sums of the two
 * weight gradients): an upper bound valid on any device,
 * 2 * min(rows, 1024) * cols * 4. */
size_t liger_layernorm_bwd_workspace(int64_t rows, int64_t cols);

/* Backward, with mean and rstd as the forward wrote them:
 *     g = dy w,  xh = (x - mean) rstd
 *     dx = dres + rstd (g - sum_j g / cols - xh sum_j g xh / cols)
 *     dw = sum_t dy xh,  db = sum_t dy
 *   dres [rows, cols] or NULL (0): the gradient of x that does not come through
 *   the norm (the residual stream's).  w NULL: 1.  dw, db [cols], each may be
 *   NULL (not wanted).  The sums over rows are fp32, in a fixed order.
 *   dx may be dy or dres; no other overlap.  rows = 0 writes zeros to dw, db.
 *   ws: at least liger_layernorm_bwd_workspace bytes, 16-byte aligned. */
int liger_layernorm_bwd(const void* dy, const void* dres, const void* x, const void* w, const float* mean,
                        const float* rstd, void* dx, void* dw, void* db, void* ws, size_t ws_bytes, int64_t rows,
                        int64_t cols, int dtype, void* stream);

/* ------------------- projection with bias, activation and residual
 * X [T, H], W [N, H], bias [N] or NULL, residual [T, N] or NULL, Y [T, N]:
 *     P = X W^T + bias,  Y = act(P) + residual
 *   act: 0 none, 1 relu, 2 gelu (p Phi(p), with erf), 3 gelu with tanh
 *   (p (1 + tanh(sqrt(2/pi) (p + 0.044715 p^3))) / 2), 4 silu (p sigmoid(p)).
 *   The sums are fp32, Y is rounded once from act(P) + residual.
 *   pre [T, N] or NULL: P kept for the backward of the activation, IEEE half
 *   precision for bf16 tensors (8 times finer than bf16 down to 2^-14, in steps of
 *   2^-24 below; values past its range are kept as its largest, where every
 *   derivative here has its limit, and with relu, whose derivative their sign
 *   decides, positive ones below 2^-24 as that), fp32 for fp32.
 *   All tensors 16-byte aligned.  residual may be Y; no other overlap.
 *   bf16 with H and N multiples of 8, 64 or more, runs on the tensor cores;
 *   fp32, and bf16 of other sizes, in fp32 FMA.  T = 0 does nothing. */
#define LIGER_ACT_NONE 0
#define LIGER_ACT_RELU 1
#define LIGER_ACT_GELU 2
#define LIGER_ACT_GELU_TANH 3
#define LIGER_ACT_SILU 4
int liger_linear_act_fwd(const void* X, const void* W, const void* bias, const void* residual, void* Y, void* pre,
                         int64_t T, int64_t H, int64_t N, int act, int dtype, void* stream);

/* Bytes of workspace liger_linear_act_bwd needs: dP where there is an
 * activation, and fp32 partial sums of db of many tokens; 0 for arguments out of
 * range. */
size_t liger_linear_act_bwd_workspace(int64_t T, int64_t H, int64_t N, int act, int dtype);

/* Backward, from dY [T, N] and pre as the forward kept it (not read, may be
 * NULL, when act is 0):
 *     dP = dY act'(P),  dX = dP W,  dW = dP^T X,  db = sum_t dP
 *   dX [T, H], dW [N, H], db [N] in dtype, each may be NULL (not wanted, and
 *   then W or X is not read).  relu'(0) = 0.  The gradient of the residual is dY.
 *   On the tensor cores dP is rounded to bf16 once, as an operand of both
 *   products (with act = 0 it is dY as it stands); db is summed in fp32 from
 *   the unrounded dP.  No output overlaps another tensor; dX is written twice
 *   (sums of dW may stand in it first).
 *   T = 0 writes zeros to dW and db.
 *   ws: at least liger_linear_act_bwd_workspace bytes, 256-byte aligned (NULL
 *   where that is 0). */
int liger_linear_act_bwd(const void* dY, const void* X, const void* W, const void* pre, void* dX, void* dW, void* db,
                         void* ws, size_t ws_bytes, int64_t T, int64_t H, int64_t N, int act, int dtype, void* stream);

/* --------------------------- rotary positions, partial and scaled
 * q [batch, seq, n_q_heads, head_dim], k [batch, seq, n_k_heads, head_dim] as
 * views: element [b, s, h, j] stands q_token_stride (b seq + s) + head_dim h +
 * j elements behind the pointer (k, and the outputs, by their own strides, each
 * at least heads * head_dim).  The first rotary_dim elements R of each head are
 * rotated by the token's position p (pos int32 [batch, seq], any value, or NULL:
 * p = s), pair i < R/2 by the angle p f_i, cos and sin both times m:
 *     a' = m (a cos - b sin),  b' = m (b cos + a sin)
 *   pairing 0: (a, b) = elements (i, i + R/2); 1: (2i, 2i + 1).  The other
 *   elements are copied (in place: left as they are).
 *   f_i by `scaling`, with f0_i = theta^(-2i/R), F = factor:
 *     0 none:   f0_i
 *     1 linear: f0_i / F
 *     2 ntk:    theta' = theta F^(R/(R-2)) in place of theta (R = 2: theta)
 *     3 bands:  with n_i = orig_len f0_i / 2 pi (turns over the original
 *               context) and c = clamp((n_i - low) / (high - low), 0, 1):
 *               f0_i (c + (1 - c) / F)                      (low < high)
 *     4 yarn:   with d(n) = R ln(orig_len / (2 pi n)) / (2 ln theta),
 *               l = max(floor(d(high)), 0), u = min(ceil(d(low)), R - 1),
 *               c = clamp((i - l) / max(u - l, 0.001), 0, 1):
 *               f0_i (1 - c + c / F)             (low, high > 0; theta > 1)
 *   m = attn_factor, or if that is 0: 0.1 ln F + 1 for yarn with F > 1, else 1.
 *   The angle is formed and reduced in double precision.
 * _bwd is the transpose (the angle negated, the same m): from the gradients of
 * the outputs to those of q and k.
 *   q_out may be q, and k_out k, with equal strides; no other overlap.  Head
 *   counts may be 0 (then the pointers are not looked at).  rotary_dim even, 2
 *   to head_dim <= 512; factor > 0; orig_len > 0 for 3 and 4.  Pointers aligned
 *   to the element size. */
#define LIGER_ROPE_NONE 0
#define LIGER_ROPE_LINEAR 1
#define LIGER_ROPE_NTK 2
#define LIGER_ROPE_BANDS 3
#define LIGER_ROPE_YARN 4
int liger_rope_scaled_fwd(const void* q, const void* k, void* q_out, void* k_out, const int32_t* pos, int64_t batch,
                          int64_t seq, int64_t n_q_heads, int64_t n_k_heads, int64_t head_dim, int64_t rotary_dim,
                          int64_t q_token_stride, int64_t k_token_stride, int64_t q_out_token_stride,
                          int64_t k_out_token_stride, int pairing, double theta, int scaling, double factor, double low,
                          double high, double orig_len, double attn_factor, int dtype, void* stream);
int liger_rope_scaled_bwd(const void* dq, const void* dk, void* dq_out, void* dk_out, const int32_t* pos, int64_t batch,
                          int64_t seq, int64_t n_q_heads, int64_t n_k_heads, int64_t head_dim, int64_t rotary_dim,
                          int64_t q_token_stride, int64_t k_token_stride, int64_t q_out_token_stride,
                          int64_t k_out_token_stride, int pairing, double theta, int scaling, double factor, double low,
                          double high, double orig_len, double attn_factor, int dtype, void* stream);

/* -------------------- token log-probabilities, entropy, alternatives
 * logits [T, V], row t at logits + t ld (ld >= V), dtype; with z = logits[t] /
 * temperature (at least 1e-30):
 *     row_max[t] = max_v logits[t, v]
 *     log_sum[t] = log sum_v exp(z_v - row_max[t] / temperature)
 *     logp[t] = z[tokens[t]] - row_max[t] / temperature - log_sum[t]
 *               (0 where tokens[t] is ignore_index)
 *     entropy[t] = -sum_v p_v log p_v,  p = softmax(z)   (p = 0 counts as 0)
 *     top_ids[t, :k] = the k largest logits' indices, largest first, equal ones
 *                      by index (-0 equals 0; NaN before all numbers)
 *     top_logp[t, :k] = the same of top_ids
 *   log sum exp z is row_max / temperature + log_sum; kept apart, nothing is lost
 *   where the logits are far from 0, or all of a row the type's lowest value.
 *   tokens int64 [T], logp float [T]: both or neither (NULL).  row_max, log_sum,
 *   entropy float [T], each may be NULL.  top_logp float, top_ids int64 [T, k]:
 *   both, with 1 <= k <= LIGER_TOP_MAX and k <= V, or NULL with k = 0.
 *   All but logp are formed at ignored tokens too.
 *   logits of -inf count as ruled out.  A row of nothing else has row_max, log_sum,
 *   logp and top_logp -inf and entropy 0.  A row with a NaN or +inf has NaN for
 *   log_sum, entropy, top_logp and logp.
 *   A token outside [0, V) that is not ignore_index: logp NaN.
 *   Pointers aligned to their element sizes; rows of 16-byte aligned starts
 *   (pointer and ld) are read fastest. */
#define LIGER_TOP_MAX 32
int liger_token_logp_fwd(const void* logits, int64_t ld, const int64_t* tokens, int64_t T, int64_t V,
                         int64_t ignore_index, float temperature, float* logp, float* row_max, float* log_sum, float* entropy,
                         int64_t k, float* top_logp, int64_t* top_ids, int dtype, void* stream);

/* The gradient of the logits from those of logp and of the entropy, with
 * row_max, log_sum and entropy as the forward wrote them:
 *     dlogits[t, v] = (g_logp[t] (1[v = tokens[t]] - p_v)
 *                      - g_entropy[t] p_v (log p_v + entropy[t])) / temperature
 *   g_logp float [T] with tokens, or NULL (0); g_entropy float [T] with
 *   entropy, or NULL (0); one of the two at least.  At ignored tokens g_logp
 *   counts as 0 and is not read.  A row whose g_logp and g_entropy are both 0 (or
 *   absent) is +0 whatever its logits are, and so is one without a logit above -inf.
 *   A token outside [0, V) that is not ignore_index: NaN in its row.
 *   dlogits [T, V], rows ldd apart (>= V); it may be logits, with ldd = ld; no
 *   other overlap. */
int liger_token_logp_bwd(const void* logits, int64_t ld, const int64_t* tokens, const float* row_max,
                         const float* log_sum, const float* entropy, const float* g_logp, const float* g_entropy, int64_t T,
                         int64_t V, int64_t ignore_index, float temperature, void* dlogits, int64_t ldd, int dtype,
                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LIGER_LAYER_H */
