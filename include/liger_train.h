/*
 * liger_train.h -- C-ABI of libliger.so, second part: operators of a
 * post-training step beside those of liger.h, whose conventions (status
 * codes, dtypes, alignment, ownership of buffers, streams, threads) hold here
 * too.
 *
 *   - block norms: the norm behind a block, its gate, the scaled residual sum
 *     and the norm before the next block, forward and backward;
 *   - SwiGLU with 8-bit activation checkpoints: the gate and up values kept
 *     for the backward in 8 bits, elementwise and in FusedLinearSwiGLU;
 *   - the label log-probabilities of a linear head, and the clipped policy
 *     loss with a KL term from the hidden states, with its gradients.
 *
 * Every call here except liger_linear_logp_fwd and liger_linear_policy_fwd_bwd
 * (which wait for their label scan; work on the workspace may be queued by then)
 * queues work only and can be captured in a
 * CUDA graph after a first call on the device.  A bounded wait that expires in a
 * kernel (see liger.h) leaves NaN in the block norms' unfinished rows and sums,
 * in logp and in the policy's loss and stats; liger_device_status names the
 * block norms' as RMSNorm's and the 8-bit FusedLinearSwiGLU's as
 * FusedLinearSwiGLU's.
 */
#ifndef LIGER_TRAIN_H
#define LIGER_TRAIN_H

#include "liger.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------------------------------------------------- block norms
 * One pass over the rows between two blocks of a decoder: the norm behind the
 * block just computed (post-norm), the block's gate, the residual sum and the
 * norm before the next block (pre-norm).
 *
 * Forward, per row t of z (the block's output) and r (the residual stream),
 * both [rows, cols]:
 *     rz = 1 / sqrt(mean_j z[t,j]^2 + eps)
 *     p[j] = z[t,j] rz w_post[j]                    (p = z when w_post is NULL)
 *     h[t,j] = res_scale r[t,j] + block_scale g[j] p[j]
 *     rh = 1 / sqrt(mean_j h[t,j]^2 + eps)
 *     y[t,j] = h[t,j] rh w_pre[j]
 *   with g = gate row t / (rows / gates), gate [gates, cols]: gates = 1 is one
 *   learned gate per channel, gates = n one gate for each of n sequences of
 *   rows / n rows; gates = 0 with gate NULL is no gate (g = 1).
 *   rows must be a multiple of gates.
 *   w_post [cols] or NULL (no post-norm; rstd_z is then not written);
 *   w_pre [cols] or NULL (no pre-norm; y and rstd_h are then not written).
 *   rstd_z, rstd_h: float [rows], each may be NULL (not stored).
 *   All arithmetic is fp32 and h, y are rounded once, each from the unrounded
 *   h (y is not formed from the stored h).
 *   h may alias r, and y may alias z; no other overlap of inputs and outputs.
 */
int liger_block_norm_fwd(const void* z, const void* r, const void* w_post, const void* gate, const void* w_pre, void* h,
                         void* y, float* rstd_z, float* rstd_h, int64_t rows, int64_t cols, int64_t gates,
                         float res_scale, float block_scale, float eps, int dtype, void* stream);

/* Bytes of workspace liger_block_norm_bwd needs (fp32 partial sums of the
 * weight and gate gradients): an upper bound valid on any device,
 * 3 * min(rows, 1024) * cols * 4. */
size_t liger_block_norm_bwd_workspace(int64_t rows, int64_t cols, int64_t gates);

/* Backward, from dh (the gradient of h that does not come through y; NULL: 0)
 * and dy, with z, h, rstd_z, rstd_h as the forward read and wrote them:
 *     u = dy w_pre,  s1 = sum_j u h
 *     D = dh + rh u - rh^3 / cols s1 h               (D = dh without w_pre)
 *     dr = res_scale D
 *     q = block_scale g w_post,  s2 = sum_j q D z
 *     dz = rz q D - rz^3 / cols s2 z                 (dz = block_scale g D without w_post)
 *     dw_pre = sum_t dy h rh
 *     dw_post = sum_t block_scale g D z rz
 *     dgate[i] = sum over the rows of gate row i of block_scale D p
 *   Required: z with w_post or gate; h, dy, rstd_h, dw_pre with w_pre; rstd_z,
 *   dw_post with w_post; dgate with gate; dh without w_pre.
 *   The sums over rows are reduced in a fixed order (deterministic run to run
 *   on one device).  dr may alias dh, and dz may alias dy; no other overlap.
 *   ws: at least liger_block_norm_bwd_workspace bytes, 16-byte aligned.
 *   rows = 0 writes zeros to dw_post, dgate and dw_pre.
 */
int liger_block_norm_bwd(const void* dh, const void* dy, const void* z, const void* h, const void* w_post,
                         const void* gate, const void* w_pre, const float* rstd_z, const float* rstd_h, void* dr,
                         void* dz, void* dw_post, void* dgate, void* dw_pre, void* ws, size_t ws_bytes, int64_t rows,
                         int64_t cols, int64_t gates, float res_scale, float block_scale, int dtype, void* stream);

/* ------------------------------------- SwiGLU with 8-bit checkpoints
 * The checkpoint of a [rows, cols] tensor x that a backward will read: int8
 * codes [rows, cols] and one scale byte for each group of 32 columns of a row
 * (the last group of a row may be shorter), scales [rows, ceil(cols / 32)].
 * For a group with m = max |x|:
 *     E = floor(log2 m),  step = 2^(E - 6),  code = clamp(rint(x / step), -127, 127),
 *     scale byte = E + 127,  x read back as code * step
 *   (rint rounds halves to even).  The step is a power of two, so x / step and
 *   code * step are exact: |x - read back| <= step / 2 (< step where |x| >
 *   127.5 step), step <= m / 64.
 *   m < 2^-111: codes 0 and scale byte 0 (the group reads back as zeros).
 *   A group that holds an infinity or NaN: scale byte 255, all of the group
 *   reads back as NaN.
 * 1 + 1/32 bytes an element, against 2 (bf16) or 4.
 */
#define LIGER_CKPT8_GROUP 32

/* Forward, elementwise on [rows, cols]: y = silu(gate) * up from the exact
 * gate and up (as liger_swiglu_fwd), and the checkpoints of both.
 *   gate, up, y: dtype, 16-byte aligned; y may alias gate or up.
 *   gate8, up8: int8 codes, 16-byte aligned; gate_scale, up_scale: scale bytes. */
int liger_swiglu_fwd_ckpt8(const void* gate, const void* up, void* y, int8_t* gate8, uint8_t* gate_scale, int8_t* up8,
                           uint8_t* up_scale, int64_t rows, int64_t cols, int dtype, void* stream);

/* Backward from the checkpoints: with g, u read back and s = sigmoid(g),
 *     dup = dy g s,  dgate = dy u s (1 + g (1 - s))
 *   dgate or dup may alias dy. */
int liger_swiglu_bwd_ckpt8(const void* dy, const int8_t* gate8, const uint8_t* gate_scale, const int8_t* up8,
                           const uint8_t* up_scale, void* dgate, void* dup, int64_t rows, int64_t cols, int dtype,
                           void* stream);

/* FusedLinearSwiGLU (liger_fused_linear_swiglu_fwd / _bwd) with the gate and
 * up products kept in 8 bits: the forward's epilogue writes out and the
 * checkpoints of g = X Wg^T and u = X Wu^T ([T, I], formed from the fp32
 * products; 2.06 bytes an element against the 4 of _fwd_save), and the
 * backward reads them instead of recomputing g and u (8 T H I flops).
 * Arguments, shapes (bf16; H >= 64, H and I multiples of 8), workspace
 * (liger_fused_linear_swiglu_workspace) and errors otherwise as
 * liger_fused_linear_swiglu_fwd_save / _bwd_saved; codes 16-byte aligned.  dWg
 * or dX is written twice: sums of the other gradients may stand in it first.
 * As there, the backward's dG and dU are rounded to bf16 once, as operands of
 * the three products, whose sums are fp32. */
int liger_fused_linear_swiglu_fwd_ckpt8(const void* X, const void* Wg, const void* Wu, void* out, int8_t* gate8,
                                        uint8_t* gate_scale, int8_t* up8, uint8_t* up_scale, int64_t T, int64_t H,
                                        int64_t I, int dtype, void* stream);
int liger_fused_linear_swiglu_bwd_ckpt8(const void* X, const void* Wg, const void* Wu, const void* dH,
                                        const int8_t* gate8, const uint8_t* gate_scale, const int8_t* up8,
                                        const uint8_t* up_scale, void* dX, void* dWg, void* dWu, void* ws,
                                        size_t ws_bytes, int64_t T, int64_t H, int64_t I, int dtype, void* stream);

/* --------------------------------- label log-probabilities of a linear head
 *     logp[t] = z_t[labels[t]] - log sum_v exp(z_t[v]),  z_t = W x_t
 * of the tokens whose label is not ignore_index, 0 on the others: what a policy
 * loss needs of the old and of the reference policy.  Forward only; the logits
 * never reach device memory on the bf16 tensor-core path (H >= 64 and a
 * multiple of 8, V >= 256); other cases run in fp32 with a [chunk x V] buffer.
 *   X [T, H], W [V, H] in dtype, labels int64 [T], logp float [T].  Off the
 *   tensor cores V is at most 4194240, and so are the rows of a chunk.
 *   ws: at least liger_linear_logp_workspace bytes, 256-byte aligned.
 * liger_linear_logp_fwd waits for a scan of the labels: a label outside [0, V)
 * that is not ignore_index returns LIGER_ERR_LABEL with logp left as it was,
 * and tokens that are ignored do not go through the GEMM where leaving them out
 * saves a tile of 256.  The _async form
 * does not wait (it can be captured): it runs all tokens, and a bad label's
 * logp is NaN. */
size_t liger_linear_logp_workspace(int64_t T, int64_t H, int64_t V, int dtype);
int liger_linear_logp_fwd(const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H, int64_t V,
                          int64_t ignore_index, float* logp, void* ws, size_t ws_bytes, int dtype, void* stream);
int liger_linear_logp_fwd_async(const void* X, const void* W, const int64_t* labels, int64_t T, int64_t H, int64_t V,
                                int64_t ignore_index, float* logp, void* ws, size_t ws_bytes, int dtype, void* stream);

/* ------------------------- clipped policy loss with a KL term of a linear head
 * T tokens in B sequences, packed: sequence b is the tokens [cu_seqlens[b],
 * cu_seqlens[b + 1]) (int32 [B + 1] on the device, not descending, within
 * [0, T]); cu_seqlens NULL: B = 1, one sequence of all T tokens.  A token is
 * valid if it lies in a sequence and its label is not ignore_index.  With lp =
 * logp[t] as above, A the token's advantage and d = ref_logp[t] - lp, a valid
 * token has
 *     r = exp(lp - old_logp[t]),  kl = exp(d) - d - 1   (0 without ref_logp)
 *     l = -min(r A, clamp(r, 1 - eps_low, 1 + eps_high) A) + beta kl
 *     dl/dlp = -(r A, or 0 where A > 0 and r > 1 + eps_high or A < 0 and r < 1 - eps_low)
 *              + beta (1 - exp(d))
 *   (A = 0: no policy term), and
 *     loss = sum over valid tokens of w l
 *     reduction 0 (token mean):    w = 1 / number of valid tokens
 *     reduction 1 (sum):           w = 1
 *     reduction 2 (sequence mean): w = 1 / (B * valid tokens of the token's sequence)
 *     D_t = grad_scale w dl/dlp (onehot(labels[t]) - softmax(z_t)),  dX = D W,  dW = D^T X
 *   No valid token: loss 0 and zero gradients.
 *   adv: float [B], or [T] with LIGER_POLICY_ADV_PER_TOKEN in flags.
 *   old_logp float [T]; ref_logp float [T], may be NULL when beta is 0 (then no
 *   kl).  Nothing of old_logp, ref_logp or a per-token adv is read at tokens that are
 *   not valid, and X may hold anything there.  0 <= eps_low <= 1, eps_high >= 0.
 *   loss: one float; stats: two floats or NULL, the mean kl and the share of
 *   clipped tokens over the valid tokens; logp: float [T] or NULL, 0 at tokens
 *   that are not valid (it must not overlap old_logp, ref_logp or adv:
 *   LIGER_ERR_SHAPE); dX [T, H], dW [V, H] in dtype, each may be NULL.  Rows
 *   of dX of tokens that are not valid are written as +0.
 *   Token chunks and the GEMM path by dtype and shape are as in
 *   liger_linear_ce_fwd_bwd, but chunk 0 is min(T, 8192) on the tensor-core
 *   path: per chunk the logits exist only in a [chunk x V] workspace buffer
 *   (up to 8192 tokens that is all of them, and dW needs no fp32 [V x H] sum).
 *   ws: at least liger_linear_policy_workspace bytes, 256-byte aligned.
 *   The call waits for a scan of the labels and sequences: a bad label returns
 *   LIGER_ERR_LABEL, bad cu_seqlens LIGER_ERR_SHAPE, with no output written,
 *   and tokens that are not valid do not go through the tensor-core GEMMs where
 *   leaving them out saves a tile of 256.  The _async form does not wait
 *   (it can be captured in a CUDA graph): all tokens go through the GEMMs, a bad
 *   label counts as ignored and bad cu_seqlens leave no valid token; either
 *   makes the loss and stats NaN.
 *   dW may differ between the two forms by rounding (the same sums over another
 *   grouping of the tokens). */
#define LIGER_POLICY_ADV_PER_TOKEN 1
size_t liger_linear_policy_workspace(int64_t T, int64_t H, int64_t V, int64_t B, int64_t chunk, int dtype);
int liger_linear_policy_fwd_bwd(const void* X, const void* W, const int64_t* labels, const int32_t* cu_seqlens,
                                const float* old_logp, const float* ref_logp, const float* adv, int64_t T, int64_t H,
                                int64_t V, int64_t B, int64_t ignore_index, int reduction, int flags, float eps_low,
                                float eps_high, float beta, float grad_scale, float* loss, float* stats, float* logp,
                                void* dX, void* dW, void* ws, size_t ws_bytes, int64_t chunk, int dtype, void* stream);
int liger_linear_policy_fwd_bwd_async(const void* X, const void* W, const int64_t* labels, const int32_t* cu_seqlens,
                                      const float* old_logp, const float* ref_logp, const float* adv, int64_t T,
                                      int64_t H, int64_t V, int64_t B, int64_t ignore_index, int reduction, int flags,
                                      float eps_low, float eps_high, float beta, float grad_scale, float* loss,
                                      float* stats, float* logp, void* dX, void* dW, void* ws, size_t ws_bytes,
                                      int64_t chunk, int dtype, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LIGER_TRAIN_H */
