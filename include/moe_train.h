/*
 * moe_train.h -- C ABI of the layer's training side (libmoe_train.so, which
 * needs libmoe.so): the router with its logits kept, the balance loss with
 * its per-expert counts, and the gradients of both back to x and W_r; the
 * tokens sorted by expert, the experts on the sorted rows and the weighted sum
 * back, each with its gradient; and the optimizer's step (their formulas stand
 * at their declarations).
 *
 * Formulas of the router, with s = sigmoid(z), z = x W_r^T [T, E] and the router of moe.h:
 *   gate weights   w_k = scale s_k / D,  D = sum_{j chosen} s_j + 1e-20;
 *                  dL/ds_k = scale / D (dw_k - sum_j dw_j s_j / D) over the
 *                  chosen experts, 0 elsewhere (the bias only chooses, and
 *                  the choice has no gradient);
 *   balance loss   over sequences q = 0 .. S - 1 (the gate configuration's
 *                  seq_aux form [OpenModelAtlas "Kimi K2 · Router", MoEGate
 *                  configuration fields]), n_q tokens that count in each:
 *                  p_ti = s_ti / (sum_j s_tj + 1e-20),
 *                  c_qi = selections of expert i by the tokens of q,
 *                  L = alpha / S sum_q sum_i E c_qi / (K n_q)
 *                      * (1 / n_q) sum_{t in q} p_ti
 *                  (an empty sequence adds 0); c has no gradient, so
 *                  dL/dp_ti = alpha / S * E c_qi / (K n_q^2) =: a_qi and
 *                  dL/ds_tj = (a_qj - sum_i a_qi p_ti) / (sum_j s_tj + 1e-20);
 *   both           dz = dL/ds * s (1 - s),
 *                  dx = dz W_r,  dW_r = dz^T x.
 *
 * The conventions of moe.h hold: device pointers owned by the caller,
 * row-major, 16-byte aligned (loss and d_loss: 4-byte); arguments are checked
 * before anything is enqueued; calls only enqueue kernels on `stream`, which
 * must belong to the current device, so they can be captured; nothing is
 * allocated; concurrent calls, and captured graphs that may run at the same
 * time, need distinct workspaces.  Results do not depend on timing: the same
 * call gives the same bits.  T is at most 2^28 - 65536 (moe_router_train: as
 * moe_router; the experts' side: T K < 2^31).  T == 0 is a no-op but for loss (0), seq_counts
 * (zeros) and dW_r (zeros).  A NaN logit of a token that counts (see
 * moe_balance) makes the loss NaN, and that token's gradient as far as it
 * depends on the logit; in tokens that do not count it is harmless.  Logits past
 * +-87, infinite ones too, are held there.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the tokens form sequences, and the loss's weight.
 *   n_seq        S, 1 .. 65535.  Empty sequences are stepped over one by one
 *                (60000 of them over 100 tokens take 16 ms, loss and gradient).
 *   seq_offsets  [S + 1] int32, ascending, within 0 .. T: sequence q holds the
 *                tokens seq_offsets[q] .. seq_offsets[q + 1] - 1.  Tokens
 *                before the first or after the last are in none: the balance
 *                loss does not see them.  NULL with S = 1: all T tokens.
 *   token_mask   [T] uint8, or NULL: tokens whose byte is 0 (padding) do not
 *                count: they are in no sum or count, and their gradient rows
 *                (dz, and so dx) are zero, that of the gate weights included.
 *   alpha        the loss's weight.                                          */
typedef struct {
    int32_t n_seq;
    const int32_t *seq_offsets;
    const uint8_t *token_mask;
    float alpha;
} moe_balance;

/* moe_router, bit for bit, that also writes the logits z [T, E] fp32 which
 * the calls below take.  Workspace as for moe_router.                        */
moe_status moe_router_train(const moe_layer_desc *desc, const void *x,
                            const float *W_r, const float *b,
                            int32_t *topk_idx, float *topk_w,
                            int32_t *expert_counts, float *logits,
                            void *workspace, size_t workspace_bytes,
                            void *stream);

/* The balance loss.  Uses T, E and K of the descriptor.
 *   logits [T, E] fp32, topk_idx [T, K] int32 (distinct ids 0 .. E - 1 in a
 *   token; other ids are counted nowhere, and an id twice counts twice; n_q
 *   counts tokens, whatever their ids)
 *   -> loss [1] fp32, seq_counts [S, E] int32 (c_qi; their sum over q is a
 *   load that moe_bias_update takes).
 * Workspace of at least moe_balance_workspace_size(desc, S) bytes (0: an
 * invalid descriptor or S).                                                  */
size_t moe_balance_workspace_size(const moe_layer_desc *desc, int32_t n_seq);
moe_status moe_balance_loss(const moe_layer_desc *desc, const float *logits,
                            const int32_t *topk_idx, const moe_balance *balance,
                            float *loss, int32_t *seq_counts, void *workspace,
                            size_t workspace_bytes, void *stream);

/* The gradient at the logits.  Uses T, E, K and scale of the descriptor.
 *   d_topk_w [T, K] fp32, or NULL: no gradient from the gate weights;
 *   balance and seq_counts (as moe_balance_loss wrote them for the same
 *   sequences), or seq_counts NULL: no gradient from the balance loss (a
 *   balance given then still masks tokens); d_loss [1] fp32: the gradient at
 *   the loss, NULL for 1.
 *   At least one of d_topk_w and seq_counts is given.
 *   -> d_logits [T, E] fp32, which may be the logits' own memory.            */
moe_status moe_gate_backward(const moe_layer_desc *desc, const float *logits,
                             const int32_t *topk_idx, const float *d_topk_w,
                             const moe_balance *balance,
                             const int32_t *seq_counts, const float *d_loss,
                             float *d_logits, void *stream);

/* The router's backward pass: moe_gate_backward, then its two products.
 *   x [T, d] and W_r [E, d] as moe_router_train took them; the others as above
 *   -> dx [T, d] (act_dtype) and dW_r [E, d] fp32, either may be NULL (both:
 *   MOE_ERR_NULL).
 * dx is accurate to its type, dW_r to fp32: with bf16 activations the
 * products run on bf16 parts of dz and W_r that carry 16 and 24 bits.
 * Workspace of at least moe_router_backward_workspace_size(desc) bytes.      */
size_t moe_router_backward_workspace_size(const moe_layer_desc *desc);
moe_status moe_router_backward(const moe_layer_desc *desc, const void *x,
                               const float *W_r, const float *logits,
                               const int32_t *topk_idx, const float *d_topk_w,
                               const moe_balance *balance,
                               const int32_t *seq_counts, const float *d_loss,
                               void *dx, float *dW_r, void *workspace,
                               size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The experts' side.  An assignment a = t K + k is token t's k-th choice; the
 * R = T K assignments are sorted by expert into rows, stably (ascending a
 * within an expert), and the experts work on the rows of x, y, ... in that
 * order:
 *   xs[pos[t,k]] = x[t]                  moe_sort_tokens
 *   y = experts(xs)                      moe_experts_forward
 *   out[t] = sum_k w[t,k] y[pos[t,k]]    moe_combine
 * and back: moe_combine_backward (dout to dy and dw, which is the d_topk_w of
 * moe_router_backward), moe_experts_backward, moe_sort_tokens_backward.
 *
 * Descriptor fields used: T, d, E, K, F and act_dtype, with 1 <= K <= 16,
 * 1 <= E <= 1024, T K < 2^31, d (F) a positive multiple of 64 and at most 2^22
 * (2^21).  E is the number of this GPU's experts: K may exceed it.  A row whose
 * place is behind expert_offsets[E], or outside 0 .. rows - 1, belongs to no
 * assignment: it is neither read nor written.  Offsets that are not ascending
 * within 0 .. rows are not detected; they are taken as if clamped to it, and what
 * comes out is not said.  Results may not overlap what a call reads, but where it
 * says so.                                                                   */

/* The order.
 *   topk_idx [T, K] int32; e0: the id of this GPU's first expert; token_mask
 *   [T] uint8, or NULL: tokens whose byte is 0 have no rows
 *   -> expert_counts [E] (nullable), expert_offsets [E + 1]: expert e holds
 *      rows expert_offsets[e] .. expert_offsets[e + 1] - 1; sorted_token [T K]
 *      (nullable): each row's token (behind the last row it is left as it
 *      was); pos [T, K]: each assignment's row, -1 for ids outside e0 .. e0 +
 *      E - 1 and for masked tokens.  An expert chosen twice by a token has two
 *      rows of it.  All int32.
 * Workspace of at least moe_dispatch_workspace_size(desc) bytes.             */
size_t moe_dispatch_workspace_size(const moe_layer_desc *desc);
moe_status moe_dispatch(const moe_layer_desc *desc, const int32_t *topk_idx,
                        int32_t e0, const uint8_t *token_mask,
                        int32_t *expert_counts, int32_t *expert_offsets,
                        int32_t *sorted_token, int32_t *pos, void *workspace,
                        size_t workspace_bytes, void *stream);

/* x [T, d] -> xs [rows, d] (act_dtype): xs[pos[t,k]] = x[t]; and its gradient,
 * dx[t] = residual[t] + sum_k dxs[pos[t,k]], summed in slot order in fp32 and
 * rounded once.  residual [T, d] may be NULL (0) or dx itself.               */
moe_status moe_sort_tokens(const moe_layer_desc *desc, const void *x,
                           const int32_t *pos, int64_t rows, void *xs,
                           void *stream);
moe_status moe_sort_tokens_backward(const moe_layer_desc *desc, const void *dxs,
                                    const int32_t *pos, const void *residual,
                                    int64_t rows, void *dx, void *stream);

/* out[t] = residual[t] + sum_k topk_w[t,k] y[pos[t,k]], summed in slot order in
 * fp32 and rounded once: y [rows, d], residual and out [T, d] (act_dtype; residual
 * NULL for 0, or out itself), topk_w [T, K] fp32.  Its gradients from dout [T, d]:
 * dy[pos[t,k]] = topk_w[t,k] dout[t], dy [rows, d]; d_topk_w[t,k] = <dout[t],
 * y[pos[t,k]]>, fp32 [T, K], 0 without a row.  dy or d_topk_w may be NULL (both:
 * MOE_ERR_NULL); y is needed for d_topk_w, topk_w for dy; dy may be y.
 * (residual's gradient is dout.)                                             */
moe_status moe_combine(const moe_layer_desc *desc, const void *y,
                       const float *topk_w, const int32_t *pos,
                       const void *residual, int64_t rows, void *out,
                       void *stream);
moe_status moe_combine_backward(const moe_layer_desc *desc, const void *dout,
                                const void *y, const float *topk_w,
                                const int32_t *pos, int64_t rows, void *dy,
                                float *d_topk_w, void *stream);

/* The SwiGLU experts on sorted rows, bf16 (act_dtype MOE_BF16, weights of
 * MOE_LAYOUT_ROWS: W->W_gate, W_up [E, F, d], W->W_down [E, d, F]):
 *   a = xs W_gate^T, b = xs W_up^T, h = a sigmoid(a) b, y = h W_down^T.
 *   xs, y [rows, d]; expert_offsets [E + 1] int32, ascending, within 0 .. rows
 *   gate_up [rows, 2 F] fp32 (a, then b, of a row) and h [rows, F] are kept for
 *   the backward call; gate_up may be NULL.
 * Sums are kept in fp32; h is rounded to bf16.  rows at most moe_experts_max_rows(desc) (0 or less: the sizes are out
 * of range; d F < 2^31).                                                      */
int64_t moe_experts_max_rows(const moe_layer_desc *desc);
moe_status moe_experts_forward(const moe_layer_desc *desc, int64_t rows,
                               const void *xs, const int32_t *expert_offsets,
                               const moe_expert_weights *W, float *gate_up,
                               void *h, void *y, void *stream);

/* Its gradients from dy [rows, d], with what the forward call was given and
 * kept:  dh = dy W_down,  db = dh a s,  da = dh b s (1 + a (1 - s)),  s =
 * sigmoid(a) (da, db rounded to bf16);
 *   dxs [rows, d] = da W_gate + db W_up, or NULL;
 *   dW_gate = da^T xs, dW_up = db^T xs [E, F, d], dW_down = dy^T h [E, d, F],
 *   all bf16, zero for an expert without rows, or all NULL.
 * Workspace of at least moe_experts_backward_workspace_size(desc, rows) bytes
 * (0: out of range).                                                          */
size_t moe_experts_backward_workspace_size(const moe_layer_desc *desc, int64_t rows);
moe_status moe_experts_backward(const moe_layer_desc *desc, int64_t rows,
                                const void *dy, const void *xs,
                                const int32_t *expert_offsets,
                                const moe_expert_weights *W,
                                const float *gate_up, const void *h, void *dxs,
                                void *dW_gate, void *dW_up, void *dW_down,
                                void *workspace, size_t workspace_bytes,
                                void *stream);

/* ------------------------------------------------------------------------
 * One AdamW step over many tensors (decoupled weight decay), t = step >= 1:
 *   g = grad_scale grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g g,
 *   param = (1 - lr weight_decay) param
 *           - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps),  eps >= 2^-40.
 * Moments in 32 bits are fp32.  In 8 bits, 128 consecutive values of a tensor share
 * a scale 2^(s - 127) (one byte s; s = 255: the block holds NaN, as after an
 * infinite or NaN moment in it); m is an E4M3 code (sign, 4 exponent bits with
 * bias 7, 3 fraction bits), v an unsigned code of 5 exponent bits with bias
 * 15 and 3 fraction bits; the value is code x scale.  A new moment x, computed in
 * fp32, is rounded to one of its two neighbours at random, up with the
 * probability that keeps the mean; so is a bf16 parameter.  Under the root, v is
 * at least b2 times the value of code 1 in the block that it was read from (an m that
 * was rounded up would else move its parameter by any amount beside a v that was
 * rounded to 0), unless |m| is over 64 times the root of that: moments that are no
 * averages of the same gradients are taken as they are.  The random bits are of
 * (seed, step, the tensor's number in `tensors`, the element i): with
 *   mix(h): h = (h ^ (h >> 16)) 0x85ebca6b, h = (h ^ (h >> 13)) 0xc2b2ae35,
 *           h ^ (h >> 16)          [A. Appleby's 32-bit mixer, public domain]
 * and all sums and products modulo 2^32,
 *   word = mix(i % 2^32 + mix(mix(mix(seed) + step) + tensor)
 *              + (i / 2^32) 0x9e3779b9);
 * m takes its low 16 bits, v its high ones, a parameter the low ones of
 * mix(word ^ 0x9e3779b9).                                                     */
typedef struct {
    int32_t param_dtype;   /* moe_dtype: MOE_F32 or MOE_BF16                  */
    int32_t grad_dtype;    /* MOE_F32 or MOE_BF16                             */
    int32_t moment_bits;   /* 32 or 8                                         */
    int32_t step;          /* t, from 1 on                                    */
    uint32_t seed;
    float lr, eps, weight_decay;
    double beta_avg, beta_sq;     /* b1, b2 in [0, 1)                         */
    const float *lr_device;       /* [1] on the device, in place of lr; or NULL */
    const int32_t *step_device;   /* likewise, in place of step: for a call that
                                     is captured and replayed                  */
    const float *grad_scale;      /* [1] on the device, or NULL for 1          */
    int32_t keep_table;    /* 0: the call writes the tensors' table first (one */
                           /* launch per 56 of them); else the table holds it, */
                           /* from a call with the same `tensors`              */
} moe_adamw_desc;

/* One tensor of n elements; 16-byte aligned pointers (scales: any).
 *   copy: bf16 [n], receives fp32 parameters rounded to nearest; or NULL (as it
 *   must be with bf16 parameters).
 *   exp_avg, exp_avg_sq: fp32 [n], or uint8 [n] codes with their scales
 *   uint8 [(n + 127) / 128] (NULL with 32 bits).                              */
typedef struct {
    void *param;
    const void *grad;
    void *exp_avg, *exp_avg_sq;
    uint8_t *exp_avg_scale, *exp_avg_sq_scale;
    void *copy;
    int64_t n;
} moe_adamw_tensor;

/* `tensors` is host memory and is read before the call returns.  A tensor may
 * be empty (n = 0); no two may overlap; at most 65536 of them, with less than
 * 2^36 elements each and 2^37 in all.  `table`: device memory of at least
 * moe_adamw_table_size(n_tensors) bytes (0: out of range), 16-byte aligned,
 * which the call writes unless keep_table says that it is written, and reads.  */
size_t moe_adamw_table_size(int32_t n_tensors);
moe_status moe_adamw(const moe_adamw_desc *desc, const moe_adamw_tensor *tensors,
                     int32_t n_tensors, void *table, size_t table_bytes,
                     void *stream);

/* 8-bit moments to the values they stand for: avg[i] and sq[i] (host arrays of
 * device pointers; an entry, or a whole array, may be NULL) receive fp32 [n] of
 * tensor i.                                                                  */
moe_status moe_adamw_moments(const moe_adamw_tensor *tensors, int32_t n_tensors,
                             float *const *avg, float *const *sq, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_TRAIN_H */
