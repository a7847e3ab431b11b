/*
 * moe_train.h -- C ABI of the router's training side (libmoe_train.so, which
 * needs libmoe.so): the router with its logits kept, the balance loss with
 * its per-expert counts, and the gradients of both back to x and W_r.
 *
 * Formulas, with s = sigmoid(z), z = x W_r^T [T, E] and the router of moe.h:
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
 * moe_router).  T == 0 is a no-op but for loss (0), seq_counts
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

#ifdef __cplusplus
}
#endif
#endif /* MOE_TRAIN_H */
