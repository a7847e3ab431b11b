// Internal launchers of the router's training side (host side).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// In libmoe.so (api.cpp): the descriptor's checks for a router call, and
// moe_router with the logits [T, E] written too.
moe_status router_check(const moe_layer_desc* desc);
moe_status router_with_logits(const moe_layer_desc* desc, const void* x, const float* W_r, const float* b,
                              int32_t* topk_idx, float* topk_w, int32_t* expert_counts, float* logits,
                              void* workspace, size_t workspace_bytes, void* stream);

// Sequences of the balance loss: q holds tokens off[q] .. off[q + 1] - 1
// (off NULL: one sequence of all tokens); mask NULL: every token counts.
struct SeqArgs {
    const int32_t* off;
    const uint8_t* mask;
    int32_t S, T, E, K;
};

// Balance loss.  part_p / part_c / part_n hold balance_slots(T, S) partial
// rows of E (p sums, counts, tokens); part_l one word per (sequence, 64
// experts); ticket one int.
int64_t balance_slots(int T, int S);
hipError_t launch_balance_loss(const SeqArgs& a, const float* z, const int32_t* idx, float alpha, float* part_p,
                               int32_t* part_c, int32_t* part_n, uint64_t* part_l, int32_t* ticket, float* loss,
                               int32_t* seq_counts, hipStream_t stream);

// d_logits; dw NULL: no gate term; counts NULL: no balance term.
hipError_t launch_gate_backward(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                const int32_t* counts, float alpha, const float* d_loss, float* dz,
                                hipStream_t stream);

// The same gradient for launch_small_products: rows [T, Es] and cols [Es, Ts]
// (E and T up to whole 16s), zero past E and T.
hipError_t launch_gate_backward_small(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                      const int32_t* counts, float alpha, const float* d_loss, float* rows, float* cols,
                                      hipStream_t stream);
// The same gradient as operands of the two products (bf16 activations):
// rows (nullable) [T, 3 Ep] = [hi | lo | hi], zero past E (Ep = E up to 64s);
// cols (nullable): its parts hi, mid, lo with hi + mid + lo == dz in
// [dw_slabs(T)][3][ceil(E/16)] blocks of 1 KiB (16 experts x 32 tokens, element
// (r, c) at ((c / 8) 16 + r) 8 + c % 8), zero past E and T; with it live
// [32 dw_slabs(T)]: 0xffff for the tokens that count, else 0.  n_tok: scratch of T floats.
int dw_slabs(int T);
hipError_t launch_gate_backward_planes(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                       const int32_t* counts, float alpha, const float* d_loss, uint16_t* rows, int Ep,
                                       uint16_t* cols, uint16_t* live, float* n_tok, hipStream_t stream);

// W_r [E, d] -> W_r^T [d, 3 Ep] = [hi | hi | lo] in the fragment-block layout.
hipError_t launch_pack_wt(const float* W, int E, int64_t d, int Ep, uint16_t* dst, hipStream_t stream);

// dW_r from cols and bf16 x: nsplit planes [E, d] whose sum it is.
struct DwPlan {
    int mb, mt, ntn, nsplit;
};
DwPlan dw_plan(int T, int E, int64_t d);
hipError_t launch_dw(const DwPlan& p, const uint16_t* cols, const uint16_t* live, const void* x, int T, int E, int64_t d,
                     float* part, hipStream_t stream);

// Both products (dx, dW_r; either nullable) in fp32 on the vector ALUs.
hipError_t launch_small_products(bool bf16, const float* rows, const float* cols, const void* x, const float* W,
                                 const uint8_t* mask, int T, int E, int64_t d, void* dx, float* dW, hipStream_t stream);

// [R, C] -> [C, Rp], columns R .. Rp - 1 and those of rows with a zero mask
// byte zero; [R, C] -> [R, Cp], columns C .. Cp - 1 zero.
hipError_t launch_transpose(const float* src, int64_t R, int64_t C, int64_t Rp, const uint8_t* mask, float* dst,
                            hipStream_t stream);
hipError_t launch_pad_rows(const float* src, int64_t R, int C, int Cp, float* dst, hipStream_t stream);
// out[i] = sum over the n planes of part[i], in plane order.
hipError_t launch_sum_planes(const float* part, int n, int64_t stride, int64_t count, float* out, hipStream_t stream);

}  // namespace moe
