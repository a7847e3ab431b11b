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
// rows of E (p sums, counts, tokens); part_l one float per (sequence, 64
// experts); ticket one int.
int balance_chunk(int T);
int64_t balance_slots(int T, int S);
hipError_t launch_balance_loss(const SeqArgs& a, const float* z, const int32_t* idx, float alpha, float* part_p,
                               int32_t* part_c, int32_t* part_n, float* part_l, int32_t* ticket, float* loss,
                               int32_t* seq_counts, hipStream_t stream);

// d_logits; dw NULL: no gate term; counts NULL: no balance term.
hipError_t launch_gate_backward(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                const int32_t* counts, float alpha, const float* d_loss, float* dz,
                                hipStream_t stream);

// [R, C] fp32 -> bf16 parts, row-major, columns C .. Cp - 1 zero: the row
// [hi | lo | hi] of 3 Cp columns (hi = rne(v), lo = rne(v - hi)).
hipError_t launch_split_rows(const float* src, int64_t R, int C, int Cp, uint16_t* dst, hipStream_t stream);
// [R, C] -> [C, Rp], columns R .. Rp - 1 zero.  fp32 -> fp32; bf16 -> bf16;
// fp32 -> three bf16 planes [C, Rp] with hi + mid + lo == v; fp32 -> rows
// [hi | hi | lo] of 3 Rp columns.
enum TransposeKind { TR_F32 = 0, TR_BF16 = 1, TR_PLANES3 = 2, TR_HHL = 3 };
hipError_t launch_transpose(TransposeKind kind, const void* src, int64_t R, int64_t C, int64_t Rp, void* dst,
                            hipStream_t stream);
// out[i] = sum over the n planes of part[i], in plane order.
hipError_t launch_sum_planes(const float* part, int n, int64_t stride, int64_t count, float* out, hipStream_t stream);

}  // namespace moe
