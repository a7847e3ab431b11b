// Internal launchers of the experts' training side and the optimizer (host side).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_train.h"
#include "launch.hpp"

namespace moe {

// ---- rows.hip
// Stable order of the assignments a = t K + k by expert.  part: nothing for
// order_blocks() == 1, else order_blocks() E ints.
int order_blocks(int64_t A);
hipError_t launch_order(const int32_t* idx, int T, int E, int e0, int K, const uint8_t* mask, int32_t* part,
                        int32_t* counts, int32_t* offsets, int32_t* sorted_token, int32_t* pos, hipStream_t stream);

// xs[pos[t,k]] = x[t] for 0 <= pos < rows; a row is `bytes` long (a multiple of 128).
hipError_t launch_spread(const void* x, const int32_t* pos, int T, int K, int64_t bytes, int64_t rows, void* xs,
                         hipStream_t stream);
// out[t] = res[t] + sum_k w[t,k] y[pos[t,k]] over 0 <= pos < rows; res and w (then 1) may be null, res may be out.
hipError_t launch_gather(DType dt, const void* y, const float* w, const int32_t* pos, const void* res, int T, int K,
                         int64_t d, int64_t rows, void* out, hipStream_t stream);
// dy[pos[t,k]] = w[t,k] dout[t], dw[t,k] = <dout[t], y[pos[t,k]]>; either may be null.
hipError_t launch_gather_backward(DType dt, const void* dout, const void* y, const float* w, const int32_t* pos, int T,
                                  int K, int64_t d, int64_t rows, void* dy, float* dw, hipStream_t stream);

// ---- experts.hip
// One grouped product over rows sorted by expert (off [E + 1]); bf16.
enum ExpertsKind { EXP_UP, EXP_DOWN, EXP_DH, EXP_DX, EXP_DW_DOWN, EXP_DW_UP };
struct ExpertsArgs {
    const int32_t* off;
    const uint16_t *A, *B, *B2;  // B2: W_up beside W_gate
    float* gu;                   // [R, 2 F]: a and b, written by EXP_UP (may be null), read by EXP_DH
    uint16_t *C, *C2;            // EXP_DW_UP: dW_gate and dW_up
    int64_t R;
    int32_t E, d, F;
};
int64_t experts_max_rows(int E, int d, int F);
hipError_t launch_experts(ExpertsKind kind, const ExpertsArgs& a, hipStream_t stream);
// EXP_DH with EXP_DW_DOWN, or EXP_DX with EXP_DW_UP.
hipError_t launch_experts_pair(ExpertsKind kind, const ExpertsArgs& a, const ExpertsArgs& dw, hipStream_t stream);

// ---- adamw.hip
int64_t adamw_table_bytes(int n);
int64_t adamw_blocks(const moe_adamw_tensor* t, int n);
hipError_t launch_adamw(const moe_adamw_desc& D, const moe_adamw_tensor* t, int n, void* table, hipStream_t stream);
hipError_t launch_adamw_moments(const moe_adamw_tensor* t, float* const* avg, float* const* sq, int n,
                                hipStream_t stream);

}  // namespace moe
