// C ABI of the experts' training side and the optimizer (include/moe_train.h):
// argument validation, workspace layout and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_train.h"
#include "experts.hpp"

using namespace moe;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
template <typename... P>
bool aligned16(P... p) {
    return (aligned(p, 16) && ...);
}
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

#define MOE_HIP(x)                                 \
    do {                                           \
        if ((x) != hipSuccess) return MOE_ERR_HIP; \
    } while (0)

constexpr int32_t kMaxTensors = 65536;
constexpr float kMinEps = 0x1p-40f;  // (far above the root of any subnormal v, which is taken as 0)
constexpr int64_t kMaxBlocks = 1 << 24;  // (a launch has less than 2^32 threads)
constexpr int32_t kMaxD = 1 << 22;  // columns of a row: byte offsets within a tile of 256 rows stay below 2^32

// The fields of a call on rows: T, d, K and the type.
moe_status check_rows(const moe_layer_desc* D, int64_t rows) {
    if (!D) return MOE_ERR_NULL;
    if (D->act_dtype != MOE_F32 && D->act_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (D->T < 0 || D->K < 1 || D->K > 16 || static_cast<int64_t>(D->T) * D->K >= (1ll << 31)) return MOE_ERR_SHAPE;
    if (D->d < 64 || D->d % 64 || D->d > kMaxD || rows < 0 || rows >= (1ll << 31)) return MOE_ERR_SHAPE;
    return MOE_OK;
}
DType type_of(const moe_layer_desc* D) { return D->act_dtype == MOE_BF16 ? DT_BF16 : DT_F32; }
int64_t row_bytes(const moe_layer_desc* D) { return static_cast<int64_t>(D->d) * (D->act_dtype == MOE_BF16 ? 2 : 4); }

moe_status check_order(const moe_layer_desc* D) {
    if (!D) return MOE_ERR_NULL;
    if (D->E < 1 || D->E > 1024 || D->T < 0 || D->K < 1 || D->K > 16) return MOE_ERR_SHAPE;
    return static_cast<int64_t>(D->T) * D->K < (1ll << 31) ? MOE_OK : MOE_ERR_SHAPE;
}
int64_t order_bytes(const moe_layer_desc* D) {
    const int nb = order_blocks(static_cast<int64_t>(D->T) * D->K);
    return nb > 1 ? static_cast<int64_t>(nb) * D->E * 4 : 16;
}

moe_status check_experts(const moe_layer_desc* D, int64_t rows) {
    if (!D) return MOE_ERR_NULL;
    if (D->act_dtype != MOE_BF16 || D->w_dtype != MOE_BF16 || D->w_layout != MOE_LAYOUT_ROWS) return MOE_ERR_UNSUPPORTED;
    if (D->E < 1 || D->E > 1024 || D->d < 64 || D->d % 64 || D->F < 64 || D->F % 64 || D->d > kMaxD || D->F > kMaxD / 2 ||
        static_cast<int64_t>(D->d) * D->F >= (1ll << 31))
        return MOE_ERR_SHAPE;
    const int64_t most = experts_max_rows(D->E, D->d, D->F);
    return most >= 0 && rows >= 0 && rows <= most ? MOE_OK : MOE_ERR_SHAPE;
}

ExpertsArgs experts_args(const moe_layer_desc* D, int64_t rows, const int32_t* off) {
    ExpertsArgs a{};
    a.off = off;
    a.R = rows;
    a.E = D->E;
    a.d = D->d;
    a.F = D->F;
    return a;
}
const uint16_t* in(const void* p) { return static_cast<const uint16_t*>(p); }
uint16_t* out(void* p) { return static_cast<uint16_t*>(p); }

moe_status check_tensors(const moe_adamw_tensor* t, int32_t n, bool eight) {
    for (int i = 0; i < n; ++i) {
        if (t[i].n < 0 || t[i].n >= (1ll << 36)) return MOE_ERR_SHAPE;
        if (t[i].n == 0) continue;
        if (!t[i].exp_avg || !t[i].exp_avg_sq) return MOE_ERR_NULL;
        if (eight && (!t[i].exp_avg_scale || !t[i].exp_avg_sq_scale)) return MOE_ERR_NULL;
        if (!aligned16(t[i].exp_avg, t[i].exp_avg_sq)) return MOE_ERR_ALIGN;
    }
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_dispatch_workspace_size(const moe_layer_desc* desc) {
    return check_order(desc) == MOE_OK ? static_cast<size_t>(order_bytes(desc)) : 0;
}

moe_status moe_dispatch(const moe_layer_desc* desc, const int32_t* topk_idx, int32_t e0, const uint8_t* token_mask,
                        int32_t* expert_counts, int32_t* expert_offsets, int32_t* sorted_token, int32_t* pos,
                        void* workspace, size_t workspace_bytes, void* stream) {
    const moe_status st = check_order(desc);
    if (st != MOE_OK) return st;
    if (e0 < 0 || e0 > INT32_MAX - desc->E) return MOE_ERR_SHAPE;
    if (!expert_offsets || !workspace || (desc->T && (!topk_idx || !pos))) return MOE_ERR_NULL;
    if (!aligned16(topk_idx, token_mask, expert_counts, expert_offsets, sorted_token, pos, workspace)) return MOE_ERR_ALIGN;
    if (workspace_bytes < static_cast<size_t>(order_bytes(desc))) return MOE_ERR_WORKSPACE;
    MOE_HIP(launch_order(topk_idx, desc->T, desc->E, e0, desc->K, token_mask, static_cast<int32_t*>(workspace),
                         expert_counts, expert_offsets, sorted_token, pos, static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

moe_status moe_sort_tokens(const moe_layer_desc* desc, const void* x, const int32_t* pos, int64_t rows, void* xs,
                           void* stream) {
    const moe_status st = check_rows(desc, rows);
    if (st != MOE_OK) return st;
    if (!aligned16(x, pos, xs)) return MOE_ERR_ALIGN;
    if (desc->T == 0 || rows == 0) return MOE_OK;
    if (!x || !pos || !xs) return MOE_ERR_NULL;
    MOE_HIP(launch_spread(x, pos, desc->T, desc->K, row_bytes(desc), rows, xs, static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

moe_status moe_sort_tokens_backward(const moe_layer_desc* desc, const void* dxs, const int32_t* pos,
                                    const void* residual, int64_t rows, void* dx, void* stream) {
    const moe_status st = check_rows(desc, rows);
    if (st != MOE_OK) return st;
    if (!aligned16(dxs, pos, residual, dx)) return MOE_ERR_ALIGN;
    if (desc->T == 0) return MOE_OK;
    if ((rows && !dxs) || !pos || !dx) return MOE_ERR_NULL;
    MOE_HIP(launch_gather(type_of(desc), dxs, nullptr, pos, residual, desc->T, desc->K, desc->d, rows, dx,
                          static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

moe_status moe_combine(const moe_layer_desc* desc, const void* y, const float* topk_w, const int32_t* pos,
                       const void* residual, int64_t rows, void* out, void* stream) {
    const moe_status st = check_rows(desc, rows);
    if (st != MOE_OK) return st;
    if (!aligned16(y, topk_w, pos, residual, out)) return MOE_ERR_ALIGN;
    if (desc->T == 0) return MOE_OK;
    if ((rows && !y) || !topk_w || !pos || !out) return MOE_ERR_NULL;
    MOE_HIP(launch_gather(type_of(desc), y, topk_w, pos, residual, desc->T, desc->K, desc->d, rows, out,
                          static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

moe_status moe_combine_backward(const moe_layer_desc* desc, const void* dout, const void* y, const float* topk_w,
                                const int32_t* pos, int64_t rows, void* dy, float* d_topk_w, void* stream) {
    const moe_status st = check_rows(desc, rows);
    if (st != MOE_OK) return st;
    if (!aligned16(dout, y, topk_w, pos, dy, d_topk_w)) return MOE_ERR_ALIGN;
    if (desc->T == 0) return MOE_OK;
    if (!dout || !pos || (!dy && !d_topk_w) || (dy && !topk_w) || (d_topk_w && rows && !y)) return MOE_ERR_NULL;
    MOE_HIP(launch_gather_backward(type_of(desc), dout, y, topk_w, pos, desc->T, desc->K, desc->d, rows, dy, d_topk_w,
                                   static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

int64_t moe_experts_max_rows(const moe_layer_desc* desc) {
    return check_experts(desc, 0) == MOE_OK ? experts_max_rows(desc->E, desc->d, desc->F) : 0;
}

moe_status moe_experts_forward(const moe_layer_desc* desc, int64_t rows, const void* xs, const int32_t* expert_offsets,
                               const moe_expert_weights* W, float* gate_up, void* h, void* y, void* stream) {
    const moe_status st = check_experts(desc, rows);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!xs || !expert_offsets || !W || !W->W_gate || !W->W_up || !W->W_down || !h || !y) return MOE_ERR_NULL;
    if (!aligned16(xs, expert_offsets, W->W_gate, W->W_up, W->W_down, gate_up, h, y)) return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ExpertsArgs a = experts_args(desc, rows, expert_offsets);
    a.A = in(xs);
    a.B = in(W->W_gate);
    a.B2 = in(W->W_up);
    a.gu = gate_up;
    a.C = out(h);
    MOE_HIP(launch_experts(EXP_UP, a, s));
    a.A = in(h);
    a.B = in(W->W_down);
    a.C = out(y);
    MOE_HIP(launch_experts(EXP_DOWN, a, s));
    return MOE_OK;
}

size_t moe_experts_backward_workspace_size(const moe_layer_desc* desc, int64_t rows) {
    if (check_experts(desc, rows) != MOE_OK) return 0;
    return static_cast<size_t>(up(std::max<int64_t>(rows, 1) * 2 * desc->F * 2, 256));
}

moe_status moe_experts_backward(const moe_layer_desc* desc, int64_t rows, const void* dy, const void* xs,
                                const int32_t* expert_offsets, const moe_expert_weights* W, const float* gate_up,
                                const void* h, void* dxs, void* dW_gate, void* dW_up, void* dW_down, void* workspace,
                                size_t workspace_bytes, void* stream) {
    const moe_status st = check_experts(desc, rows);
    if (st != MOE_OK) return st;
    const bool dw = dW_gate || dW_up || dW_down;
    if (dw && !(dW_gate && dW_up && dW_down)) return MOE_ERR_NULL;
    if (!aligned16(dy, xs, expert_offsets, gate_up, h, dxs, dW_gate, dW_up, dW_down, workspace)) return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (rows == 0) {
        if (!dw) return MOE_OK;
        const int64_t n = static_cast<int64_t>(desc->E) * desc->d * desc->F / 2;  // of 32 bits
        for (void* p : {dW_gate, dW_up, dW_down}) MOE_HIP(launch_fill_i32(static_cast<int32_t*>(p), 0, n, s));
        return MOE_OK;
    }
    if (!dw && !dxs) return MOE_ERR_NULL;
    if (!dy || !expert_offsets || !W || !W->W_down || !gate_up || !workspace) return MOE_ERR_NULL;
    if ((dxs && (!W->W_gate || !W->W_up)) || (dw && (!xs || !h))) return MOE_ERR_NULL;
    if (!aligned16(W->W_gate, W->W_up, W->W_down)) return MOE_ERR_ALIGN;
    if (workspace_bytes < moe_experts_backward_workspace_size(desc, rows)) return MOE_ERR_WORKSPACE;
    ExpertsArgs dh = experts_args(desc, rows, expert_offsets), dx = dh, dd = dh, du = dh;
    dh.A = in(dy);
    dh.B = in(W->W_down);
    dh.gu = const_cast<float*>(gate_up);
    dh.C = out(workspace);
    dd.A = in(dy);
    dd.B = in(h);
    dd.C = out(dW_down);
    dx.A = in(workspace);
    dx.B = in(W->W_gate);
    dx.B2 = in(W->W_up);
    dx.C = out(dxs);
    du.A = in(workspace);
    du.B = in(xs);
    du.C = out(dW_gate);
    du.C2 = out(dW_up);
    MOE_HIP(dw ? launch_experts_pair(EXP_DH, dh, dd, s) : launch_experts(EXP_DH, dh, s));
    MOE_HIP(dw && dxs ? launch_experts_pair(EXP_DX, dx, du, s)
                      : dw ? launch_experts(EXP_DW_UP, du, s) : launch_experts(EXP_DX, dx, s));
    return MOE_OK;
}

size_t moe_adamw_table_size(int32_t n_tensors) {
    return n_tensors < 0 || n_tensors > kMaxTensors ? 0 : static_cast<size_t>(up(adamw_table_bytes(n_tensors) + 1, 256));
}

moe_status moe_adamw(const moe_adamw_desc* desc, const moe_adamw_tensor* tensors, int32_t n_tensors, void* table,
                     size_t table_bytes, void* stream) {
    if (!desc || (n_tensors > 0 && !tensors)) return MOE_ERR_NULL;
    if (n_tensors < 0 || n_tensors > kMaxTensors || (desc->step < 1 && !desc->step_device)) return MOE_ERR_SHAPE;
    auto beta = [](double b) { return b >= 0.0 && b < 1.0; };
    if (!beta(desc->beta_avg) || !beta(desc->beta_sq) || !(desc->eps >= kMinEps)) return MOE_ERR_SHAPE;
    auto type = [](int32_t t) { return t == MOE_F32 || t == MOE_BF16; };
    if (!type(desc->param_dtype) || !type(desc->grad_dtype) || (desc->moment_bits != 32 && desc->moment_bits != 8))
        return MOE_ERR_UNSUPPORTED;
    if (!aligned(desc->lr_device, 4) || !aligned(desc->step_device, 4) || !aligned(desc->grad_scale, 4)) return MOE_ERR_ALIGN;
    const moe_status st = check_tensors(tensors, n_tensors, desc->moment_bits == 8);
    if (st != MOE_OK) return st;
    for (int i = 0; i < n_tensors; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        if (!t.param || !t.grad) return MOE_ERR_NULL;
        if (t.copy && desc->param_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
        if (!aligned16(t.param, t.grad, t.copy)) return MOE_ERR_ALIGN;
    }
    const int64_t blocks = adamw_blocks(tensors, n_tensors);
    if (blocks == 0) return MOE_OK;
    if (blocks >= kMaxBlocks) return MOE_ERR_SHAPE;
    if (!table) return MOE_ERR_NULL;
    if (!aligned16(table)) return MOE_ERR_ALIGN;
    if (table_bytes < static_cast<size_t>(adamw_table_bytes(n_tensors))) return MOE_ERR_WORKSPACE;
    MOE_HIP(launch_adamw(*desc, tensors, n_tensors, table, static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

moe_status moe_adamw_moments(const moe_adamw_tensor* tensors, int32_t n_tensors, float* const* avg, float* const* sq,
                             void* stream) {
    if (n_tensors < 0) return MOE_ERR_SHAPE;
    if (n_tensors > 0 && (!tensors || (!avg && !sq))) return MOE_ERR_NULL;
    const moe_status st = check_tensors(tensors, n_tensors, true);
    if (st != MOE_OK) return st;
    for (int i = 0; i < n_tensors; ++i)
        if (tensors[i].n && !aligned16(avg ? avg[i] : nullptr, sq ? sq[i] : nullptr)) return MOE_ERR_ALIGN;
    MOE_HIP(launch_adamw_moments(tensors, avg, sq, n_tensors, static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

}  // extern "C"
