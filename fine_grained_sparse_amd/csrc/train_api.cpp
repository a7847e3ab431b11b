// C ABI of the router's training side (include/moe_train.h): argument
// validation, workspace layout and launches.  libmoe_train.so; the router and
// the grouped GEMM are libmoe.so's.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/moe_train.h"
#include "launch.hpp"
#include "train.hpp"

using namespace moe;

namespace {

constexpr int64_t kAlign = 256;
// Both products as one launch on the vector ALUs up to this many tokens and
// this T E d.  Whole passes (balance loss, gradient) against the matrix units,
// whose operands take four launches more: bf16 43 / 55 us at 301 x 48 x 1024
// (T x E x d), 55 / 55 at 1024 x 64 x 1024, 76 / 54 at 2048 x 32 x 512, 75 / 81
// at 64 x 384 x 7168, 100 / 84 at 128 x 384 x 7168; fp32 41 / 58 at 77 x 20 x
// 320, 68 / 86 at 1024 x 256 x 1024.
constexpr int64_t kSmallT = 1024, kSmallTEd = 200000000;
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

#define MOE_HIP(x)                                 \
    do {                                           \
        if ((x) != hipSuccess) return MOE_ERR_HIP; \
    } while (0)

struct Arena {
    int64_t off = 0;
    int64_t take(int64_t bytes) {
        const int64_t o = off;
        off = up(off + std::max<int64_t>(bytes, 1), kAlign);
        return o;
    }
};

template <typename P>
P* at(void* ws, int64_t off) {
    return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

// The router's own checks, and a T whose launches stay below 2^32 threads, as a
// launch must (16 threads a token; 32 above 512 experts, whose logits fill the
// memory before).  Token numbers that a kernel forms past the last one then fit
// in 31 bits too.
constexpr int32_t kMaxT = (1 << 28) - 65536;
moe_status check_desc(const moe_layer_desc* D) {
    const moe_status st = router_check(D);
    return st == MOE_OK && D->T > kMaxT ? MOE_ERR_SHAPE : st;
}

moe_status check_balance(const moe_balance* b) {
    if (b->n_seq < 1 || b->n_seq > 65535) return MOE_ERR_SHAPE;
    if (!b->seq_offsets && b->n_seq != 1) return MOE_ERR_NULL;
    if (!aligned16(b->seq_offsets) || !aligned16(b->token_mask)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

SeqArgs seq_args(const moe_layer_desc* D, const moe_balance* b) {
    SeqArgs a{};
    a.off = b ? b->seq_offsets : nullptr;
    a.mask = b ? b->token_mask : nullptr;
    a.S = b ? b->n_seq : 1;
    a.T = D->T;
    a.E = D->E;
    a.K = D->K;
    return a;
}

struct BalancePlan {
    int64_t o_p, o_c, o_n, o_l, o_ticket, total;
};
BalancePlan balance_plan(const moe_layer_desc* D, int S) {
    BalancePlan p{};
    Arena ar;
    const int64_t slots = balance_slots(D->T, S);
    p.o_p = ar.take(slots * D->E * 4);
    p.o_c = ar.take(slots * D->E * 4);
    p.o_n = ar.take(slots * 4);
    p.o_l = ar.take(cdiv(D->E, 64) * S * 8);
    p.o_ticket = ar.take(4);
    p.total = ar.off;
    return p;
}

struct BackPlan {
    bool bf16, small;
    int64_t Ep, Tp;  // E and T in whole 64-column K steps
    TileCfg xcfg;
    DwPlan dw;       // bf16
    int nsplit;      // planes of dW_r
    int64_t o_dz, o_rows, o_wt, o_cols, o_live, o_ntok, o_xt, o_part, total;
};
BackPlan back_plan(const moe_layer_desc* D) {
    BackPlan p{};
    p.bf16 = D->act_dtype == MOE_BF16;
    const int64_t T = D->T, E = D->E, d = D->d;
    p.small = T <= kSmallT && T * E * d <= kSmallTEd;
    p.Ep = up(E, 64);
    p.Tp = up(T, 64);
    Arena ar;
    if (p.small) {
        p.o_rows = ar.take(T * up(E, 16) * 4);
        p.o_cols = ar.take(up(E, 16) * up(T, 16) * 4);
    } else if (p.bf16) {
        p.xcfg = T > 64 ? TILE_WIDE : TILE_SMALL;
        p.dw = dw_plan(D->T, D->E, d);
        p.nsplit = p.dw.nsplit;
        p.o_rows = ar.take(T * 3 * p.Ep * 2);
        p.o_wt = ar.take(d * 3 * p.Ep * 2);
        p.o_cols = ar.take(3 * cdiv(E, 16) * dw_slabs(D->T) * 1024);
        p.o_live = ar.take(static_cast<int64_t>(dw_slabs(D->T)) * 64);
        p.o_ntok = ar.take(T * 4);
        p.o_part = ar.take(p.nsplit > 1 ? p.nsplit * E * d * 4 : 1);
    } else {
        p.xcfg = TILE_SMALL;
        // dW_r has few output tiles and a long K (the tokens): split K until
        // about 512 workgroups are in flight, at least 8 K steps each
        const int64_t wgs = cdiv(E, tile_bm(TILE_SMALL)) * cdiv(d, 256);
        p.nsplit = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({16, cdiv(512, wgs), p.Tp / 32 / 8})));
        p.o_dz = ar.take(T * E * 4);
        p.o_rows = ar.take(T * p.Ep * 4);
        p.o_wt = ar.take(d * p.Ep * 4);
        p.o_cols = ar.take(E * p.Tp * 4);
        p.o_xt = ar.take(d * p.Tp * 4);
        p.o_part = ar.take(p.nsplit > 1 ? p.nsplit * E * d * 4 : 1);
    }
    p.total = ar.off;
    return p;
}

GemmArgs dense(const void* A, int64_t lda, const void* B, int64_t ldb, int64_t K, void* C, int64_t ldc, int M, int N) {
    GemmArgs g{};
    g.g[0].seg[0] = GemmSeg{A, B, nullptr, lda, ldb, static_cast<int32_t>(K), 0};
    g.g[0].nseg = 1;
    g.g[0].N = N;
    g.g[0].C = C;
    g.g[0].ldc = ldc;
    g.M = M;
    g.nsplit = 1;
    return g;
}

// The checks shared by the two backward calls; *idle: nothing to do but the
// zeros of an empty batch.
moe_status check_backward(const moe_layer_desc* D, const float* logits, const int32_t* idx, const float* dw,
                          const moe_balance* b, const int32_t* counts, const float* d_loss, bool* idle) {
    const moe_status st = check_desc(D);
    if (st != MOE_OK) return st;
    *idle = D->T == 0;
    if (counts && !b) return MOE_ERR_NULL;
    if (b) {
        const moe_status sb = check_balance(b);
        if (sb != MOE_OK) return sb;
    }
    if (!aligned16(counts) || !aligned(d_loss, 4)) return MOE_ERR_ALIGN;
    if (*idle) return MOE_OK;
    if (!logits || !idx || (!dw && !counts)) return MOE_ERR_NULL;
    if (!aligned16(logits) || !aligned16(idx) || !aligned16(dw)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_router_train(const moe_layer_desc* desc, const void* x, const float* W_r, const float* b,
                            int32_t* topk_idx, float* topk_w, int32_t* expert_counts, float* logits, void* workspace,
                            size_t workspace_bytes, void* stream) {
    return router_with_logits(desc, x, W_r, b, topk_idx, topk_w, expert_counts, logits, workspace, workspace_bytes,
                              stream);
}

size_t moe_balance_workspace_size(const moe_layer_desc* desc, int32_t n_seq) {
    if (check_desc(desc) != MOE_OK || n_seq < 1 || n_seq > 65535) return 0;
    return static_cast<size_t>(balance_plan(desc, n_seq).total);
}

moe_status moe_balance_loss(const moe_layer_desc* desc, const float* logits, const int32_t* topk_idx,
                            const moe_balance* balance, float* loss, int32_t* seq_counts, void* workspace,
                            size_t workspace_bytes, void* stream) {
    moe_status st = check_desc(desc);
    if (st != MOE_OK) return st;
    if (!balance || !loss || !seq_counts) return MOE_ERR_NULL;
    st = check_balance(balance);
    if (st != MOE_OK) return st;
    if (!aligned(loss, 4) || !aligned16(seq_counts)) return MOE_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (desc->T == 0) {
        MOE_HIP(launch_fill_i32(seq_counts, 0, static_cast<int64_t>(balance->n_seq) * desc->E, s));
        MOE_HIP(launch_fill_i32(reinterpret_cast<int32_t*>(loss), 0, 1, s));  // the bits of +0.0
        return MOE_OK;
    }
    if (!logits || !topk_idx || !workspace) return MOE_ERR_NULL;
    if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(workspace)) return MOE_ERR_ALIGN;
    const BalancePlan p = balance_plan(desc, balance->n_seq);
    if (workspace_bytes < static_cast<size_t>(p.total)) return MOE_ERR_WORKSPACE;
    MOE_HIP(launch_balance_loss(seq_args(desc, balance), logits, topk_idx, balance->alpha, at<float>(workspace, p.o_p),
                                at<int32_t>(workspace, p.o_c), at<int32_t>(workspace, p.o_n),
                                at<uint64_t>(workspace, p.o_l), at<int32_t>(workspace, p.o_ticket), loss, seq_counts, s));
    return MOE_OK;
}

moe_status moe_gate_backward(const moe_layer_desc* desc, const float* logits, const int32_t* topk_idx,
                             const float* d_topk_w, const moe_balance* balance, const int32_t* seq_counts,
                             const float* d_loss, float* d_logits, void* stream) {
    bool idle = false;
    const moe_status st = check_backward(desc, logits, topk_idx, d_topk_w, balance, seq_counts, d_loss, &idle);
    if (st != MOE_OK || idle) return st;
    if (!d_logits) return MOE_ERR_NULL;
    if (!aligned16(d_logits)) return MOE_ERR_ALIGN;
    MOE_HIP(launch_gate_backward(seq_args(desc, balance), logits, topk_idx, d_topk_w, desc->scale, seq_counts,
                                 balance ? balance->alpha : 0.f, d_loss, d_logits, static_cast<hipStream_t>(stream)));
    return MOE_OK;
}

size_t moe_router_backward_workspace_size(const moe_layer_desc* desc) {
    if (check_desc(desc) != MOE_OK) return 0;
    return static_cast<size_t>(back_plan(desc).total);
}

moe_status moe_router_backward(const moe_layer_desc* desc, const void* x, const float* W_r, const float* logits,
                               const int32_t* topk_idx, const float* d_topk_w, const moe_balance* balance,
                               const int32_t* seq_counts, const float* d_loss, void* dx, float* dW_r, void* workspace,
                               size_t workspace_bytes, void* stream) {
    bool idle = false;
    const moe_status st = check_backward(desc, logits, topk_idx, d_topk_w, balance, seq_counts, d_loss, &idle);
    if (st != MOE_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t T = desc->T, E = desc->E, d = desc->d;
    if (!aligned16(dx) || !aligned16(dW_r)) return MOE_ERR_ALIGN;
    if (idle) {
        if (dW_r) MOE_HIP(launch_fill_i32(reinterpret_cast<int32_t*>(dW_r), 0, E * d, s));
        return MOE_OK;
    }
    if ((!dx && !dW_r) || (dx && !W_r) || (dW_r && !x) || !workspace) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(W_r) || !aligned16(workspace)) return MOE_ERR_ALIGN;
    const BackPlan p = back_plan(desc);
    if (workspace_bytes < static_cast<size_t>(p.total)) return MOE_ERR_WORKSPACE;
    const SeqArgs sa = seq_args(desc, balance);
    const uint8_t* mask = sa.mask;
    const float alpha = balance ? balance->alpha : 0.f;
    float* part = p.nsplit > 1 ? at<float>(workspace, p.o_part) : dW_r;  // (the small products need none)
    if (p.bf16 && !p.small) {
        uint16_t* rows = dx ? at<uint16_t>(workspace, p.o_rows) : nullptr;
        uint16_t* cols = dW_r ? at<uint16_t>(workspace, p.o_cols) : nullptr;
        const int Ep = static_cast<int>(p.Ep);
        MOE_HIP(launch_gate_backward_planes(sa, logits, topk_idx, d_topk_w, desc->scale, seq_counts, alpha, d_loss, rows,
                                            Ep, cols, at<uint16_t>(workspace, p.o_live), at<float>(workspace, p.o_ntok), s));
        if (dx) {
            uint16_t* wt = at<uint16_t>(workspace, p.o_wt);
            MOE_HIP(launch_pack_wt(W_r, desc->E, d, Ep, wt, s));
            const GemmArgs g = dense(rows, 3 * p.Ep, wt, 3 * p.Ep, 3 * p.Ep, dx, d, desc->T, desc->d);
            MOE_HIP(launch_gemm(g, DT_BF16, false, EPI_STORE, p.xcfg, static_cast<int>(cdiv(T, tile_bm(p.xcfg))),
                                desc->d, true, s));
        }
        if (dW_r) MOE_HIP(launch_dw(p.dw, cols, at<uint16_t>(workspace, p.o_live), x, desc->T, desc->E, d, part, s));
    } else if (p.small) {
        float* rows = at<float>(workspace, p.o_rows);
        float* cols = at<float>(workspace, p.o_cols);
        MOE_HIP(launch_gate_backward_small(sa, logits, topk_idx, d_topk_w, desc->scale, seq_counts, alpha, d_loss, rows,
                                           cols, s));
        MOE_HIP(launch_small_products(p.bf16, rows, cols, x, W_r, mask, desc->T, desc->E, d, dx, dW_r, s));
        return MOE_OK;
    } else {
        float* dz = at<float>(workspace, p.o_dz);
        MOE_HIP(launch_gate_backward(sa, logits, topk_idx, d_topk_w, desc->scale, seq_counts, alpha, d_loss, dz, s));
        if (dx) {
            float* rows = at<float>(workspace, p.o_rows);
            float* wt = at<float>(workspace, p.o_wt);
            MOE_HIP(launch_pad_rows(dz, T, desc->E, static_cast<int>(p.Ep), rows, s));
            MOE_HIP(launch_transpose(W_r, E, d, p.Ep, nullptr, wt, s));
            const GemmArgs g = dense(rows, p.Ep, wt, p.Ep, p.Ep, dx, d, desc->T, desc->d);
            MOE_HIP(launch_gemm(g, DT_F32, false, EPI_STORE, p.xcfg, static_cast<int>(cdiv(T, tile_bm(p.xcfg))),
                                desc->d, false, s));
        }
        if (dW_r) {
            float* dzt = at<float>(workspace, p.o_cols);
            float* xt = at<float>(workspace, p.o_xt);
            MOE_HIP(launch_transpose(dz, T, E, p.Tp, nullptr, dzt, s));
            MOE_HIP(launch_transpose(static_cast<const float*>(x), T, d, p.Tp, mask, xt, s));
            GemmArgs g = dense(dzt, p.Tp, xt, p.Tp, p.Tp, part, d, desc->E, desc->d);
            g.nsplit = p.nsplit;
            g.split_stride = E * d;
            MOE_HIP(launch_gemm(g, DT_F32, false, EPI_STORE, TILE_SMALL, static_cast<int>(cdiv(E, tile_bm(TILE_SMALL))),
                                desc->d, false, s));
        }
    }
    if (dW_r && p.nsplit > 1) MOE_HIP(launch_sum_planes(part, p.nsplit, E * d, E * d, dW_r, s));
    return MOE_OK;
}

}  // extern "C"
