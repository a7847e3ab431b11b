// Expert projections with 4-bit weights: C = epi(A * B^T) over the tile
// table of the dispatch, A in bf16, the routed experts' B as OCP E2M1 codes
// (sign, two exponent bits of bias 1, one mantissa bit: 0, .5, 1, 1.5, 2, 3,
// 4, 6) with one E8M0 exponent per 32 consecutive columns of a row, the
// shared experts' B (riding in the same launch) in packed bf16.
//
// element (r, c) = code(r, c) * 2^(s(r, c / 32) - 127).  The product has two
// significant bits, so v_cvt_scalef32_pk_bf16_fp4 turns two codes and their
// scale into two bf16 operands without rounding, and the bf16 MFMA
// accumulates exact products in fp32: the 4 bits cost no accuracy beyond the
// weights' own, and half a VALU instruction per weight.
//
// Packed layout (MOE_LAYOUT_FRAG16, include/moe.h): blocks of 16 rows x 128
// columns, 1 KiB of codes and 64 bytes of scales.  Lane l of a block holds
// row l % 16, columns 32 (l / 16) .. + 31: one scale group, so a lane needs
// one scale byte per 16 bytes of codes.  The four MFMAs of a block take
// columns 32 g + 8 s .. + 7 from lane group g in step s for both operands: a
// permutation of K that the dot product does not see.
//
// Bound by the weights' bytes (0.53 per weight) until an expert has some 60
// rows, from there by the MFMAs and the conversions beside them.  The sums
// stay in fp32 through the K split and the combine; H is rounded, to the bf16
// the next MFMA takes (as in the bf16 and FP8 layers; norm-wise 1.6e-3, about
// the output's own rounding), and in latent layers x_lat and the sum R to two
// bf16 parts, 16 bits.
#include "common.hpp"
#include "jobs.hpp"
#include "launch.hpp"

#include <type_traits>

namespace moe {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Eight codes of one scale group -> one bf16 operand.
__device__ __forceinline__ uint4 fp4x8_to_bf16(uint32_t q, float scale) {
#define MOE_CVT(byte) __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, byte))
    return make_uint4(MOE_CVT(0), MOE_CVT(1), MOE_CVT(2), MOE_CVT(3));
#undef MOE_CVT
}

// 16 bytes read once: the weights, streamed past the cached activations.
__device__ __forceinline__ uint4 ldg16_once(const char* p) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ float silu_times(float g, float u) { return g / (1.0f + expf(-g)) * u; }

__device__ __forceinline__ void store4(bf16_t* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                                              f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// v as two bf16 parts, hi at p and the rest at p + lo (16 of v's bits; lo 0: hi alone).
__device__ __forceinline__ void store_parts(bf16_t* p, int64_t lo, const float (&v)[4]) {
    store4(p, v);
    if (!lo) return;
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = v[i] - bf16_to_f32(f32_to_bf16(v[i]));
    store4(p + lo, r);
}

// ---- few rows: weights streamed once, K split over the waves of a workgroup

// acc[j] += (row block j of the weights) * (activation rows), over the
// 128-column blocks k0, k0 + step, .. < kend.  w[j] / sc[j]: this lane's place
// in block 0 of row block j; x: this lane's row at column 32 (lane / 16).
// Everything comes straight from memory to the registers of the one wave that
// uses it, the next block's loads in flight while a block is used.  TWO: the
// activations come in two parts, the second xlo bytes behind the first, and
// every weight meets both.
// D blocks are in flight.  D = 1 leaves the registers for more waves, which
// then hide each other's latency: better where a wave has few blocks.
template <int RB, bool TWO>
struct Fp4Load {
    uint4 q[RB], x[TWO ? 8 : 4];
    uint32_t e[RB];
};
template <int RB, int D, bool TWO = false>
__device__ __forceinline__ void fp4_stream(f32x4 (&acc)[RB], const char* const (&w)[RB], const uint8_t* const (&sc)[RB],
                                           const char* x, int k0, int step, int kend, int64_t xlo = 0) {
    if (k0 >= kend) return;
    auto load = [&](Fp4Load<RB, TWO>& l, int k) {
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            l.q[j] = ldg16_once(w[j] + static_cast<int64_t>(k) * 1024);
            l.e[j] = sc[j][k * 64];
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            l.x[s] = ldg16(x + static_cast<int64_t>(k) * 256 + s * 16);
            if constexpr (TWO) l.x[4 + s] = ldg16(x + xlo + static_cast<int64_t>(k) * 256 + s * 16);
        }
    };
    auto use = [&](const Fp4Load<RB, TWO>& l) {
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            const float scale = __uint_as_float(l.e[j] << 23);
            const uint32_t c[4] = {l.q[j].x, l.q[j].y, l.q[j].z, l.q[j].w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint4 f = fp4x8_to_bf16(c[s], scale);
                acc[j] = Mfma<bf16_t>::run(f, l.x[s], acc[j]);
                if constexpr (TWO) acc[j] = Mfma<bf16_t>::run(f, l.x[4 + s], acc[j]);
            }
        }
    };
    if constexpr (D == 1) {
        for (int k = k0; k < kend; k += step) {
            Fp4Load<RB, TWO> l;
            load(l, k);
            use(l);
        }
    } else {
        Fp4Load<RB, TWO> l[D];
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (k0 + u * step < kend) load(l[u], k0 + u * step);
        for (int k = k0; k < kend; k += D * step) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                __builtin_amdgcn_sched_barrier(0);  // (left alone, the loads sink to their uses)
                if (k + u * step < kend) {
                    use(l[u]);
                    if (k + (D + u) * step < kend) load(l[u], k + (D + u) * step);
                }
            }
        }
    }
}
// The same for packed bf16 weights, over 32-column blocks, U in flight; x at column
// 8 (lane / 16).
template <int RB, int U, bool TWO = false>
__device__ __forceinline__ void bf16_stream(f32x4 (&acc)[RB], const char* const (&w)[RB], const char* x, int k0, int step,
                                            int kend, int64_t xlo = 0) {
    if (k0 >= kend) return;
    uint4 q[U][RB], xv[U], xl[TWO ? U : 1];
    auto load = [&](int u, int k) {
        if (k >= kend) return;  // (uniform)
#pragma unroll
        for (int j = 0; j < RB; ++j) q[u][j] = ldg16_once(w[j] + static_cast<int64_t>(k) * 1024);
        xv[u] = ldg16(x + static_cast<int64_t>(k) * 64);
        if constexpr (TWO) xl[u] = ldg16(x + xlo + static_cast<int64_t>(k) * 64);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, k0 + u * step);
    for (int k = k0; k < kend; k += U * step) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            __builtin_amdgcn_sched_barrier(0);
            if (k + u * step < kend) {
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    acc[j] = Mfma<bf16_t>::run(q[u][j], xv[u], acc[j]);
                    if constexpr (TWO) acc[j] = Mfma<bf16_t>::run(q[u][j], xl[u], acc[j]);
                }
                load(u, k + (U + u) * step);
            }
        }
    }
}

// A direct launch (no tile table: batches of up to kDirectT tokens): who
// shares an expert is found by each wave from the T K chosen ids themselves,
// which saves the launch of a dispatch and the wait for its tables.
struct DirectArgs {
    const int32_t* idx;  // [A] chosen ids
    int32_t A, K, e0, E; // A = T K; this slice's experts are e0 .. e0 + E - 1
    int32_t nsh;         // leading blocks that compute the shared experts
    int32_t h_rows;      // 1: activation row of assignment a is a (H), 0: a / K (tokens)
};
constexpr int kDirectT = 16, kDirectA = kDirectT * 16;

// Assignment a leads its expert's rows r0 .. r0 + 15 (those are the
// assignments to the same expert, in order) when its own rank among them is a
// multiple of 16; rows[] of this wave receives them.  Returns their number, 0
// if a leads none; *e the local expert.
__device__ __forceinline__ int direct_rows(const DirectArgs& d, int a, int* rows, int* e) {
    const int lane = threadIdx.x & 63;
    int id[kDirectA / 64];
#pragma unroll
    for (int i = 0; i < kDirectA / 64; ++i) id[i] = i * 64 + lane < d.A ? d.idx[i * 64 + lane] : d.idx[0];
    const int mine = d.idx[a];
    *e = mine - d.e0;
    if (static_cast<unsigned>(*e) >= static_cast<unsigned>(d.E)) return 0;
    int before = 0, total = 0;
    uint64_t m[kDirectA / 64];
#pragma unroll
    for (int i = 0; i < kDirectA / 64; ++i) {
        m[i] = __ballot(i * 64 + lane < d.A && id[i] == mine);
        const int off = a - i * 64;
        before += off >= 64 ? __popcll(m[i]) : off > 0 ? __popcll(m[i] & ((1ull << off) - 1)) : 0;
        total += __popcll(m[i]);
    }
    if (before & 15) return 0;
    int rank = -before;
#pragma unroll
    for (int i = 0; i < kDirectA / 64; ++i) {
        const int r = rank + __popcll(m[i] & ((1ull << lane) - 1));
        if (((m[i] >> lane) & 1) && r >= 0 && r < 16) rows[r] = i * 64 + lane;
        rank += __popcll(m[i]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return min(16, total - before);
}

// 16 activation rows x (16 RB) weight rows per workgroup (SwiGLU: RB/2 row
// blocks of the gate and the same RB/2 of the up matrix; a direct launch's
// shared blocks: RB/2 of these, so that the bf16 blocks are no heavier than
// the FP4 ones).  The NW waves split K, block by block in turn, with no
// barrier in the K loop; their partial sums meet in LDS at the end, added in
// wave order.  Small workgroups, because only many waves with loads of their
// own in flight keep the HBM busy.  Measured, 7168 x 2048: 16 tokens over 384
// experts and a shared one (direct), up 274 us for 1.76 GB and down 147 for 0.90,
// 6.0 to 6.5 TB/s, where a large copy reaches 4.7; 256 tokens over 48 experts
// up 115 to 128 us and down 67 to 70 for 0.75 and 0.37 GB, 5.3 to 6.5 TB/s; one
// token's up, 184 MB, 30 us.
// TWO: the routed experts' activation rows hold two parts, K columns each.
template <typename TC, int EPI, int NW, int D, bool DIRECT, bool TWO>
__global__ __launch_bounds__(64 * NW) void k_fp4_rows16(const GemmArgs a, const DirectArgs dir) {
    constexpr int BM = 16, RB = 4, NJ = EPI == EPI_SWIGLU ? RB / 2 : RB, BNO = 16 * NJ;
    __shared__ f32x4 red[NW][RB][64];
    __shared__ int rows_of[NW][16];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, grp = lane >> 4;

    int gi, expert = 0, rows, n0, row, crow;  // this lane's activation row and its row of C
    if constexpr (DIRECT) {
        const int b = static_cast<int>(blockIdx.x);
        if (b < dir.nsh) {
            gi = 1;
            rows = dir.A / dir.K;
            n0 = b * (BNO / 2);
            row = crow = r16 < rows ? r16 : 0;
        } else {
            gi = 0;
            const int k = b - dir.nsh;
            n0 = (k % a.ntn) * BNO;
            rows = direct_rows(dir, k / a.ntn, rows_of[wid], &expert);
            if (!rows) return;
            crow = rows_of[wid][r16 < rows ? r16 : 0];
            row = dir.h_rows ? crow : crow / dir.K;
        }
    } else {
        Job jb;
        // (the bf16 shared pairs, four times the bytes of a routed one, first:
        // 1040 us against 1080, 64 tokens over 384 experts and a shared one)
        if (!pick_job<BM, BNO>(a, jb, 0x7fffffff)) return;
        gi = jb.gi;
        expert = jb.expert;
        rows = jb.rows;
        n0 = jb.n0;
        crow = jb.row0 + (r16 < rows ? r16 : 0);  // (rows past the tile's repeat its first)
        const int32_t* map = gi ? a.g[1].rowmap : a.g[0].rowmap;
        row = map ? map[crow] : crow;
    }
    const GemmGroup& G = gi ? a.g[1] : a.g[0];
    const int K = G.seg[0].K;
    const char* x = static_cast<const char*>(G.seg[0].A) + static_cast<int64_t>(row) * G.seg[0].lda * 2;
    int nj = NJ;  // output row blocks of this tile
    if constexpr (DIRECT) nj = gi ? NJ / 2 : NJ;

    f32x4 acc[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto block_of = [&](int j) { return min(n0 / 16 + j, G.N / 16 - 1); };  // clamped to the matrix
    if (gi == 0) {
        const int kb = K / 128;
        const int64_t eb = static_cast<int64_t>(expert) * G.b_estride, es = static_cast<int64_t>(expert) * G.s_estride;
        const char* w[RB];
        const uint8_t* sc[RB];
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            const bool up = EPI == EPI_SWIGLU && j >= NJ;
            const int64_t blk = static_cast<int64_t>(block_of(j % NJ)) * kb;
            w[j] = static_cast<const char*>(up ? G.seg[0].Bu : G.seg[0].B) + eb + blk * 1024 + lane * 16;
            sc[j] = (up ? G.bsu : G.bs) + es + blk * 64 + lane;
        }
        fp4_stream<RB, D, TWO>(acc, w, sc, x + grp * 64, wid, NW, kb, K * 2);
    } else {
        constexpr int RS = DIRECT ? RB / 2 : RB, NS = EPI == EPI_SWIGLU ? RS / 2 : RS;
        const char* w[RS];
        f32x4 part[RS];
#pragma unroll
        for (int j = 0; j < RS; ++j) {
            const void* m = (EPI == EPI_SWIGLU && j >= NS) ? G.seg[0].Bu : G.seg[0].B;
            w[j] = static_cast<const char*>(m) + static_cast<int64_t>(block_of(j % NS)) * (K / 32) * 1024 + lane * 16;
            part[j] = acc[j];
        }
        bf16_stream<RS, DIRECT ? 4 : 1>(part, w, x + grp * 16, wid, NW, K / 32);
#pragma unroll
        for (int j = 0; j < RS; ++j) acc[EPI == EPI_SWIGLU && j >= NS ? NJ + j - NS : j] = part[j];
    }

    // accumulator j of a lane: activation row lane % 16, weight rows
    // 4 (lane / 16) .. + 3 of row block j
#pragma unroll
    for (int j = 0; j < RB; ++j) red[wid][j][lane] = acc[j];
    __syncthreads();
    if (wid >= nj) return;
    auto total = [&](int j) {
        f32x4 v = red[0][j][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            const f32x4 o = red[w][j][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += o[i];
        }
        return v;
    };
    const f32x4 g = total(wid);
    float v[4] = {g[0], g[1], g[2], g[3]};
    if (EPI == EPI_SWIGLU) {
        const f32x4 u = total(wid + NJ);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu_times(v[i], u[i]);
    }
    const int col = n0 + wid * 16 + grp * 4;
    if (r16 < rows && col < G.N) store4(static_cast<TC*>(G.C) + static_cast<int64_t>(crow) * G.ldc + col, v);
}

// Dense maps of a few rows (the latent form's): C = A B^T over up to two K
// segments of packed bf16 (their rows of A in one or two parts), 16 rows x 32 columns per workgroup, K split over
// the waves as above.  lo: C is written in two parts, that far apart.
constexpr int kDenseNW = 8;
__global__ __launch_bounds__(64 * kDenseNW) void k_dense_rows16(const GemmArgs a, int64_t lo) {
    constexpr int RB = 2;
    __shared__ f32x4 red[kDenseNW][RB][64];
    const GemmGroup& G = a.g[0];
    const int lane = threadIdx.x & 63, r16 = lane & 15, grp = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * RB, row0 = blockIdx.y * 16;
    const int64_t row = min(row0 + r16, a.M - 1);
    f32x4 acc[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < G.nseg; ++i) {
        const GemmSeg& S = i ? G.seg[1] : G.seg[0];
        const int kb = S.K / 32;
        const char* w[RB];
#pragma unroll
        for (int j = 0; j < RB; ++j)
            w[j] = static_cast<const char*>(S.B) + static_cast<int64_t>(min(n0 / 16 + j, G.N / 16 - 1)) * kb * 1024 + lane * 16;
        const char* x = static_cast<const char*>(S.A) + row * S.lda * 2 + grp * 16;
        if (S.two)
            bf16_stream<RB, 4, true>(acc, w, x, wid, kDenseNW, kb, S.K * 2);
        else
            bf16_stream<RB, 4>(acc, w, x, wid, kDenseNW, kb);
    }
#pragma unroll
    for (int j = 0; j < RB; ++j) red[wid][j][lane] = acc[j];
    __syncthreads();
    if (wid >= RB) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kDenseNW; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += red[w][wid][lane][j];
    const int col = n0 + wid * 16 + grp * 4;
    if (row0 + r16 < a.M && col < G.N) store_parts(static_cast<bf16_t*>(G.C) + row * G.ldc + col, lo, v);
}

// Down projection and combine of a single token in one: block (n, t) forms
// out[t, 16 n .. 16 n + 15] = shared + sum_k w_k (W_down[e_k] H[t K + k]),
// the waves taking the token's experts (or parts of their K) in turn, each
// weighting its own sum in fp32.  The one activation row fills one of the
// MFMA's 16, which costs nothing here: the weights' bytes set the pace.  91 MB
// in 21.8 us (4.2 TB/s; a launch of this length is a third latency).  Against
// the down projection and the combine apart, whole layers of 7168 x 2048: 55.6
// / 57.3 us at one token; at two every token streams the weights it shares with
// the other for itself, 92 / 84 us, so fp4_fused asks for one.
constexpr int kFusedNW = 8;
__global__ __launch_bounds__(64 * kFusedNW) void k_fp4_down_combine(const GemmArgs a, const DirectArgs d,
                                                                   const float* __restrict__ wt,
                                                                   bf16_t* __restrict__ out, int64_t ldo, int64_t lo) {
    __shared__ f32x4 red[kFusedNW][64];
    const int lane = threadIdx.x & 63, grp = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = blockIdx.x, t = blockIdx.y;
    const GemmGroup &G = a.g[0], &S = a.g[1];
    const int kb = G.seg[0].K / 128;
    const int parts = d.K >= kFusedNW ? 1 : kFusedNW / d.K, per = (kb + parts - 1) / parts;
    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
    if (S.N) {  // first: its weights' addresses wait for no id
        const int ks = S.seg[0].K / 32;
        f32x4 acc[1] = {sum};
        const char* const w[1] = {static_cast<const char*>(S.seg[0].B) + static_cast<int64_t>(n) * ks * 1024 + lane * 16};
        bf16_stream<1, 4>(acc, w, static_cast<const char*>(S.seg[0].A) + static_cast<int64_t>(t) * S.seg[0].lda * 2 + grp * 16,
                       wid, kFusedNW, ks);
        sum = acc[0];
    }
    for (int i = wid; i < d.K * parts; i += kFusedNW) {
        const int as = t * d.K + i / parts, p = i % parts;
        const int e = d.idx[as] - d.e0;
        if (static_cast<unsigned>(e) >= static_cast<unsigned>(d.E)) continue;
        f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
        const int64_t blk = static_cast<int64_t>(n) * kb;
        const char* const w[1] = {static_cast<const char*>(G.seg[0].B) + e * G.b_estride + blk * 1024 + lane * 16};
        const uint8_t* const sc[1] = {G.bs + e * G.s_estride + blk * 64 + lane};
        const char* x = static_cast<const char*>(G.seg[0].A) + static_cast<int64_t>(as) * G.seg[0].lda * 2 + grp * 64;
        fp4_stream<1, 4>(acc, w, sc, x, p * per, 1, min(kb, (p + 1) * per));
        const float c = wt[as];
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = fmaf(c, acc[0][j], sum[j]);
    }
    red[wid][lane] = sum;
    __syncthreads();
    if (wid || (lane & 15)) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kFusedNW; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += red[w][lane][j];
    store_parts(out + t * ldo + n * 16 + grp * 4, lo, v);
}

// Many rows: BM = 16 MT activation rows x 256 weight rows per workgroup
// (SwiGLU: 128 of the gate and the same 128 of the up matrix), each wave all
// BM rows x 64 weight rows.  The activations, which every wave needs, go
// through LDS in stages of 128 columns (two buffers, filled through registers
// loaded two stages ahead, one barrier a stage); each wave's own weights go
// straight to its registers.  A code is converted once and used by MT MFMAs.
// LDS row r keeps its 16-byte chunk c at c ^ (r % 16), so the 16 rows that a
// fragment read touches at one chunk lie in 16 different bank groups.
// TWO (rows of two parts, K columns each): every K block takes two stages, one
// for either part, and its weights come through the caches twice.
// Measured, 2048 tokens over 48 of 384 experts of 7168 x 2048 and a shared one
// (43 rows an expert): up 296 to 322 us, down 168 to 182 us, 361 GFLOP together
// at 0.72 to 0.78 PFLOP/s (a large bf16 product of the library: 1.37) while
// 2.1 GB stream past, 0.8 of them for the shared pairs.
template <typename TC, int EPI, int MT, bool ONCE, bool TWO>
struct Fp4Tile {
    static constexpr int BM = 16 * MT, RB = 4, NJ = EPI == EPI_SWIGLU ? RB / 2 : RB;
    static constexpr int BNO = 4 * 16 * NJ;            // output columns per workgroup
    static constexpr int STAGE = BM * 256;             // bytes
    static constexpr int XL = STAGE / 16 / 256;        // 16-byte pieces per thread and stage

    __device__ __forceinline__ static void run(const GemmArgs& a, const Job& jb, char* lds) {
        const GemmGroup& G = jb.gi ? a.g[1] : a.g[0];
        const int tid = threadIdx.x, lane = tid & 63;
        const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int r16 = lane & 15, grp = lane >> 4;
        const int K = G.seg[0].K, kb = (K + 127) / 128;
        const int two = TWO && jb.gi == 0 ? 1 : 0, nst = kb << two;  // stage st: K block st >> two, part st & two

        // this thread's pieces of a stage: row (tid / 16) + 16 i, chunk tid % 16
        const char* xs[XL];
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int r = (tid >> 4) + 16 * i;
            const int p = jb.row0 + (r < jb.rows ? r : 0);
            const int64_t arow = G.rowmap ? G.rowmap[p] : p;
            xs[i] = static_cast<const char*>(G.seg[0].A) + arow * G.seg[0].lda * 2;
        }
        const int chunk = tid & 15;
        const int wpos = (tid >> 4) * 256 + ((chunk ^ (tid >> 4)) << 4);
        uint4 xr[2][XL];
        auto load_x = [&](int st, int i) {
            int off = min((st >> two) * 256 + chunk * 16, K * 2 - 16);  // (past the end; the last stage may hold 64 columns)
            if (TWO) off += (st & two) * K * 2;
            return ldg16(xs[i] + off);
        };
        auto write_x = [&](int st, int i, const uint4& v) {
            *reinterpret_cast<uint4*>(lds + (st & 1) * STAGE + wpos + i * 16 * 256) = v;
        };
        auto read_x = [&](int st, int c, uint4 (&x)[MT]) {  // chunk c of rows r16 + 16 i
            const char* b = lds + (st & 1) * STAGE + r16 * 256 + ((c ^ r16) << 4);
#pragma unroll
            for (int i = 0; i < MT; ++i) x[i] = *reinterpret_cast<const uint4*>(b + i * 16 * 256);
        };

        int rb[RB];
#pragma unroll
        for (int j = 0; j < RB; ++j) rb[j] = min(jb.n0 / 16 + wid * NJ + j % NJ, G.N / 16 - 1);
        f32x4 acc[RB][MT];
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

        // Loads run two stages ahead: stage st issues those of st + 2 into the
        // registers that its own came through, and writes st + 1, loaded a
        // whole stage ago, to the other buffer.  A stage has 16 steps of MT
        // MFMAs and does a little of this after each: a burst of loads or of
        // LDS writes holds up the MFMAs behind it.
        auto tick = [&](int st, auto par, int k) {
            constexpr int P = decltype(par)::value;
#pragma unroll
            for (int i = 0; i < XL; ++i) {
                if (k == 1 + i) xr[P][i] = load_x(st + 2, i);
                if (k == 8 + i) write_x(st + 1, i, xr[1 - P][i]);
            }
        };
        auto stages = [&](auto&& body) {
#pragma unroll
            for (int i = 0; i < XL; ++i) {
                xr[0][i] = load_x(0, i);
                xr[1][i] = load_x(1, i);
            }
#pragma unroll
            for (int i = 0; i < XL; ++i) write_x(0, i, xr[0][i]);
            __syncthreads();
            int st = 0;
            for (; st + 1 < nst; st += 2) {
                body(st, std::integral_constant<int, 0>{});
                __syncthreads();
                body(st + 1, std::integral_constant<int, 1>{});
                __syncthreads();
            }
            if (st < nst) body(st, std::integral_constant<int, 0>{});
        };
        if (jb.gi == 0) {
            const int64_t eb = static_cast<int64_t>(jb.expert) * G.b_estride;
            const int64_t es = static_cast<int64_t>(jb.expert) * G.s_estride;
            const char* w[RB];
            const uint8_t* sc[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                const bool up = EPI == EPI_SWIGLU && j >= NJ;
                w[j] = static_cast<const char*>(up ? G.seg[0].Bu : G.seg[0].B) + eb +
                       static_cast<int64_t>(rb[j]) * kb * 1024 + lane * 16;
                sc[j] = (up ? G.bsu : G.bs) + es + static_cast<int64_t>(rb[j]) * kb * 64 + lane;
            }
            uint4 q[2][RB];
            uint32_t e[2][RB];
            auto load_w = [&](int st, int j, uint4& o, uint32_t& oe) {
                const int k = min(st, nst - 1) >> two;
                o = ONCE ? ldg16_once(w[j] + static_cast<int64_t>(k) * 1024) : ldg16(w[j] + static_cast<int64_t>(k) * 1024);
                oe = sc[j][k * 64];
            };
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                load_w(0, j, q[0][j], e[0][j]);
                load_w(1, j, q[1][j], e[1][j]);
            }
            stages([&](int st, auto par) {
                constexpr int P = decltype(par)::value;
                uint4 x[2][MT], f[2];
                read_x(st, 4 * grp, x[0]);
                auto convert = [&](int k) {  // fragment k: slab k / RB, row block k % RB
                    const uint4& c = q[P][k % RB];
                    const uint32_t cw = k / RB == 0 ? c.x : k / RB == 1 ? c.y : k / RB == 2 ? c.z : c.w;
                    return fp4x8_to_bf16(cw, __uint_as_float(e[P][k % RB] << 23));
                };
                f[0] = convert(0);
                __builtin_amdgcn_sched_barrier(0);  // (left alone, loads sink to their uses)
#pragma unroll
                for (int k = 0; k < 4 * RB; ++k) {
                    const int s = k / RB, j = k % RB;
                    if (j == 0 && s < 3) read_x(st, 4 * grp + s + 1, x[(s + 1) & 1]);
                    if (k + 1 < 4 * RB) f[(k + 1) & 1] = convert(k + 1);
#pragma unroll
                    for (int i = 0; i < MT; ++i) acc[j][i] = Mfma<bf16_t>::run(f[k & 1], x[s & 1][i], acc[j][i]);
                    // the next fragment's conversions, and the next slab's reads, between the MFMAs
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, (4 + MT - 1) / MT, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    tick(st, par, k);
                    // only now, past the codes' last use: loaded earlier, they would sit in other registers
                    // and be copied back at the loop's end, a copy that waits for every load in flight
                    if (s == 3) load_w(st + 2, j, q[P][j], e[P][j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            });
        } else {
            const int nsl = K / 32;  // 32-column blocks, loaded four ahead
            const char* w[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                w[j] = static_cast<const char*>((EPI == EPI_SWIGLU && j >= NJ) ? G.seg[0].Bu : G.seg[0].B) +
                       static_cast<int64_t>(rb[j]) * nsl * 1024 + lane * 16;
            uint4 q[4][RB];
            auto load_w = [&](int sl, int j) { return ldg16(w[j] + static_cast<int64_t>(min(sl, nsl - 1)) * 1024); };
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int j = 0; j < RB; ++j) q[s][j] = load_w(s, j);
            stages([&](int st, auto par) {
                uint4 x[2][MT];
                read_x(st, grp, x[0]);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (s < 3) read_x(st, 4 * (s + 1) + grp, x[(s + 1) & 1]);
                    const bool use = 4 * st + s < nsl;  // (uniform: the last stage may hold two blocks)
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int j = 0; j < RB; ++j) {
                        if (use)
#pragma unroll
                            for (int i = 0; i < MT; ++i) acc[j][i] = Mfma<bf16_t>::run(q[s][j], x[s & 1][i], acc[j][i]);
                        __builtin_amdgcn_sched_barrier(0);
                        tick(st, par, s * RB + j);
                        q[s][j] = load_w(4 * st + s + 4, j);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            });
        }

        // acc[j][i] of a lane: row 16 i + lane % 16, weight rows 4 (lane / 16) .. + 3 of row block j
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = 16 * i + r16;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int col = jb.n0 + (wid * NJ + j) * 16 + grp * 4;
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = EPI == EPI_SWIGLU ? silu_times(acc[j][i][k], acc[(j + NJ) % RB][i][k]) : acc[j][i][k];
                if (r < jb.rows && col < G.N)
                    store4(static_cast<TC*>(G.C) + static_cast<int64_t>(jb.row0 + r) * G.ldc + col, v);
            }
        }
    }
};

// A tile with fewer rows (an expert's last) runs the body of the next quarter
// of BM.
template <typename TC, int EPI, int MT, bool ONCE, bool TWO>
__global__ __launch_bounds__(256, 2) void k_fp4_tile(const GemmArgs a) {
    using Tile = Fp4Tile<TC, EPI, MT, ONCE, TWO>;
    __shared__ __attribute__((aligned(1024))) char lds[2 * Tile::STAGE];
    Job jb;
    // (48 experts of 7168 x 2048 and a shared one, shared pairs first or last:
    // 276 / 310 us at 512 tokens, which make 128 of them in the up projection;
    // 536 / 513 at 2048, where they would fill every CU)
    if (!pick_job<Tile::BM, Tile::BNO>(a, jb, 256)) return;
    if (jb.rows <= Tile::BM / 4)
        Fp4Tile<TC, EPI, MT / 4, ONCE, TWO>::run(a, jb, lds);
    else if (jb.rows <= Tile::BM / 2)
        Fp4Tile<TC, EPI, MT / 2, ONCE, TWO>::run(a, jb, lds);
    else if (jb.rows <= Tile::BM / 4 * 3)
        Fp4Tile<TC, EPI, MT / 4 * 3, ONCE, TWO>::run(a, jb, lds);
    else
        Tile::run(a, jb, lds);
}

// Row-major codes and scales -> blocks of 16 rows x 128 columns: one thread
// per 16 bytes of codes, which are a lane's share of a block as they stand,
// and their scale byte.
__global__ __launch_bounds__(256) void k_pack_fp4(const uint4* __restrict__ src, const uint8_t* __restrict__ ssrc,
                                                  uint4* __restrict__ dst, uint8_t* __restrict__ sdst, int64_t pieces,
                                                  int rows, int cols) {
    const int64_t per = static_cast<int64_t>(rows) * cols / 32;  // pieces per matrix
    const int kb = cols / 128, pc = cols / 32;
    for (int64_t q = blockIdx.x * 256ll + threadIdx.x; q < pieces; q += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t m = q / per, rem = q % per, blk = rem / 64;
        const int l = static_cast<int>(rem % 64);
        const int64_t i = blk / kb, j = blk % kb;
        const int64_t from = m * per + (i * 16 + (l & 15)) * pc + j * 4 + (l >> 4);
        dst[q] = src[from];
        sdst[q] = ssrc[from];
    }
}

// fp32 [rows, n] -> bf16 [rows, 2 n]: a row's upper parts, then what they leave.
__global__ __launch_bounds__(256) void k_two_parts(const float4* __restrict__ src, int64_t pieces, int n,
                                                   bf16_t* __restrict__ dst) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < pieces; i += static_cast<int64_t>(gridDim.x) * 256) {
        const float4 f = src[i];
        const float v[4] = {f.x, f.y, f.z, f.w};
        const int64_t r = i / (n / 4), c = i % (n / 4) * 4;
        store_parts(dst + r * 2 * n + c, n, v);
    }
}

template <typename TC, int EPI, bool TWO>
hipError_t launch_t(const GemmArgs& args, int bm, bool once, int max_tiles, int max_n, hipStream_t stream) {
    const int bno = (bm == 16 ? 64 : 256) / (EPI == EPI_SWIGLU ? 2 : 1);
    GemmArgs a = args;
    a.ntn = (max_n + bno - 1) / bno;
    if (static_cast<int64_t>(max_tiles) * a.ntn >= (int64_t{1} << 31) - 64) return hipErrorInvalidValue;
    const dim3 grid(job_blocks(max_tiles, a.ntn));
    if (bm == 16)
        hipLaunchKernelGGL((k_fp4_rows16<TC, EPI, 4, 1, false, TWO>), grid, dim3(256), 0, stream, a, DirectArgs{});
    else if (once && !TWO)
        hipLaunchKernelGGL((k_fp4_tile<TC, EPI, 4, !TWO, TWO>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_fp4_tile<TC, EPI, 4, false, TWO>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

// One K segment per group; the routed matrices in whole 16 x 128 blocks, the
// shared ones in whole 16 x 32 blocks and 64-column steps.
bool fp4_fits(const GemmArgs& a, Epi epi, bool two) {
    const GemmGroup &R = a.g[0], &S = a.g[1];
    if (two && (epi != EPI_SWIGLU || R.seg[0].lda < 2ll * R.seg[0].K)) return false;
    return a.nsplit == 1 && R.nseg == 1 && R.N > 0 && R.N % 16 == 0 && R.seg[0].K > 0 && R.seg[0].K % 128 == 0 && R.bs &&
           (epi != EPI_SWIGLU || R.bsu) && (!S.N || (S.nseg == 1 && S.N % 16 == 0 && S.seg[0].K % 64 == 0));
}

}  // namespace

// 64-row tiles from 8 rows per expert, or from 4 when shared experts, whose
// every 16 tokens would be another pass over their weights, ride along; where
// the 64-row tiles of the up projection are fewer than the CUs, from 16.
// Measured (16-row against 64-row tiles), 7168 x 2048: 48 of 384 experts alone
// 202 / 212 us at 5.3 rows, 218 / 219 at 8, 255 / 225 at 10.7, 324 / 235 at 16;
// 384 experts and a shared one 1337 / 1318 us at 2.7 rows, 1495 / 1418 at 4,
// 1613 / 1460 at 5.3, 2090 / 1599 at 10.7; 48 experts of 1024 x 256 and a shared
// one (96 tiles) 33 / 36 us at 5.3, 32 / 40 at 10.7, 53 / 48 at 21.  128-row
// tiles lost to 64-row ones even at 341 rows (1.40 against 1.35 ms): their
// accumulators leave room for one wave per SIMD.
int fp4_bm(int64_t rows, int E, int F, bool shared) {
    const bool few = static_cast<int64_t>(E) * ((F + 127) / 128) < 256;
    return rows < (few ? 16 : shared ? 4 : 8) * static_cast<int64_t>(E) ? 16 : 64;
}

hipError_t launch_gemm_fp4(const GemmArgs& args, Epi epi, bool two, int bm, bool once, int max_tiles, int max_n,
                           hipStream_t stream) {
    if (max_tiles <= 0 || max_n <= 0) return hipSuccess;
    if ((bm != 16 && bm != 64) || !args.tiles || !fp4_fits(args, epi, two)) return hipErrorInvalidValue;
    if (two) return launch_t<bf16_t, EPI_SWIGLU, true>(args, bm, once, max_tiles, max_n, stream);
    if (epi == EPI_SWIGLU) return launch_t<bf16_t, EPI_SWIGLU, false>(args, bm, once, max_tiles, max_n, stream);
    return launch_t<float, EPI_STORE, false>(args, bm, once, max_tiles, max_n, stream);
}

bool fp4_direct(int64_t T) { return T <= kDirectT; }
bool fp4_fused(int64_t T) { return T == 1; }

hipError_t launch_fp4_direct(const GemmArgs& args, Epi epi, bool two, const int32_t* idx, int T, int K, int e0, int E,
                             hipStream_t stream) {
    if (T < 1 || T > kDirectT || K < 1 || K > kDirectA / kDirectT || !fp4_fits(args, epi, two)) return hipErrorInvalidValue;
    const int bno = epi == EPI_SWIGLU ? 32 : 64;
    GemmArgs a = args;
    a.ntn = (a.g[0].N + bno - 1) / bno;
    const int nsh = a.g[1].N ? (a.g[1].N + bno / 2 - 1) / (bno / 2) : 0;
    const DirectArgs d{idx, T * K, K, e0, E, nsh, epi == EPI_SWIGLU ? 0 : 1};
    const dim3 grid(static_cast<unsigned>(nsh + T * K * a.ntn));
    // (two parts: one block of K in flight leaves two workgroups to a CU; two in
    // flight took 99 us against 96 at 8 tokens, 132 / 128 at 16, 50 / 52 at one)
    if (two)
        hipLaunchKernelGGL((k_fp4_rows16<bf16_t, EPI_SWIGLU, 8, 1, true, true>), grid, dim3(512), 0, stream, a, d);
    else if (epi == EPI_SWIGLU)
        hipLaunchKernelGGL((k_fp4_rows16<bf16_t, EPI_SWIGLU, 8, 2, true, false>), grid, dim3(512), 0, stream, a, d);
    else
        hipLaunchKernelGGL((k_fp4_rows16<float, EPI_STORE, 4, 1, true, false>), grid, dim3(256), 0, stream, a, d);
    return hipGetLastError();
}

hipError_t launch_fp4_down_combine(const GemmArgs& args, const int32_t* idx, const float* w, int T, int K, int e0, int E,
                                   uint16_t* out, int64_t ldo, int64_t lo, hipStream_t stream) {
    if (T < 1 || K < 1 || !fp4_fits(args, EPI_STORE, false) || (args.g[1].N && args.g[1].N != args.g[0].N))
        return hipErrorInvalidValue;
    const DirectArgs d{idx, T * K, K, e0, E, 0, 1};
    hipLaunchKernelGGL(k_fp4_down_combine, dim3(args.g[0].N / 16, T), dim3(64 * kFusedNW), 0, stream, args, d, w, out,
                       ldo, lo);
    return hipGetLastError();
}

hipError_t launch_dense_rows16(const GemmArgs& a, int64_t lo, hipStream_t stream) {
    const GemmGroup& G = a.g[0];
    if (a.nsplit != 1 || a.M < 1 || G.nseg < 1 || G.nseg > 2 || G.N < 16 || G.N % 16) return hipErrorInvalidValue;
    for (int i = 0; i < G.nseg; ++i)
        if (G.seg[i].K < 32 || G.seg[i].K % 32 || (G.seg[i].two && G.seg[i].lda < 2ll * G.seg[i].K))
            return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_dense_rows16, dim3((G.N + 31) / 32, (a.M + 15) / 16), dim3(64 * kDenseNW), 0, stream, a, lo);
    return hipGetLastError();
}

hipError_t launch_two_parts(const float* src, int64_t rows, int n, uint16_t* dst, hipStream_t stream) {
    if (rows < 1 || n < 4 || n % 4) return hipErrorInvalidValue;
    const int64_t pieces = rows * (n / 4), blocks = (pieces + 255) / 256;
    hipLaunchKernelGGL(k_two_parts, dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)), dim3(256), 0, stream,
                       reinterpret_cast<const float4*>(src), pieces, n, dst);
    return hipGetLastError();
}

hipError_t launch_pack_fp4(const uint8_t* src, const uint8_t* ssrc, uint8_t* dst, uint8_t* sdst, int64_t count,
                           int rows, int cols, hipStream_t stream) {
    if (count <= 0 || rows <= 0 || cols <= 0) return hipSuccess;
    if (rows % 16 || cols % 128) return hipErrorInvalidValue;
    const int64_t pieces = count * rows * (cols / 32);
    const int64_t blocks = (pieces + 255) / 256;
    hipLaunchKernelGGL(k_pack_fp4, dim3(static_cast<unsigned>(blocks < 16384 ? blocks : 16384)), dim3(256), 0, stream,
                       reinterpret_cast<const uint4*>(src), ssrc, reinterpret_cast<uint4*>(dst), sdst, pieces, rows, cols);
    return hipGetLastError();
}

}  // namespace moe
