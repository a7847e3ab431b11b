// The SwiGLU experts on rows sorted by expert, forward and backward: six grouped
// products in bf16 with fp32 accumulators.  With a = x W_gate^T, b = x W_up^T,
// s = sigmoid(a), h = a s b of an expert's rows:
//   EXP_UP       a, b and h                     rows x (2 F),  K = d
//   EXP_DOWN     y = h W_down^T                 rows x d,      K = F
//   EXP_DH       dh = dy W_down, and from it    rows x F,      K = d
//                db = dh a s,  da = dh b s (1 + a (1 - s))
//   EXP_DX       dx = da W_gate + db W_up       rows x d,      K = 2 F
//   EXP_DW_DOWN  dW_down = dy^T h               d x F,         K = rows
//   EXP_DW_UP    [dW_gate; dW_up] = [da; db]^T x   2 F x d,    K = rows
// h, da and db are rounded to bf16, as the activations of the layer are.  a and b are
// kept in fp32 between the calls: in bf16 they would add as much to the gradients' error as
// all else (dW_gate and dx of normal rows: 3.1e-3 of the 2-norm against 2.4e-3, of
// which 1.7e-3 is the result's own rounding), and they are 2% of the bytes at 683 rows an expert.
#include <type_traits>

#include "common.hpp"
#include "experts.hpp"

namespace moe {
namespace {

// An operand of a product C[m, n] = sum_k A[m, k] B[n, k] lies in memory either
// with its k side by side (rows: a row of the matrix is one m or n) or with its m
// or n side by side (columns: a row is one k; read transposed from LDS).
//
// A block of four waves holds a tile of BM x 256 in registers, over slabs of 32
// k.  A slab of both operands is (BM + 256) x 64 bytes and goes from global
// memory straight into one of four LDS slots (global_load_lds_dwordx4, 1 KiB per
// wave and instruction).  In the middle of slab b every wave waits for its loads of
// b + 1, issued two slabs before, and meets the others: after that b + 1 may be
// read, and the slot of b - 1, which nobody reads any more, takes b + 3.
// A wave holds the A fragments of a slab, and B's one ahead of their products; those of
// A are replaced one by one under the slab's last products.
//
// Rows operand: a 1 KiB block holds 16 rows x 32 k; 16-byte chunk c of row r at r
// 64 + (c ^ (r / 2 % 4)) 16, so that four neighbouring lanes load 64 bytes of a
// row, and eight lanes that read one chunk of eight rows meet all banks once.
// Columns operand: a block holds 2 k x 256 columns; 32-byte chunk c of row r at c
// ^ (r % 4 + 4 (r / 8 % 2)) (see k_dw).
// A lane has four neighbouring columns of each product; two of them are exchanged
// between the lanes of neighbouring groups of 16 for eight: 16-byte stores.
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void dma(const char* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma(const char* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
// This wave's loads but the newest N, and its reads of LDS, have landed; then all waves'.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// What rows behind an expert's last one are read as in the columns operands.
__device__ const uint4 kZero16 = {0, 0, 0, 0};

struct Job {  // a tile: its expert, that expert's rows, and the tile's place in C
    int e, r0, rows, m0, nt;
};

template <int KIND, int BM>
struct Tile {
    static constexpr bool kDw = KIND == EXP_DW_DOWN || KIND == EXP_DW_UP;
    static constexpr bool kACol = kDw, kBCol = kDw || KIND == EXP_DH || KIND == EXP_DX;
    static constexpr bool kPair = KIND == EXP_UP;          // 128 columns of W_gate and the same of W_up
    static constexpr int kWM = BM == 256 ? 2 : 1, kWN = 4 / kWM;
    static constexpr int MI = BM / 16 / kWM, NJ = 16 / kWN;  // fragments of a wave
    static constexpr int NA = BM / 16, NB = 16;              // 1 KiB blocks of a slab
    static constexpr int kSlot = (NA + NB) * 1024;
    static constexpr int LA = NA / 4, LB = NB / 4, NL = LA + LB;  // loads of a wave
    static constexpr int kN = kPair ? 128 : 256;                // columns of C per tile
};

// The tile of job `lin`, expert by expert, M tiles side by side; rows == 0: none.
template <int KIND, int BM>
__device__ __forceinline__ Job find_job(const ExpertsArgs& a, int ntm, int ntn) {
    const int lane = threadIdx.x & 63;
    auto clamped = [&](int e) { return static_cast<int>(min(max(static_cast<int64_t>(a.off[e]), int64_t(0)), a.R)); };
    // blocks go to the eight XCDs round robin: each takes one stretch of the list
    if (Tile<KIND, BM>::kDw) {
        const int total = a.E * ntm * ntn, lin = xcd_slot_pair(static_cast<int>(blockIdx.x), total, total);
        if (lin < 0) return Job{0, 0, 0, 0, -1};
        const int e = lin / (ntm * ntn), in = lin % (ntm * ntn);
        const int r0 = clamped(e), r1 = clamped(e + 1);
        return Job{e, r0, max(r1 - r0, 0), in % ntm * BM, in / ntm};
    }
    // tiles of all experts, then those before this one's
    int total = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        int n = e < a.E ? max(clamped(e + 1) - clamped(e), 0) : 0;
        n = (n + BM - 1) / BM;
#pragma unroll
        for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
        total += n;
    }
    const int lin = xcd_slot_pair(static_cast<int>(blockIdx.x), total * ntn, total * ntn);
    if (lin < 0) return Job{0, 0, 0, 0, -1};
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        const int r0 = e < a.E ? clamped(e) : 0, rows = e < a.E ? max(clamped(e + 1) - r0, 0) : 0;
        const int n = (rows + BM - 1) / BM;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(incl, o);
            if (lane >= o) incl += v;
        }
        const int first = before + incl - n;
        const uint64_t mine = __ballot(n > 0 && first * ntn <= lin && lin < (first + n) * ntn);
        if (mine) {
            const int l = __ffsll(static_cast<unsigned long long>(mine)) - 1;
            const int in = lin - __shfl(first, l) * ntn, m = __shfl(n, l);
            return Job{e0 + l, __shfl(r0, l), __shfl(rows, l), in % m * BM, in / m};
        }
        before += __shfl(incl, 63);
    }
    return Job{0, 0, 0, 0, -1};
}

__device__ __forceinline__ float sigmoid(float a) { return 1.f / (1.f + __expf(-a)); }

__device__ __forceinline__ uint4 pack8v(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int KIND, int BM>
__global__ __launch_bounds__(256, BM == 256 ? 1 : 2) void k_experts(const ExpertsArgs a, int ntm, int ntn) {
    using S = Tile<KIND, BM>;
    constexpr int MI = S::MI, NJ = S::NJ;
    __shared__ __attribute__((aligned(1024))) char lds[4 * S::kSlot];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, grp = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wid / S::kWN, wn = wid % S::kWN;
    Job job = find_job<KIND, BM>(a, ntm, ntn);
    if (job.nt < 0) return;
    job.e = __builtin_amdgcn_readfirstlane(job.e);
    job.r0 = __builtin_amdgcn_readfirstlane(job.r0);
    job.rows = __builtin_amdgcn_readfirstlane(job.rows);
    job.m0 = __builtin_amdgcn_readfirstlane(job.m0);
    job.nt = __builtin_amdgcn_readfirstlane(job.nt);
    const int64_t d = a.d, F = a.F;
    const int n0 = job.nt * S::kN;

    // Leading dimensions, extents and the operands' first bytes.
    const int64_t lda = KIND == EXP_UP || KIND == EXP_DH || KIND == EXP_DW_DOWN ? d : KIND == EXP_DOWN ? F : 2 * F;
    const int64_t ldb = KIND == EXP_DOWN || KIND == EXP_DH || KIND == EXP_DW_DOWN ? F : d;
    const int N = KIND == EXP_UP || KIND == EXP_DH || KIND == EXP_DW_DOWN ? a.F : a.d;
    const int M = KIND == EXP_DW_DOWN ? a.d : KIND == EXP_DW_UP ? 2 * a.F : job.rows;
    const int K = S::kDw ? job.rows : KIND == EXP_UP || KIND == EXP_DH ? a.d : KIND == EXP_DOWN ? a.F : 2 * a.F;
    const int slabs = (K + 31) / 32;
    const char* A = reinterpret_cast<const char*>(a.A + job.r0 * lda);
    const char* B = reinterpret_cast<const char*>(a.B + (S::kDw ? job.r0 * ldb : job.e * F * d));
    const char* B2 = reinterpret_cast<const char*>(KIND == EXP_UP || KIND == EXP_DX ? a.B2 + job.e * F * d : a.B);
    if (!S::kACol) A += job.m0 * lda * 2;

    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(lds)));
    auto fl = [](int r) { return (r & 3) | ((r >> 1) & 4); };
    // Where a lane reads its 16 bytes of a load: from the operand's base, slab 0.
    // Past the last m, n or column the last one is read again (its results are
    // not stored).
    uint32_t oa[S::LA], ob[S::LB];
#pragma unroll
    for (int k = 0; k < S::LA; ++k) {
        const int q = wid + 4 * k;
        if (S::kACol) {
            const int r = 2 * q + (lane >> 5), c = ((((lane & 31) >> 1) ^ fl(r)) << 1) | (lane & 1);
            oa[k] = static_cast<uint32_t>(r * lda + min(job.m0 + c * 8, M - 8)) * 2;
        } else {
            const int r = lane >> 2, c = (lane & 3) ^ ((lane >> 3) & 3);
            oa[k] = static_cast<uint32_t>(min(q * 16 + r, M - 1 - job.m0) * lda + c * 8) * 2;
        }
    }
#pragma unroll
    for (int k = 0; k < S::LB; ++k) {
        const int q = wid + 4 * k;
        if (S::kBCol) {
            const int r = 2 * q + (lane >> 5), c = ((((lane & 31) >> 1) ^ fl(r)) << 1) | (lane & 1);
            ob[k] = static_cast<uint32_t>(r * ldb + min(n0 + c * 8, N - 8)) * 2;
        } else {
            const int r = lane >> 2, c = (lane & 3) ^ ((lane >> 3) & 3);
            // EXP_UP: half of a wave's fragments are of W_gate, the other half the same of W_up
            const int f = S::kPair ? q / NJ * (NJ / 2) + q % (NJ / 2) : q;
            ob[k] = static_cast<uint32_t>(min(n0 + f * 16 + r, N - 1) * ldb + c * 8) * 2;
        }
    }
    // Slab b's k-th load of this wave.  Every call issues one instruction, so that
    // counting the newest ones is enough to wait for the others.
    auto load = [&](int b, int k) {
        const bool isA = k < S::LA;
        const int q = wid + 4 * (isA ? k : k - S::LA);
        const uint32_t dst = lds0 + (b & 3) * S::kSlot + (isA ? q : S::NA + q) * 1024;
        const uint32_t off = isA ? oa[isA ? k : 0] : ob[isA ? 0 : k - S::LA];
        const char* base;
        if (isA) {
            base = A + static_cast<int64_t>(b) * (S::kACol ? 32 * lda * 2 : 64);
        } else if (KIND == EXP_DX) {  // [W_gate; W_up], F rows each (a multiple of 32)
            const int64_t row = static_cast<int64_t>(b) * 32;
            base = row < F ? B + row * ldb * 2 : B2 + (row - F) * ldb * 2;
        } else if (S::kPair) {
            base = ((q & (NJ / 2)) ? B2 : B) + static_cast<int64_t>(b) * 64;
        } else {
            base = B + static_cast<int64_t>(b) * (S::kBCol ? 32 * ldb * 2 : 64);
        }
        if (S::kDw && (b + 1) * 32 > K) {  // the last rows: zeros behind them
            const bool in = b * 32 + 2 * q + (lane >> 5) < K;
            dma(in ? base + off : reinterpret_cast<const char*>(&kZero16), dst);
        } else {
            dma(base, off, dst);
        }
    };
    auto tr = [&](uint32_t at) {
        return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                             (__attribute__((address_space(3))) s16x4*)(lds + at)));
    };
    auto read_a = [&](int b, int i) -> uint4 {
        const uint32_t o = (b & 3) * S::kSlot;
        if (S::kACol) {
            uint2 h[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 8 * grp + (r16 >> 2) + 4 * u;
                h[u] = tr(o + r * 512 + (((wm * MI + i) ^ fl(r)) << 5) + (r16 & 3) * 8);
            }
            return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
        }
        return *reinterpret_cast<const uint4*>(lds + o + (wm * MI + i) * 1024 + r16 * 64 + ((grp ^ ((r16 >> 1) & 3)) << 4));
    };
    auto read_b = [&](int b, int j) -> uint4 {
        const uint32_t o = (b & 3) * S::kSlot + S::NA * 1024;
        const int f = wn * NJ + j;
        if (S::kBCol) {
            uint2 h[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 8 * grp + (r16 >> 2) + 4 * u;
                h[u] = tr(o + r * 512 + ((f ^ fl(r)) << 5) + (r16 & 3) * 8);
            }
            return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
        }
        return *reinterpret_cast<const uint4*>(lds + o + f * 1024 + r16 * 64 + ((grp ^ ((r16 >> 1) & 3)) << 4));
    };

    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (slabs > 0) {
        uint4 fa[MI], fb[2];
#pragma unroll
        for (int b = 0; b < 3; ++b)
            if (b < slabs)
#pragma unroll
                for (int k = 0; k < S::NL; ++k) load(b, k);
        // slab b has landed: `newer` later ones may be on their way
        auto arrive = [&](int newer) {
            __builtin_amdgcn_sched_barrier(0);
            if (newer >= 2) wait_and_meet<2 * S::NL>();
            else if (newer == 1) wait_and_meet<S::NL>();
            else wait_and_meet<0>();
            __builtin_amdgcn_sched_barrier(0);
        };
        arrive(slabs - 1);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = read_a(0, i);
        fb[0] = read_b(0, 0);
        for (int b = 0; b < slabs; ++b) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if (j == NJ / 2 && b + 1 < slabs) arrive(min(1, slabs - 2 - b));
                __builtin_amdgcn_sched_barrier(0);
                fb[(j + 1) & 1] = j + 1 < NJ ? read_b(b, j + 1) : read_b(b + 1, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    acc[i][j] = Mfma<bf16_t>::run(fb[j & 1], fa[i], acc[i][j]);
                    if (j == NJ - 1) {
                        __builtin_amdgcn_sched_barrier(0);
                        fa[i] = read_a(b + 1, i);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (j >= NJ / 2) {
#pragma unroll
                        for (int k = 0; k < S::NL; ++k)
                            if (k * (MI * NJ / 2) / S::NL == (j - NJ / 2) * MI + i) {
                                __builtin_amdgcn_sched_barrier(0);
                                if (b + 3 < slabs) load(b + 3, k);
                                __builtin_amdgcn_sched_barrier(0);
                            }
                    }
                }
            }
        }
    }

    // A lane's part of fragments j and j + 1 of row 16 i + r16: columns 16 j + nl .. + 7,
    // nl = 16 (grp % 2) + 8 (grp / 2), once the odd groups' j and the even groups' j + 1 are exchanged.
    const int nl = 16 * (grp & 1) + 8 * (grp >> 1);
    auto eight = [&](int i, int j, float (&v)[8]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][j][u]), __float_as_uint(acc[i][j + 1][u]),
                                                            false, false);
            v[u] = __uint_as_float(q[0]);
            v[4 + u] = __uint_as_float(q[1]);
        }
    };
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m = job.m0 + (wm * MI + i) * 16 + r16;
        if (KIND == EXP_UP) {
            const int64_t row = job.r0 + m;
#pragma unroll
            for (int j = 0; j < NJ / 2; j += 2) {
                const int n = n0 + (wn * NJ / 2 + j) * 16 + nl;
                float g[8], u[8], h[8];
                eight(i, j, g);
                eight(i, j + NJ / 2, u);
                if (m >= M || n >= N) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = g[e] * sigmoid(g[e]) * u[e];
                if (a.gu) {
                    pack8(a.gu + row * 2 * F + n, g);
                    pack8(a.gu + row * 2 * F + F + n, u);
                }
                stg16(a.C + row * F + n, pack8v(h));
            }
        } else if (KIND == EXP_DH) {
            const int64_t row = job.r0 + m;
#pragma unroll
            for (int j = 0; j < NJ; j += 2) {
                const int n = n0 + (wn * NJ + j) * 16 + nl;
                float dh[8], g[8], u[8], dg[8], du[8];
                eight(i, j, dh);
                if (m >= M || n >= N) continue;
                unpack8(a.gu + row * 2 * F + n, g);
                unpack8(a.gu + row * 2 * F + F + n, u);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float s = sigmoid(g[e]);
                    du[e] = dh[e] * g[e] * s;
                    dg[e] = dh[e] * u[e] * s * (1.f + g[e] * (1.f - s));
                }
                stg16(a.C + row * 2 * F + n, pack8v(dg));
                stg16(a.C + row * 2 * F + F + n, pack8v(du));
            }
        } else {
            bf16_t* out;
            if (KIND == EXP_DW_DOWN)
                out = a.C + (job.e * d + m) * F;
            else if (KIND == EXP_DW_UP)
                out = m < a.F ? a.C + (job.e * F + m) * d : a.C2 + (job.e * F + m - F) * d;
            else
                out = a.C + (job.r0 + m) * d;
#pragma unroll
            for (int j = 0; j < NJ; j += 2) {
                const int n = n0 + (wn * NJ + j) * 16 + nl;
                float v[8];
                eight(i, j, v);
                if (m >= M || n >= N) continue;
                stg16(out + n, pack8v(v));
            }
        }
    }
}

// Blocks of a launch: at least one per tile, whatever the experts' row counts.
template <int KIND, int BM>
int64_t tiles(int64_t R, int64_t E, int64_t d, int64_t F, int* ntm, int* ntn) {
    using S = Tile<KIND, BM>;
    const int64_t N = KIND == EXP_UP || KIND == EXP_DH || KIND == EXP_DW_DOWN ? F : d;
    *ntn = static_cast<int>((N + S::kN - 1) / S::kN);
    *ntm = KIND == EXP_DW_DOWN ? static_cast<int>((d + BM - 1) / BM) : static_cast<int>((2 * F + BM - 1) / BM);
    const int64_t mt = S::kDw ? E * *ntm : R < E ? R : (R - E) / BM + E;  // sum of ceil(n_e / BM), sum n_e = R
    return mt * *ntn;
}

constexpr int64_t kMaxTiles = 1 << 23;  // a launch has less than 2^32 threads

template <int KIND, int BM>
hipError_t launch(const ExpertsArgs& a, hipStream_t stream) {
    int ntm, ntn;
    const int64_t n = tiles<KIND, BM>(a.R, a.E, a.d, a.F, &ntm, &ntn);
    if (n > kMaxTiles) return hipErrorInvalidValue;
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL((k_experts<KIND, BM>), dim3(job_blocks(static_cast<int>(n), 1)), dim3(256), 0, stream, a, ntm, ntn);
    return hipGetLastError();
}

// Rows of an M tile: 64 while experts hold fewer than kTall rows on average.
constexpr int64_t kTall = 128;
bool tall(const ExpertsArgs& a) { return a.R >= kTall * a.E; }

}  // namespace

// The most rows that every launch can take.
int64_t experts_max_rows(int E, int d, int F) {
    const int64_t ntn = ((d > F ? d : F) + 127) / 128;
    const int64_t most = (kMaxTiles / ntn - E) * 64;
    if (static_cast<int64_t>(E) * ((2ll * F + 255) / 256) * ((d + 255) / 256) > kMaxTiles) return -1;
    return most < 0 ? -1 : most < (1ll << 31) - 256 ? most : (1ll << 31) - 256;
}

hipError_t launch_experts(ExpertsKind kind, const ExpertsArgs& a, hipStream_t stream) {
    if (a.E < 1 || a.R < 0 || a.d % 64 || a.F % 64 || a.d < 64 || a.F < 64) return hipErrorInvalidValue;
    switch (kind) {
        case EXP_UP: return tall(a) ? launch<EXP_UP, 256>(a, stream) : launch<EXP_UP, 64>(a, stream);
        case EXP_DOWN: return tall(a) ? launch<EXP_DOWN, 256>(a, stream) : launch<EXP_DOWN, 64>(a, stream);
        case EXP_DH: return tall(a) ? launch<EXP_DH, 256>(a, stream) : launch<EXP_DH, 64>(a, stream);
        case EXP_DX: return tall(a) ? launch<EXP_DX, 256>(a, stream) : launch<EXP_DX, 64>(a, stream);
        case EXP_DW_DOWN: return launch<EXP_DW_DOWN, 256>(a, stream);
        case EXP_DW_UP: return launch<EXP_DW_UP, 256>(a, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace moe
