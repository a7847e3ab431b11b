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
// which 1.7e-3 is the result's own rounding).  That costs 3% more bytes at 683 rows an expert (a and b are 6%
// of the 17.8 GB of all six products there) and 8 F bytes a row that are kept until the backward call.
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "experts.hpp"

namespace moe {
namespace {

// An operand of a product C[m, n] = sum_k A[m, k] B[n, k] lies in memory either
// with its k side by side (rows: a row of the matrix is one m or n) or with its m
// or n side by side (columns: a row is one k; read transposed from LDS).
//
// A block of eight waves holds a tile of 256 x 256 in registers.  Stages of 64 k of
// both operands go from global memory straight into LDS (global_load_lds_dwordx4,
// 1 KiB per wave and instruction): A into two slots, B, the weights, which come
// from further away, into three.  While the products of a stage run, a wave asks
// for the next stage of A and the one after the next of B, one load every eight
// products; near its end it waits for its loads of the next stage and meets the
// other waves: after that the next stage may be read, and this one, which all
// have in registers by then, be overwritten.  Half a stage (32 k) is one step of
// products; its fragments are read from LDS under the products before: those of B
// two ahead, those of A each after its last use.
//
// Rows operand: a 1 KiB block holds 8 rows x 64 k; 16-byte chunk c of row r at r 128 +
// (c ^ r) 16: a load takes whole lines of 128 bytes (segments of 64 bytes reach half
// the L2's rate: 16 against 33 TB/s, measured by itself), and eight lanes that read a
// chunk of eight rows meet all banks once.
// Columns operand: a block holds 2 k x 256 columns; 32-byte chunk c of row r at c
// ^ (r % 4 + 4 (r / 8 % 2)) (see k_dw).
// A lane has four neighbouring columns of each product; two of them are exchanged
// between the lanes of neighbouring groups of 16 for eight: 16-byte stores.
//
// Blocks stay for all their tiles: the first loads of the next one are on their
// way while a tile is stored.
typedef short s16x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from base + off (src) to LDS at slot + AT + 16 lane.
template <int AT>
__device__ __forceinline__ void dma(const char* base, uint32_t off, uint32_t slot) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(slot)), "v"(off), "s"(base), "n"(AT) : "memory", "m0", "scc");
}
template <int AT>
__device__ __forceinline__ void dma(const char* src, uint32_t slot) {
    asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(__builtin_amdgcn_readfirstlane(slot)), "v"(src), "n"(AT) : "memory", "m0", "scc");
}
// This wave's vector memory operations but the newest N, and its reads of LDS, are done; then all waves'.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
// The same without regard to loads and stores.
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// What rows behind an expert's last one are read as in the columns operands.
__device__ const uint4 kZero16 = {0, 0, 0, 0};

constexpr int kCUs = 256, kWaves = 8, kBM = 256;
constexpr int kLds = 160 * 1024;  // two stages of A, three of B

template <int KIND>
struct Tile {
    static constexpr bool kDw = KIND == EXP_DW_DOWN || KIND == EXP_DW_UP;
    static constexpr bool kACol = kDw, kBCol = kDw || KIND == EXP_DH || KIND == EXP_DX;
    static constexpr bool kPair = KIND == EXP_UP;          // 128 columns of W_gate and the same of W_up
    static constexpr int kWM = 2, kWN = 4;                   // waves
    static constexpr int MI = kBM / 16 / kWM, NJ = 16 / kWN;  // fragments of a wave
    static constexpr int kA = kBM * 128, kB = 256 * 128;      // bytes of a stage
    static constexpr int LA = 4, LB = 4;                     // loads of a wave and stage
    static constexpr int kN = kPair ? 128 : 256;             // columns of C per tile
};

// A block's tiles: it takes every gridDim.x / 8-th of its XCD's stretch of the list
// (blocks go to the eight XCDs round robin), which has the experts in order, an expert's
// M tiles side by side, so that the tiles which share weights run together.
struct Jobs {
    int lin, end, step;               // this tile, past the stretch, to the next one
    int lo, each;                     // kDw: of each expert's tiles, this XCD's first and how many
    int e, r0, rows, first, n;        // its expert, that one's rows, the M tiles before and of it
    int m0, nt;                       // the tile's first row (of the expert's, or of C) and N tile
};
__device__ __forceinline__ int row_at(const ExpertsArgs& a, int e) {  // (e is the same for all lanes)
    const int v = reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(reinterpret_cast<uintptr_t>(a.off))[e];
    return __builtin_amdgcn_readfirstlane(static_cast<int>(min(max(static_cast<int64_t>(v), int64_t(0)), a.R)));
}

template <int KIND>
__device__ __forceinline__ void place(const ExpertsArgs& a, int ntm, int ntn, Jobs& j) {
    if (Tile<KIND>::kDw) {
        const int e = j.lin / j.each, in = j.lo + j.lin - e * j.each;
        j.e = e;
        j.r0 = row_at(a, e);
        j.rows = max(row_at(a, e + 1) - j.r0, 0);
        // along the shorter side of C first: an XCD reads all of the smaller operand, and a part of the other
        const int major = in / min(ntm, ntn), minor = in - major * min(ntm, ntn);
        j.nt = ntm <= ntn ? major : minor;
        j.m0 = (ntm <= ntn ? minor : major) * kBM;
    } else {
        const int in = j.lin - j.first * ntn;
        j.nt = in / j.n;
        j.m0 = (in - j.nt * j.n) * kBM;
    }
}

// The block's first tile; false: it has none.
template <int KIND>
__device__ __forceinline__ bool first_job(const ExpertsArgs& a, int ntm, int ntn, int slot, Jobs& j) {
    const int lane = threadIdx.x & 63, xcd = blockIdx.x & 7;
    j.step = gridDim.x >> 3;
    if (Tile<KIND>::kDw) {
        // An expert's tiles take as long as it has rows: every XCD has an eighth of each expert's, unless there are
        // few (48 experts of 7168 x 2048, 683 rows on average, a quarter up or down: 2.48 -> 2.16 ms and 1.21 -> 1.13).
        const int t = ntm * ntn;
        if (t >= 64) {
            j.lo = static_cast<int>(static_cast<int64_t>(t) * xcd / 8);
            j.each = static_cast<int>(static_cast<int64_t>(t) * (xcd + 1) / 8) - j.lo;
            j.lin = slot;
            j.end = a.E * j.each;
        } else {
            const int total = a.E * t, per = (total + 7) >> 3;
            j.lo = 0;
            j.each = t;
            j.lin = xcd * per + slot;
            j.end = min(total, (xcd + 1) * per);
        }
        if (j.lin >= j.end) return false;
        place<KIND>(a, ntm, ntn, j);
        return true;
    }
    // a lane per expert, 64 experts at a time
    struct Rows {
        int r0, rows, n;
    };
    auto rows_of = [&](int e0) {
        const int e = e0 + lane;
        Rows r{0, 0, 0};
        if (e < a.E) {
            auto clamped = [&](int i) { return static_cast<int>(min(max(static_cast<int64_t>(a.off[i]), int64_t(0)), a.R)); };
            const int end = clamped(e + 1);
            r.r0 = clamped(e);
            r.rows = max(end - r.r0, 0);
            r.n = (r.rows + kBM - 1) / kBM;
        }
        return r;
    };
    const Rows head = rows_of(0);
    int total = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        int n = e0 == 0 ? head.n : rows_of(e0).n;
#pragma unroll
        for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
        total += n;
    }
    total = __builtin_amdgcn_readfirstlane(total) * ntn;
    const int per = (total + 7) >> 3;
    j.lin = xcd * per + slot;
    j.end = min(total, (xcd + 1) * per);
    if (j.lin >= j.end) return false;
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const Rows r = e0 == 0 ? head : rows_of(e0);
        int incl = r.n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(incl, o);
            if (lane >= o) incl += v;
        }
        const int first = before + incl - r.n;
        const uint64_t mine = __ballot(r.n > 0 && first * ntn <= j.lin && j.lin < (first + r.n) * ntn);
        if (mine) {
            const int l = __ffsll(static_cast<unsigned long long>(mine)) - 1;
            j.e = e0 + l;
            j.r0 = __builtin_amdgcn_readlane(r.r0, l);
            j.rows = __builtin_amdgcn_readlane(r.rows, l);
            j.n = __builtin_amdgcn_readlane(r.n, l);
            j.first = __builtin_amdgcn_readlane(first, l);
            place<KIND>(a, ntm, ntn, j);
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}
template <int KIND>
__device__ __forceinline__ bool next_job(const ExpertsArgs& a, int ntm, int ntn, Jobs& j) {
    j.lin += j.step;
    if (j.lin >= j.end) return false;
    if (!Tile<KIND>::kDw)
        while (j.lin >= (j.first + j.n) * ntn) {
            if (++j.e >= a.E) return false;
            j.first += j.n;
            j.r0 = row_at(a, j.e);
            j.rows = max(row_at(a, j.e + 1) - j.r0, 0);
            j.n = (j.rows + kBM - 1) / kBM;
        }
    place<KIND>(a, ntm, ntn, j);
    return true;
}

__device__ __forceinline__ float sigmoid(float a) { return 1.f / (1.f + __expf(-a)); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {  // rounded to nearest even
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}
__device__ __forceinline__ uint4 pack8v(const float (&v)[8]) {
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// The value of the lane 8 further on among its 16.
__device__ __forceinline__ uint32_t row_ror8(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x128, 0xf, 0xf, true));
}
__device__ __forceinline__ uint4 row_ror8(uint4 v) {
    return make_uint4(row_ror8(v.x), row_ror8(v.y), row_ror8(v.z), row_ror8(v.w));
}

// f(0), f(1), .. f(N - 1), each a constant.
template <typename F, int... I>
__device__ __forceinline__ void for_each(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_each(F&& f) {
    for_each(f, std::make_integer_sequence<int, N>());
}

template <int KIND>
__device__ __forceinline__ void run(const ExpertsArgs& a, int ntm, int ntn, int slot, char* lds) {
    using S = Tile<KIND>;
    constexpr int MI = S::MI, NJ = S::NJ, LA = S::LA, LB = S::LB;
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, grp = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wid / S::kWN, wn = wid % S::kWN;
    Jobs job;
    if (!first_job<KIND>(a, ntm, ntn, slot, job)) return;
    const int64_t d = a.d, F = a.F;
    const int64_t lda = KIND == EXP_UP || KIND == EXP_DH || KIND == EXP_DW_DOWN ? d : KIND == EXP_DOWN ? F : 2 * F;
    const int64_t ldb = KIND == EXP_DOWN || KIND == EXP_DH || KIND == EXP_DW_DOWN ? F : d;
    const int N = KIND == EXP_UP || KIND == EXP_DH || KIND == EXP_DW_DOWN ? a.F : a.d;

    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(lds)));
    auto fl = [](int r) { return (r & 3) | ((r >> 1) & 4); };

    // The operands of a tile: first bytes, the lane's offset of each load, extents.
    // Past the last m, n or column the last one is read again (its results are
    // not stored).
    const char *A, *B, *B2;
    uint32_t oa[LA], ob[LB];
    int M, K, stages;
    auto setup = [&](const Jobs& j) {
        M = KIND == EXP_DW_DOWN ? a.d : KIND == EXP_DW_UP ? 2 * a.F : j.rows;
        K = S::kDw ? j.rows : KIND == EXP_UP || KIND == EXP_DH ? a.d : KIND == EXP_DOWN ? a.F : 2 * a.F;
        stages = (K + 63) >> 6;
        A = reinterpret_cast<const char*>(a.A + (j.r0 + (S::kACol ? 0 : j.m0)) * lda);
        B = reinterpret_cast<const char*>(a.B + (S::kDw ? j.r0 * ldb : j.e * F * d));
        // EXP_DX: [W_gate; W_up], F rows each (a multiple of 64)
        B2 = reinterpret_cast<const char*>(KIND == EXP_UP || KIND == EXP_DX ? a.B2 + j.e * F * d : a.B);
        if (KIND == EXP_DX) B2 -= F * ldb * 2;
        const int n0 = j.nt * S::kN;
        auto columns = [&](int k, int64_t ld, int c0, int end) {  // of k row 2 (wid + 4 k) + lane / 32
            const int r = 2 * (wid + kWaves * k) + (lane >> 5), c = ((((lane & 31) >> 1) ^ fl(r)) << 1) | (lane & 1);
            return static_cast<uint32_t>(r * ld + min(c0 + c * 8, end - 8)) * 2;
        };
#pragma unroll
        for (int k = 0; k < LA; ++k) {
            const int r = lane >> 3, c = (lane & 7) ^ r;
            oa[k] = S::kACol ? columns(k, lda, j.m0, M)
                             : static_cast<uint32_t>(min((wid + kWaves * k) * 8 + r, M - 1 - j.m0) * lda + c * 8) * 2;
        }
#pragma unroll
        for (int k = 0; k < LB; ++k) {
            const int q = wid + kWaves * k, r = lane >> 3, c = (lane & 7) ^ r;
            // EXP_UP: half of a wave's fragments (two blocks each) are of W_gate, the other half the same of W_up
            const int f = S::kPair ? q / (2 * NJ) * NJ + q % NJ : q;
            ob[k] = S::kBCol ? columns(k, ldb, n0, N)
                             : static_cast<uint32_t>(min(n0 + f * 8 + r, N - 1) * ldb + c * 8) * 2;
        }
    };
    // Stage s's K-th load of this wave, of A or B, to a slot.  Every call issues one
    // instruction, so that counting the newest ones is enough to wait for the others.
    // LAST: it may be the last stage, whose rows (of columns operands) behind the end are zeros.
    auto one = [&](auto k_, auto last_, const char* base, uint32_t off, int s, uint32_t slot) {
        constexpr int k = decltype(k_)::value;
        if (S::kDw && decltype(last_)::value) {
            const bool in = s * 64 + 2 * (wid + kWaves * k) + (lane >> 5) < K;
            dma<k * kWaves * 1024>(in ? base + off : reinterpret_cast<const char*>(&kZero16), slot);
        } else {
            dma<k * kWaves * 1024>(base, off, slot);
        }
    };
    const uint32_t lds_w = lds0 + wid * 1024;
    auto load_a = [&](int s, int slot, auto k, auto last) {
        one(k, last, A + s * (S::kACol ? 128 * lda : 128), oa[decltype(k)::value], s, lds_w + slot * S::kA);
    };
    auto load_b = [&](int s, int slot, auto k_, auto last) {
        constexpr int k = decltype(k_)::value;
        const bool up = KIND == EXP_DX ? s * 64 >= a.F : S::kPair && ((wid + kWaves * k) & NJ);
        one(k_, last, (up ? B2 : B) + s * (S::kBCol ? 128 * ldb : 128), ob[k], s, lds_w + 2 * S::kA + slot * S::kB);
    };
    // Fragment f of half h of the stage at `o`.  (Columns: a lane's rows are 8 grp + r16 / 4 and that + 4, alike in f.)
    const uint32_t lt = (8 * grp + (r16 >> 2)) * 512 + (((r16 >> 2) | ((grp & 1) << 2)) << 5) + (r16 & 3) * 8;
    const uint32_t lr = r16 * 128, lc = (grp ^ (r16 & 3)) | (r16 & 4);
    auto read = [&](bool col, uint32_t o, int f, int h) -> uint4 {
        if (col) {
            typedef __attribute__((address_space(3))) s16x4* P;
            const P q = (P)(lds + o + (lt ^ (f << 5)));
            const uint2 v0 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(q + h * 2048));
            const uint2 v1 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(q + h * 2048 + 256));
            return make_uint4(v0.x, v0.y, v1.x, v1.y);
        }
        return *reinterpret_cast<const uint4*>(lds + o + f * 2048 + lr + ((lc ^ (4 * h)) << 4));
    };
    // Fragments of A's rows per wave: an expert's last tile has fewer, in steps of kStep, and the waves share them.
    constexpr int kStep = MI / 4;
    int mi = MI;
    auto read_a = [&](int slot, int i, int h) { return read(S::kACol, slot * S::kA, wm * mi + i, h); };
    auto read_b = [&](int slot, int j, int h) { return read(S::kBCol, 2 * S::kA + slot * S::kB, wn * NJ + j, h); };

    // The loads that go out while stage s runs, in 2 NJ portions: A of s + 1, then B
    // of s + 2 (to bslot).  Portions 0 and 1 belong to the last quarter of stage s - 1.
    // SURE: those stages exist and are not the last one.
    constexpr int LATE = NJ - 2;
    static_assert(LA + LB == 2 * NJ && LA >= 2, "a load a portion, the first two of A");
    auto portion = [&](int s, auto p_, int bslot, auto sure_) {
        constexpr int p = decltype(p_)::value;
        constexpr bool SURE = decltype(sure_)::value;
        if constexpr (p < LA) {
            if (SURE || s + 1 < stages) load_a(s + 1, (s + 1) & 1, p_, std::bool_constant<!SURE>());
        } else {
            if (SURE || s + 2 < stages) load_b(s + 2, bslot, std::integral_constant<int, p - LA>(), std::bool_constant<!SURE>());
        }
    };
    // A tile's first loads: stage 0, B of stage 1, portions 0 and 1 of stage 0.
    constexpr int kFirst = LB + 2;  // those behind stage 0's, of two stages or more
    auto begin = [&]() {
        if (stages == 0) return;
        for_each<LA>([&](auto k) { load_a(0, 0, k, std::true_type()); });
        for_each<LB>([&](auto k) { load_b(0, 0, k, std::true_type()); });
        if (stages > 1) for_each<LB>([&](auto k) { load_b(1, 1, k, std::true_type()); });
        portion(0, std::integral_constant<int, 0>(), 2, std::false_type());
        portion(0, std::integral_constant<int, 1>(), 2, std::false_type());
    };

    setup(job);
    begin();
    int stored = 0;  // stores of the tile before, all behind these loads (0: none, or some other number)
    constexpr int kStores = KIND == EXP_UP ? 0 : MI * NJ / 2 * (KIND == EXP_DH ? 2 : 1);
    for (;;) {
        f32x4 acc[MI][NJ];
        if (!S::kDw) mi = kStep * min((M - job.m0 + kBM / 4 - 1) / (kBM / 4), 4);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (stages > 0) {
            uint4 fa[MI], fb[4];  // (fb: a ring, two fragments ahead)
            if (stages > 1) {
                if (kStores && kFirst + kStores < 64 && stored) wait_and_meet<(kFirst + kStores) & 63>();
                else wait_and_meet<kFirst>();
            } else {
                if (kStores && kStores < 64 && stored) wait_and_meet<kStores & 63>();
                else wait_and_meet<0>();
            }
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[i] = read_a(0, i, 0);
            fb[0] = read_b(0, 0, 0);
            fb[1] = read_b(0, 1, 0);
            int bs = 0;  // B slot of stage s
            // half H of stage s
            auto half = [&](int s, auto h_, auto sure) {
                constexpr int H = decltype(h_)::value;
                const int bnext = bs == 2 ? 0 : bs + 1, bprev = bs == 0 ? 2 : bs - 1;
                for_each<NJ>([&](auto j_) {
                    constexpr int j = decltype(j_)::value;
                    if (H == 1 && j == LATE && (decltype(sure)::value || s + 1 < stages)) {
                        // stage s + 1 has landed, and nobody reads stage s any more
                        if (decltype(sure)::value || s + 2 < stages) wait_and_meet<LB>();
                        else wait_and_meet<0>();
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        if (!S::kDw && g > 0 && mi <= g * kStep) break;  // (uniform)
#pragma unroll
                        for (int i = g * kStep; i < (g + 1) * kStep; ++i) {
                            acc[i][j] = Mfma<bf16_t>::run(fb[j & 3], fa[i], acc[i][j]);
                            __builtin_amdgcn_sched_barrier(0);
                            if (i == 0) fb[(j + 2) & 3] = j < LATE ? read_b(bs, j + 2, H) : read_b(H ? bnext : bs, j - LATE, H ^ 1);
                            if (j == NJ - 1) fa[i] = read_a((s + H) & 1, i, H ^ 1);
                            __builtin_amdgcn_sched_barrier(0);
                            // B of s + 2 takes the slot of stage s - 1, that of s + 3 the slot of s
                            if (i == kStep - 1) {
                                if constexpr (H == 0) portion(s, std::integral_constant<int, j + 2>(), bprev, sure);
                                else if constexpr (j < LATE) portion(s, std::integral_constant<int, NJ + 2 + j>(), bprev, sure);
                                else portion(s + 1, std::integral_constant<int, j - LATE>(), bs, sure);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                });
                if (H) bs = bnext;
            };
            using H0 = std::integral_constant<int, 0>;
            using H1 = std::integral_constant<int, 1>;
            // (stages that the loads of stage s reach: s + 2, of kDw not the last one)
            int s = 0;
            for (; s < stages - (S::kDw ? 3 : 2); ++s) {
                half(s, H0(), std::true_type());
                half(s, H1(), std::true_type());
            }
            for (; s < stages; ++s) {
                half(s, H0(), std::false_type());
                if (!S::kDw || K - s * 64 > 32) half(s, H1(), std::false_type());
            }
        }

        const Jobs at = job;
        const int m_end = M;
        const bool again = next_job<KIND>(a, ntm, ntn, job);
        if (again) {
            meet();  // nobody reads this tile's stages any more
            setup(job);
            begin();
        }
        const int n0 = at.nt * S::kN;
        stored = at.m0 + kBM <= m_end && n0 + S::kN <= N;

        // A lane's part of fragments j and j + 1 of row 16 i + r16: columns 16 j + nl .. + 7,
        // nl = 16 (grp % 2) + 8 (grp / 2), once the odd groups' j and the even groups' j + 1 are exchanged.
        const int nl = 16 * (grp & 1) + 8 * (grp >> 1);
        auto eight = [&](int i, int j, float (&v)[8]) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][j][u]),
                                                                __float_as_uint(acc[i][j + 1][u]), false, false);
                v[u] = __uint_as_float(q[0]);
                v[4 + u] = __uint_as_float(q[1]);
            }
        };
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // (or all of acc is moved at once, and spilled)
            if (!S::kDw && i >= mi) break;  // (uniform)
            const int m = at.m0 + (wm * mi + i) * 16 + r16;
            if (KIND == EXP_UP) {
                const int64_t row = at.r0 + m;
#pragma unroll
                for (int j = 0; j < NJ / 2; j += 2) {
                    const int n = n0 + (wn * NJ / 2 + j) * 16 + nl;
                    float g[8], u[8], h[8];
                    eight(i, j, g);
                    eight(i, j + NJ / 2, u);
                    if (m >= m_end || n >= N) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] = g[e] * sigmoid(g[e]) * u[e];
                    if (a.gu) {
                        pack8(a.gu + row * 2 * F + n, g);
                        pack8(a.gu + row * 2 * F + F + n, u);
                    }
                    stg16(a.C + row * F + n, pack8v(h));
                }
            } else if (KIND == EXP_DH) {
                const int64_t row = at.r0 + m;
#pragma unroll
                for (int j = 0; j < NJ; j += 2) {
                    const int n = n0 + (wn * NJ + j) * 16 + nl;
                    float dh[8], g[8], u[8], dg[8], du[8];
                    eight(i, j, dh);
                    if (m >= m_end || n >= N) continue;
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
                // Half of what a lane has goes to the lane of row r16 ^ 8, so that eight lanes write 128
                // bytes of a row: half-written lines of the L2 reach only part of the memory's rate.
                uint4 p[2];
#pragma unroll
                for (int j = 0; j < NJ; j += 2) {
                    const auto q0 = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][0], acc[i][j][1]),
                                                                     pack2(acc[i][j + 1][0], acc[i][j + 1][1]), false, false);
                    const auto q1 = __builtin_amdgcn_permlane16_swap(pack2(acc[i][j][2], acc[i][j][3]),
                                                                     pack2(acc[i][j + 1][2], acc[i][j + 1][3]), false, false);
                    p[j / 2] = make_uint4(q0[0], q1[0], q0[1], q1[1]);
                }
                const bool low = r16 < 8;
                const uint4 get = row_ror8(low ? p[1] : p[0]);
                const int n = n0 + wn * NJ * 16 + (low ? 0 : 32) + nl;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int mu = m - r16 + (r16 & 7) + 8 * u;
                    if (mu >= m_end || n >= N) continue;
                    bf16_t* out;
                    if (KIND == EXP_DW_DOWN)
                        out = a.C + (at.e * d + mu) * F;
                    else if (KIND == EXP_DW_UP)
                        out = mu < a.F ? a.C + (at.e * F + mu) * d : a.C2 + (at.e * F + mu - F) * d;
                    else
                        out = a.C + (at.r0 + mu) * d;
                    stg16(out + n, low == (u == 0) ? p[u] : get);
                }
            }
        }
        if (!again) return;
    }
}

// One product, or two that do not wait for each other: a block goes from its tiles of the
// first to those of the second, and blocks that have none of the first come first in the
// second.  Two in one for few tiles, where launches and idle CUs count; with
// many, blocks that reach the second at different times share less in the L2.  Forward
// and backward, four launches in all against six: 40 / 54 us at 96 rows, 32 experts of 512 x
// 256; 188 / 194 at 2000, 32 of 1024 x 1024; 552 / 571 at 4096, 48 of 2048 x 1024 (3600 tiles in the larger
// pair); but 2840 / 2690 at 2048, 48 of 7168 x 2048 (23000).
constexpr int kNone = -1;
template <int FIRST, int SECOND>
__global__ __launch_bounds__(64 * kWaves, 2) void k_experts(const ExpertsArgs a, int ntm, int ntn, const ExpertsArgs a2,
                                                            int ntm2, int ntn2) {
    __shared__ __attribute__((aligned(1024))) char lds[kLds];
    const int slot = blockIdx.x >> 3;
    run<FIRST>(a, ntm, ntn, slot, lds);
    if constexpr (SECOND != kNone) {
        meet();  // nobody reads the first's stages any more
        run<SECOND>(a2, ntm2, ntn2, static_cast<int>(gridDim.x >> 3) - 1 - slot, lds);
    }
}

// The most tiles that a product can have, whatever the experts' row counts.
template <int KIND>
int64_t tiles(int64_t R, int64_t E, int64_t d, int64_t F, int* ntm, int* ntn) {
    using S = Tile<KIND>;
    const int64_t N = KIND == EXP_UP || KIND == EXP_DH || KIND == EXP_DW_DOWN ? F : d;
    *ntn = static_cast<int>((N + S::kN - 1) / S::kN);
    *ntm = KIND == EXP_DW_DOWN ? static_cast<int>((d + kBM - 1) / kBM) : static_cast<int>((2 * F + kBM - 1) / kBM);
    const int64_t mt = S::kDw ? E * *ntm : R < E ? R : (R - E) / kBM + E;  // sum of ceil(n_e / kBM), sum n_e = R
    return mt * *ntn;
}

constexpr int64_t kMaxTiles = 1 << 26;  // (tile numbers are 32 bits)
constexpr int64_t kFewTiles = 16 * kCUs;  // of two products in one launch

template <int FIRST, int SECOND = kNone>
hipError_t launch(const ExpertsArgs& a, const ExpertsArgs& a2, hipStream_t stream) {
    int ntm, ntn, ntm2 = 0, ntn2 = 0;
    const int64_t n = tiles<FIRST>(a.R, a.E, a.d, a.F, &ntm, &ntn);
    int64_t n2 = 0;
    if constexpr (SECOND != kNone) n2 = tiles<SECOND>(a2.R, a2.E, a2.d, a2.F, &ntm2, &ntn2);
    if (n > kMaxTiles || n2 > kMaxTiles) return hipErrorInvalidValue;
    if (n + n2 == 0) return hipSuccess;
    // whole eights of blocks: one for every XCD's stretch
    const int64_t blocks = (n + n2 + 7) / 8 * 8;
    const unsigned grid = static_cast<unsigned>(blocks < kCUs ? blocks : kCUs);
    hipLaunchKernelGGL((k_experts<FIRST, SECOND>), dim3(grid), dim3(64 * kWaves), 0, stream, a, ntm, ntn, a2, ntm2, ntn2);
    return hipGetLastError();
}

}  // namespace

// The most rows that every launch can take.
int64_t experts_max_rows(int E, int d, int F) {
    const int64_t ntn = ((d > F ? d : F) + 127) / 128;
    const int64_t most = (kMaxTiles / ntn - E) * kBM;
    if (static_cast<int64_t>(E) * ((2ll * F + 255) / 256) * ((d + 255) / 256) > kMaxTiles) return -1;
    return most < 0 ? -1 : most < (1ll << 31) - 256 ? most : (1ll << 31) - 256;
}

hipError_t launch_experts(ExpertsKind kind, const ExpertsArgs& a, hipStream_t stream) {
    if (a.E < 1 || a.R < 0 || a.d % 64 || a.F % 64 || a.d < 64 || a.F < 64) return hipErrorInvalidValue;
    switch (kind) {
        case EXP_UP: return launch<EXP_UP>(a, a, stream);
        case EXP_DOWN: return launch<EXP_DOWN>(a, a, stream);
        case EXP_DH: return launch<EXP_DH>(a, a, stream);
        case EXP_DX: return launch<EXP_DX>(a, a, stream);
        case EXP_DW_UP: return launch<EXP_DW_UP>(a, a, stream);
        case EXP_DW_DOWN: return launch<EXP_DW_DOWN>(a, a, stream);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_experts_pair(ExpertsKind kind, const ExpertsArgs& a, const ExpertsArgs& dw, hipStream_t stream) {
    if (a.E < 1 || a.R < 0 || a.d % 64 || a.F % 64 || a.d < 64 || a.F < 64) return hipErrorInvalidValue;
    int m, n;
    const int64_t both = kind == EXP_DH ? tiles<EXP_DH>(a.R, a.E, a.d, a.F, &m, &n) + tiles<EXP_DW_DOWN>(a.R, a.E, a.d, a.F, &m, &n)
                                        : tiles<EXP_DX>(a.R, a.E, a.d, a.F, &m, &n) + tiles<EXP_DW_UP>(a.R, a.E, a.d, a.F, &m, &n);
    if (kind == EXP_DH && both <= kFewTiles) return launch<EXP_DH, EXP_DW_DOWN>(a, dw, stream);
    if (kind == EXP_DX && both <= kFewTiles) return launch<EXP_DX, EXP_DW_UP>(a, dw, stream);
    const hipError_t err = launch_experts(kind, a, stream);
    return err != hipSuccess ? err : launch_experts(kind == EXP_DH ? EXP_DW_DOWN : EXP_DW_UP, dw, stream);
}

}  // namespace moe
