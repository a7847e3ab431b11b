// The router's training side: balance loss with per-sequence expert counts,
// and the gradient of the loss and of the gate weights at the logits.
// Formulas: include/moe_train.h.
//
// Every kernel here reads or writes the logits [T, E] once and is bound by
// that traffic.  A wave owns a token: lane l holds experts 128 j + 2 l and
// + 1, so a row is read in 512-byte pieces and its sums are one butterfly.
#include "common.hpp"
#include "launch.hpp"
#include "train.hpp"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

// sigmoid with the hardware exp2 and reciprocal: e = exp(-z) = 2^p 2^r with
// p = -z log2(e) rounded and r its rounding error, so that e carries about
// one ulp at any z.  Returns s and 1 - s = e s (no cancellation near s = 1).
// Logits past +-87 are held there (s is 1.6e-38 or 1); a NaN stays one (the
// maximum and minimum that pass it on cost what the others do).
struct Sigm {
    float s, c;
};
__device__ __forceinline__ Sigm sigm(float z) {
    constexpr float kL = 1.44269502f, kLlo = 1.92596303e-8f, kLn2 = 0.693147181f;
    const float m = -__builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -87.f), 87.f);
    const float p = m * kL;
    const float r = fmaf(m, kLlo, fmaf(m, kL, -p));
    float e = __builtin_amdgcn_exp2f(p);
    e = fmaf(e, r * kLn2, e);
    Sigm o;
    o.s = __builtin_amdgcn_rcpf(1.f + e);
    o.c = e * o.s;
    return o;
}

// Sums over the 16 lanes of a row, and over the wave, in every lane: lane
// moves inside the adds (partners at distance 1, 2, then the mirrored half
// and row, whose sums are complete by then) and two half-wave swaps, where
// shuffles through LDS took six round trips.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __uint_as_float(static_cast<uint32_t>(
                   __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float row16_sum(float v) {
    v = add_dpp<0xB1>(v);   // quad_perm [1,0,3,2]
    v = add_dpp<0x4E>(v);   // quad_perm [2,3,0,1]
    v = add_dpp<0x141>(v);  // row_half_mirror
    return add_dpp<0x140>(v);  // row_mirror
}
__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A lane's two neighbours e, e + 1 of a row of E, which may start at any
// 4-byte address (odd E).  FULL: both exist in every lane; otherwise the pair
// is read where it fits and what lies past the row is 0.
typedef float f32x2_any __attribute__((ext_vector_type(2), aligned(4)));
template <bool FULL>
__device__ __forceinline__ float2 load2(const float* p, int e, int E) {
    if (FULL) {
        const f32x2_any v = *reinterpret_cast<const f32x2_any*>(p + e);
        return make_float2(v[0], v[1]);
    }
    if (E < 2) return make_float2(e == 0 ? p[0] : 0.f, 0.f);  // (uniform)
    const f32x2_any v = *reinterpret_cast<const f32x2_any*>(p + min(e, E - 2));
    return make_float2(e <= E - 2 ? v[0] : e == E - 1 ? v[1] : 0.f, e <= E - 2 ? v[1] : 0.f);
}
template <bool FULL>
__device__ __forceinline__ void store2(float* p, int e, int E, float a, float b) {
    if (FULL || e + 1 < E) {
        f32x2_any v;
        v[0] = a;
        v[1] = b;
        *reinterpret_cast<f32x2_any*>(p + e) = v;
    } else if (e < E) {
        p[e] = a;
    }
}
// A lane's 2 J2 experts of a row: 128 j + 2 lane and + 1; E lies in the last
// of the J2 pieces, so only that one looks at its end.
template <int J2>
__device__ __forceinline__ void load_row(const float* p, int lane, int E, float (&o)[2 * J2]) {
#pragma unroll
    for (int j = 0; j < J2; ++j) {
        const int e = j * 128 + lane * 2;
        const float2 v = j + 1 < J2 ? load2<true>(p, e, E) : load2<false>(p, e, E);
        o[2 * j] = v.x;
        o[2 * j + 1] = v.y;
    }
}
template <int J2>
__device__ __forceinline__ bool in_row(int j, int lane, int E) {  // element j of the lane lies in the row
    return (j >> 1) + 1 < J2 || (j >> 1) * 128 + lane * 2 + (j & 1) < E;
}

__device__ __forceinline__ int seq_lo(const SeqArgs& a, int q) { return a.off ? min(max(a.off[q], 0), a.T) : 0; }
__device__ __forceinline__ int seq_hi(const SeqArgs& a, int q) { return a.off ? min(max(a.off[q + 1], 0), a.T) : a.T; }

// The first sequence that ends after token t (S if none does).
__device__ __forceinline__ int seq_of(const SeqArgs& a, int t) {
    if (!a.off) return 0;
    if (a.S <= 64) {  // one look at all of them
        const int l = threadIdx.x & 63;
        return __popcll(__ballot(l < a.S && seq_hi(a, l < a.S ? l : 0) <= t));
    }
    int lo = 0, hi = a.S;
    while (lo < hi) {
        const int m = (lo + hi) >> 1;
        if (seq_hi(a, m) > t)
            hi = m;
        else
            lo = m + 1;
    }
    return lo;
}

constexpr int kMaxE = 1024;

// This wave's share of the sums of p over tokens lo .. hi - 1 of one sequence,
// kTok tokens at a time for each of the block's NW waves.
template <int J2, int NW, int kTok>
__device__ __forceinline__ void score_sums(const SeqArgs& a, const float* __restrict__ z, int lo, int hi, int wid, int lane,
                                           float (&acc)[2 * J2]) {
#pragma unroll
    for (int j = 0; j < 2 * J2; ++j) acc[j] = 0.f;
    for (int t = lo + wid * kTok; t < hi; t += NW * kTok) {
        float v[kTok][2 * J2], sum[kTok];
        bool live[kTok];
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            const int tu = min(t + u, hi - 1);
            live[u] = t + u < hi && (!a.mask || a.mask[tu]);
            load_row<J2>(z + static_cast<int64_t>(tu) * a.E, lane, a.E, v[u]);
        }
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            sum[u] = 0.f;
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) {
                v[u][j] = in_row<J2>(j, lane, a.E) ? sigm(v[u][j]).s : 0.f;
                sum[u] += v[u][j];
            }
        }
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            if (!live[u]) continue;  // (uniform; its scores may be NaN)
            const float inv = 1.f / (wave_sum(sum[u]) + 1e-20f);
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) acc[j] = fmaf(v[u][j], inv, acc[j]);
        }
    }
}

// The selections of each expert by the tokens that count, added to hist.
template <int NW>
__device__ __forceinline__ void count_choices(const SeqArgs& a, const int32_t* __restrict__ idx, int lo, int hi, int tid,
                                              int* hist) {
    for (int i = tid; i < (hi - lo) * a.K; i += 64 * NW) {
        const unsigned e = static_cast<unsigned>(idx[static_cast<int64_t>(lo) * a.K + i]);
        if (e < static_cast<unsigned>(a.E) && (!a.mask || a.mask[lo + i / a.K])) atomicAdd(&hist[e], 1);
    }
}

// One block per chunk of 64 tokens.  For every sequence q that the chunk c
// meets, the sums of p and the counts over their common tokens go to partial
// row c + q: along the ascending sequences c + q grows with every (chunk,
// sequence) pair that meets, so the rows are distinct and at most chunks + S,
// and the blocks' work does not depend on the sequences.  A wave takes up to
// four tokens at a time, so that their rows are in flight together.  Bound by
// reading z: 235 MB (65521 x 896) in 56 us, 4.2 TB/s; 16384 x 384, which the
// caches hold, takes 14 us, mostly the latency of one round.
constexpr int kChunk = 64;
// Tokens in hand (more experts: fewer, for the registers' sake; 65521 x 896:
// k_balance_partial 56 us with one, 64 with two, 69 with four, which suit the
// gradient) and waves of a block (65521 x 896: 64 us with 8 waves, 71 with 16;
// 16384 x 384: 15.6 / 14.0).
constexpr int toks(int j2) { return j2 <= 4 ? 4 : 2; }
constexpr int partial_toks(int j2) { return j2 <= 4 ? 4 : 1; }
constexpr int partial_waves(int j2) { return j2 <= 4 ? 16 : 8; }
template <int J2>
__global__ __launch_bounds__(64 * partial_waves(J2)) void k_balance_partial(const SeqArgs a, const float* __restrict__ z,
                                                         const int32_t* __restrict__ idx, float* __restrict__ part_p,
                                                         int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
                                                         uint64_t* __restrict__ part_l, int32_t* __restrict__ ticket) {
    constexpr int NW = partial_waves(J2), kTok = partial_toks(J2);
    __shared__ float sp[NW][J2 * 128];
    __shared__ int hist[kMaxE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = blockIdx.x, c0 = c * kChunk, c1 = min(a.T, c0 + kChunk);
    // for k_balance_final: no share is there yet
    if (c == 0 && tid == 0) *ticket = 0;
    for (int64_t i = c * 64ll * NW + tid; i < (a.E + 63) / 64 * a.S; i += gridDim.x * 64ll * NW) part_l[i] = 0;
    for (int q = seq_of(a, c0); q < a.S && seq_lo(a, q) < c1; ++q) {
        const int lo = max(seq_lo(a, q), c0), hi = min(seq_hi(a, q), c1);
        if (lo >= hi) continue;
        const int64_t slot = c + q;
        for (int e = tid; e < a.E; e += 64 * NW) hist[e] = 0;
        float acc[2 * J2];
        score_sums<J2, NW, kTok>(a, z, lo, hi, wid, lane, acc);
        __syncthreads();
        count_choices<NW>(a, idx, lo, hi, tid, hist);
#pragma unroll
        for (int j = 0; j < J2; ++j)
            *reinterpret_cast<float2*>(&sp[wid][j * 128 + lane * 2]) = make_float2(acc[2 * j], acc[2 * j + 1]);
        if (wid == 0) {
            const int t = lo + lane;
            const uint64_t live = __ballot(t < hi && (!a.mask || a.mask[t < hi ? t : lo]));
            if (lane == 0) part_n[slot] = __popcll(live);
        }
        __syncthreads();
        for (int e = tid; e < a.E; e += 64 * NW) {
            float p = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) p += sp[w][e];
            part_p[slot * a.E + e] = p;
            part_c[slot * a.E + e] = hist[e];
        }
        __syncthreads();
    }
}

// Block (64 experts, sequence): the 16 waves take the sequence's partial
// rows in turn, their sums meet in LDS in wave order; the counts go out, and
// the block's share of the loss goes to part_l.  The last block to finish
// adds the shares up in a fixed order: a launch of its own for that would cost
// more than this kernel.  A share is one atomic word that says itself that it is there (kThere),
// so the last block needs no order between other blocks' shares and tickets: it
// reads a word until it is there, and its block has stored it by then or is
// just about to.  (An acquire-release ticket instead writes back and invalidates
// the L2 in every block: 173 -> 180 us for loss and gradient of 65521 x 896 in 37
// sequences, 230 -> 310 of 16384 x 256 in 4000.)  Latency-bound: 7.8 us at
// 16384 x 384 x 4 sequences, 12.7 at 65521 x 896 x 37 (8 MB of partial rows).
constexpr uint64_t kThere = 1ull << 32;
__global__ __launch_bounds__(1024) void k_balance_final(const SeqArgs a, const float* __restrict__ part_p,
                                                        const int32_t* __restrict__ part_c,
                                                        const int32_t* __restrict__ part_n, float alpha,
                                                        uint64_t* part_l, int32_t* ticket, float* __restrict__ loss,
                                                        int32_t* __restrict__ seq_counts) {
    __shared__ float sp[16][64];
    __shared__ int sc[16][64], sn[16];
    __shared__ int last;
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int q = blockIdx.y, e = blockIdx.x * 64 + lane;
    const int lo = seq_lo(a, q), hi = seq_hi(a, q);
    float p = 0.f;
    int cnt = 0, n = 0;
    if (lo < hi) {
        const int cl = (hi - 1) / kChunk;
#pragma unroll 8
        for (int c = lo / kChunk + wid; c <= cl; c += 16) {
            const int64_t slot = c + q;
            if (e < a.E) {
                p += part_p[slot * a.E + e];
                cnt += part_c[slot * a.E + e];
            }
            n += part_n[slot];
        }
    }
    sp[wid][lane] = p;
    sc[wid][lane] = cnt;
    if (lane == 0) sn[wid] = n;
    __syncthreads();
    if (wid == 0) {
        for (int w = 1; w < 16; ++w) {
            p += sp[w][lane];
            cnt += sc[w][lane];
            n += sn[w];
        }
        if (e < a.E) seq_counts[static_cast<int64_t>(q) * a.E + e] = cnt;
        const float l = wave_sum(p * static_cast<float>(cnt));
        if (lane == 0) {
            const float nf = static_cast<float>(n);
            const float f = n > 0 ? static_cast<float>(a.E) / (static_cast<float>(a.K) * nf) / nf : 0.f;
            __hip_atomic_store(part_l + static_cast<int64_t>(q) * gridDim.x + blockIdx.x,
                               kThere | __float_as_uint(l * f), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const int total = static_cast<int>(gridDim.x * gridDim.y);
            last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    const int total = static_cast<int>(gridDim.x * gridDim.y);
    float l = 0.f;
    for (int i = threadIdx.x; i < total; i += 1024) {
        uint64_t v = 0;
        while (!(v & kThere)) v = __hip_atomic_load(part_l + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        l += __uint_as_float(static_cast<uint32_t>(v));
    }
    l = wave_sum(l);
    __syncthreads();
    if (lane == 0) sp[0][wid] = l;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.f;
        for (int w = 0; w < 16; ++w) t += sp[0][w];
        *loss = t * (alpha / static_cast<float>(a.S));
    }
}

// The whole loss of a small batch in one block: no partial rows, no second
// launch, but 2 us for every 64 tokens and every sequence, in a row.  One block
// against two launches, replayed from a graph: 6.4 / 8.0 us at 128 x 32 (T x E),
// 8.1 / 9.3 at 128 x 256, 11.0 / 11.3 at 128 x 512, 10.3 / 14.0 at 64 x 128 in four
// sequences, but 11.9 / 9.7 at 301 x 48 in two and 20 / 10 at 256 x 32 in eight; a
// call of the binding takes 3 us less.
constexpr int kSmallT = 128, kSmallS = 4, kSmallJ2 = 4;  // (J2: its sums fill 32 of the 64 KiB of LDS)
template <int J2>
__global__ __launch_bounds__(1024) void k_balance_small(const SeqArgs a, const float* __restrict__ z,
                                                        const int32_t* __restrict__ idx, float alpha,
                                                        float* __restrict__ loss, int32_t* __restrict__ seq_counts) {
    constexpr int NW = 16;
    __shared__ float sp[NW][J2 * 128], red[NW];
    __shared__ int hist[J2 * 128], sn;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    float total = 0.f;
    for (int q = 0; q < a.S; ++q) {
        const int lo = seq_lo(a, q), hi = seq_hi(a, q);
        if (tid < a.E) hist[tid] = 0;
        if (tid == 0) sn = 0;
        float acc[2 * J2];
        score_sums<J2, NW, partial_toks(J2)>(a, z, lo, hi, wid, lane, acc);
#pragma unroll
        for (int j = 0; j < J2; ++j)
            *reinterpret_cast<float2*>(&sp[wid][j * 128 + lane * 2]) = make_float2(acc[2 * j], acc[2 * j + 1]);
        __syncthreads();
        count_choices<NW>(a, idx, lo, hi, tid, hist);
        for (int t = lo + wid * 64; t < hi; t += 64 * NW) {
            const uint64_t live = __ballot(t + lane < hi && (!a.mask || a.mask[t + lane]));
            if (lane == 0) atomicAdd(&sn, __popcll(live));
        }
        __syncthreads();
        float l = 0.f;
        if (tid < a.E) {
            float p = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) p += sp[w][tid];
            const int cnt = hist[tid];
            seq_counts[static_cast<int64_t>(q) * a.E + tid] = cnt;
            l = p * static_cast<float>(cnt);
        }
        l = wave_sum(l);
        if (lane == 0) red[wid] = l;
        __syncthreads();
        if (tid == 0) {
            const int n = sn;
            const float nf = static_cast<float>(n);
            float t = 0.f;
            for (int w = 0; w < NW; ++w) t += red[w];
            total += n > 0 ? t * (static_cast<float>(a.E) / (static_cast<float>(a.K) * nf) / nf) : 0.f;
        }
    }
    if (tid == 0) *loss = total * (alpha / static_cast<float>(a.S));
}

// n_q, for the gradient: the number of tokens of a sequence that count, and not
// that of its choices over K, as a token may hold ids that no count has.
// Without a mask it is the sequence's length; with one its bytes are counted:
// by each block of the gradient for the sequences of its own tokens, or, for
// many tokens, once by k_seq_tokens, which leaves n_q (as float) at q's first
// token and at the first token of each of the gradient's waves.  The gradient
// unmasked / counting in its blocks / with k_seq_tokens, in us: 15 / 16.6 / 20 at
// 16384 x 384 in four sequences, 98 / 116 / 110 at 65521 x 896 in 37 and
// 104 / 136 / 111 in one, 328 / 2327 / 435 at 1048576 x 128 (of which k_seq_tokens 50).
constexpr int kSeqTokensT = 32768;

// This wave's share (of its block's NW) of the tokens that count among lo ..
// hi - 1: the mask in whole 16-byte pieces, single bytes at both ends.
template <int NW>
__device__ __forceinline__ int live_share(const uint8_t* mask, int lo, int hi, int tid) {
    const int p0 = lo / 16 + (lo % 16 != 0), p1 = hi / 16;  // pieces that lie inside
    int n = 0;
    if (p0 < p1) {
#pragma unroll 4
        for (int p = p0 + tid; p < p1; p += 64 * NW) {
            const uint4 v = *reinterpret_cast<const uint4*>(mask + static_cast<int64_t>(p) * 16);
            const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)  // the bytes that are not zero
                n += __popc((d[i] | ((d[i] & 0x7f7f7f7fu) + 0x7f7f7f7fu)) & 0x80808080u);
        }
        if (tid < 16) {
            if (lo + tid < p0 * 16) n += mask[lo + tid] != 0;
            if (p1 * 16 + tid < hi) n += mask[p1 * 16 + tid] != 0;
        }
    } else if (lo + tid < hi) {  // (30 tokens at most)
        n = mask[lo + tid] != 0;
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) n += __shfl_xor(n, o);
    return n;
}

// One block per 1024 tokens, a token per thread.  The part of a sequence that
// lies in the block comes from a running count of the block's mask bytes, what
// the first and the last token's sequences hold outside of it from reading
// that.  Latency: 6 us at 65521 tokens (six steps of the search, two reads).
__global__ __launch_bounds__(1024) void k_seq_tokens(const SeqArgs a, int tok, float* __restrict__ n_tok, int64_t stride) {
    __shared__ int upto[1025], wave_n[16], outer[2], ends[4];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int b0 = blockIdx.x * 1024, b1 = min(a.T, b0 + 1024), t = b0 + tid;
    const uint64_t live = __ballot(t < b1 && a.mask[t < b1 ? t : b0]);
    int l = 0, h = a.S;  // the first sequence that ends after t
    while (l < h) {
        const int m = (l + h) >> 1;
        if (seq_hi(a, m) > t)
            h = m;
        else
            l = m + 1;
    }
    int lo = 0, hi = 0;  // t's sequence (none: 0, 0)
    if (t < b1 && l < a.S && seq_lo(a, l) <= t) {
        lo = seq_lo(a, l);
        hi = seq_hi(a, l);
    }
    if (lane == 0) wave_n[wid] = __popcll(live);
    if (tid < 2) outer[tid] = 0;
    if (tid == 0) ends[0] = lo, ends[1] = hi;
    if (t == b1 - 1) ends[2] = lo, ends[3] = hi;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wid; ++w) before += wave_n[w];
    upto[tid] = before + __popcll(live & ((1ull << lane) - 1));
    if (tid == 1023) upto[1024] = before + __popcll(live);
    const int lo0 = ends[0], hi0 = ends[1], lo1 = ends[2], hi1 = ends[3];
    int n = live_share<16>(a.mask, lo0, min(hi0, b0), tid);
    if (lane == 0) atomicAdd(&outer[0], n);
    n = live_share<16>(a.mask, b1, max(hi1, b1), tid);
    if (lane == 0) atomicAdd(&outer[1], n);
    __syncthreads();
    if (lo >= hi || (t % tok && t != lo)) return;  // (a wave of the gradient asks for no other)
    n = upto[min(hi, b1) - b0] - upto[max(lo, b0) - b0] + (lo < b0 ? outer[0] : 0) + (hi > b1 ? outer[1] : 0);
    n_tok[t * stride] = static_cast<float>(n);
}

// Where k_gate_backward leaves dz as the two products' operands instead.
struct PlaneArgs {
    float *rows32, *cols32;  // (small products) dz as [T][Es] and as [Es][Ts], zero past E and T
    int32_t Es, Ts;          // E and T in whole 16s
    bf16_t* rows;   // [T][3 Ep]: hi | lo | hi of a token's row, zero past E
    bf16_t* cols;   // [Tb][3][Eb] blocks of 16 experts x 32 tokens of its parts hi, mid, lo (hi + mid + lo == dz):
                    // element (r, c) of a block at ((c / 8) 16 + r) 8 + c % 8, zero past E and T; a slab of tokens
                    // lies together
    uint16_t* live; // [32 Tb]: 0xffff for the tokens that count, else 0
    int32_t Ep, Eb, Tb;
};

enum GateOut { GATE_ROWS = 0, GATE_SMALL = 1, GATE_PLANES = 2 };

// A wave takes a few consecutive tokens.  The gate term touches only the K
// chosen experts of each: lane 16 u + k computes token u's slot k, and the
// values reach the lanes that own the experts through a row in LDS that is
// zero between tokens.  dz may be z's memory, and n_tok lie in dz: a wave reads
// both at its own tokens only, before it writes them.  Bound by its one reading
// of z and writing of dz: 470 MB (65521 x 896) in 95 us, 4.9 TB/s, a large
// copy's rate here.  (Rows whose every lane asked whether its pair lies inside
// took 146 us, those with four tokens in hand at 14 pairs a lane 225: 193
// registers, two waves per SIMD.)
template <int J2, int OUT>
__global__ __launch_bounds__(256) void k_gate_backward(const SeqArgs a, const float* z,
                                                       const int32_t* __restrict__ idx, const float* __restrict__ dw,
                                                       float scale, const int32_t* __restrict__ counts, float alpha,
                                                       const float* __restrict__ d_loss, float* dz,
                                                       const PlaneArgs pl, const float* n_tok, int64_t n_stride) {
    constexpr int kTok = toks(J2);
    __shared__ float rows[4][J2 * 128];
    __shared__ int n_at[4 * kTok];  // n_q, at the first of the block's tokens that is in q
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float* row = rows[wid];
    const int b0 = blockIdx.x * 4 * kTok, t0 = b0 + wid * kTok;
    if (counts && a.mask && !n_tok) {
        const int b1 = min(a.T, b0 + 4 * kTok);
        if (threadIdx.x < 4 * kTok) n_at[threadIdx.x] = 0;
        __syncthreads();
        for (int q = b0 < b1 ? seq_of(a, b0) : a.S; q < a.S && seq_lo(a, q) < b1; ++q) {
            const int lo = seq_lo(a, q), hi = seq_hi(a, q);
            if (lo >= hi) continue;
            const int n = live_share<4>(a.mask, lo, hi, threadIdx.x);
            if (lane == 0) atomicAdd(&n_at[max(lo, b0) - b0], n);
        }
        __syncthreads();
    }
    if (OUT == GATE_ROWS && t0 >= a.T) return;

    bool live[kTok];
#pragma unroll
    for (int u = 0; u < kTok; ++u) live[u] = t0 + u < a.T && (!a.mask || a.mask[min(t0 + u, a.T - 1)]);

    // the gate term, in lane 16 u + k
    float gv = 0.f;
    int ge = -1;
    if (dw) {
        for (int e = lane; e < J2 * 128; e += 64) row[e] = 0.f;
        const int u = lane >> 4, k = lane & 15, t = min(t0 + u, a.T - 1);
        bool use = false;
#pragma unroll
        for (int v = 0; v < kTok; ++v) use = use || (u == v && live[v]);
        use = use && k < a.K;
        const int64_t i = static_cast<int64_t>(t) * a.K + (k < a.K ? k : 0);
        const int e = idx[i];
        const bool ok = use && static_cast<unsigned>(e) < static_cast<unsigned>(a.E);
        const Sigm s = sigm(ok ? z[static_cast<int64_t>(t) * a.E + e] : 0.f);
        const float g = ok ? dw[i] : 0.f, sc = ok ? s.s : 0.f;
        const float den = row16_sum(sc) + 1e-20f;
        // g - mean in two passes: with few or alike g the first mean leaves little
        // but its rounding error, which the second removes.  sum dev s is mean 1e-20
        // without one (den holds 1e-20 more than the scores), not 0.
        const float mean = row16_sum(g * sc) / den, dev = g - mean;
        gv = scale / den * (dev - (row16_sum(ok ? dev * sc : 0.f) - mean * 1e-20f) / den) * (s.s * s.c);
        ge = ok ? e : -1;
    }

    float d[kTok][2 * J2];
#pragma unroll
    for (int u = 0; u < kTok; ++u)
#pragma unroll
        for (int j = 0; j < 2 * J2; ++j) d[u][j] = 0.f;
    if (counts && t0 < a.T) {
        float s[kTok][2 * J2], inv[kTok];
        const float n_first = n_tok ? n_tok[t0 * n_stride] : 0.f;
#pragma unroll
        for (int u = 0; u < kTok; ++u) load_row<J2>(z + static_cast<int64_t>(min(t0 + u, a.T - 1)) * a.E, lane, a.E, s[u]);
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) {
                const Sigm g = sigm(s[u][j]);
                s[u][j] = in_row<J2>(j, lane, a.E) ? g.s : 0.f;
                d[u][j] = s[u][j] * g.c;  // s (1 - s)
                sum += s[u][j];
            }
            inv[u] = 1.f / (wave_sum(sum) + 1e-20f);
        }
        bool done[kTok];
#pragma unroll
        for (int u = 0; u < kTok; ++u) done[u] = false;
        for (int q = seq_of(a, t0); q < a.S && seq_lo(a, q) < min(t0 + kTok, a.T); ++q) {
            const int qlo = seq_lo(a, q), qhi = seq_hi(a, q);
            if (qlo >= qhi) continue;
            const int32_t* cr = counts + static_cast<int64_t>(q) * a.E;
            float co[2 * J2];  // a_q of this lane's experts
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j)
                co[j] = in_row<J2>(j, lane, a.E) ? static_cast<float>(cr[(j >> 1) * 128 + lane * 2 + (j & 1)]) : 0.f;
            const float n = n_tok ? (qlo <= t0 ? n_first : n_tok[qlo * n_stride])
                                  : static_cast<float>(a.mask ? n_at[max(qlo, b0) - b0] : qhi - qlo);
            const float g = alpha * (d_loss ? *d_loss : 1.f) / static_cast<float>(a.S);
            const float f = n > 0.f ? g * (static_cast<float>(a.E) / (static_cast<float>(a.K) * n) / n) : 0.f;
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) co[j] *= f;
#pragma unroll
            for (int u = 0; u < kTok; ++u) {
                if (t0 + u < qlo || t0 + u >= qhi || done[u]) continue;  // (uniform)
                done[u] = true;
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < 2 * J2; ++j) dot = fmaf(co[j], s[u][j], dot);
                const float mean = wave_sum(dot) * inv[u];
#pragma unroll
                for (int j = 0; j < 2 * J2; ++j) d[u][j] *= (co[j] - mean) * inv[u];
            }
        }
#pragma unroll
        for (int u = 0; u < kTok; ++u)
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) d[u][j] = done[u] && live[u] ? d[u][j] : 0.f;
    }
    if (dw) {
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            const bool mine = ge >= 0 && (lane >> 4) == u;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (mine) atomicAdd(&row[ge], gv);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int j = 0; j < J2; ++j) {
                const float2 v = *reinterpret_cast<const float2*>(&row[j * 128 + lane * 2]);
                d[u][2 * j] += v.x;
                d[u][2 * j + 1] += v.y;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (mine) row[ge] = 0.f;
        }
    }
    if constexpr (OUT == GATE_ROWS) {
#pragma unroll
        for (int u = 0; u < kTok; ++u)
            if (t0 + u < a.T) {
                float* o = dz + static_cast<int64_t>(t0 + u) * a.E;
#pragma unroll
                for (int j = 0; j < J2; ++j) {
                    if (j + 1 < J2)
                        store2<true>(o, j * 128 + lane * 2, a.E, d[u][2 * j], d[u][2 * j + 1]);
                    else
                        store2<false>(o, j * 128 + lane * 2, a.E, d[u][2 * j], d[u][2 * j + 1]);
                }
            }
    } else if constexpr (OUT == GATE_SMALL) {
        if (t0 >= pl.Ts) return;
#pragma unroll
        for (int j = 0; j < 2 * J2; ++j) {
            const int e = (j >> 1) * 128 + lane * 2 + (j & 1);
            if (e >= pl.Es) continue;
#pragma unroll
            for (int u = 0; u < kTok; ++u) {
                if (t0 + u < a.T) pl.rows32[static_cast<int64_t>(t0 + u) * pl.Es + e] = d[u][j];
                pl.cols32[static_cast<int64_t>(e) * pl.Ts + t0 + u] = d[u][j];
            }
        }
    } else {
        bf16_t hi[kTok][2 * J2], mid[kTok][2 * J2], lo[kTok][2 * J2];
#pragma unroll
        for (int u = 0; u < kTok; ++u)
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) {
                hi[u][j] = f32_to_bf16(d[u][j]);
                const float r = d[u][j] - bf16_to_f32(hi[u][j]);
                mid[u][j] = f32_to_bf16(r);
                lo[u][j] = f32_to_bf16(r - bf16_to_f32(mid[u][j]));
            }
        auto pair = [](bf16_t x, bf16_t y) { return x | (static_cast<uint32_t>(y) << 16); };
        if (pl.rows) {
#pragma unroll
            for (int u = 0; u < kTok; ++u)
                if (t0 + u < a.T) {
                    uint32_t* o = reinterpret_cast<uint32_t*>(pl.rows + static_cast<int64_t>(t0 + u) * 3 * pl.Ep);
#pragma unroll
                    for (int j = 0; j < J2; ++j) {
                        const int e = j * 128 + lane * 2;
                        if (e >= pl.Ep) continue;
                        const uint32_t h = pair(hi[u][2 * j], hi[u][2 * j + 1]);
                        o[e / 2] = h;
                        o[(pl.Ep + e) / 2] = pair(mid[u][2 * j], mid[u][2 * j + 1]);
                        o[(2 * pl.Ep + e) / 2] = h;
                    }
                }
        }
        if (pl.cols && t0 < pl.Tb * 32) {
            if (lane < kTok) {
                bool l = false;
#pragma unroll
                for (int u = 0; u < kTok; ++u) l = l || (lane == u && live[u]);
                pl.live[t0 + lane] = l ? 0xffffu : 0u;
            }
            const int64_t plane = static_cast<int64_t>(pl.Eb) * 512;
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) {
                const int e = (j >> 1) * 128 + lane * 2 + (j & 1);
                if (e >= pl.Eb * 16) continue;
                bf16_t* o = pl.cols + (static_cast<int64_t>(t0 / 32) * 3 * pl.Eb + e / 16) * 512 + ((t0 % 32) / 8 * 16 + e % 16) * 8 + t0 % 8;
                if constexpr (kTok == 4) {
                    *reinterpret_cast<uint2*>(o) = make_uint2(pair(hi[0][j], hi[1][j]), pair(hi[2][j], hi[3][j]));
                    *reinterpret_cast<uint2*>(o + plane) = make_uint2(pair(mid[0][j], mid[1][j]), pair(mid[2][j], mid[3][j]));
                    *reinterpret_cast<uint2*>(o + 2 * plane) = make_uint2(pair(lo[0][j], lo[1][j]), pair(lo[2][j], lo[3][j]));
                } else {
                    *reinterpret_cast<uint32_t*>(o) = pair(hi[0][j], hi[1][j]);
                    *reinterpret_cast<uint32_t*>(o + plane) = pair(mid[0][j], mid[1][j]);
                    *reinterpret_cast<uint32_t*>(o + 2 * plane) = pair(lo[0][j], lo[1][j]);
                }
            }
        }
    }
}

// W_r [E, d] -> the packed right operand of dx: W_r^T as [d, 3 Ep] in the
// fragment-block layout of 16 x 32, its rows [hi | hi | lo]: with dz's hi | lo |
// hi a plain K = 3 Ep product gives the three terms that 16 bits of either
// side need.  A wave reads 64 columns of eight rows and writes their 16-byte
// pieces.  27 MB (384 x 7168) in 6 to 7 us.
__global__ __launch_bounds__(256) void k_pack_wt(const float* __restrict__ W, int E, int64_t d, int Ep,
                                                 bf16_t* __restrict__ dst) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + lane;  // (d is a multiple of 64)
    const int e0 = blockIdx.y * 32 + w * 8, kb = 3 * Ep / 32;
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bf16_t hh[2], ll[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int e = e0 + 2 * i + b;
            const float v = e < E ? W[e * d + n] : 0.f;
            hh[b] = f32_to_bf16(v);
            ll[b] = f32_to_bf16(v - bf16_to_f32(hh[b]));
        }
        h[i] = hh[0] | (static_cast<uint32_t>(hh[1]) << 16);
        l[i] = ll[0] | (static_cast<uint32_t>(ll[1]) << 16);
    }
    const uint4 hv = make_uint4(h[0], h[1], h[2], h[3]), lv = make_uint4(l[0], l[1], l[2], l[3]);
    bf16_t* o = dst + ((n / 16) * kb + blockIdx.y) * 512 + (w * 16 + n % 16) * 8;
    stg16(o, hv);
    stg16(o + Ep / 32 * 512, hv);
    stg16(o + 2 * (Ep / 32) * 512, lv);
}

// dW_r = dz^T x, split over the tokens: job (split, M tile, N tile) adds up
// (32 MB experts) x (256 columns) over its tokens into its plane of `part`;
// the four waves hold (16 MB) x 128 each.  dz comes in three bf16 parts that
// carry all its bits (each product with the bf16 x is then exact in the fp32
// accumulator), so a tile of M x N moves 3 M + N values per token, least with
// N the longer side.  Both operands of an MFMA want eight consecutive tokens
// per lane: k_gate_backward writes dz that way, in whole fragments of 1 KiB; x
// is row-major and is read transposed from LDS (ds_read_b64_tr_b16: a group of
// 16 lanes reads 4 rows x 16 columns, lane i receives column i).  32-byte
// chunk c of slab row r of x sits at c ^ f(r), f = r % 4 + 4 (r / 8 % 2), so the
// rows that lanes 0 - 31 read lie in different banks.
//
// With 192 accumulators a SIMD has one wave, so nothing but the order of its
// own instructions hides a latency.  Slabs of 32 tokens come straight into a
// ring of three LDS buffers (DMA: staging them in registers left the compiler
// too few, and it copied the accumulators once a slab).  In the middle of slab
// b every wave waits for its own loads of b + 1, which have had a slab's time,
// and meets the others: after that b + 1 may be read, and b - 1, which nobody
// reads any more, makes room for b + 2.  The first fragments of b + 1 are read
// under the last products of b.  Between them the loads go out one or two at a
// time: a burst of them holds up the MFMAs behind it.
// 16384 x 384 x 7168 (T x E x d): 270 GFLOP of partial products in 246 us from
// rest, 278 back to back (1.1 and 0.97 PFLOP/s; 87% of the CUs have a block,
// whose matrix pipes are then 61% busy).  On the way there: 507 us with 384 x
// 128 tiles and dz straight into registers, 559 with both operands through LDS
// one slab ahead, 359 with three buffers and register staging, 316 with the
// loads by DMA in one burst.
// x of a token that does not count may hold anything: its fragments are
// masked by `live` after the read.
typedef short s16x4 __attribute__((ext_vector_type(4)));
struct DwArgs {
    const bf16_t* cols;    // PlaneArgs::cols, ::live
    const uint16_t* live;
    const bf16_t* x;
    float* part;
    int64_t d;
    int32_t T, E, Eb, Tb, ntn, mt, nsplit;
};
// 16 (4) bytes per lane from base + off (src) to LDS at lds + 16 (4) lane.
// Nothing waits for these but wait_loads(), and no register is their target.
// (A write of m0 needs a wait state before a load to LDS reads it.)
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <int MB>
__global__ __launch_bounds__(256, 1) void k_dw(const DwArgs a) {
    constexpr int NA = 6 * MB, LA = (NA + 3) / 4;           // 1 KiB blocks of dz per slab, and per wave
    constexpr int XO = NA * 1024, LO = XO + 16384, BUF = LO + 256;  // x, live (64 bytes, four times)
    __shared__ __attribute__((aligned(1024))) char lds[3 * BUF];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, grp = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wid >> 1, wn = wid & 1;
    // split-major job order, a contiguous stretch of it per XCD: the blocks of
    // an XCD share the parts of dz they stream
    const int jobs = a.ntn * a.mt * a.nsplit;
    const int job = xcd_slot_pair(static_cast<int>(blockIdx.x), jobs, jobs);
    if (job < 0) return;
    const int sp = job / (a.ntn * a.mt), mt = job % a.mt;
    const int64_t n0 = static_cast<int64_t>(job / a.mt % a.ntn) * 256;
    const int per = (a.Tb + a.nsplit - 1) / a.nsplit;
    const int b0 = min(a.Tb, sp * per), b1 = min(a.Tb, b0 + per);
    const int eb0 = mt * 2 * MB;  // this tile's first block of 16 experts

    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(lds)));
    auto fl = [](int r) { return (r & 3) | ((r >> 1) & 4); };
    // x: block q of a slab is its rows 2 q and 2 q + 1; lane l fills position
    // l % 32 of row 2 q + l / 32
    const int xrow = lane >> 5;
    // Slab b to buffer `buf`: wave w moves blocks w, w + 4, .. of dz (block q:
    // part q / (2 MB), experts 16 (q % (2 MB)) ..) and of x.  Past the last slab
    // the last one is read again; past the ends of dz's blocks, of x's rows
    // and of its columns likewise (nothing of it is stored, or its dz is 0).
    constexpr int NL = LA + 5;  // loads per wave and slab
    auto load = [&](int b, int buf, int k) {  // the k-th of them
        const int bc = min(b, a.Tb - 1);
        const uint32_t dst = lds0 + buf * BUF;
        if (k < LA) {
            const int q = min(wid + 4 * k, NA - 1);
            const int64_t blk = static_cast<int64_t>(bc) * 3 * a.Eb + q / (2 * MB) * a.Eb + min(eb0 + q % (2 * MB), a.Eb - 1);
            dma16(a.cols + blk * 512, lane * 16, dst + q * 1024);
        } else if (k < LA + 4) {
            const int q = wid + 4 * (k - LA), r = 2 * q + xrow;
            const int c = ((((lane & 31) >> 1) ^ fl(r)) << 1) | (lane & 1);  // logical 16-byte chunk
            const int64_t row = min(bc * 32 + r, a.T - 1), col = min(n0 + c * 8, a.d - 8);
            dma16(a.x + row * a.d + col, dst + XO + q * 1024);
        } else {
            dma4(a.live + bc * 32, (lane & 15) * 4, dst + LO);
        }
    };
    auto load_all = [&](int b, int buf) {
#pragma unroll
        for (int k = 0; k < NL; ++k) load(b, buf, k);
    };
    auto read_a = [&](int buf, int p, uint4 (&f)[MB]) {
        const char* o = lds + buf * BUF + (p * 2 * MB + wm * MB) * 1024 + lane * 16;
#pragma unroll
        for (int i = 0; i < MB; ++i) f[i] = *reinterpret_cast<const uint4*>(o + i * 1024);
    };
    auto read_live = [&](int buf) { return *reinterpret_cast<const uint4*>(lds + buf * BUF + LO + grp * 16); };
    // rows 8 grp + r16 / 4 and + 4 of columns 16 j ..: 8 bytes per lane
    auto read_x = [&](int buf, int j) {
        uint2 h[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * grp + (r16 >> 2) + 4 * i;
            const char* q = lds + buf * BUF + XO + r * 512 + (((wn * 8 + j) ^ fl(r)) << 5) + (r16 & 3) * 8;
            h[i] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                 (__attribute__((address_space(3))) s16x4*)(q)));
        }
        return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
    };

    f32x4 acc[MB][8];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (b0 < b1) {
        load_all(b0, 0);
        wait_loads();
        __syncthreads();
        load_all(b0 + 1, 1);
        uint4 f[3][MB], xf[2], lm;
#pragma unroll
        for (int p = 0; p < 3; ++p) read_a(0, p, f[p]);
        xf[0] = read_x(0, 0);
        lm = read_live(0);
        int buf = 0;
        for (int b = b0; b < b1; ++b) {
            const int next = buf == 2 ? 0 : buf + 1, third = buf == 0 ? 2 : buf - 1;
            uint4 ln = lm;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j == 4) {
                    wait_loads();
                    __syncthreads();
                }
                xf[(j + 1) & 1] = j < 7 ? read_x(buf, j + 1) : read_x(next, 0);
                if (j == 7) ln = read_live(next);
                __builtin_amdgcn_sched_barrier(0);
                const uint4 x = make_uint4(xf[j & 1].x & lm.x, xf[j & 1].y & lm.y, xf[j & 1].z & lm.z, xf[j & 1].w & lm.w);
#pragma unroll
                for (int p = 0; p < 3; ++p) {
#pragma unroll
                    for (int i = 0; i < MB; ++i) acc[i][j] = Mfma<bf16_t>::run(x, f[p][i], acc[i][j]);
                    __builtin_amdgcn_sched_barrier(0);
                    if (j == 7) read_a(next, p, f[p]);
                    // the loads of b + 2 a few at a time: issued together they hold up the MFMAs behind them
                    if (j >= 4)
#pragma unroll
                        for (int k = 0; k < NL; ++k)
                            if (k * 12 / NL == (j - 4) * 3 + p) load(b + 2, third, k);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            lm = ln;
            buf = next;
        }
        wait_loads();  // no load may reach the LDS after the block has left it
    }
    // acc[i][j] of a lane: expert 16 i + lane % 16, columns 16 j + 4 (lane / 16) .. + 3
    float* out = a.part + sp * a.E * a.d;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int e = (eb0 + wm * MB + i) * 16 + r16;
        if (e >= a.E) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t n = n0 + (wn * 8 + j) * 16 + grp * 4;
            if (n < a.d)
                *reinterpret_cast<float4*>(out + e * a.d + n) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        }
    }
}

// Both products of a small router in one launch, on the vector ALUs: fp32
// FMAs.  Blocks of 16 rows (tokens for dx, experts for dW_r) x 64 columns, a
// column per lane; the 16 waves split the sum (its steps wait for memory, so
// few of them in a row), and each step of it takes one line of x or W_r and 16
// neighbours of dz (of its rows for dW_r, of its transpose for dx), the same
// for the whole wave.  4.4 us at 77 x 20 x 320 (T x E x d) fp32, 13 us at 301 x 48
// x 1024 bf16, where the matrix units' route takes four launches more.
constexpr int kSmallNW = 16;
template <typename TX>
__device__ __forceinline__ void small_rows(const float* __restrict__ A, int64_t lda, int n, const TX* __restrict__ B,
                                           int64_t d, const uint8_t* mask, int wid, float (&acc)[16]) {
    const int k0 = static_cast<int>(static_cast<int64_t>(n) * wid / kSmallNW);
    const int k1 = static_cast<int>(static_cast<int64_t>(n) * (wid + 1) / kSmallNW);
#pragma unroll 4
    for (int k = k0; k < k1; ++k) {
        float b = Elem<TX>::to_f32(B[k * d]);
        if (mask && !mask[k]) b = 0.f;
        const float* p = A + k * lda;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = fmaf(p[i], b, acc[i]);
    }
}
template <typename TX>
__global__ __launch_bounds__(64 * kSmallNW) void k_small_products(const float* __restrict__ rows, const float* __restrict__ cols,
                                                        int Es, int Ts, const TX* __restrict__ x,
                                                        const float* __restrict__ W, const uint8_t* __restrict__ mask,
                                                        int T, int E, int64_t d, int xblocks, TX* __restrict__ dx,
                                                        float* __restrict__ dW) {
    __shared__ float red[kSmallNW][16][64];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t ntn = d / 64;
    const bool isx = static_cast<int>(blockIdx.x) < xblocks;
    const int64_t b = isx ? blockIdx.x : blockIdx.x - xblocks;
    const int64_t col = (b % ntn) * 64 + lane;
    const int r0 = static_cast<int>(b / ntn) * 16;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    if (isx)
        small_rows<float>(cols + r0, Ts, E, W + col, d, nullptr, wid, acc);
    else
        small_rows<TX>(rows + r0, Es, T, x + col, d, mask, wid, acc);
#pragma unroll
    for (int i = 0; i < 16; ++i) red[wid][i][lane] = acc[i];
    __syncthreads();
    static_assert(kSmallNW == 16, "a row per wave");
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSmallNW; ++w) v += red[w][wid][lane];
    if (isx) {
        if (r0 + wid < T) dx[(r0 + wid) * d + col] = Elem<TX>::from_f32(v);
    } else {
        if (r0 + wid < E) dW[(r0 + wid) * d + col] = v;
    }
}

// Operands of the fp32 products, which run on the fp32 MFMAs of the router's
// own tile: full fp32, where planes of bf16 would need six products a side.
// [R, C] fp32 -> [C, Rp], columns R .. Rp - 1 zero, and those of rows that do
// not count (mask); 64 x 64 tiles through LDS.
__global__ __launch_bounds__(256) void k_transpose(const float* __restrict__ src, int64_t R, int64_t C, int64_t Rp,
                                                   const uint8_t* __restrict__ mask, float* __restrict__ dst) {
    __shared__ float tile[64][65];
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 64;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int64_t c0 = static_cast<int64_t>(blockIdx.y) * 64; c0 < C; c0 += static_cast<int64_t>(gridDim.y) * 64) {
        for (int i = w; i < 64; i += 4) {
            const int64_t r = r0 + i, c = c0 + lane;
            tile[i][lane] = r < R && c < C && (!mask || mask[r]) ? src[r * C + c] : 0.f;
        }
        __syncthreads();
        for (int i = w; i < 64; i += 4) {
            const int64_t c = c0 + i, r = r0 + lane;
            if (c < C && r < Rp) dst[c * Rp + r] = tile[lane][i];
        }
        __syncthreads();
    }
}
// [R, C] fp32 -> [R, Cp], columns C .. Cp - 1 zero.
__global__ __launch_bounds__(256) void k_pad_rows(const float* __restrict__ src, int64_t n, int C, int Cp,
                                                  float* __restrict__ dst) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int c = static_cast<int>(i % Cp);
        dst[i] = c < C ? src[i / Cp * C + c] : 0.f;
    }
}

__global__ __launch_bounds__(256) void k_sum_planes(const float4* __restrict__ part, int n, int64_t stride4,
                                                    int64_t count4, float4* __restrict__ out) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < count4; i += static_cast<int64_t>(gridDim.x) * 256) {
        float4 v = part[i];
        for (int p = 1; p < n; ++p) {
            const float4 o = part[p * stride4 + i];
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
        }
        out[i] = v;
    }
}

unsigned grid_of(int64_t threads, int64_t most) {
    const int64_t b = (threads + 255) / 256;
    return static_cast<unsigned>(b < most ? b : most);
}

}  // namespace

int dw_slabs(int T) { return static_cast<int>((static_cast<int64_t>(T) + 31) / 32); }

int64_t balance_slots(int T, int S) { return (static_cast<int64_t>(T) + kChunk - 1) / kChunk + S; }

// The kernels hold 2 J2 experts per lane, J2 = ceil(E / 128).
#define MOE_FOR_E(E, CALL)             \
    switch (((E) + 127) / 128) {       \
        case 1: CALL(1); break;        \
        case 2: CALL(2); break;        \
        case 3: CALL(3); break;        \
        case 4: CALL(4); break;        \
        case 5: CALL(5); break;        \
        case 6: CALL(6); break;        \
        case 7: CALL(7); break;        \
        case 8: CALL(8); break;        \
        default: return hipErrorInvalidValue; \
    }

hipError_t launch_balance_loss(const SeqArgs& a, const float* z, const int32_t* idx, float alpha, float* part_p,
                               int32_t* part_c, int32_t* part_n, uint64_t* part_l, int32_t* ticket, float* loss,
                               int32_t* seq_counts, hipStream_t stream) {
    if (a.T < 1 || a.E < 1 || a.E > kMaxE || a.S < 1 || a.S > 65535) return hipErrorInvalidValue;
    const int j2 = (a.E + 127) / 128;
    if (a.T <= kSmallT && a.S <= kSmallS && j2 <= kSmallJ2) {
#define MOE_CALL(J2) hipLaunchKernelGGL(k_balance_small<J2>, dim3(1), dim3(1024), 0, stream, a, z, idx, alpha, loss, seq_counts)
        switch (j2) {
            case 1: MOE_CALL(1); break;
            case 2: MOE_CALL(2); break;
            case 3: MOE_CALL(3); break;
            default: MOE_CALL(4); break;
        }
#undef MOE_CALL
        return hipGetLastError();
    }
    const dim3 grid((a.T + kChunk - 1) / kChunk);
#define MOE_CALL(J2) \
    hipLaunchKernelGGL(k_balance_partial<J2>, grid, dim3(64 * partial_waves(J2)), 0, stream, a, z, idx, part_p, part_c, \
                       part_n, part_l, ticket)
    MOE_FOR_E(a.E, MOE_CALL);
#undef MOE_CALL
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_balance_final, dim3((a.E + 63) / 64, a.S), dim3(1024), 0, stream, a, part_p, part_c,
                       part_n, alpha, part_l, ticket, loss, seq_counts);
    return hipGetLastError();
}

template <int OUT>
static hipError_t launch_gate(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                              const int32_t* counts, float alpha, const float* d_loss, float* dz, const PlaneArgs& pl,
                              int64_t tokens, float* n_tok, int64_t n_stride, hipStream_t stream) {
    if (a.T < 1 || a.E < 1 || a.E > kMaxE || a.K > 16) return hipErrorInvalidValue;
    const int tok = toks((a.E + 127) / 128), per = 4 * tok;
    if (!counts || !a.mask || a.T <= kSeqTokensT) n_tok = nullptr;
    if (n_tok) {
        hipLaunchKernelGGL(k_seq_tokens, dim3((a.T + 1023) / 1024), dim3(1024), 0, stream, a, tok, n_tok, n_stride);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    const dim3 grid(static_cast<unsigned>((tokens + per - 1) / per));
#define MOE_CALL(J2)                                                                                                  \
    hipLaunchKernelGGL((k_gate_backward<J2, OUT>), grid, dim3(256), 0, stream, a, z, idx, dw, scale, counts, alpha, \
                       d_loss, dz, pl, n_tok, n_stride)
    MOE_FOR_E(a.E, MOE_CALL);
#undef MOE_CALL
    return hipGetLastError();
}

hipError_t launch_gate_backward(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                const int32_t* counts, float alpha, const float* d_loss, float* dz,
                                hipStream_t stream) {
    // dz itself takes n_q at each token's first logit, unless z may be the same memory
    const uintptr_t o = reinterpret_cast<uintptr_t>(dz), i = reinterpret_cast<uintptr_t>(z);
    const uintptr_t bytes = static_cast<uintptr_t>(a.T) * a.E * 4;
    float* n_tok = o < i + bytes && i < o + bytes ? nullptr : dz;
    return launch_gate<GATE_ROWS>(a, z, idx, dw, scale, counts, alpha, d_loss, dz, PlaneArgs{}, a.T, n_tok, a.E, stream);
}

hipError_t launch_gate_backward_small(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                      const int32_t* counts, float alpha, const float* d_loss, float* rows, float* cols,
                                      hipStream_t stream) {
    PlaneArgs pl{};
    pl.rows32 = rows;
    pl.cols32 = cols;
    pl.Es = (a.E + 15) / 16 * 16;
    pl.Ts = (a.T + 15) / 16 * 16;
    return launch_gate<GATE_SMALL>(a, z, idx, dw, scale, counts, alpha, d_loss, nullptr, pl, pl.Ts, nullptr, 0, stream);
}

hipError_t launch_gate_backward_planes(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                       const int32_t* counts, float alpha, const float* d_loss, uint16_t* rows, int Ep,
                                       uint16_t* cols, uint16_t* live, float* n_tok, hipStream_t stream) {
    if (Ep % 64 || Ep < a.E || Ep >= a.E + 64) return hipErrorInvalidValue;
    PlaneArgs pl{};
    pl.rows = rows;
    pl.cols = cols;
    pl.live = live;
    pl.Ep = Ep;
    pl.Eb = (a.E + 15) / 16;
    pl.Tb = dw_slabs(a.T);
    return launch_gate<GATE_PLANES>(a, z, idx, dw, scale, counts, alpha, d_loss, nullptr, pl,
                                    static_cast<int64_t>(pl.Tb) * 32, n_tok, 1, stream);
}

hipError_t launch_pack_wt(const float* W, int E, int64_t d, int Ep, uint16_t* dst, hipStream_t stream) {
    if (d % 64 || Ep % 64) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_pack_wt, dim3(static_cast<unsigned>(d / 64), Ep / 32), dim3(256), 0, stream, W, E, d, Ep, dst);
    return hipGetLastError();
}

DwPlan dw_plan(int T, int E, int64_t d) {
    DwPlan p{};
    // M tiles of 32 MB experts, MB <= 6 (192 of a lane's registers are then
    // accumulators, at one wave per SIMD)
    const int rb = (E + 31) / 32;
    p.mt = (rb + 5) / 6;
    p.mb = (rb + p.mt - 1) / p.mt;
    p.ntn = static_cast<int>((d + 255) / 256);
    // one block per CU at a time: the fewest splits that fill 85% of the 256
    // CUs over whole rounds (each split costs a pass over [E, d] more), or the
    // fullest of the 16
    const int64_t jobs = static_cast<int64_t>(p.mt) * p.ntn;
    const int most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, (T + 31) / 32 / 4)));
    double best = 0;
    for (int n = 1; n <= most; ++n) {
        const int64_t b = jobs * n, rounds = (b + 255) / 256;
        const double full = static_cast<double>(b) / static_cast<double>(rounds * 256);
        if (full > best) {
            best = full;
            p.nsplit = n;
        }
        if (full >= 0.85) break;
    }
    return p;
}

hipError_t launch_dw(const DwPlan& p, const uint16_t* cols, const uint16_t* live, const void* x, int T, int E, int64_t d,
                     float* part, hipStream_t stream) {
    if (T < 1 || E < 1 || d < 64 || d % 8) return hipErrorInvalidValue;
    const DwArgs a{cols, live, static_cast<const bf16_t*>(x), part, d, T, E, (E + 15) / 16, dw_slabs(T), p.ntn, p.mt,
                   p.nsplit};
    const int64_t jobs = static_cast<int64_t>(p.ntn) * p.mt * p.nsplit;
    if (jobs >= (int64_t{1} << 30)) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>((jobs + 7) / 8 * 8 + 16));
    switch (p.mb) {
#define MOE_CALL(MB)                                                        \
    case MB:                                                                \
        hipLaunchKernelGGL(k_dw<MB>, grid, dim3(256), 0, stream, a); \
        break
        MOE_CALL(1);
        MOE_CALL(2);
        MOE_CALL(3);
        MOE_CALL(4);
        MOE_CALL(5);
        MOE_CALL(6);
#undef MOE_CALL
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch_small_products(bool bf16, const float* rows, const float* cols, const void* x, const float* W,
                                 const uint8_t* mask, int T, int E, int64_t d, void* dx, float* dW, hipStream_t stream) {
    if (T < 1 || E < 1 || d % 64) return hipErrorInvalidValue;
    const int64_t ntn = d / 64, xb = dx ? (static_cast<int64_t>(T) + 15) / 16 * ntn : 0, wb = dW ? (E + 15) / 16 * ntn : 0;
    if (xb + wb < 1 || xb + wb >= (int64_t{1} << 31)) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(xb + wb));
    const int Es = (E + 15) / 16 * 16, Ts = (T + 15) / 16 * 16;
    if (bf16)
        hipLaunchKernelGGL(k_small_products<bf16_t>, grid, dim3(64 * kSmallNW), 0, stream, rows, cols, Es, Ts,
                           static_cast<const bf16_t*>(x), W, mask, T, E, d, static_cast<int>(xb),
                           static_cast<bf16_t*>(dx), dW);
    else
        hipLaunchKernelGGL(k_small_products<float>, grid, dim3(64 * kSmallNW), 0, stream, rows, cols, Es, Ts,
                           static_cast<const float*>(x), W, mask, T, E, d, static_cast<int>(xb),
                           static_cast<float*>(dx), dW);
    return hipGetLastError();
}

hipError_t launch_transpose(const float* src, int64_t R, int64_t C, int64_t Rp, const uint8_t* mask, float* dst,
                            hipStream_t stream) {
    if (Rp >= (int64_t{1} << 31) * 64) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>((Rp + 63) / 64), static_cast<unsigned>(std::min<int64_t>((C + 63) / 64, 65535)));
    hipLaunchKernelGGL(k_transpose, grid, dim3(256), 0, stream, src, R, C, Rp, mask, dst);
    return hipGetLastError();
}

hipError_t launch_pad_rows(const float* src, int64_t R, int C, int Cp, float* dst, hipStream_t stream) {
    hipLaunchKernelGGL(k_pad_rows, dim3(grid_of(R * Cp, 8192)), dim3(256), 0, stream, src, R * Cp, C, Cp, dst);
    return hipGetLastError();
}

hipError_t launch_sum_planes(const float* part, int n, int64_t stride, int64_t count, float* out, hipStream_t stream) {
    if (count % 4 || stride % 4) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_sum_planes, dim3(grid_of(count / 4, 8192)), dim3(256), 0, stream,
                       reinterpret_cast<const float4*>(part), n, stride / 4, count / 4, reinterpret_cast<float4*>(out));
    return hipGetLastError();
}

}  // namespace moe
