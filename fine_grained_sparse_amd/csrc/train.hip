// The router's training side: balance loss with per-sequence expert counts,
// and the gradient of the loss and of the gate weights at the logits.
// Formulas: include/moe_train.h.
//
// Every kernel here reads or writes the logits [T, E] once and is bound by
// that traffic.  A wave owns a token: lane l holds experts 128 j + 2 l and
// + 1, so a row is read in 512-byte pieces and its sums are one butterfly.
#include "common.hpp"
#include "train.hpp"

namespace moe {
namespace {

// sigmoid with the hardware exp2 and reciprocal: e = exp(-z) = 2^p 2^r with
// p = -z log2(e) rounded and r its rounding error, so that e carries about
// one ulp at any z.  Returns s and 1 - s = e s (no cancellation near s = 1).
// Logits past +-87 are held there (s is 1.6e-38 or 1).
struct Sigm {
    float s, c;
};
__device__ __forceinline__ Sigm sigm(float z) {
    constexpr float kL = 1.44269502f, kLlo = 1.92596303e-8f, kLn2 = 0.693147181f;
    const float m = -fminf(fmaxf(z, -87.f), 87.f);
    const float p = m * kL;
    const float r = fmaf(m, kLlo, fmaf(m, kL, -p));
    float e = __builtin_amdgcn_exp2f(p);
    e = fmaf(e, r * kLn2, e);
    Sigm o;
    o.s = __builtin_amdgcn_rcpf(1.f + e);
    o.c = e * o.s;
    return o;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// Two neighbours of a row, which may start at any 4-byte address (odd E).
typedef float f32x2_any __attribute__((ext_vector_type(2), aligned(4)));
__device__ __forceinline__ float2 load2(const float* p, int e, int E) {
    if (e + 1 < E) {
        const f32x2_any v = *reinterpret_cast<const f32x2_any*>(p + e);
        return make_float2(v[0], v[1]);
    }
    return make_float2(e < E ? p[e] : 0.f, 0.f);
}
__device__ __forceinline__ void store2(float* p, int e, int E, float a, float b) {
    if (e + 1 < E) {
        f32x2_any v;
        v[0] = a;
        v[1] = b;
        *reinterpret_cast<f32x2_any*>(p + e) = v;
    } else if (e < E) {
        p[e] = a;
    }
}

__device__ __forceinline__ int seq_lo(const SeqArgs& a, int q) { return a.off ? min(max(a.off[q], 0), a.T) : 0; }
__device__ __forceinline__ int seq_hi(const SeqArgs& a, int q) { return a.off ? min(max(a.off[q + 1], 0), a.T) : a.T; }

// The first sequence that ends after token t (S if none does).
__device__ __forceinline__ int seq_of(const SeqArgs& a, int t) {
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

// One block per chunk of C tokens (C <= 64).  For every sequence q that the
// chunk c meets, the sums of p and the counts over their common tokens go to
// partial row c + q: along the ascending sequences c + q grows with every
// (chunk, sequence) pair that meets, so the rows are distinct and at most
// chunks + S.  The balance over blocks does not depend on the sequences.
template <int J2>
__global__ __launch_bounds__(256) void k_balance_partial(const SeqArgs a, int C, const float* __restrict__ z,
                                                         const int32_t* __restrict__ idx, float* __restrict__ part_p,
                                                         int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
                                                         int32_t* __restrict__ ticket) {
    __shared__ float sp[4][kMaxE];
    __shared__ int hist[kMaxE];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int c = blockIdx.x, c0 = c * C, c1 = min(a.T, c0 + C);
    if (c == 0 && tid == 0) *ticket = 0;  // for k_balance_final
    for (int q = seq_of(a, c0); q < a.S && seq_lo(a, q) < c1; ++q) {
        const int lo = max(seq_lo(a, q), c0), hi = min(seq_hi(a, q), c1);
        if (lo >= hi) continue;
        const int64_t slot = c + q;
        for (int e = tid; e < a.E; e += 256) hist[e] = 0;
        float acc[2 * J2];
#pragma unroll
        for (int j = 0; j < 2 * J2; ++j) acc[j] = 0.f;
        for (int t = lo + wid; t < hi; t += 4) {
            if (a.mask && !a.mask[t]) continue;
            const float* row = z + static_cast<int64_t>(t) * a.E;
            float s[2 * J2], sum = 0.f;
#pragma unroll
            for (int j = 0; j < J2; ++j) {
                const int e = j * 128 + lane * 2;
                const float2 v = load2(row, e, a.E);
                s[2 * j] = e < a.E ? sigm(v.x).s : 0.f;
                s[2 * j + 1] = e + 1 < a.E ? sigm(v.y).s : 0.f;
                sum += s[2 * j] + s[2 * j + 1];
            }
            const float inv = 1.f / (wave_sum(sum) + 1e-20f);
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) acc[j] = fmaf(s[j], inv, acc[j]);
        }
        __syncthreads();
        const int64_t i1 = static_cast<int64_t>(hi) * a.K;
        for (int64_t i = static_cast<int64_t>(lo) * a.K + tid; i < i1; i += 256) {
            const unsigned e = static_cast<unsigned>(idx[i]);
            if (e < static_cast<unsigned>(a.E) && (!a.mask || a.mask[i / a.K])) atomicAdd(&hist[e], 1);
        }
#pragma unroll
        for (int j = 0; j < J2; ++j) {
            sp[wid][j * 128 + lane * 2] = acc[2 * j];
            sp[wid][j * 128 + lane * 2 + 1] = acc[2 * j + 1];
        }
        if (wid == 0) {
            const int t = lo + lane;
            const uint64_t live = __ballot(t < hi && (!a.mask || a.mask[t < hi ? t : lo]));
            if (lane == 0) part_n[slot] = __popcll(live);
        }
        __syncthreads();
        for (int e = tid; e < a.E; e += 256) {
            part_p[slot * a.E + e] = (sp[0][e] + sp[1][e]) + (sp[2][e] + sp[3][e]);
            part_c[slot * a.E + e] = hist[e];
        }
        __syncthreads();
    }
}

// Block (64 experts, sequence): the 16 waves take the sequence's partial
// rows in turn, their sums meet in LDS in wave order; the counts go out, and
// the block's share of the loss goes to part_l.  The last block to finish
// adds the shares up in a fixed order.
__global__ __launch_bounds__(1024) void k_balance_final(const SeqArgs a, int C, const float* __restrict__ part_p,
                                                        const int32_t* __restrict__ part_c,
                                                        const int32_t* __restrict__ part_n, float alpha,
                                                        float* part_l, int32_t* ticket, float* __restrict__ loss,
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
        const int cl = (hi - 1) / C;
#pragma unroll 4
        for (int c = lo / C + wid; c <= cl; c += 16) {
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
            __hip_atomic_store(part_l + static_cast<int64_t>(q) * gridDim.x + blockIdx.x, l * f, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
            const int total = static_cast<int>(gridDim.x * gridDim.y);
            last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    const int total = static_cast<int>(gridDim.x * gridDim.y);
    float l = 0.f;
    for (int i = threadIdx.x; i < total; i += 1024)
        l += __hip_atomic_load(part_l + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

// A wave per token, kTW consecutive tokens per wave.  The gate term touches
// only the K chosen experts: lane k < K computes its own and adds it to a
// row in LDS (zero between tokens), from which the owning lanes take it.
constexpr int kTW = 4;
template <int J2>
__global__ __launch_bounds__(256) void k_gate_backward(const SeqArgs a, const float* __restrict__ z,
                                                       const int32_t* __restrict__ idx, const float* __restrict__ dw,
                                                       float scale, const int32_t* __restrict__ counts, float alpha,
                                                       const float* __restrict__ d_loss, float* __restrict__ dz) {
    __shared__ float rows[4][kMaxE];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    float* row = rows[wid];
    for (int e = lane; e < kMaxE; e += 64) row[e] = 0.f;
    __syncthreads();
    const int t0 = (blockIdx.x * 4 + wid) * kTW, t1 = min(a.T, t0 + kTW);
    if (t0 >= t1) return;
    float co[2 * J2];  // a_q of this lane's experts, for the sequence in hand
    int q = -1, qlo = 0, qhi = 0;
    for (int t = t0; t < t1; ++t) {
        float* out = dz + static_cast<int64_t>(t) * a.E;
        if (a.mask && !a.mask[t]) {
#pragma unroll
            for (int j = 0; j < J2; ++j) store2(out, j * 128 + lane * 2, a.E, 0.f, 0.f);
            continue;
        }
        const float* zr = z + static_cast<int64_t>(t) * a.E;
        float d[2 * J2];
        bool member = false;
        if (counts) {
            if (q < 0 || t >= qhi) {
                q = seq_of(a, t);
                qlo = q < a.S ? seq_lo(a, q) : a.T;
                qhi = q < a.S ? seq_hi(a, q) : a.T;
                if (q < a.S) {
                    const int32_t* cr = counts + static_cast<int64_t>(q) * a.E;
                    float total = 0.f;
#pragma unroll
                    for (int j = 0; j < J2; ++j) {
                        const int e = j * 128 + lane * 2;
                        co[2 * j] = e < a.E ? static_cast<float>(cr[e]) : 0.f;
                        co[2 * j + 1] = e + 1 < a.E ? static_cast<float>(cr[e + 1]) : 0.f;
                        total += co[2 * j] + co[2 * j + 1];
                    }
                    // K n_q is the sum of the counts
                    const float n = wave_sum(total) / static_cast<float>(a.K);
                    const float g = alpha * (d_loss ? *d_loss : 1.f) / static_cast<float>(a.S);
                    const float f = n > 0.f ? g * (static_cast<float>(a.E) / (static_cast<float>(a.K) * n) / n) : 0.f;
#pragma unroll
                    for (int j = 0; j < 2 * J2; ++j) co[j] *= f;
                }
            }
            member = q < a.S && t >= qlo;
        }
        if (member) {
            float s[2 * J2], sum = 0.f, dot = 0.f;
#pragma unroll
            for (int j = 0; j < J2; ++j) {
                const int e = j * 128 + lane * 2;
                const float2 v = load2(zr, e, a.E);
                const Sigm s0 = sigm(v.x), s1 = sigm(v.y);
                s[2 * j] = s0.s * s0.c;
                s[2 * j + 1] = s1.s * s1.c;
                const float x0 = e < a.E ? s0.s : 0.f, x1 = e + 1 < a.E ? s1.s : 0.f;
                sum += x0 + x1;
                dot = fmaf(co[2 * j], x0, fmaf(co[2 * j + 1], x1, dot));
            }
            const float inv = 1.f / (wave_sum(sum) + 1e-20f);
            const float mean = wave_sum(dot) * inv;
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) d[j] = (co[j] - mean) * inv * s[j];
        } else {
#pragma unroll
            for (int j = 0; j < 2 * J2; ++j) d[j] = 0.f;
        }
        if (dw) {
            const bool use = lane < a.K;
            const int64_t i = static_cast<int64_t>(t) * a.K + (use ? lane : 0);
            const int e = idx[i];
            const bool ok = use && static_cast<unsigned>(e) < static_cast<unsigned>(a.E);
            const Sigm s = sigm(ok ? zr[e] : 0.f);
            const float g = ok ? dw[i] : 0.f, sc = ok ? s.s : 0.f;
            const float den = wave_sum(sc) + 1e-20f;
            const float mean = wave_sum(g * sc) / den;
            if (ok) atomicAdd(&row[e], scale / den * (g - mean) * (s.s * s.c));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int j = 0; j < J2; ++j) {
                d[2 * j] += row[j * 128 + lane * 2];
                d[2 * j + 1] += row[j * 128 + lane * 2 + 1];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (ok) row[e] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < J2; ++j) store2(out, j * 128 + lane * 2, a.E, d[2 * j], d[2 * j + 1]);
    }
}

__global__ __launch_bounds__(256) void k_split_rows(const float* __restrict__ src, int64_t R, int C, int Cp,
                                                    bf16_t* __restrict__ dst) {
    const int64_t n = R * Cp;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / Cp;
        const int c = static_cast<int>(i % Cp);
        const float v = c < C ? src[r * C + c] : 0.f;
        const bf16_t h = f32_to_bf16(v), l = f32_to_bf16(v - bf16_to_f32(h));
        bf16_t* o = dst + r * 3 * Cp + c;
        o[0] = h;
        o[Cp] = l;
        o[2 * Cp] = h;
    }
}

// 64 x 64 tiles through LDS.
template <int KIND>
__global__ __launch_bounds__(256) void k_transpose(const void* __restrict__ src, int64_t R, int64_t C, int64_t Rp,
                                                   void* __restrict__ dst) {
    __shared__ float tile[64][65];
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 64, c0 = static_cast<int64_t>(blockIdx.y) * 64;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int i = w; i < 64; i += 4) {
        const int64_t r = r0 + i, c = c0 + lane;
        float v = 0.f;
        if (r < R && c < C)
            v = KIND == TR_BF16 ? bf16_to_f32(static_cast<const bf16_t*>(src)[r * C + c])
                                : static_cast<const float*>(src)[r * C + c];
        tile[i][lane] = v;
    }
    __syncthreads();
    for (int i = w; i < 64; i += 4) {
        const int64_t c = c0 + i, r = r0 + lane;
        if (c >= C || r >= Rp) continue;
        const float v = tile[lane][i];
        if (KIND == TR_F32) {
            static_cast<float*>(dst)[c * Rp + r] = v;
            continue;
        }
        bf16_t* o = static_cast<bf16_t*>(dst);
        const bf16_t h = f32_to_bf16(v);
        if (KIND == TR_BF16) {
            o[c * Rp + r] = h;
            continue;
        }
        const float r1 = v - bf16_to_f32(h);
        const bf16_t m = f32_to_bf16(r1);
        if (KIND == TR_PLANES3) {
            o[c * Rp + r] = h;
            o[(C + c) * Rp + r] = m;
            o[(2 * C + c) * Rp + r] = f32_to_bf16(r1 - bf16_to_f32(m));
        } else {
            o[c * 3 * Rp + r] = h;
            o[c * 3 * Rp + Rp + r] = h;
            o[c * 3 * Rp + 2 * Rp + r] = m;
        }
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

int balance_chunk(int T) { return T >= 32768 ? 64 : 32; }
int64_t balance_slots(int T, int S) { return (static_cast<int64_t>(T) + balance_chunk(T) - 1) / balance_chunk(T) + S; }

// The kernels hold 2 J2 experts per lane: the smallest that reaches E.
#define MOE_FOR_E(E, CALL)   \
    do {                     \
        if ((E) <= 128)      \
            CALL(1);         \
        else if ((E) <= 256) \
            CALL(2);         \
        else if ((E) <= 384) \
            CALL(3);         \
        else if ((E) <= 512) \
            CALL(4);         \
        else if ((E) <= 896) \
            CALL(7);         \
        else                 \
            CALL(8);         \
    } while (0)

hipError_t launch_balance_loss(const SeqArgs& a, const float* z, const int32_t* idx, float alpha, float* part_p,
                               int32_t* part_c, int32_t* part_n, float* part_l, int32_t* ticket, float* loss,
                               int32_t* seq_counts, hipStream_t stream) {
    if (a.T < 1 || a.E < 1 || a.E > kMaxE || a.S < 1 || a.S > 65535) return hipErrorInvalidValue;
    const int C = balance_chunk(a.T);
    const dim3 grid((a.T + C - 1) / C);
#define MOE_CALL(J2)                                                                                             \
    hipLaunchKernelGGL(k_balance_partial<J2>, grid, dim3(256), 0, stream, a, C, z, idx, part_p, part_c, part_n, \
                       ticket)
    MOE_FOR_E(a.E, MOE_CALL);
#undef MOE_CALL
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_balance_final, dim3((a.E + 63) / 64, a.S), dim3(1024), 0, stream, a, C, part_p, part_c,
                       part_n, alpha, part_l, ticket, loss, seq_counts);
    return hipGetLastError();
}

hipError_t launch_gate_backward(const SeqArgs& a, const float* z, const int32_t* idx, const float* dw, float scale,
                                const int32_t* counts, float alpha, const float* d_loss, float* dz,
                                hipStream_t stream) {
    if (a.T < 1 || a.E < 1 || a.E > kMaxE) return hipErrorInvalidValue;
    const dim3 grid((a.T + 4 * kTW - 1) / (4 * kTW));
#define MOE_CALL(J2)                                                                                               \
    hipLaunchKernelGGL(k_gate_backward<J2>, grid, dim3(256), 0, stream, a, z, idx, dw, scale, counts, alpha, d_loss, \
                       dz)
    MOE_FOR_E(a.E, MOE_CALL);
#undef MOE_CALL
    return hipGetLastError();
}

hipError_t launch_split_rows(const float* src, int64_t R, int C, int Cp, uint16_t* dst, hipStream_t stream) {
    if (R <= 0) return hipSuccess;
    hipLaunchKernelGGL(k_split_rows, dim3(grid_of(R * Cp, 8192)), dim3(256), 0, stream, src, R, C, Cp, dst);
    return hipGetLastError();
}

hipError_t launch_transpose(TransposeKind kind, const void* src, int64_t R, int64_t C, int64_t Rp, void* dst,
                            hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>((Rp + 63) / 64), static_cast<unsigned>((C + 63) / 64));
    if (grid.y > 65535u || Rp >= (int64_t{1} << 31)) return hipErrorInvalidValue;
#define MOE_CALL(K) hipLaunchKernelGGL(k_transpose<K>, grid, dim3(256), 0, stream, src, R, C, Rp, dst)
    switch (kind) {
        case TR_F32: MOE_CALL(TR_F32); break;
        case TR_BF16: MOE_CALL(TR_BF16); break;
        case TR_PLANES3: MOE_CALL(TR_PLANES3); break;
        case TR_HHL: MOE_CALL(TR_HHL); break;
    }
#undef MOE_CALL
    return hipGetLastError();
}

hipError_t launch_sum_planes(const float* part, int n, int64_t stride, int64_t count, float* out, hipStream_t stream) {
    if (count % 4 || stride % 4) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_sum_planes, dim3(grid_of(count / 4, 8192)), dim3(256), 0, stream,
                       reinterpret_cast<const float4*>(part), n, stride / 4, count / 4, reinterpret_cast<float4*>(out));
    return hipGetLastError();
}

}  // namespace moe
