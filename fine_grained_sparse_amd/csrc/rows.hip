// Rows of the experts' training side: the tokens' order by expert, the copy of
// each token to its experts' rows, the weighted sum back, and the gradients of
// both.
#include "common.hpp"
#include "experts.hpp"

namespace moe {
namespace {

// ---------------------------------------------------------------- the order
// A stable counting sort of the assignments a = t K + k by expert.  A block of
// 16 waves takes `per` consecutive assignments, a wave 1/16 of them, 64 at a
// time: lanes with the same expert find each other by one ballot per bit of the
// id, so an assignment's place among the wave's is a popcount, and only one
// lane per expert touches the wave's running counts (LDS).  The
// order never depends on timing, and an expert chosen twice by a token has two
// places.  What is not this call's (foreign ids, masked tokens) counts as
// expert E and is dropped.
constexpr int kOrderWaves = 16, kOrderBlock = 64 * kOrderWaves;

// Block-wide exclusive scan over 1024 threads; *total: the sum.
__device__ __forceinline__ int order_scan(int x, int* total, int* sh) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 63) sh[w] = incl;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kOrderWaves; ++i) {
        const int v = sh[i];
        before += i < w ? v : 0;
        sum += v;
    }
    *total = sum;
    return before + incl - x;
}

__device__ __forceinline__ int local_expert(const int32_t* idx, const uint8_t* mask, int64_t a, int64_t end, int E,
                                            int e0, int K) {
    if (a >= end) return E;
    const unsigned e = static_cast<unsigned>(idx[a]) - static_cast<unsigned>(e0);
    if (e >= static_cast<unsigned>(E) || (mask && !mask[static_cast<uint32_t>(a) / static_cast<uint32_t>(K)])) return E;
    return static_cast<int>(e);
}

// SINGLE: the whole sort in one block.  Otherwise the block's counts go to
// part[block][E] and the places among its own to pos; k_order_finish adds what
// comes before.
template <bool SINGLE>
__global__ __launch_bounds__(kOrderBlock) void k_order(const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
                                                       int64_t A, int E, int e0, int K, int bits, int64_t per,
                                                       int32_t* __restrict__ part, int32_t* __restrict__ counts,
                                                       int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_token,
                                                       int32_t* pos) {
    extern __shared__ int run[];  // [16][E + 1]: each wave's running counts, then where its own begin
    __shared__ int sh[kOrderWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, E1 = E + 1;
    const int64_t b0 = blockIdx.x * per, b1 = min(A, b0 + per);
    const int64_t seg = (per / kOrderWaves + 63) / 64 * 64;  // (per is a whole number of 1024)
    const int64_t a0 = b0 + w * seg, a1 = min(b1, a0 + seg);
    for (int i = tid; i < kOrderWaves * E1; i += kOrderBlock) run[i] = 0;
    __syncthreads();
    int* const mine = run + w * E1;
    for (int64_t c = a0; c < a1; c += 64) {
        const int e = local_expert(idx, mask, c + lane, a1, E, e0, K);
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const uint64_t v = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? v : ~v;
        }
        const int before = __popcll(same & ((1ull << lane) - 1ull)), all = __popcll(same);
        const int base = mine[e];
        __builtin_amdgcn_wave_barrier();
        if (before == all - 1) mine[e] = base + all;  // (the last of them; all have read by then: one wave)
        __builtin_amdgcn_wave_barrier();
        if (c + lane < a1) pos[c + lane] = e < E ? base + before : -1;
    }
    __syncthreads();
    int cnt = 0;
    if (tid < E)
        for (int i = 0; i < kOrderWaves; ++i) {
            const int v = run[i * E1 + tid];
            run[i * E1 + tid] = cnt;
            cnt += v;
        }
    if (!SINGLE && tid < E) part[static_cast<int64_t>(blockIdx.x) * E + tid] = cnt;
    int off = 0;
    if (SINGLE) {
        int total;
        off = order_scan(tid < E ? cnt : 0, &total, sh);
        if (tid < E) {
            if (counts) counts[tid] = cnt;
            offsets[tid] = off;
            for (int i = 0; i < kOrderWaves; ++i) run[i * E1 + tid] += off;
        }
        if (tid == 0) offsets[E] = total;
    }
    __syncthreads();
    for (int64_t c = a0; c < a1; c += 64) {
        const int64_t a = c + lane;
        const int e = local_expert(idx, mask, a, a1, E, e0, K);
        if (e < E) {
            const int p = pos[a] + mine[e];
            pos[a] = p;
            if (SINGLE && sorted_token) sorted_token[p] = static_cast<int32_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(K));
        }
    }
}

// Every block sums the counts of all blocks, and those before it, for itself:
// one launch less than a scan of its own, and part stays in the L2.
__global__ __launch_bounds__(kOrderBlock) void k_order_finish(const int32_t* __restrict__ idx,
                                                              const uint8_t* __restrict__ mask, int64_t A, int E, int e0,
                                                              int K, int64_t per, const int32_t* __restrict__ part,
                                                              int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ sorted_token, int32_t* pos) {
    __shared__ int begin[1024], all[1024], sh[kOrderWaves];
    const int tid = threadIdx.x;
    begin[tid] = all[tid] = 0;
    __syncthreads();
    int width = 64;  // threads that take the experts; the others take other blocks' counts
    while (width < E) width <<= 1;
    const int e = tid & (width - 1), groups = kOrderBlock / width;
    if (e < E) {
        int c = 0, f = 0;
#pragma unroll 8
        for (int b = tid / width; b < static_cast<int>(gridDim.x); b += groups) {
            const int v = part[static_cast<int64_t>(b) * E + e];
            f += b < static_cast<int>(blockIdx.x) ? v : 0;
            c += v;
        }
        atomicAdd(&all[e], c);  // (whole numbers: in any order)
        atomicAdd(&begin[e], f);
    }
    __syncthreads();
    const int cnt = all[tid], before = begin[tid];
    int total;
    const int off = order_scan(cnt, &total, sh);
    begin[tid] = off + before;
    if (blockIdx.x == 0) {
        if (tid < E) {
            if (counts) counts[tid] = cnt;
            offsets[tid] = off;
        }
        if (tid == 0) offsets[E] = total;
    }
    __syncthreads();
    const int64_t b0 = blockIdx.x * per, b1 = min(A, b0 + per);
    for (int64_t a = b0 + tid; a < b1; a += kOrderBlock) {
        const int x = local_expert(idx, mask, a, b1, E, e0, K);
        if (x < E) {
            const int p = pos[a] + begin[x];
            pos[a] = p;
            if (sorted_token) sorted_token[p] = static_cast<int32_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(K));
        }
    }
}

// ------------------------------------------------------- to the rows and back
// n / c for n < 2^31 by a multiplication: (n m) >> (31 + s) with s = ceil(log2 c),
// m = ceil(2^(31 + s) / c) < 2^32; exact (the error n (m c - 2^(31+s)) / (c 2^(31+s)) is
// below 1 / c).
struct Div {
    uint32_t m, s, c;
    explicit Div(uint32_t c_) : c(c_) {
        s = 0;
        while ((1u << s) < c) ++s;
        m = static_cast<uint32_t>(((1ull << (31 + s)) + c - 1) / c);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> (31 + s));
    }
};

// 16 bytes that are read, or written, once in the call, past the caches.  16384 tokens of 7168
// bf16 columns, top-8: sorted and summed back in turn 415 + 366 us, 408 + 428 with cached stores
// (which the next kernel pays for), 405 + 410 with neither, each by itself; the weighted sum and its
// gradients in turn 404 + 822, 468 + 794 with cached stores.  (x itself is read through the
// caches: 355 against 402 us.)  5.1 to 5.8 TB/s; a large copy reaches 4.9 here.
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 once(const uint4* p) {
    const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
    return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void once(uint4* p, uint4 v) {
    __builtin_nontemporal_store((u32x4_t{v.x, v.y, v.z, v.w}), reinterpret_cast<u32x4_t*>(p));
}

__device__ __forceinline__ bool row_ok(int p, int64_t rows) { return p >= 0 && p < rows; }

// A thread carries 16 bytes of a token's row to its K places.
template <int KM>
__global__ __launch_bounds__(256) void k_spread(const uint4* __restrict__ x, const int32_t* __restrict__ pos, uint32_t n,
                                                Div chunks, int K, int64_t rows, uint4* __restrict__ xs) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const uint32_t t = chunks(i), c = i - t * chunks.c;
    const uint4 v = x[i];
#pragma unroll
    for (int k = 0; k < KM; ++k)
        if (k < K) {
            const int p = pos[static_cast<int64_t>(t) * K + k];
            if (row_ok(p, rows)) once(xs + static_cast<int64_t>(p) * chunks.c + c, v);
        }
}

template <typename T> struct Chunk;  // the values of 16 bytes
template <> struct Chunk<bf16_t> {
    static constexpr int N = 8;
    __device__ __forceinline__ static void get(uint4 v, float (&o)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(u[i] << 16);
            o[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static uint4 put(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Chunk<float> {
    static constexpr int N = 4;
    __device__ __forceinline__ static void get(uint4 v, float (&o)[4]) {
        o[0] = __uint_as_float(v.x);
        o[1] = __uint_as_float(v.y);
        o[2] = __uint_as_float(v.z);
        o[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static uint4 put(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};

// A thread sums 16 bytes' worth of columns of a token over its K rows, all of
// which are asked for before the first is used; in slot order, in fp32.
template <typename T, int KM>
__global__ __launch_bounds__(256) void k_gather(const uint4* __restrict__ y, const float* __restrict__ w,
                                                const int32_t* __restrict__ pos, const uint4* res, uint32_t n, Div chunks,
                                                int K, int64_t rows, uint4* out) {
    constexpr int N = Chunk<T>::N;
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const uint32_t t = chunks(i), c = i - t * chunks.c;
    uint4 v[KM];
    bool ok[KM];
    float wk[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k) {
        ok[k] = false;
        if (k < K) {
            const int64_t a = static_cast<int64_t>(t) * K + k;
            const int p = pos[a];
            ok[k] = row_ok(p, rows);
            if (ok[k]) v[k] = once(y + static_cast<int64_t>(p) * chunks.c + c);
            wk[k] = w ? w[a] : 1.f;
        }
    }
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    if (res) Chunk<T>::get(res[i], acc);
#pragma unroll
    for (int k = 0; k < KM; ++k)
        if (ok[k]) {
            float f[N];
            Chunk<T>::get(v[k], f);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = fmaf(wk[k], f[e], acc[e]);
        }
    out[i] = Chunk<T>::put(acc);
}

// The gradients of the weighted sum in one pass over y: G threads take KM of a
// token's rows (several tokens per wave for short rows, several waves for long
// ones), hold 16 bytes of dout at a time and go over the rows with it.  dy of a
// row is written where y of it was read, which may be the same memory.  Eight rows a time, so that dout is read
// once or twice; one (a block of 1024) where the tokens are too few to fill the chip:
// 10.1 -> 5.4 us at 64 tokens of 7168 columns, top-8.  4001 tokens of 3584, top-16: 176 us (sixteen
// rows a time, which spilled: 256), 5.2 TB/s.
template <typename T, int KM, bool DY, bool DW>
__global__ __launch_bounds__(KM == 1 ? 1024 : 256) void k_gather_backward(const uint4* __restrict__ dout, const uint4* y,
                                                          const float* __restrict__ w, const int32_t* __restrict__ pos,
                                                          int64_t T0, int64_t Tn, uint32_t C, int K, int G, int64_t rows,
                                                          uint4* dy, float* __restrict__ dw) {
    constexpr int N = Chunk<T>::N;
    __shared__ float sh[16][KM];
    const int g = threadIdx.x & (G - 1), k0 = blockIdx.y * KM;
    const int64_t t = T0 + static_cast<int64_t>(blockIdx.x) * (blockDim.x / G) + threadIdx.x / G;
    const bool live = t < Tn;
    int p[KM];
    float wk[KM], s[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k) {
        p[k] = -1;
        wk[k] = s[k] = 0.f;
        if (k0 + k < K && live) {
            const int v = pos[t * K + k0 + k];
            if (row_ok(v, rows)) p[k] = v;
            if (DY) wk[k] = w[t * K + k0 + k];
        }
    }
    if (live)
        for (uint32_t c = g; c < C; c += G) {
            float o[N];
            Chunk<T>::get(dout[t * C + c], o);
            uint4 v[KM];
            if (DW) {
#pragma unroll
                for (int k = 0; k < KM; ++k)
                    if (p[k] >= 0) v[k] = once(y + static_cast<int64_t>(p[k]) * C + c);
            }
#pragma unroll
            for (int k = 0; k < KM; ++k) {
                if (p[k] < 0) continue;
                if (DY) {
                    float q[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) q[e] = wk[k] * o[e];
                    once(dy + static_cast<int64_t>(p[k]) * C + c, Chunk<T>::put(q));
                }
                if (DW) {
                    float f[N];
                    Chunk<T>::get(v[k], f);
#pragma unroll
                    for (int e = 0; e < N; ++e) s[k] = fmaf(f[e], o[e], s[k]);
                }
            }
        }
    if (!DW) return;
    const int half = G < 64 ? G : 64;
#pragma unroll
    for (int k = 0; k < KM; ++k)
        for (int off = half / 2; off; off >>= 1) s[k] += __shfl_xor(s[k], off);
    if (G <= 64) {
#pragma unroll
        for (int k = 0; k < KM; ++k)
            if (live && k0 + k < K && g == k) dw[t * K + k0 + k] = s[k];  // (G >= 8)
        return;
    }
    const int wv = threadIdx.x >> 6;  // (G == blockDim.x)
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < KM; ++k) sh[wv][k] = s[k];
    __syncthreads();
    if (live && threadIdx.x < KM && k0 + static_cast<int>(threadIdx.x) < K) {
        float v = 0.f;
        for (int i = 0; i < G / 64; ++i) v += sh[i][threadIdx.x];
        dw[t * K + k0 + threadIdx.x] = v;
    }
}

constexpr int64_t kPerLaunch = (1ll << 31) - 256;  // chunks of 16 bytes a launch goes over

}  // namespace

// One block up to kOrderSingle assignments, else up to kOrderBlocks of at least 1024:
// 5.6 / 6.7 us (one block / two launches) at 2048 over 32 experts, 7.8 / 7.0 at 4096; 6.7 / 7.6 and
// 10.1 / 7.8 over 384; 131072 assignments 12.7 us with 64 blocks, 15.5 with 32, 12.9 with 128.
constexpr int64_t kOrderSingle = 2048, kOrderBlocks = 64;
static int64_t order_per(int64_t A) {  // assignments per block
    return ((A + kOrderBlocks - 1) / kOrderBlocks + 1023) / 1024 * 1024;
}
int order_blocks(int64_t A) {
    if (A <= kOrderSingle) return 1;
    const int64_t per = order_per(A);
    return static_cast<int>((A + per - 1) / per);
}

hipError_t launch_order(const int32_t* idx, int T, int E, int e0, int K, const uint8_t* mask, int32_t* part,
                        int32_t* counts, int32_t* offsets, int32_t* sorted_token, int32_t* pos, hipStream_t stream) {
    if (E < 1 || E > 1024 || K < 1 || T < 0) return hipErrorInvalidValue;
    const int64_t A = static_cast<int64_t>(T) * K;
    int bits = 0;
    while ((E >> bits) != 0) ++bits;  // ids 0 .. E
    const int nb = order_blocks(A);
    const size_t lds = static_cast<size_t>(kOrderWaves) * (E + 1) * 4;
    const bool ask = lds + kOrderWaves * 4 > 64 * 1024;  // (with k_order's own array, more than a launch has unasked)
    if (nb == 1) {
        const int64_t per = (A + 1023) / 1024 * 1024;
        if (ask) {
            const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_order<true>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
            if (err != hipSuccess) return err;
        }
        hipLaunchKernelGGL(k_order<true>, dim3(1), dim3(kOrderBlock), lds, stream, idx, mask, A, E, e0, K, bits, per,
                           part, counts, offsets, sorted_token, pos);
        return hipGetLastError();
    }
    if (ask) {
        const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_order<false>),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (err != hipSuccess) return err;
    }
    const int64_t per = order_per(A);
    hipLaunchKernelGGL(k_order<false>, dim3(nb), dim3(kOrderBlock), lds, stream, idx, mask, A, E, e0, K, bits, per, part,
                       counts, offsets, sorted_token, pos);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_order_finish, dim3(nb), dim3(kOrderBlock), 0, stream, idx, mask, A, E, e0, K, per, part, counts,
                       offsets, sorted_token, pos);
    return hipGetLastError();
}

hipError_t launch_spread(const void* x, const int32_t* pos, int T, int K, int64_t bytes, int64_t rows, void* xs,
                         hipStream_t stream) {
    if (K < 1 || K > 16 || bytes % 16 || bytes / 16 >= (1 << 30)) return hipErrorInvalidValue;
    const int64_t C = bytes / 16, step = kPerLaunch / C;
    for (int64_t t = 0; t < T; t += step) {  // (one launch but for rows of over 34 GB)
        const int64_t nt = T - t < step ? T - t : step;
        const uint32_t n = static_cast<uint32_t>(nt * C);
        const uint4* src = static_cast<const uint4*>(x) + t * C;
        const dim3 grid(static_cast<unsigned>((n + 255ull) / 256));
        if (K <= 8)
            hipLaunchKernelGGL(k_spread<8>, grid, dim3(256), 0, stream, src, pos + t * K, n, Div(C), K, rows,
                               static_cast<uint4*>(xs));
        else
            hipLaunchKernelGGL(k_spread<16>, grid, dim3(256), 0, stream, src, pos + t * K, n, Div(C), K, rows,
                               static_cast<uint4*>(xs));
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

template <typename T>
static hipError_t gather_t(const void* y, const float* w, const int32_t* pos, const void* res, int64_t tokens, int K,
                           int64_t C, int64_t rows, void* out, hipStream_t stream) {
    const int64_t step = kPerLaunch / C;
    for (int64_t t = 0; t < tokens; t += step) {
        const int64_t nt = tokens - t < step ? tokens - t : step;
        const uint32_t n = static_cast<uint32_t>(nt * C);
        const uint4* r = res ? static_cast<const uint4*>(res) + t * C : nullptr;
        uint4* o = static_cast<uint4*>(out) + t * C;
        const dim3 grid(static_cast<unsigned>((n + 255ull) / 256));
        if (K <= 8)
            hipLaunchKernelGGL((k_gather<T, 8>), grid, dim3(256), 0, stream, static_cast<const uint4*>(y),
                               w ? w + t * K : nullptr, pos + t * K, r, n, Div(C), K, rows, o);
        else
            hipLaunchKernelGGL((k_gather<T, 16>), grid, dim3(256), 0, stream, static_cast<const uint4*>(y),
                               w ? w + t * K : nullptr, pos + t * K, r, n, Div(C), K, rows, o);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

hipError_t launch_gather(DType dt, const void* y, const float* w, const int32_t* pos, const void* res, int T, int K,
                         int64_t d, int64_t rows, void* out, hipStream_t stream) {
    const int64_t C = d * (dt == DT_BF16 ? 2 : 4) / 16;
    if (K < 1 || K > 16 || d % 8 || C >= (1 << 30)) return hipErrorInvalidValue;
    return dt == DT_BF16 ? gather_t<bf16_t>(y, w, pos, res, T, K, C, rows, out, stream)
                         : gather_t<float>(y, w, pos, res, T, K, C, rows, out, stream);
}

template <typename T, int KM>
static hipError_t gather_backward_t(const void* dout, const void* y, const float* w, const int32_t* pos, int64_t tokens,
                                    int K, uint32_t C, int64_t rows, void* dy, float* dw, hipStream_t stream) {
    // threads per token, in blocks of at least 256: no more than a row's chunks
    // up to a wave, then a block per token
    int G = 8;
    while (G < 64 && G < static_cast<int>(C)) G <<= 1;
    if (C > 64) G = KM == 1 && C > 256 ? 1024 : 256;
    const int block = G < 256 ? 256 : G, groups = (K + KM - 1) / KM;
    const int64_t per = block / G, most = (1ll << 31) / block / groups;  // (a launch has less than 2^32 threads)
    auto f = dy && dw ? k_gather_backward<T, KM, true, true>
                      : dy ? k_gather_backward<T, KM, true, false> : k_gather_backward<T, KM, false, true>;
    for (int64_t t = 0; t < tokens; t += most * per) {
        const int64_t blocks = (tokens - t + per - 1) / per;
        hipLaunchKernelGGL(f, dim3(static_cast<unsigned>(blocks < most ? blocks : most), groups), dim3(block), 0, stream,
                           static_cast<const uint4*>(dout), static_cast<const uint4*>(y), w, pos, t, tokens, C, K, G, rows,
                           static_cast<uint4*>(dy), dw);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

constexpr int64_t kFewRows = 2048;  // rows that take a block each (of over 64 chunks)

hipError_t launch_gather_backward(DType dt, const void* dout, const void* y, const float* w, const int32_t* pos, int T,
                                  int K, int64_t d, int64_t rows, void* dy, float* dw, hipStream_t stream) {
    const int64_t C = d * (dt == DT_BF16 ? 2 : 4) / 16;
    if (K < 1 || K > 16 || d % 8 || C >= (1 << 30)) return hipErrorInvalidValue;
    const uint32_t c = static_cast<uint32_t>(C);
    const bool few = C > 64 && static_cast<int64_t>(T) * K <= kFewRows;
    if (dt == DT_BF16)
        return few ? gather_backward_t<bf16_t, 1>(dout, y, w, pos, T, K, c, rows, dy, dw, stream)
                   : gather_backward_t<bf16_t, 8>(dout, y, w, pos, T, K, c, rows, dy, dw, stream);
    return few ? gather_backward_t<float, 1>(dout, y, w, pos, T, K, c, rows, dy, dw, stream)
               : gather_backward_t<float, 8>(dout, y, w, pos, T, K, c, rows, dy, dw, stream);
}

}  // namespace moe
