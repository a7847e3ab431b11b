// One AdamW step over many tensors: decoupled weight decay, moments in fp32 or
// in 8 bits.
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2   (g scaled by grad_scale)
//   p <- (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit moments.  128 consecutive values share a power of two (E8M0).  m is E4M3 (sign, 4
// exponent bits, bias 7, 3 fraction bits), scaled so that the block's largest value lies in
// [128, 256); v, never negative, has 5 exponent bits (bias 15) and 3 fraction
// bits, the largest in [2^15, 2^16).  v keeps no root: the average is linear in
// v, and rounded at random it keeps its mean, while rounded to nearest a
// change of 1 - b2 = 1e-3 would never leave a value of 3 fraction bits.  Under the root a
// code of 0 counts as the smallest one above it, 2^-33 to 2^-32 of the block's largest v:
// beside a v that was rounded to 0, an m that was rounded up moved its parameter by up to 1390
// lr (values of 1e-5 to 1e-7 of their block's largest; 1.9 lr now, 1.1 with fp32 moments).  Not beside
// an m too large for so small a v: a state that was given so, and is no average of
// gradients, is taken as it is.  The random bits are a hash of (seed, step, tensor,
// element): the same step gives the same bits, whatever the launch.  A product or sum of
// the moments is rounded by itself (no fused multiply-add), so that the codes are those of
// the formula in fp32.
// bf16 parameters are rounded at random too: lr of a step is mostly below half
// a step of bf16.
#include <cmath>

#include "common.hpp"
#include "experts.hpp"

namespace moe {
namespace {

constexpr int kPerThread = 8, kSpan = 256 * kPerThread, kTurns = 4;
constexpr int64_t kChunk = static_cast<int64_t>(kSpan) * kTurns;  // elements of a block

// The tensors' table in device memory: an entry each, then each one's first block.
constexpr int kPiece = 56;  // entries that a launch writes, from its arguments
struct Piece {
    moe_adamw_tensor t[kPiece];
    uint32_t first[kPiece];
    int32_t at, n;
};
__global__ __launch_bounds__(64) void k_adamw_table(const Piece p, moe_adamw_tensor* __restrict__ table,
                                                    uint32_t* __restrict__ first) {
    const int i = threadIdx.x;
    if (i < p.n) {
        table[p.at + i] = p.t[i];
        first[p.at + i] = p.first[i];
    }
}

struct Step {
    float b1, b2, n1, n2;      // b, 1 - b
    double beta1, beta2, c1, c2;  // c: 1 - beta^step, of a step that the host knows
    float lr, eps, wd;
    int32_t step;
    uint32_t seed;
    const float* lr_dev;
    const int32_t* step_dev;
    const float* grad_scale;
};

// A. Appleby's 32-bit mixer (public domain).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85ebca6bu;
    h = (h ^ (h >> 13)) * 0xc2b2ae35u;
    return h ^ (h >> 16);
}

// Block -> tensor: the last whose first block is not behind it (an empty one has the
// first block of the one after it).  Two loads deep up to 4096 tensors.
__device__ __forceinline__ int find_tensor(const uint32_t* __restrict__ first, int n, uint32_t block) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 63) / 64, i = lane * step;
        const bool before = i < n && first[lo + i] <= block;  // (lane 0's always is)
        const int last = 63 - __clzll(__ballot(before));
        lo += last * step;
        n = min(step, n - last * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The largest over the 16 lanes that share a block of 128 values.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o)));
    return v;
}

// E8M0 code of a block whose largest magnitude has these bits: that value then
// has exponent TOP; 255 for one with infinities or NaN.
template <int TOP>
__device__ __forceinline__ int scale_code(uint32_t bits) {
    const int e = static_cast<int>(bits >> 23);
    return e == 255 ? 255 : max(e - TOP, 0);
}

// (As native vectors: the structures of unpack8 and pack8 gave 4.9 TB/s where these give 5.2.)
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void all8(const float* p, float (&o)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p + 4 * h);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[4 * h + k] = __uint_as_float(v[k]);
    }
}
__device__ __forceinline__ void all8(const bf16_t* p, float (&o)[8]) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        o[2 * k] = __uint_as_float(v[k] << 16);
        o[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
    }
}
__device__ __forceinline__ void all8(float* p, const float (&v)[8], int) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4_t*>(p + 4 * h) = u32x4_t{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                                         __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
}
__device__ __forceinline__ void all8(bf16_t* p, const float (&v)[8], int) { pack8(p, v); }

template <typename T>
__device__ __forceinline__ void get8(const T* p, int64_t i, int live, float (&o)[8]) {
    if (live == 8) {
        all8(p + i, o);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = k < live ? Elem<T>::to_f32(p[i + k]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int64_t i, int live, const float (&v)[8]) {
    if (live == 8) {
        all8(p + i, v, 0);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < live) p[i + k] = Elem<T>::from_f32(v[k]);
    }
}
__device__ __forceinline__ uint2 codes8(const uint8_t* p, int64_t i, int live) {
    if (live == 8) return *reinterpret_cast<const uint2*>(p + i);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < live) w[k >> 2] |= static_cast<uint32_t>(p[i + k]) << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void codes8(uint8_t* p, int64_t i, int live, uint2 v) {
    if (live == 8) {
        *reinterpret_cast<uint2*>(p + i) = v;
    } else {
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < live) p[i + k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
    }
}

// A code's bits, from bit 20 on (m's sign at bit 31), are those of a float that is 2^-120
// (m) or 2^-112 (v) of its scaled value, subnormals included.  Values of blocks
// with scale 255 are NaN; that is seen to apart.
constexpr int kShiftM = 120 - 127, kShiftV = 112 - 127;  // beside the scale's code
__device__ __forceinline__ float value_m(uint32_t top, int s) {  // top: the code in bits 24 to 31
    return ldexpf(__uint_as_float(static_cast<uint32_t>(static_cast<int32_t>(top) >> 4) & 0x87f00000u), s + kShiftM);
}
__device__ __forceinline__ float value_v(uint32_t top, int s) {
    return ldexpf(__uint_as_float((top >> 4) & 0x0ff00000u), s + kShiftV);
}
// ... and back, 16 random bits (bits 8 to 23 of rnd, above 0x80) deciding between a
// value's two neighbours; the code is bits 24 to 31.
__device__ __forceinline__ uint32_t code_v(float x, int s, uint32_t rnd) {
    return (__float_as_uint(ldexpf(fabsf(x), -s - kShiftV)) << 4) + rnd;
}
__device__ __forceinline__ uint32_t code_m(float x, int s, uint32_t rnd) {
    return ((__float_as_uint(ldexpf(fabsf(x), -s - kShiftM)) << 4) + rnd) | (__float_as_uint(x) & 0x80000000u);
}
// Byte 3 of four words, in order.
__device__ __forceinline__ uint32_t tops(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(b, a, 0x0c0c0703u) | __builtin_amdgcn_perm(d, c, 0x07030c0cu);
}

// bf16 in bits 16 to 31, 16 random bits deciding; infinities and NaN are seen to apart.
__device__ __forceinline__ uint32_t bf16_at_random(float x, uint32_t rnd16) { return __float_as_uint(x) + rnd16; }

// moe_adamw_tensor with pointers that the compiler knows to be of global memory.
#define MOE_GLOBAL __attribute__((address_space(1)))
struct Entry {
    MOE_GLOBAL char *param, *grad, *avg, *sq;
    MOE_GLOBAL uint8_t *avg_scale, *sq_scale;
    MOE_GLOBAL char* copy;
    int64_t n;
};
static_assert(sizeof(Entry) == sizeof(moe_adamw_tensor), "one layout");

// x b + y and x y with every operation rounded (__fmul_rn and its like are contracted).
__device__ __forceinline__ float average(float x, float b, float y) {
#pragma clang fp contract(off)
    const float q = x * b;
    return q + y;
}
__device__ __forceinline__ float product(float x, float y) {
#pragma clang fp contract(off)
    return x * y;
}

// An m over this many times the root of v's smallest code does not belong to a v below it: of averages of the
// same gradients it is at most (1 - b1) / sqrt((1 - b2) (1 - b1^2 / b2)) times the root of v (7.3 with 0.9 and
// 0.999), and a code that rounding adds to it is 10 such roots at most.
constexpr float kMostM = 64.f;

template <typename TP, typename TG, bool EIGHT>
__global__ __launch_bounds__(256) void k_adamw(const moe_adamw_tensor* __restrict__ table,
                                               const uint32_t* __restrict__ first, int tensors, const Step S) {
    const int tid = threadIdx.x;
    const int ti = find_tensor(first, tensors, blockIdx.x);
    const Entry t = reinterpret_cast<const Entry*>(table)[ti];
    const int64_t n = t.n, c0 = static_cast<int64_t>(blockIdx.x - first[ti]) * kChunk;
    const float lr = S.lr_dev ? *S.lr_dev : S.lr;
    const int step = S.step_dev ? *S.step_dev : S.step;
    const float gs = S.grad_scale ? *S.grad_scale : 1.f;
    const float keep = static_cast<float>(1.0 - static_cast<double>(lr) * S.wd);
    double d1 = S.c1, d2 = S.c2;
    if (S.step_dev) {
        double q1 = 1.0, q2 = 1.0, s1 = S.beta1, s2 = S.beta2;
        for (uint32_t k = static_cast<uint32_t>(max(step, 1)); k; k >>= 1, s1 *= s1, s2 *= s2)
            if (k & 1) q1 *= s1, q2 *= s2;
        d1 = 1.0 - q1;
        d2 = 1.0 - q2;
    }
    const float rate = static_cast<float>(static_cast<double>(lr) / d1);
    const float root = static_cast<float>(1.0 / sqrt(d2));
    const uint32_t key0 = mix(mix(mix(S.seed) + static_cast<uint32_t>(step)) + static_cast<uint32_t>(ti));
    TP* const p = (TP*)t.param;
    const TG* const g = (const TG*)t.grad;
    void *const avg = (void*)t.avg, *const sq = (void*)t.sq;
    uint8_t *const avg_scale = (uint8_t*)t.avg_scale, *const sq_scale = (uint8_t*)t.sq_scale;
    bf16_t* const copy = (bf16_t*)t.copy;
#pragma unroll 1
    for (int r = 0; r < kTurns; ++r) {
        const int64_t i = c0 + r * kSpan + tid * kPerThread;
        const int live = static_cast<int>(min(max(n - i, int64_t(0)), int64_t(8)));
        if (c0 + r * kSpan >= n) break;  // (uniform)
        float pv[8], gv[8], m[8], v[8];
        get8(p, i, live, pv);
        get8(g, i, live, gv);
        int sm = 0, sv = 0;
        float least = 0.f;
        if (EIGHT) {
            uint2 cm = make_uint2(0, 0), cv = cm;
            if (live) {
                cm = codes8(static_cast<const uint8_t*>(avg), i, live);
                cv = codes8(static_cast<const uint8_t*>(sq), i, live);
                sm = avg_scale[i >> 7];
                sv = sq_scale[i >> 7];
            }
            const uint32_t wm[2] = {cm.x, cm.y}, wv[2] = {cv.x, cv.y};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                m[k] = value_m(wm[k >> 2] << (24 - 8 * (k & 3)), sm);
                v[k] = value_v(wv[k >> 2] << (24 - 8 * (k & 3)), sv);
            }
            least = ldexpf(S.b2, sv + kShiftV - 129);  // b2 times code 1
            if (__any(sm == 255 || sv == 255)) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    m[k] = sm == 255 ? __builtin_nanf("") : m[k];
                    v[k] = sv == 255 ? __builtin_nanf("") : v[k];
                }
            }
        } else {
            get8(static_cast<const float*>(avg), i, live, m);
            get8(static_cast<const float*>(sq), i, live, v);
        }
        uint32_t low = ~0u;  // (bits of floats that are not negative; NaN's are the largest)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float gk = gv[k] * gs;
            m[k] = average(m[k], S.b1, gk * S.n1);
            v[k] = average(v[k], S.b2, product(gk * S.n2, gk));
            low = min(low, __float_as_uint(v[k]));
        }
        auto update = [&](int k, float x) {
            pv[k] = pv[k] * keep - rate * m[k] * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(x) * root + S.eps);
        };
        // (a branch, rarely taken: 600 M bf16 parameters 1309 -> 1330 us; with the choice in every update 1281 -> 1321)
        if (EIGHT && __any(low < __float_as_uint(least))) {
            const float most = kMostM * __builtin_amdgcn_sqrtf(least);
#pragma unroll
            for (int k = 0; k < 8; ++k) update(k, v[k] < least && fabsf(m[k]) <= most ? least : v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) update(k, v[k]);
        }
        constexpr bool kHash = EIGHT || sizeof(TP) == 2;
        uint32_t word[8];
        if (kHash) {
            const uint32_t key = key0 + static_cast<uint32_t>(i >> 32) * 0x9e3779b9u;
#pragma unroll
            for (int k = 0; k < 8; ++k) word[k] = mix(static_cast<uint32_t>(i) + k + key);
        }
        if (EIGHT) {
            uint32_t am = 0, av = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= live) m[k] = v[k] = 0.f;
                am = max(am, __float_as_uint(m[k]) & 0x7fffffffu);
                av = max(av, __float_as_uint(v[k]) & 0x7fffffffu);
            }
            sm = scale_code<7>(max16(am));
            sv = scale_code<15>(max16(av));
            uint32_t cm[8], cv[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                cm[k] = code_m(m[k], sm, __builtin_amdgcn_perm(word[k], 0x80u, 0x0c050400u));
                cv[k] = code_v(v[k], sv, __builtin_amdgcn_perm(word[k], 0x80u, 0x0c070600u));
            }
            const uint32_t wm[2] = {tops(cm[0], cm[1], cm[2], cm[3]), tops(cm[4], cm[5], cm[6], cm[7])};
            const uint32_t wv[2] = {tops(cv[0], cv[1], cv[2], cv[3]), tops(cv[4], cv[5], cv[6], cv[7])};
            if (live) {
                codes8(static_cast<uint8_t*>(avg), i, live, make_uint2(wm[0], wm[1]));
                codes8(static_cast<uint8_t*>(sq), i, live, make_uint2(wv[0], wv[1]));
                if ((tid & 15) == 0) {
                    avg_scale[i >> 7] = static_cast<uint8_t>(sm);
                    sq_scale[i >> 7] = static_cast<uint8_t>(sv);
                }
            }
        } else {
            put8(static_cast<float*>(avg), i, live, m);
            put8(static_cast<float*>(sq), i, live, v);
        }
        if (sizeof(TP) == 2) {
            uint32_t b[8];
            bool odd = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                b[k] = bf16_at_random(pv[k], mix(word[k] ^ 0x9e3779b9u) & 0xffffu);
                odd |= !(fabsf(pv[k]) < __builtin_inff());
            }
            if (__any(odd)) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (!(fabsf(pv[k]) < __builtin_inff())) b[k] = static_cast<uint32_t>(f32_to_bf16(pv[k])) << 16;
            }
            if (live == 8) {
                auto two = [&](int k) { return __builtin_amdgcn_perm(b[k + 1], b[k], 0x07060302u); };
                stg16(reinterpret_cast<char*>(p) + i * 2, make_uint4(two(0), two(2), two(4), two(6)));
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < live) reinterpret_cast<uint16_t*>(p)[i + k] = static_cast<uint16_t>(b[k] >> 16);
            }
        } else {
            put8(reinterpret_cast<float*>(p), i, live, pv);
            if (copy) put8(copy, i, live, pv);
        }
    }
}

constexpr int kTensors = 48;  // of a launch: their table is a kernel argument
struct MomentsTable {
    const uint8_t *m[kTensors], *v[kTensors], *ms[kTensors], *vs[kTensors];
    float *om[kTensors], *ov[kTensors];
    int64_t len[kTensors];
    uint32_t first[kTensors];
    int32_t n;
};

// Codes to the values they stand for.
__global__ __launch_bounds__(256) void k_moments(const MomentsTable T) {
    int lo = 0, hi = T.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (T.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const int64_t n = T.len[lo], c0 = static_cast<int64_t>(blockIdx.x - T.first[lo]) * kChunk;
    // four values a thread and turn, so that a wave's stores are whole lines
    auto one = [&](const uint8_t* codes, const uint8_t* scales, float* out, auto value) {
        if (!out) return;
        uint32_t w[2 * kTurns];
        int s[2 * kTurns];
#pragma unroll
        for (int r = 0; r < 2 * kTurns; ++r) {
            const int64_t i = c0 + r * 1024 + threadIdx.x * 4;
            if (i + 4 <= n) {
                w[r] = *reinterpret_cast<const uint32_t*>(codes + i);
                s[r] = scales[i >> 7];
            }
        }
#pragma unroll
        for (int r = 0; r < 2 * kTurns; ++r) {
            const int64_t i = c0 + r * 1024 + threadIdx.x * 4;
            if (i + 4 <= n)
                *reinterpret_cast<float4*>(out + i) = make_float4(value(w[r] << 24, s[r]), value(w[r] << 16, s[r]),
                                                                  value(w[r] << 8, s[r]), value(w[r], s[r]));
            else
                for (int64_t k = i; k < n; ++k) out[k] = value(static_cast<uint32_t>(codes[k]) << 24, scales[k >> 7]);
        }
    };
    one(T.m[lo], T.ms[lo], T.om[lo], [](uint32_t c, int s) { return s == 255 ? __builtin_nanf("") : value_m(c, s); });
    one(T.v[lo], T.vs[lo], T.ov[lo], [](uint32_t c, int s) { return s == 255 ? __builtin_nanf("") : value_v(c, s); });
}

template <typename TP, typename TG>
void enqueue(bool eight, const moe_adamw_tensor* t, const uint32_t* f, int n, const Step& S, unsigned blocks,
             hipStream_t stream) {
    if (eight)
        hipLaunchKernelGGL((k_adamw<TP, TG, true>), dim3(blocks), dim3(256), 0, stream, t, f, n, S);
    else
        hipLaunchKernelGGL((k_adamw<TP, TG, false>), dim3(blocks), dim3(256), 0, stream, t, f, n, S);
}

}  // namespace

int64_t adamw_table_bytes(int n) { return static_cast<int64_t>(n) * (sizeof(moe_adamw_tensor) + 4); }
int64_t adamw_blocks(const moe_adamw_tensor* t, int n) {
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i) blocks += (t[i].n + kChunk - 1) / kChunk;
    return blocks;
}

hipError_t launch_adamw(const moe_adamw_desc& D, const moe_adamw_tensor* t, int n, void* table, hipStream_t stream) {
    moe_adamw_tensor* const entries = static_cast<moe_adamw_tensor*>(table);
    uint32_t* const first = reinterpret_cast<uint32_t*>(entries + n);
    const int64_t blocks = adamw_blocks(t, n);
    if (blocks == 0) return hipSuccess;
    if (!D.keep_table) {
        int64_t at = 0;
        for (int i = 0; i < n; i += kPiece) {
            Piece p;
            p.at = i;
            p.n = n - i < kPiece ? n - i : kPiece;
            for (int k = 0; k < p.n; ++k) {
                p.t[k] = t[i + k];
                p.first[k] = static_cast<uint32_t>(at);
                at += (t[i + k].n + kChunk - 1) / kChunk;
            }
            hipLaunchKernelGGL(k_adamw_table, dim3(1), dim3(64), 0, stream, p, entries, first);
            const hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
    }
    Step S{};
    S.beta1 = D.beta_avg;
    S.beta2 = D.beta_sq;
    S.b1 = static_cast<float>(D.beta_avg);
    S.b2 = static_cast<float>(D.beta_sq);
    S.n1 = static_cast<float>(1.0 - D.beta_avg);
    S.n2 = static_cast<float>(1.0 - D.beta_sq);
    S.c1 = 1.0 - std::pow(D.beta_avg, D.step);
    S.c2 = 1.0 - std::pow(D.beta_sq, D.step);
    S.lr = D.lr;
    S.eps = D.eps;
    S.wd = D.weight_decay;
    S.step = D.step;
    S.seed = D.seed;
    S.lr_dev = D.lr_device;
    S.step_dev = D.step_device;
    S.grad_scale = D.grad_scale;
    const bool p16 = D.param_dtype == MOE_BF16, g16 = D.grad_dtype == MOE_BF16, eight = D.moment_bits == 8;
    const unsigned b = static_cast<unsigned>(blocks);
    if (p16) g16 ? enqueue<bf16_t, bf16_t>(eight, entries, first, n, S, b, stream) : enqueue<bf16_t, float>(eight, entries, first, n, S, b, stream);
    else g16 ? enqueue<float, bf16_t>(eight, entries, first, n, S, b, stream) : enqueue<float, float>(eight, entries, first, n, S, b, stream);
    return hipGetLastError();
}

hipError_t launch_adamw_moments(const moe_adamw_tensor* t, float* const* avg, float* const* sq, int n,
                                hipStream_t stream) {
    MomentsTable T{};
    int64_t blocks = 0;
    auto flush = [&]() {
        if (T.n == 0) return hipSuccess;
        hipLaunchKernelGGL(k_moments, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, T);
        T.n = 0;
        blocks = 0;
        return hipGetLastError();
    };
    for (int i = 0; i < n; ++i) {
        float *om = avg ? avg[i] : nullptr, *ov = sq ? sq[i] : nullptr;
        if (t[i].n == 0 || (!om && !ov)) continue;
        const int64_t nb = (t[i].n + kChunk - 1) / kChunk;
        if (T.n == kTensors || blocks + nb >= (1 << 24)) {
            const hipError_t err = flush();
            if (err != hipSuccess) return err;
        }
        const int k = T.n++;
        T.m[k] = static_cast<const uint8_t*>(t[i].exp_avg);
        T.v[k] = static_cast<const uint8_t*>(t[i].exp_avg_sq);
        T.ms[k] = t[i].exp_avg_scale;
        T.vs[k] = t[i].exp_avg_sq_scale;
        T.om[k] = om;
        T.ov[k] = ov;
        T.len[k] = t[i].n;
        T.first[k] = static_cast<uint32_t>(blocks);
        blocks += nb;
    }
    return flush();
}

}  // namespace moe
