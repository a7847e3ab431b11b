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
#include "common.hpp"
#include "jobs.hpp"
#include "launch.hpp"

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

// 16 rows x (16 RB) weight rows per workgroup (SwiGLU: RB/2 row blocks of
// the gate and the same RB/2 of the up matrix).  The four waves split K,
// block by block in turn, so the weights and the activations go from memory
// straight to the registers of the one wave that uses them, with no barrier
// in the K loop; their partial sums meet in LDS at the end, added in wave
// order.
template <typename TC, int EPI, int RB>
__global__ __launch_bounds__(256) void k_fp4_rows16(const GemmArgs a) {
    constexpr int BM = 16, NJ = EPI == EPI_SWIGLU ? RB / 2 : RB, BNO = 16 * NJ;
    static_assert(RB == 4, "four waves reduce the four row blocks");
    __shared__ f32x4 red[4][RB][64];
    Job jb;
    if (!pick_job<BM, BNO>(a, jb)) return;
    const GemmGroup& G = jb.gi ? a.g[1] : a.g[0];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, grp = lane >> 4;
    const int K = G.seg[0].K;

    // activation row of this lane (rows past the tile's repeat its first)
    const int p = jb.row0 + (r16 < jb.rows ? r16 : 0);
    const int64_t arow = G.rowmap ? G.rowmap[p] : p;
    const char* xa = static_cast<const char*>(G.seg[0].A) + arow * G.seg[0].lda * 2;

    int rb[RB];  // this tile's 16-row blocks of the weights, clamped to the matrix
#pragma unroll
    for (int j = 0; j < RB; ++j) rb[j] = min(jb.n0 / 16 + j % NJ, G.N / 16 - 1);
    f32x4 acc[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (jb.gi == 0) {
        const int kb = K / 128;
        const int64_t eb = static_cast<int64_t>(jb.expert) * G.b_estride, es = static_cast<int64_t>(jb.expert) * G.s_estride;
        const char* w[RB];
        const uint8_t* sc[RB];
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            const bool up = EPI == EPI_SWIGLU && j >= NJ;
            w[j] = static_cast<const char*>(up ? G.seg[0].Bu : G.seg[0].B) + eb + static_cast<int64_t>(rb[j]) * kb * 1024 + lane * 16;
            sc[j] = (up ? G.bsu : G.bs) + es + static_cast<int64_t>(rb[j]) * kb * 64 + lane;
        }
        xa += grp * 64;
        for (int k = wid; k < kb; k += 4) {
            uint4 q[RB], x[4];
            uint32_t e[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                q[j] = ldg16_once(w[j] + static_cast<int64_t>(k) * 1024);
                e[j] = sc[j][k * 64];
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) x[s] = ldg16(xa + k * 256 + s * 16);
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                const float scale = __uint_as_float(e[j] << 23);
                const uint32_t c[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                for (int s = 0; s < 4; ++s) acc[j] = Mfma<bf16_t>::run(fp4x8_to_bf16(c[s], scale), x[s], acc[j]);
            }
        }
    } else {
        const int kb = K / 32;
        xa += grp * 16;
        for (int k = wid; k < kb; k += 4) {
            uint4 q[RB];
            const uint4 x = ldg16(xa + k * 64);
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                const void* m = (EPI == EPI_SWIGLU && j >= NJ) ? G.seg[0].Bu : G.seg[0].B;
                q[j] = ldg16_once(static_cast<const char*>(m) + (static_cast<int64_t>(rb[j]) * kb + k) * 1024 + lane * 16);
            }
#pragma unroll
            for (int j = 0; j < RB; ++j) acc[j] = Mfma<bf16_t>::run(q[j], x, acc[j]);
        }
    }

    // accumulator j of a lane: activation row lane % 16, weight rows
    // 4 (lane / 16) .. + 3 of row block j
#pragma unroll
    for (int j = 0; j < RB; ++j) red[wid][j][lane] = acc[j];
    __syncthreads();
    if (wid >= NJ) return;
    auto total = [&](int j) {
        f32x4 v = red[0][j][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
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
    const int col = jb.n0 + wid * 16 + grp * 4;
    if (r16 < jb.rows && col < G.N)
        store4(static_cast<TC*>(G.C) + static_cast<int64_t>(jb.row0 + r16) * G.ldc + col, v);
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

constexpr int kRB = 4;

}  // namespace

int fp4_bm() { return 16; }

hipError_t launch_gemm_fp4(const GemmArgs& args, Epi epi, int max_tiles, int max_n, hipStream_t stream) {
    if (max_tiles <= 0 || max_n <= 0) return hipSuccess;
    if (!fp4_grid_fits(max_tiles, max_n) || args.nsplit != 1 || !args.tiles) return hipErrorInvalidValue;
    const GemmGroup& R = args.g[0];
    if (R.nseg != 1 || R.N % 16 || R.seg[0].K % 128 || !R.bs || (epi == EPI_SWIGLU && !R.bsu)) return hipErrorInvalidValue;
    if (args.g[1].N && (args.g[1].nseg != 1 || args.g[1].N % 16 || args.g[1].seg[0].K % 32)) return hipErrorInvalidValue;
    GemmArgs a = args;
    const int bno = epi == EPI_SWIGLU ? 8 * kRB : 16 * kRB;
    a.ntn = (max_n + bno - 1) / bno;
    const dim3 grid(job_blocks(max_tiles, a.ntn));
    if (epi == EPI_SWIGLU)
        hipLaunchKernelGGL((k_fp4_rows16<bf16_t, EPI_SWIGLU, kRB>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_fp4_rows16<float, EPI_STORE, kRB>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

bool fp4_grid_fits(int64_t max_tiles, int64_t max_n) {
    return max_tiles * ((max_n + 31) / 32) < (int64_t{1} << 31) - 64;
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
