// Products of few rows with weights in 4 bits and group scales, and the gated
// MLP block of few rows: y = x W^T, h = act(x W0^T) * (x W1^T).
//
// A wave takes 16 weight rows and a stretch of K. Per 128 elements of K every
// lane loads 16 bytes of codes (32 elements of one row: lane l has row l % 16,
// part l / 16), converts them to BF16 exactly, and four 16x16x32 matrix
// instructions multiply them with up to 16 rows of x. K's order inside the
// instructions is free as long as both operands agree, so a lane multiplies the
// elements it loaded. The waves of a workgroup share the K of the same weight
// rows; their FP32 sums are added in LDS in a fixed order.
//   mxfp4  the conversion instruction applies the scale 2^(s - 127);
//   nvfp4  E2M1 times E4M3 is exact in BF16: FP32 product, packed;
//   int4   the code is put into a BF16's upper mantissa bits, 16 + q, and the
//          group's sum is s (sum (16 + q) x - (16 + z) sum x) with the sum of x
//          from the matrix core too, all in FP32: the errors are those of an
//          FP32 sum whose weights are at most 31 instead of 15. Groups of less
//          than 128 elements would put several groups into one instruction;
//          there the lanes exchange their words first (a 4 x 4 transposition
//          over the wave's four parts), so that an instruction covers 32
//          consecutive elements.
#include <type_traits>

#include "bg_internal.hpp"
#include "gate.hpp"
#include "mma_common.hpp"

#pragma clang fp contract(off)

namespace bg {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int BLOCK = 128;    // K of a wave's load

struct GemvParams {
    const uint16_t* x;
    W4Operand w[2];
    uint16_t* y;
    int R, N, K, group;
};

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Lane part g, word i -> lane part i, word g.
__device__ __forceinline__ void exchange(uint32_t (&w)[4]) {
    auto swap32 = [](uint32_t& a, uint32_t& b) {
        const auto p = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        a = p[0], b = p[1];
    };
    auto swap16 = [](uint32_t& a, uint32_t& b) {
        const auto p = __builtin_amdgcn_permlane16_swap(a, b, false, false);
        a = p[0], b = p[1];
    };
    swap32(w[0], w[2]);
    swap32(w[1], w[3]);
    swap16(w[0], w[1]);
    swap16(w[2], w[3]);
}

// Eight int4 codes -> 16 + q in BF16, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 int4_pairs(uint32_t w) {
    const u32x4 v = {((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                     ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u};
    return __builtin_bit_cast(bf16x8, v);
}
// Eight elements of x in that order.
__device__ __forceinline__ bf16x8 x_pairs(u32x4 v) {
    const u32x4 p = {__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                     __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
    return __builtin_bit_cast(bf16x8, p);
}

__device__ __forceinline__ bf16x8 mxfp4_values(uint32_t w, float scale) {
    bf16x8 v;
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    const u32x4 u = {__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                     __builtin_bit_cast(uint32_t, d)};
    return __builtin_bit_cast(bf16x8, u);
}

__device__ __forceinline__ bf16x8 nvfp4_values(uint32_t w, float scale) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const u32x4 u = {pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale),
                     pack_bf16x2(c.x * scale, c.y * scale), pack_bf16x2(d.x * scale, d.y * scale)};
    return __builtin_bit_cast(bf16x8, u);
}

// What a lane holds of 128 elements of K of its weight row.
struct Held {
    u32x4 codes;
    uint32_t scale;     // mxfp4: the byte; nvfp4: two bytes; int4: s in the upper half, z in the lower
};

// GB: 32-element blocks of a 128-element load that certainly share a group
// (int4: 1, 2 or 4).
template <int FORMAT, int GB, int WAVES, bool GATED, int ACT>
__global__ void __launch_bounds__(WAVES * 64)
gemv_w4_kernel(GemvParams p) {
    constexpr int SETS = GATED ? 2 : 1, DEEP = GATED ? 2 : 4;
    constexpr bool INT4 = FORMAT == BG_W4_INT4, EXCHANGE = INT4 && GB < 4;
    constexpr int PAD = 20;                     // floats between weight rows: 16 sums, aligned, over all banks
    __shared__ __attribute__((aligned(16))) float sums[SETS][WAVES][16][PAD];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16, r0 = blockIdx.y * 16;
    const int part = lane >> 4;
    const int64_t row = min(n0 + (lane & 15), p.N - 1);
    const uint16_t* x = p.x + (int64_t)min(r0 + (lane & 15), p.R - 1) * p.K;

    const int blocks = (p.K + BLOCK - 1) / BLOCK;
    const int per = (blocks + WAVES - 1) / WAVES;
    const int first = min(wave * per, blocks), last = min(first + per, blocks);

    f32x4 acc[SETS] = {};

    // past the end of K: codes and scales that are finite; x is zero there
    auto load = [&](const W4Operand& w, int b) {
        Held h;
        const int k = b * BLOCK + part * 32;
        const bool in = k < p.K;
        const int kc = in ? k : 0;
        h.codes = *reinterpret_cast<const u32x4*>(w.codes + row * (p.K / 2) + kc / 2);
        if constexpr (FORMAT == BG_W4_MXFP4) {
            const uint32_t s = w.scales[row * (p.K / 32) + kc / 32];
            h.scale = in ? s : 127u;
        } else if constexpr (FORMAT == BG_W4_NVFP4) {
            const uint32_t s = *reinterpret_cast<const uint16_t*>(w.scales + row * (p.K / 16) + kc / 16);
            h.scale = in ? s : 0u;
        } else {
            const int64_t at = row * (p.K / p.group) + kc / p.group;
            const uint32_t s = reinterpret_cast<const uint16_t*>(w.scales)[at];
            const uint32_t z = w.zeros != nullptr ? w.zeros[at] : 8u;
            h.scale = in ? s << 16 | z : 0u;
        }
        return h;
    };

    for (int b0 = first; b0 < last; b0 += DEEP) {
        Held held[DEEP][SETS];
#pragma unroll
        for (int d = 0; d < DEEP; ++d)
#pragma unroll
            for (int s = 0; s < SETS; ++s) held[d][s] = load(p.w[s], min(b0 + d, last - 1));
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const int b = b0 + d;
            if (b >= last) break;
            u32x4 xv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = b * BLOCK + (EXCHANGE ? 32 * i + 8 * part : 32 * part + 8 * i);
                xv[i] = k < p.K ? *reinterpret_cast<const u32x4*>(x + k) : u32x4{0u, 0u, 0u, 0u};
            }
            if constexpr (!INT4) {
#pragma unroll
                for (int s = 0; s < SETS; ++s) {
                    const Held& h = held[d][s];
                    f32x2 e4m3 = {};
                    if constexpr (FORMAT == BG_W4_NVFP4) e4m3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(h.scale, 1.0f, false);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bf16x8 v = FORMAT == BG_W4_MXFP4
                                             ? mxfp4_values(h.codes[i], __builtin_bit_cast(float, h.scale << 23))
                                             : nvfp4_values(h.codes[i], i < 2 ? e4m3.x : e4m3.y);
                        acc[s] = mfma16(__builtin_bit_cast(bf16x8, xv[i]), v, acc[s]);
                    }
                }
            } else {
                const u32x4 ones4 = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
                const bf16x8 ones = __builtin_bit_cast(bf16x8, ones4);
                uint32_t codes[SETS][4], scale[SETS][4];
#pragma unroll
                for (int s = 0; s < SETS; ++s) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) codes[s][i] = held[d][s].codes[i], scale[s][i] = held[d][s].scale;
                    if constexpr (EXCHANGE) {
                        exchange(codes[s]);
                        exchange(scale[s]);
                    }
                }
#pragma unroll
                for (int g = 0; g < 4; g += GB) {
                    f32x4 sum = {}, prod[SETS] = {};
#pragma unroll
                    for (int i = g; i < g + GB; ++i) {
                        const bf16x8 xs = x_pairs(xv[i]);
                        sum = mfma16(xs, ones, sum);
#pragma unroll
                        for (int s = 0; s < SETS; ++s) prod[s] = mfma16(xs, int4_pairs(codes[s][i]), prod[s]);
                    }
#pragma unroll
                    for (int s = 0; s < SETS; ++s) {
                        const float by = bf16_hi(scale[s][g]), off = 16.0f + (float)(scale[s][g] & 0xFFFFu);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[s][e] = __builtin_fmaf(by, __builtin_fmaf(-off, sum[e], prod[s][e]), acc[s][e]);
                    }
                }
            }
        }
    }

#pragma unroll
    for (int s = 0; s < SETS; ++s) *reinterpret_cast<f32x4*>(&sums[s][wave][lane & 15][4 * part]) = acc[s];
    __syncthreads();
    const int n = tid & 15, r = tid >> 4;
    if (tid < 256 && n0 + n < p.N && r0 + r < p.R) {
        float v[SETS];
#pragma unroll
        for (int s = 0; s < SETS; ++s) {
            v[s] = sums[s][0][n][r];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v[s] += sums[s][w][n][r];
            if constexpr (FORMAT == BG_W4_NVFP4) v[s] *= p.w[s].scale_2;
        }
        const float out = GATED ? gate<ACT>(v[0]) * v[SETS - 1] : v[0];
        p.y[(int64_t)(r0 + r) * p.N + n0 + n] = (uint16_t)pack_bf16x2(out, 0.0f);
    }
}

template <int FORMAT, int GB, bool GATED, int ACT>
hipError_t launch(const GemvParams& p, hipStream_t stream) {
    constexpr int WAVES = 8;
    const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)((p.R + 15) / 16));
    hipLaunchKernelGGL((gemv_w4_kernel<FORMAT, GB, WAVES, GATED, ACT>), grid, dim3(WAVES * 64), 0, stream, p);
    return hipGetLastError();
}

template <bool GATED, int ACT>
hipError_t launch_format(const GemvParams& p, int format, hipStream_t stream) {
    if (format == BG_W4_MXFP4) return launch<BG_W4_MXFP4, 4, GATED, ACT>(p, stream);
    if (format == BG_W4_NVFP4) return launch<BG_W4_NVFP4, 4, GATED, ACT>(p, stream);
    if (p.group % 128 == 0) return launch<BG_W4_INT4, 4, GATED, ACT>(p, stream);
    if (p.group % 64 == 0) return launch<BG_W4_INT4, 2, GATED, ACT>(p, stream);
    return launch<BG_W4_INT4, 1, GATED, ACT>(p, stream);
}

}  // namespace

hipError_t launch_gemv_w4(const GemvProblem& q, hipStream_t stream) {
    const GemvParams p{q.x, {q.w[0], q.w[1]}, q.y, (int)q.R, (int)q.N, (int)q.K, (int)q.group};
    if (!q.gated) return launch_format<false, BG_SILU>(p, q.format, stream);
    return q.act == BG_SILU ? launch_format<true, BG_SILU>(p, q.format, stream)
                            : launch_format<true, BG_GELU_TANH>(p, q.format, stream);
}

}  // namespace bg
