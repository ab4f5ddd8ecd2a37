// Products of few rows with weights in 4 bits and group scales, and the gated
// MLP block of few rows: y = x W^T, h = act(x W0^T) * (x W1^T).
//
// A wave takes 16 weight rows and stretches of K. Per 128 elements of K every
// lane loads 16 bytes of codes (32 elements of one row: lane l has row l % 16,
// part l / 16), converts them to BF16 exactly, and four 16x16x32 matrix
// instructions multiply them with up to 16 rows of x. K's order inside the
// instructions is free as long as both operands agree, so a lane multiplies the
// elements it loaded. The waves of a workgroup share the K of the same weight
// rows; their FP32 sums are added in LDS in a fixed order.
//   mxfp4  the conversion instruction applies the scale 2^(s - 127); what passes
//          BF16 (codes of 2 and more under the bytes 253 and 254) makes the sum
//          infinite or NaN, and such sums are computed again (sum_of_terms);
//   nvfp4  E2M1 times E4M3 is exact in BF16: FP32 product, packed;
//   int4   the code is put into a BF16's upper mantissa bits, 16 + q, and the
//          group's sum is s (sum (16 + q) x - (16 + z) sum x) with the sum of x
//          from the matrix core too, all in FP32: the errors are those of an
//          FP32 sum with weights of up to 31 beside one of 16 + z (24 without
//          zero points, 271 at most). Groups of less than 128 elements would put
//          several groups into one instruction; there the lanes exchange their
//          words first (a 4 x 4 transposition over the wave's four parts), so
//          that an instruction covers 32 consecutive elements.
//
// Bound by the weights' bytes, and for more rows by x, which every workgroup
// reads whole: 7168 x 16384 MXFP4 (62 MB) takes 15.1 us for one row (4.1 TB/s; the
// codes alone, read the same way without a use, take 10.7) and 21.8 us for 16,
// where 224 workgroups read 115 MB of x besides (16.0 us without that). What
// made it so, one row and 16: x loaded from global memory by every wave 27 and
// 51 us (its loads wait behind the codes', which the counter retires in order);
// through LDS, one chunk of K for all waves, 38 and 43 us with scales loaded and
// shifted where they are read (the next loads waited for them); with scales of
// four blocks in one load and nothing between the loads 15 and 22 us. Codes two
// stretches ahead instead of one gain nothing (14.6 and 22.2 us, and short K lose).
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
    int R, N, K, group, groups;     // groups: of a row
    int act;
    uint32_t per_group;   // int4: 2^32 over the group's 32-element blocks, rounded up: exact for K <= 2^20 (0 for one block)
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

// Eight E2M1 codes.
__device__ __forceinline__ void e2m1_values(uint32_t w, f32x2 (&v)[4]) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
}

__device__ __forceinline__ bf16x8 nvfp4_values(uint32_t w, float scale) {
    f32x2 v[4];
    e2m1_values(w, v);
    const u32x4 u = {pack_bf16x2(v[0].x * scale, v[0].y * scale), pack_bf16x2(v[1].x * scale, v[1].y * scale),
                     pack_bf16x2(v[2].x * scale, v[2].y * scale), pack_bf16x2(v[3].x * scale, v[3].y * scale)};
    return __builtin_bit_cast(bf16x8, u);
}

// Four bytes p[at ..] of an array of size > 0 bytes on a 16-byte boundary, still
// to be shifted down by `shift` bits. Those past its end are anything; no aligned
// word is read that holds none of it.
__device__ __forceinline__ uint32_t bytes_at(const uint8_t* p, int64_t at, int64_t size, uint32_t& shift) {
    typedef uint32_t Word __attribute__((aligned(1)));
    const int64_t from = min(at, (size + 3) / 4 * 4 - 4);
    shift = 8 * (uint32_t)(at - from);
    return *reinterpret_cast<const Word*>(p + from);
}

// One sum of the definition, term by term in 64 bits, for those that came out
// infinite or NaN: of factors in BF16, which does not hold MXFP4's largest weights
// (4 * 2^126 and up), of int4's difference of two sums, which infinities and
// values next to FP32's range do not survive, or of nvfp4's sum before its second
// scale. One thread takes it, 0.7 to 0.9 us for 32 elements of K, and a NaN ends
// it: rows of x that are NaN, or memory that nobody wrote, cost 1 us; one infinity
// at the end of 7168 x 16384 costs 570 (int4 760) us.
template <int FORMAT>
__device__ float sum_of_terms(const GemvParams& p, const W4Operand& w, const uint16_t* x, int64_t n) {
    const uint8_t* codes = w.codes + n * (p.K / 2);
    double sum = 0.0;
#pragma unroll 1
    for (int k = 0; k < p.K && sum == sum; k += 32) {
        const u32x4 c = *reinterpret_cast<const u32x4*>(codes + k / 2);
        double scale = 0.0;
        float zero = 8.0f;
        if constexpr (FORMAT == BG_W4_INT4) {
            const int64_t at = n * p.groups + k / p.group;
            scale = bf16_lo(reinterpret_cast<const uint16_t*>(w.scales)[at]);
            if (w.zeros != nullptr) zero = w.zeros[at];
        } else if constexpr (FORMAT == BG_W4_MXFP4) {
            const uint32_t e = w.scales[n * (p.K / 32) + k / 32];
            scale = e == 255u ? __builtin_nan("") : __builtin_bit_cast(double, (uint64_t)(e + (1023 - 127)) << 52);
        }
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const u32x4 xv = *reinterpret_cast<const u32x4*>(x + k + 8 * i);
            f32x2 v[4];
            if constexpr (FORMAT == BG_W4_INT4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = f32x2{(float)(c[i] >> 8 * j & 15u) - zero, (float)(c[i] >> (8 * j + 4) & 15u) - zero};
            } else {
                e2m1_values(c[i], v);
            }
            if constexpr (FORMAT == BG_W4_NVFP4) {
                const f32x2 s = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.scales[n * (p.K / 16) + k / 16 + i / 2], 1.0f, false);
                scale = (double)s.x * w.scale_2;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum = __builtin_fma((double)v[j].x * scale, (double)bf16_lo(xv[j]), sum);
                sum = __builtin_fma((double)v[j].y * scale, (double)bf16_hi(xv[j]), sum);
            }
        }
    }
    return (float)sum;
}

// A workgroup is KW x NW waves: wave (kw, nw) takes 16 weight rows (of both
// matrices where gated) and every KW-th stretch of SPAN elements of K. x goes
// through LDS, one chunk of KW stretches at a time for all waves, double buffered;
// the codes and scales of the next stretch are in flight in registers while one is
// multiplied.
// RP: rows of x that LDS holds (R <= RP, or 16 at a time).
// GB: 32-element blocks of a 128-element block that certainly share a group
// (int4: 1, 2 or 4).
constexpr int SPAN = 4 * BLOCK;

template <int FORMAT, int GB, int RP, int KW, int NW, bool GATED>
__global__ void __launch_bounds__(KW * NW * 64)
gemv_w4_kernel(GemvParams p) {
    constexpr int MATS = GATED ? 2 : 1;
    constexpr bool INT4 = FORMAT == BG_W4_INT4, EXCHANGE = INT4 && GB < 4;
    constexpr int NT = KW * NW * 64, ROWS = 16 * NW;      // weight rows of the workgroup
    constexpr int CHUNK = KW * SPAN, PITCH = CHUNK + 8;        // 16 rows of x: all banks
    constexpr int XREGS = (RP * CHUNK / 8 + NT - 1) / NT;
    constexpr int PAD = 20;                                    // floats between weight rows of the sums
    constexpr int XBYTES = 2 * RP * PITCH * 2, SBYTES = MATS * KW * NW * 16 * PAD * 4;
    // words that hold a block's scales: mxfp4 4 bytes, nvfp4 8, int4 one per group
    constexpr int WORDS = FORMAT == BG_W4_MXFP4 ? 1 : FORMAT == BG_W4_NVFP4 ? 2 : 4 / GB;
    __shared__ __attribute__((aligned(16))) uint8_t lds[XBYTES > SBYTES ? XBYTES : SBYTES];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = wave % KW, nw = wave / KW;
    const int n0 = blockIdx.x * ROWS + nw * 16, r0 = blockIdx.y * 16;
    const int part = lane >> 4;
    const int rows = min(p.R - r0, RP);
    const bool zeros = INT4 && p.w[0].zeros != nullptr;
    const int row = min(n0 + (lane & 15), p.N - 1);

    const int spans = (p.K + SPAN - 1) / SPAN, chunks = (spans + KW - 1) / KW;

    struct Stage {
        u32x4 codes[MATS][4];
        // of block `part` of the stretch, as loaded (nothing may wait for them
        // before the next loads are issued): four bytes and a shift, or s and z
        uint32_t scale[MATS][WORDS], more[MATS][WORDS];
    };
    auto load = [&](Stage& t, int chunk) {
        const int k0 = min(chunk * KW + kw, spans - 1) * SPAN;
#pragma unroll
        for (int s = 0; s < MATS; ++s) {
            const W4Operand& w = p.w[s];
            const int64_t r = row;
            const uint8_t* codes = w.codes + r * (p.K / 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + i * BLOCK + part * 32;
                t.codes[s][i] = *reinterpret_cast<const u32x4*>(codes + (k < p.K ? k / 2 : 0));
            }
            const int k = k0 + part * BLOCK;
            if constexpr (FORMAT == BG_W4_MXFP4) {
                const int64_t per = p.K / 32;
                t.scale[s][0] = bytes_at(w.scales, r * per + (k < p.K ? k / 32 : 0), p.N * per, t.more[s][0]);
            } else if constexpr (FORMAT == BG_W4_NVFP4) {
                const int64_t per = p.K / 16;
                const int64_t from = r * per + (k < p.K ? k / 16 : 0);
                t.scale[s][0] = bytes_at(w.scales, from, p.N * per, t.more[s][0]);
                t.scale[s][WORDS - 1] = bytes_at(w.scales, from + 4, p.N * per, t.more[s][WORDS - 1]);
            } else {
                const int64_t per = p.groups;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    const int ki = k + i * (BLOCK / WORDS);
                    const int64_t at = r * per + (ki < p.K ? (p.per_group ? (int)__umulhi((uint32_t)ki / 32, p.per_group) : ki / 32) : 0);
                    t.scale[s][i] = reinterpret_cast<const uint16_t*>(w.scales)[at];
                    t.more[s][i] = zeros ? w.zeros[at] : 8u;
                }
            }
        }
    };

    // x: zeros past the end of K; int4 in the order of its codes
    u32x4 xr[XREGS];
    auto load_x = [&](int chunk) {
#pragma unroll
        for (int i = 0; i < XREGS; ++i) {
            const int q = tid + i * NT, r = q / (CHUNK / 8), k = chunk * CHUNK + q % (CHUNK / 8) * 8;
            xr[i] = *reinterpret_cast<const u32x4*>(p.x + (int64_t)(r0 + min(r, rows - 1)) * p.K + min(k, p.K - 8));
        }
    };
    auto store_x = [&](int chunk) {
        uint16_t* buf = reinterpret_cast<uint16_t*>(lds) + (chunk & 1) * (RP * PITCH);
#pragma unroll
        for (int i = 0; i < XREGS; ++i) {
            const int q = tid + i * NT, r = q / (CHUNK / 8), c = q % (CHUNK / 8);
            const u32x4 v = chunk * CHUNK + c * 8 < p.K ? xr[i] : u32x4{0u, 0u, 0u, 0u};
            if (r < RP) *reinterpret_cast<u32x4*>(buf + r * PITCH + c * 8) = INT4 ? __builtin_bit_cast(u32x4, x_pairs(v)) : v;
        }
    };

    f32x4 acc[MATS] = {};

    auto multiply = [&](const Stage& t, int chunk) {
        const int k0 = (chunk * KW + kw) * SPAN;
        if (k0 >= p.K) return;
        const uint16_t* buf = reinterpret_cast<const uint16_t*>(lds) + (chunk & 1) * (RP * PITCH) +
                              min(lane & 15, RP - 1) * PITCH + kw * SPAN + (EXCHANGE ? 8 * part : 32 * part);
        // every lane gets the scales of all four blocks
        uint32_t scale[MATS][WORDS][4];
#pragma unroll
        for (int s = 0; s < MATS; ++s)
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    scale[s][w][i] = INT4 ? t.scale[s][w] << 16 | t.more[s][w] : t.scale[s][w] >> (t.more[s][w] & 31);
                exchange(scale[s][w]);
            }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            bf16x8 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = *reinterpret_cast<const bf16x8*>(buf + b * BLOCK + (EXCHANGE ? 32 : 8) * i);
            if constexpr (!INT4) {
                const bool in = k0 + b * BLOCK + part * 32 < p.K;
#pragma unroll
                for (int s = 0; s < MATS; ++s) {
                    if constexpr (FORMAT == BG_W4_MXFP4) {
                        const uint32_t e = in ? scale[s][0][b] >> (8 * part) & 255u : 127u;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[s] = mfma16(x[i], mxfp4_values(t.codes[s][b][i], __builtin_bit_cast(float, e << 23)), acc[s]);
                    } else {
                        const uint32_t e = in ? scale[s][part >> 1 ? WORDS - 1 : 0][b] >> (16 * (part & 1)) : 0u;
                        const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(e, 1.0f, false);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[s] = mfma16(x[i], nvfp4_values(t.codes[s][b][i], i < 2 ? f.x : f.y), acc[s]);
                    }
                }
            } else {
                const u32x4 ones4 = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
                const bf16x8 ones = __builtin_bit_cast(bf16x8, ones4);
                uint32_t codes[MATS][4];
#pragma unroll
                for (int s = 0; s < MATS; ++s) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) codes[s][i] = t.codes[s][b][i];
                    if constexpr (EXCHANGE) exchange(codes[s]);
                }
#pragma unroll
                for (int g = 0; g < 4; g += GB) {
                    f32x4 sum = {}, prod[MATS] = {};
#pragma unroll
                    for (int i = g; i < g + GB; ++i) {
                        sum = mfma16(x[i], ones, sum);
#pragma unroll
                        for (int s = 0; s < MATS; ++s) prod[s] = mfma16(x[i], int4_pairs(codes[s][i]), prod[s]);
                    }
#pragma unroll
                    for (int s = 0; s < MATS; ++s) {
                        // past the end of K the group read is another one, perhaps infinite
                        const uint32_t h = k0 + b * BLOCK + g * 32 < p.K ? scale[s][g / GB][b] : 0u;
                        const float by = bf16_hi(h), off = 16.0f + (float)(h & 0xFFFFu);
#pragma unroll
                        for (int e = 0; e < (RP == 1 ? 1 : 4); ++e)      // row 0 is element 0
                            acc[s][e] = __builtin_fmaf(by, __builtin_fmaf(-off, sum[e], prod[s][e]), acc[s][e]);
                    }
                }
            }
        }
    };

    // Loads have no condition around them: the compiler counts what is in flight.
    if (chunks > 0) {
        Stage a, b;
        load_x(0);
        load(a, 0);
        store_x(0);
        lds_barrier();
        auto turn = [&](const Stage& now, Stage& next, int c) {
            load_x(c + 1);
            load(next, c + 1);
            multiply(now, c);
            store_x(c + 1);
            lds_barrier();
        };
        int c = 0;
        for (; c + 2 < chunks; c += 2) {
            turn(a, b, c);
            turn(b, a, c + 1);
        }
        if (c + 1 < chunks) {
            turn(a, b, c);
            multiply(b, c + 1);
        } else {
            multiply(a, c);
        }
        lds_barrier();
    }

    float* sums = reinterpret_cast<float*>(lds);
    auto at = [&](int s, int w, int n, int r) { return sums + ((s * (KW * NW) + w) * 16 + n) * PAD + r; };
#pragma unroll
    for (int s = 0; s < MATS; ++s) *reinterpret_cast<f32x4*>(at(s, wave, lane & 15, 4 * part)) = acc[s];
    __syncthreads();
    // The sum of output q and matrix m.
    auto sum = [&](int q, int m) {
        const int n = q % ROWS, r = q / ROWS, w0 = n / 16 * KW;      // weight row n: wave n / 16 of N
        float v = *at(m, w0, n & 15, r);
#pragma unroll
        for (int w = 1; w < KW; ++w) v += *at(m, w0 + w, n & 15, r);
        if constexpr (FORMAT == BG_W4_NVFP4) v *= p.w[m].scale_2;
        return v;
    };
    auto store = [&](int q, const float (&v)[MATS]) {
        float out = v[0];
        if constexpr (GATED) out = (p.act == BG_SILU ? gate<BG_SILU>(v[0]) : gate<BG_GELU_TANH>(v[0])) * v[MATS - 1];
        p.y[(int64_t)(r0 + q / ROWS) * p.N + blockIdx.x * ROWS + q % ROWS] = (uint16_t)pack_bf16x2(out, 0.0f);
    };
    auto finite = [](float v) { return __builtin_fabsf(v) < __builtin_inff(); };
    bool again = false;
    for (int q = tid; q < rows * ROWS; q += NT) {
        if (blockIdx.x * ROWS + q % ROWS >= (unsigned)p.N) continue;
        float v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            v[m] = sum(q, m);
            again |= !finite(v[m]);
        }
        store(q, v);
    }
    if (!again) return;
    // Behind the stores, so that a launch without such sums does not fetch the code:
    // 1 x 11008 x 2048 int4 gated 9.3 us, with it before the store 9.4.
    for (int q = tid; q < rows * ROWS; q += NT) {
        const int n = q % ROWS, r = q / ROWS;
        if (blockIdx.x * ROWS + n >= (unsigned)p.N) continue;
        float v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            v[m] = sum(q, m);
            if (!finite(v[m])) v[m] = sum_of_terms<FORMAT>(p, p.w[m], p.x + (int64_t)(r0 + r) * p.K, blockIdx.x * ROWS + n);
        }
        store(q, v);
    }
}

template <int FORMAT, int GB, int RP, int KW, int NW, bool GATED>
hipError_t launch_kernel(const GemvParams& p, hipStream_t stream) {
    constexpr int ROWS = 16 * NW;
    const dim3 grid((unsigned)((p.N + ROWS - 1) / ROWS), (unsigned)((p.R + 15) / 16));
    hipLaunchKernelGGL((gemv_w4_kernel<FORMAT, GB, RP, KW, NW, GATED>), grid, dim3(KW * NW * 64), 0, stream, p);
    return hipGetLastError();
}

// Waves of a workgroup (KW x NW) by the 16-row groups of weights against the
// compute units, the stretches of K, and the rows of x in LDS. Measured us:
//  up to one group per unit, 8 x 1 where K has six stretches or more and 16 rows
//  of x are not held (their chunk would not fit), else 4 x 1. One row, MXFP4:
//  2048 x 11008 6.3 with 8 x 1, 6.8 with 4 x 1, 8.9 with 4 x 2; 512 x 2048 3.7, 3.1,
//  3.6. 16 rows: 4096 x 7168 4 x 1 9.3, 4 x 2 10.2, 2 x 2 9.9.
//  Up to two, 8 x 1 for up to four rows (7168 x 16384, one row, int4: 19.3; 4 x 1
//  20.6, 4 x 2 19.7), 4 x 2 above (8 rows MXFP4 18.5, 4 x 1 21.8, 2 x 2 19.0; 16 rows
//  21.9, 29.2, 22.6): two groups of weight rows then share x.
//  More: 4 x 1 up to four rows (11008 x 2048, one row: 5.3; 8 x 1 7.3, 2 x 2 5.7), 2 x 2
//  above (12287 x 2080, 8 rows: 6.8; 4 x 1 8.5, 4 x 2 7.7; 32000 x 2048, 16 rows: 13.0;
//  4 x 1 25.1, 4 x 2 16.0).
//  Gated, twice the weights in flight: 8 x 1 up to one group per unit (4096 x 11008,
//  one row int4: 15.8; 4 x 1 17.7), and 4 x 1 up to eight rows past it (11008 x 4096, 8
//  rows int4: 19.5; 2 x 2 22.1, 8 x 1 22.8).
template <int FORMAT, int GB, int RP, bool GATED>
hipError_t launch_rows(const GemvParams& p, uint32_t cus, hipStream_t stream) {
    const uint32_t groups = ((uint32_t)p.N + 15) / 16, spans = ((uint32_t)p.K + SPAN - 1) / SPAN;
    if constexpr (RP < 16) {
        if (spans >= 6 && groups <= (RP <= 4 && !GATED ? 2 : 1) * cus)
            return launch_kernel<FORMAT, GB, RP, 8, 1, GATED>(p, stream);
    }
    if (groups <= cus || RP <= 4 || (GATED && RP <= 8)) return launch_kernel<FORMAT, GB, RP, 4, 1, GATED>(p, stream);
    if constexpr (RP > 4 && !(GATED && RP <= 8)) {
        if (groups <= 2 * cus) return launch_kernel<FORMAT, GB, RP, 4, 2, GATED>(p, stream);
        return launch_kernel<FORMAT, GB, RP, 2, 2, GATED>(p, stream);
    }
    return hipErrorInvalidValue;
}

template <int FORMAT, int GB, bool GATED>
hipError_t launch(const GemvParams& p, uint32_t cus, hipStream_t stream) {
    if (p.R == 1) return launch_rows<FORMAT, GB, 1, GATED>(p, cus, stream);
    if (p.R <= 4) return launch_rows<FORMAT, GB, 4, GATED>(p, cus, stream);
    if (p.R <= 8) return launch_rows<FORMAT, GB, 8, GATED>(p, cus, stream);
    return launch_rows<FORMAT, GB, 16, GATED>(p, cus, stream);
}

template <bool GATED>
hipError_t launch_format(const GemvParams& p, int format, uint32_t cus, hipStream_t stream) {
    if (format == BG_W4_MXFP4) return launch<BG_W4_MXFP4, 4, GATED>(p, cus, stream);
    if (format == BG_W4_NVFP4) return launch<BG_W4_NVFP4, 4, GATED>(p, cus, stream);
    if (p.group % 128 == 0) return launch<BG_W4_INT4, 4, GATED>(p, cus, stream);
    if (p.group % 64 == 0) return launch<BG_W4_INT4, 2, GATED>(p, cus, stream);
    return launch<BG_W4_INT4, 1, GATED>(p, cus, stream);
}

}  // namespace

hipError_t launch_gemv_w4(const GemvProblem& q, hipStream_t stream) {
    const uint32_t blocks = q.group / 32;
    const GemvParams p{q.x, {q.w[0], q.w[1]}, q.y, (int)q.R, (int)q.N, (int)q.K, (int)q.group, (int)(q.K / q.group), q.act,
                       blocks > 1 ? (uint32_t)((((uint64_t)1 << 32) + blocks - 1) / blocks) : 0u};
    return q.gated ? launch_format<true>(p, q.format, q.cus, stream) : launch_format<false>(p, q.format, q.cus, stream);
}

}  // namespace bg
