// MXFP4 on gfx950: quantisation, reading back, and the dense and grouped
// products on the block-scaled FP4 matrix cores.
//
// Format (OCP Microscaling Formats v1.0): 32 consecutive K elements share one
// E8M0 scale byte s, element = e2m1(code) * 2^(s - 127), s = 255 is NaN.
#include "bg_internal.hpp"
#include "tile_order.hpp"

#pragma clang fp contract(off)

namespace bg {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    bf16x2 v = {(__bf16)lo, (__bf16)hi};   // v_cvt_pk_bf16_f32: round to nearest even
    return __builtin_bit_cast(uint32_t, v);
}

// ---------------------------------------------------------------------------
// Quantisation. Four lanes share a block of 32 elements, eight each: one
// 16-byte load of BF16 (two of FP32), the block's largest magnitude over the
// four lanes by two lane exchanges, four bytes of codes and a quarter of the
// scale byte out. The magnitudes are compared as their bit patterns, which
// order as the values do, with infinities and NaN above every number; the
// scale byte is then the exponent field less 2, and 255 comes out of it for
// infinities and NaN by itself. The elements are multiplied by a power of two
// (exact: a result below the smallest normal number rounds to the zero code
// either way), and rounded by the conversion instruction (nearest, ties to
// even, saturating at 6).
// ---------------------------------------------------------------------------

template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t at, float (&v)[8]) {
    if constexpr (F32) {
        const float* p = static_cast<const float*>(x) + at;
        if constexpr (VEC) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = a[i], v[i + 4] = b[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[i];
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + at;
        if constexpr (VEC) {
            const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __builtin_bit_cast(float, a[i] << 16);
                v[2 * i + 1] = __builtin_bit_cast(float, a[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(float, (uint32_t)p[i] << 16);
        }
    }
}

// Eight elements -> four code bytes; `scale` is the block's byte.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t field = top >> 23;
    scale = field == 255 ? 255u : field < 2 ? 0u : field - 2;
    if (field == 255) return 0;
    const float up = __builtin_bit_cast(float, (254u - scale) << 23);   // 2^(127 - scale)
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * up, v[1] * up, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * up, v[3] * up, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * up, v[5] * up, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * up, v[7] * up, 1.0f, 3);
    return w;
}

// A wave takes 512 elements of a row at a time.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256)
mxfp4_quantize_kernel(MxQuantProblem p, uint32_t segs, uint64_t waves) {
    const int lane = threadIdx.x & 63;
    for (uint64_t w = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < waves; w += (uint64_t)gridDim.x * 4) {
        const uint64_t r = w / segs;
        const uint32_t col = (uint32_t)(w - r * segs) * 512 + lane * 8;
        if (col >= p.K) continue;                 // K % 32 == 0: whole blocks of four lanes
        const int64_t src = p.rows != nullptr ? p.rows[r] : (int64_t)r;
        float v[8] = {};
        if (src >= 0 && src < (int64_t)p.M) load8<F32, VEC>(p.x, src * p.ldx + col, v);
        uint32_t scale;
        const uint32_t word = quantize8(v, scale);
        *reinterpret_cast<uint32_t*>(p.codes + r * (p.K / 2) + col / 2) = word;
        if ((lane & 3) == 0) p.scales[r * (p.K / 32) + col / 32] = (uint8_t)scale;
    }
}

// ---------------------------------------------------------------------------
// Reading back: four code bytes, eight values, per lane and step.
// ---------------------------------------------------------------------------

// 2^(s - 127) as FP32 (s = 0: the subnormal 2^-127; s = 255: NaN).
__device__ __forceinline__ float e8m0(uint32_t s) {
    return __builtin_bit_cast(float, s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

template <bool F32>
__global__ void __launch_bounds__(256)
mxfp4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, void* out, uint64_t units) {
    for (uint64_t u = (uint64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (uint64_t)gridDim.x * 256) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + 4 * u);
        const float s = e8m0(scales[u >> 2]);
        f32x2 v[4];
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        if constexpr (F32) {
            float* o = static_cast<float*>(out) + 8 * u;
            *reinterpret_cast<f32x4*>(o) = f32x4{v[0].x * s, v[0].y * s, v[1].x * s, v[1].y * s};
            *reinterpret_cast<f32x4*>(o + 4) = f32x4{v[2].x * s, v[2].y * s, v[3].x * s, v[3].y * s};
        } else {
            u32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[i].x * s, v[i].y * s);
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + 8 * u) = r;
        }
    }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------

// The rows of one tile: expert e (0 without groups), its first row and how
// many rows from there on are the tile's (none: the tile does not exist).
struct TileRows {
    int e, row0, rows;
};

// Tile `tile` of the experts' row ranges cut into tiles of tm rows, expert by
// expert. Every lane of the wave takes part and gets the same answer. The
// offsets are clamped to 0 .. S and an end before its start counts as empty,
// so no offsets lead outside the operands.
__device__ __forceinline__ TileRows group_tile(const int32_t* offsets, int E, int S, int tm, int tile, int lane) {
    const int per = (E + 63) >> 6;
    const int e0 = min(lane * per, E), e1 = min(e0 + per, E);
    int mine = 0;
    int prev = min(max(offsets[e0], 0), S);
    for (int e = e0; e < e1; ++e) {
        const int next = min(max(offsets[e + 1], 0), S);
        mine += (max(next - prev, 0) + tm - 1) / tm;
        prev = next;
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    const uint64_t past = __ballot(upto > tile);
    if (past == 0) return TileRows{0, 0, 0};
    const int owner = __builtin_ctzll(past);
    int left = tile - (__shfl(upto, owner) - __shfl(mine, owner));
    const int f0 = min(owner * per, E), f1 = min(f0 + per, E);
    prev = min(max(offsets[f0], 0), S);
    for (int e = f0; e < f1; ++e) {
        const int next = min(max(offsets[e + 1], 0), S);
        const int n = max(next - prev, 0), t = (n + tm - 1) / tm;
        if (left < t) return TileRows{e, prev + left * tm, min(tm, n - left * tm)};
        left -= t;
        prev = next;
    }
    return TileRows{0, 0, 0};
}

// The plain form of the product: one wave per 32 x 32 tile, operands straight
// from memory. Lane l of the instruction holds 32 consecutive K elements (one
// block, 16 bytes, and its scale byte) of row l % 32, blocks 2t and 2t + 1 in
// the two halves of the wave.
__global__ void __launch_bounds__(256)
mx_gemm_kernel(MxGemmProblem p, int tiles_n) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tm = blockIdx.x / tiles_n, tn = blockIdx.x % tiles_n;
    TileRows t{0, tm * 32, min(32, (int)p.M - tm * 32)};
    if (p.offsets != nullptr) t = group_tile(p.offsets, (int)p.E, (int)p.M, 32, tm, lane);
    if (t.rows <= 0) return;
    const int n0 = tn * 128 + wave * 32;
    if (n0 >= (int)p.N) return;
    const int blocks = (int)(p.K / 32);
    const int64_t ra = t.row0 + min(lane & 31, t.rows - 1);
    const int64_t rb = (int64_t)t.e * p.N + min(n0 + (lane & 31), (int)p.N - 1);
    const uint8_t *a = p.A + ra * (p.K / 2), *b = p.B + rb * (p.K / 2);
    const uint8_t *sa = p.SFA + ra * blocks, *sb = p.SFB + rb * blocks;
    f32x16 acc = {};
    for (int c = lane >> 5; c - (lane >> 5) < blocks; c += 2) {
        u32x4 wa = {}, wb = {};
        int ea = 127, eb = 127;
        if (c < blocks) {
            wa = *reinterpret_cast<const u32x4*>(a + (int64_t)c * 16);
            wb = *reinterpret_cast<const u32x4*>(b + (int64_t)c * 16);
            ea = sa[c];
            eb = sb[c];
        }
        const i32x8 fa = {(int)wa.x, (int)wa.y, (int)wa.z, (int)wa.w, 0, 0, 0, 0};
        const i32x8 fb = {(int)wb.x, (int)wb.y, (int)wb.z, (int)wb.w, 0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb, fa, acc, 4, 4, 0, eb, 0, ea);
    }
    const int m = lane & 31;
    if (m >= t.rows) return;
    uint16_t* out = p.C + (int64_t)(t.row0 + m) * p.N;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int n = n0 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
        if (n < (int)p.N) out[n] = (uint16_t)pack_bf16x2(acc[v], 0.0f);
    }
}

// Workgroups of a kernel that loops over the rest (a launch holds fewer than 2^32 threads).
uint32_t grid_of(uint64_t groups) { return (uint32_t)(groups < (1u << 20) ? groups : (1u << 20)); }

// A grid of one workgroup of 256 threads per tile.
bool tiles_fit(uint64_t tiles) { return tiles < (1u << 24); }

}  // namespace

hipError_t launch_mxfp4_quantize(const MxQuantProblem& p, hipStream_t stream) {
    const uint32_t segs = (p.K + 511) / 512;
    const uint64_t waves = (uint64_t)p.R * segs;
    const dim3 grid(grid_of((waves + 3) / 4));
    const bool f32 = p.type == BG_F32;
    const bool vec = (uint64_t)p.ldx * (f32 ? 4 : 2) % 16 == 0;
    auto k = f32 ? (vec ? mxfp4_quantize_kernel<true, true> : mxfp4_quantize_kernel<true, false>)
                 : (vec ? mxfp4_quantize_kernel<false, true> : mxfp4_quantize_kernel<false, false>);
    k<<<grid, 256, 0, stream>>>(p, segs, waves);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, void* out, int type, uint32_t M,
                                   uint32_t K, hipStream_t stream) {
    const uint64_t units = (uint64_t)M * (K / 8);
    const dim3 grid(grid_of((units + 255) / 256));
    if (type == BG_F32)
        mxfp4_dequantize_kernel<true><<<grid, 256, 0, stream>>>(codes, scales, out, units);
    else
        mxfp4_dequantize_kernel<false><<<grid, 256, 0, stream>>>(codes, scales, out, units);
    return hipGetLastError();
}

hipError_t launch_gemm_mxfp4(const MxGemmProblem& p, hipStream_t stream) {
    const int tiles_n = (int)((p.N + 127) / 128);
    // every expert may end in a partly filled tile
    const uint64_t tiles_m = p.offsets != nullptr ? p.M / 32 + (p.E < p.M ? p.E : p.M) : (p.M + 31) / 32;
    if (!tiles_fit(tiles_m * tiles_n)) return hipErrorInvalidValue;
    mx_gemm_kernel<<<dim3((uint32_t)(tiles_m * tiles_n)), 256, 0, stream>>>(p, tiles_n);
    return hipGetLastError();
}

}  // namespace bg
