// MXFP4 on gfx950: quantisation, reading back, and the dense and grouped
// products on the block-scaled FP4 matrix cores.
//
// Format (OCP Microscaling Formats v1.0): 32 consecutive K elements share one
// E8M0 scale byte s, element = e2m1(code) * 2^(s - 127), s = 255 is NaN.
#include <type_traits>

#include "bg_internal.hpp"
#include "mx_tiles.hpp"
#include "tile_order.hpp"

#pragma clang fp contract(off)

namespace bg {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
// the same at any address: global memory takes unaligned accesses
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
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
// infinities and NaN by itself. The conversion instruction divides by the
// scale and rounds (nearest, ties to even, saturating at 6), straight from
// BF16 pairs or FP32.
//
// Bound by memory: 5120 x 11008 in 28.1 us from BF16 and 49.5 us from FP32 over
// three inputs in turn (5.1 and 5.2 TB/s; a copy reaches 4.8), 22.8 us with the
// BF16 input still in the last-level cache. 36080 rows of 2048 gathered from
// 4510 take 28.3 us: a token is read, converted and written once per listing.
// With values unpacked and scaled one by one, a 64-bit division per wave and one
// piece per wave the vector units were the limit: 28.9 us (cached input) and
// 35.5 us (gathered); one piece per wave alone 25.0 and 30.7.
// ---------------------------------------------------------------------------

// Eight elements as loaded: FP32 in eight words, BF16 in pairs in four.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t at, uint32_t (&v)[F32 ? 8 : 4]) {
    if constexpr (F32) {
        const uint32_t* p = static_cast<const uint32_t*>(x) + at;
        if constexpr (VEC) {
            const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *reinterpret_cast<const u32x4*>(p + 4);
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
            for (int i = 0; i < 4; ++i) v[i] = a[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
        }
    }
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t w) {     // of the lane's group of four, by permutation
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)w, CTRL, 0xF, 0xF, true);
}

// Eight elements -> four code bytes; `scale` is the block's byte.
template <bool F32>
__device__ __forceinline__ uint32_t quantize8(const uint32_t (&v)[F32 ? 8 : 4], uint32_t& scale) {
    uint32_t top = 0;
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, v[i] & 0x7FFFFFFFu);
    } else {
        u16x2 t = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
        top = (uint32_t)max(t.x, t.y) << 16;
    }
    top = max(top, quad<0xB1>(top));
    top = max(top, quad<0x4E>(top));
    const uint32_t field = top >> 23;
    scale = field == 255 ? 255u : field < 2 ? 0u : field - 2;
    // the conversion divides by a power of two of which it sees the exponent field: 0 is 2^-127
    const float by = __builtin_bit_cast(float, scale << 23);
    uint32_t w = 0;
    if constexpr (F32) {
        auto f = [&](int i) { return __builtin_bit_cast(float, v[i]); };
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(0), f(1), by, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(2), f(3), by, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(4), f(5), by, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(6), f(7), by, 3);
    } else {
        auto f = [&](int i) { return __builtin_bit_cast(bf16x2, v[i]); };
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, f(0), by, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, f(1), by, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, f(2), by, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, f(3), by, 3);
    }
    return field == 255 ? 0u : w;
}

// A wave takes two pieces of 512 elements at a time, their loads in flight
// together; per_seg is 2^32 / segs rounded up, for the division (2^32 - 1 where
// segs is 1).
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256)
mxfp4_quantize_kernel(MxQuantProblem p, uint32_t segs, uint32_t per_seg, uint32_t waves) {
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int U = 2, N = F32 ? 8 : 4;
    for (uint64_t w0 = ((uint64_t)blockIdx.x * 4 + wave) * U; w0 < waves; w0 += (uint64_t)gridDim.x * 4 * U) {
        uint32_t v[U][N] = {}, r[U], col[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w = (uint32_t)min(w0 + u, (uint64_t)waves - 1);
            uint32_t q = (uint32_t)(((uint64_t)w * per_seg) >> 32);      // off by one at most
            if ((uint64_t)q * segs > w) --q;
            else if (w - q * segs >= segs) ++q;
            r[u] = q;
            col[u] = (w - q * segs) * 512 + lane * 8;
            in[u] = w0 + u < waves && col[u] < p.K;       // K % 32 == 0: whole blocks of four lanes
        }
        int64_t src[U];
#pragma unroll
        for (int u = 0; u < U; ++u) src[u] = p.rows != nullptr ? p.rows[r[u]] : (int64_t)r[u];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (in[u] && src[u] >= 0 && src[u] < (int64_t)p.M) load8<F32, VEC>(p.x, src[u] * p.ldx + col[u], v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t scale;
            const uint32_t word = quantize8<F32>(v[u], scale);
            if (!in[u]) continue;
            *reinterpret_cast<uint32_t*>(p.codes + (uint64_t)r[u] * (p.K / 2) + col[u] / 2) = word;
            if ((lane & 3) == 0) p.scales[(uint64_t)r[u] * (p.K / 32) + col[u] / 32] = (uint8_t)scale;
        }
    }
}

// ---------------------------------------------------------------------------
// Reading back: four code bytes, eight values, per lane and step; 5120 x 11008
// to BF16 in 21.8 us (6.5 TB/s), to FP32 in 44.6 us (5.7 TB/s): the writes.
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

// The experts' row ranges cut into tiles of tm rows, expert by expert; the
// tile of this workgroup's turn j on XCD x. Every XCD takes one contiguous
// stretch of the tiles that exist, so the tiles of an expert meet its weights
// in one L2. Every lane of the wave takes part and gets the same answer. The
// offsets are clamped to 0 .. S and an end before its start counts as empty,
// so no offsets lead outside the operands.
__device__ __forceinline__ TileRows group_tile(const int32_t* offsets, int E, int S, int tm, int x, int j, int lane) {
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
    const int stretch = (__shfl(upto, 63) + 7) >> 3, tile = x * stretch + j;
    const uint64_t past = __ballot(upto > tile);
    if (past == 0 || j >= stretch) return TileRows{0, 0, 0};
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

// Workgroups of a kernel that loops over the rest (a launch holds fewer than 2^32 threads).
uint32_t grid_of(uint64_t groups) { return (uint32_t)(groups < (1u << 20) ? groups : (1u << 20)); }

// Compile-time loops over a constant's values.
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (N > 0) {
        static_for<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A barrier that orders LDS only: a full fence would also wait for the direct
// loads in flight, which are counted by hand.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A pointer every lane holds the same value of, in scalar registers.
__device__ __forceinline__ void* uniform_ptr(const void* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
}

// Buffer resource from a row on: loads take a scalar and a 32-bit vector offset.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(p), (short)0, 0xFFFFFFFF, 0x00020000);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)((__attribute__((address_space(3))) const uint8_t*)p);
}

// Scheduling of one part of a step: NM matrix instructions, each followed by
// an LDS read while the NR reads last.
template <int NM, int NR>
__device__ __forceinline__ void interleave() {
    constexpr int R = (NR + NM - 1) / NM;
#pragma unroll
    for (int q = 0; q < NM; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (q * R < NR) __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    }
}

constexpr int STEP = 8;                         // blocks per K step: 128 bytes of every row, one cache line

// Swizzled 16-byte slot of block c in row `row` of a staged tile of eight
// blocks a row: the rows that the lanes of one 16-byte LDS read touch spread
// over all banks. An involution in c.
__device__ __forceinline__ int block_slot(int row, int c) { return c ^ ((row ^ (row >> 3)) & 7); }

// Direct global -> LDS staging of ROWS rows' codes, 128 bytes a row and step,
// shared out over NW waves. One instruction moves 64 x 16 bytes, eight rows,
// into one contiguous KB of LDS. Rows past the last are clamped to it. Where a
// wave has a surplus instruction it loads the last stretch again, so every
// wave issues the same number.
// The loads are inline assembly: the compiler's wait insertion cannot tell the
// stages apart and would wait for them at every LDS read. Their completion is
// tracked with s_waitcnt vmcnt before the barrier that precedes their first use.
template <int ROWS, int NW>
struct MxStager {
    static constexpr int SEGS = ROWS / 8, PER = (SEGS + NW - 1) / NW;
    uint32_t off[PER];   // byte offsets from the tile's first row at step 0
    uint32_t end;        // offset of the operand's last block
    __amdgpu_buffer_rsrc_t rsrc;

    __device__ __forceinline__ static int seg(int wave, int j) { return min(wave + j * NW, SEGS - 1); }
    // the block a lane fetches of its row: it lands in slot lane % 8
    __device__ __forceinline__ static int block(int wave, int j, int lane) {
        return block_slot(seg(wave, j) * 8 + lane / 8, lane % 8);
    }

    // data: the tile's first row; last: the last row that exists, and left: the
    // bytes of the operand, from there on
    __device__ __forceinline__ void init(const uint8_t* data, int last, int64_t left, uint32_t blocks, int wave, int lane) {
        rsrc = resource(data);
        end = (uint32_t)min(left - 16, (int64_t)0xFFFFFFF0);
#pragma unroll
        for (int j = 0; j < PER; ++j)
            off[j] = (uint32_t)min(seg(wave, j) * 8 + lane / 8, last) * (blocks * 16) +
                     (uint32_t)block(wave, j, lane) * 16;
    }

    // The codes of the step that starts at block c0. If the step reaches past
    // the rows' end (RAGGED may), what is fetched there is the next row's, or
    // the operand's last block again; it is multiplied with zeros.
    template <bool RAGGED>
    __device__ __forceinline__ void issue(uint32_t c0, uint8_t* lds, int wave) const {
        const uint32_t s = c0 * 16;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t v = RAGGED ? min(off[j] + s, end) : off[j], c = RAGGED ? 0 : s;
            asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(v), "s"(rsrc), "s"(c),
                         "{m0}"(lds_addr(lds) + seg(wave, j) * 1024));
        }
    }
};

// How the scales of a tile's rows come to LDS, by K alone:
enum ScalePath : int {
    WHOLE = 0,     // K % 256 == 0, at least a group of steps: rows four-byte aligned
    SHIFTED = 1,   // any other K >= 512: rows start at any byte
    SHORT = 2,     // K < 512
};
template <int Q>
constexpr ScalePath scale_path(uint32_t K) {
    return K < 512 ? SHORT : K % (STEP * 32) == 0 && K >= Q * STEP * 32 ? WHOLE : SHIFTED;
}

// Scales of the BM rows of A and the BN rows of B of a tile, a group of Q steps
// (two or four) at a time as [row][GROUP] bytes in LDS, by direct loads of 16
// bytes a lane. A step's 8 bytes of scales touch a cache line, as many as its
// 128 bytes of codes; groups cut the lines a row and step touches from 2 to 1.5
// (pairs) or 1.25 (fours), and that made every tile faster that kept its stages:
// 64 x 64 tiles, 128 x 7168 x 16384, 27 us step by step, 20.8 in pairs, 19.2 in
// fours; 128 x 128 tiles, 4096 x 4096 x 8192, 88.8 us in pairs and 82.4 in
// fours; the experts' tiles of 32 x 128, 16 x 8 of 256 of 2048 x 2048, 41.0 and
// 39.7. Fours stay out where their buffers cost a stage or a second workgroup
// (256 x 128 tiles 78.9 us in pairs with three stages, 80.0 in fours with two),
// registers (256 x 256: 72.5 and 76.2) or, with 32 x 64, nothing is gained.
// A last group that ends past the row starts earlier, so that it ends with it.
// SHIFTED (pairs): the loads start at the four-byte word that holds a row's
// first scale, and one more word a row ([row][4] behind the others) holds the
// up to three scales that the shift pushes out; a lane joins its four out of
// two words. (The same through registers and LDS writes: 4096 x 4096 x 8224 in
// 92 us.) The last word may reach up to three bytes past the last scale of the
// whole operand: never past the word that holds it.
// SHORT: through registers, a step at a time, zero past the row's end.
template <int BM, int BN, int NW, int PATH, int Q>
struct ScaleStager {
    static constexpr int GROUP = Q * STEP, LANES = GROUP / 16, RPL = 64 / LANES;     // lanes per row, rows per load
    // a load's rows belong to one operand: fewer rows of A take one of their own
    static constexpr int PAD = BM < RPL ? RPL : BM;
    static constexpr int SEGS = (PAD + BN) / RPL, SPER = (SEGS + NW - 1) / NW;
    static constexpr int PER = PATH == WHOLE ? SPER : PATH == SHIFTED ? 2 * SPER : 0;
    static_assert(PAD % RPL == 0 && BN % RPL == 0, "whole loads");
    static_assert(LANES == 1 || (LANES == 2 && PATH == WHOLE), "pairs, or fours of whole steps");
    static constexpr int REST = (PAD + BN) * GROUP;                // where the fifth words start
    static constexpr int BYTES = REST + (PATH == SHIFTED ? (PAD + BN) * 4 : 0);
    static constexpr int WORDS = (BM + BN) * 2, WPER = (WORDS + NW * 64 - 1) / (NW * 64);
    uint32_t off[PATH == SHORT ? WPER : SPER], lim[SPER];
    uint32_t reg[PATH == SHORT ? WPER : 1];
    __amdgpu_buffer_rsrc_t rsrc[PATH == SHORT ? 1 : SPER];
    const uint8_t *sa, *sb;

    __device__ __forceinline__ static int seg(int wave, int j) { return min(wave + j * NW, SEGS - 1); }

    // a, b: the tile's first rows; last_*: the last row that exists, from
    // there on; left_*: bytes of the operand from there on
    __device__ __forceinline__ void init(const uint8_t* a, const uint8_t* b, int last_a, int last_b, int64_t left_a,
                                         int64_t left_b, uint32_t blocks, int wave, int lane) {
        if constexpr (PATH != SHORT) {
#pragma unroll
            for (int j = 0; j < SPER; ++j) {
                const int r = seg(wave, j) * RPL, at = lane / LANES;
                const bool is_a = r < PAD;
                const uint8_t* first = is_a ? a : b;
                const uint32_t odd = PATH == SHIFTED ? (uint32_t)(reinterpret_cast<uintptr_t>(first) & 3) : 0;
                rsrc[j] = resource(first - odd);
                off[j] = odd + (uint32_t)(is_a ? min(r + at, last_a) : min(r - PAD + at, last_b)) * blocks + lane % LANES * 16;
                // offset of the word that holds the operand's last scale
                lim[j] = (uint32_t)min(odd + (is_a ? left_a : left_b) - 1, (int64_t)0x7FFFFFFF) & ~3u;
            }
        } else {
            sa = a;
            sb = b;
#pragma unroll
            for (int j = 0; j < WPER; ++j) {
                const int r = min((j * NW + wave) * 64 + lane, WORDS - 1) / 2;
                off[j] = (uint32_t)(r < BM ? min(r, last_a) : min(r - BM, last_b)) * blocks;
            }
        }
    }
    // first block of the group that a step's scales are staged with
    __device__ __forceinline__ static uint32_t group_start(int step, uint32_t blocks) {
        const uint32_t c = (uint32_t)step / Q * GROUP;
        return PATH == SHORT ? c : min(c, blocks - GROUP);
    }
    __device__ __forceinline__ void issue(uint32_t c0, uint8_t* lds, int wave) const {
        const uint32_t c = PATH == SHIFTED ? c0 & ~3u : c0;
#pragma unroll
        for (int j = 0; j < (PATH == SHORT ? 0 : SPER); ++j) {
            const uint32_t v = PATH == SHIFTED ? (off[j] + (c0 & 3)) & ~3u : off[j];
            asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(v), "s"(rsrc[j]), "s"(c),
                         "{m0}"(lds_addr(lds) + seg(wave, j) * 1024));
            if constexpr (PATH == SHIFTED)
                asm volatile("buffer_load_dword %0, %1, %2 offen lds" ::"v"(min(v + 16, lim[j] - c)), "s"(rsrc[j]), "s"(c),
                             "{m0}"(lds_addr(lds) + REST + seg(wave, j) * 256));
        }
    }
    // SHORT: the word of a step's scales that starts at the lane's block, or
    // the row's last whole word where that is past it; nothing waits for the load
    __device__ __forceinline__ static uint32_t word_block(int step, int w) { return (uint32_t)(step * STEP + (w & 1) * 4); }
    __device__ __forceinline__ void fetch(int step, uint32_t blocks, int wave, int lane) {
#pragma unroll
        for (int j = 0; j < WPER; ++j) {
            const int w = min((j * NW + wave) * 64 + lane, WORDS - 1);
            const uint8_t* q = (w / 2 < BM ? sa : sb) + off[j];
            if (blocks >= 4) {
                reg[j] = *reinterpret_cast<const u32_any*>(q + min(word_block(step, w), blocks - 4));
            } else {
                reg[j] = 0;
                for (uint32_t b = 0; b < blocks; ++b) reg[j] |= (uint32_t)q[b] << (8 * b);
            }
        }
    }
    __device__ __forceinline__ void store(int step, uint32_t blocks, uint8_t* lds, int wave, int lane) const {
#pragma unroll
        for (int j = 0; j < WPER; ++j) {
            const int w = min((j * NW + wave) * 64 + lane, WORDS - 1);
            const uint32_t c = word_block(step, w), past = c - min(c, max(blocks, 4u) - 4);
            const int row = w / 2 + (w / 2 < BM ? 0 : PAD - BM);
            *reinterpret_cast<uint32_t*>(lds + row * GROUP + step % Q * STEP + (w & 1) * 4) =
                past < 4 ? reg[j] >> (8 * past) : 0u;
        }
    }
    // Into v: the four scales from byte `at` of a group on (the step's part of
    // it and the lane's half) of the N rows row, row + 32, ..., whose first
    // scale lies `odd` bytes into its word.
    template <int N>
    __device__ __forceinline__ static void read(const uint8_t* lds, int row, uint32_t at, uint32_t odd, int (&v)[N]) {
        if constexpr (PATH != SHIFTED) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const int*>(lds + row * GROUP + at + 32 * GROUP * i);
        } else {
            const uint32_t o = at + odd, w = o >> 2;
            const bool l4 = w < 4, h4 = w < 3;
            const uint8_t* lo = lds + (l4 ? row * GROUP + w * 4 : REST + row * 4);
            const uint8_t* hi = lds + (h4 ? row * GROUP + w * 4 + 4 : REST + row * 4);
            const int ls = l4 ? 32 * GROUP : 128, hs = h4 ? 32 * GROUP : 128;
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = (int)__builtin_amdgcn_alignbyte(*reinterpret_cast<const uint32_t*>(hi + hs * i),
                                                       *reinterpret_cast<const uint32_t*>(lo + ls * i), o & 3);
        }
    }
};

// Tile kernel. A workgroup of WM x WN waves owns a BM x BN tile of C and walks
// K in steps of 256 elements, four matrix instructions deep: lane l of
// instruction s holds block 4 (l / 32) + s of row l % 32 (the order of K inside
// a product is free as long as A and B agree), so the four scale bytes a lane
// needs for a step are one aligned word, and the instruction picks byte s of
// it: no vector instruction touches codes or scales between LDS and the matrix
// cores. The steps' codes go through a ring of STAGES buffers in LDS, the
// scales through buffers of a group of Q steps, filled by direct loads.
// Where K ends inside a step, A's blocks past the end and all scales there
// become zero in registers.
// The matrix instruction takes B first, so a lane ends up with four
// consecutive columns of one row of C.
//
// Medians of a kernel trace: 4096 x 4096 x 8192 in 72.6 us (3.8 PFLOP/s; on
// another card 82.8), 5120 x 11008 x 2048 in 80.2 us (2.9; 88.8), 1015 x 12288 x
// 2048 / 2080 in 22.1 / 29.8 us, 128 x 7168 x 16384 in 21.4 us (18.0 without a
// trace), 16 x 8 of 256 experts of 2048 x 2048 in 37.1 us (the weights at 5 TB/s).
// What bounds them, as far as it is known. Power takes a fifth of the large
// ones: on zeros the same launches take 55.8 instead of 69.6 us and 65.3 instead
// of 83.1 us, and the clock, at 2.4 GHz on short kernels, falls to 1.8 .. 2.1 GHz;
// the matrix cores are busy in 42% and 32% of the cycles. For 128 x 7168 x 16384
// (11% of the cycles) the cause is not known: its time is the same on zeros, a
// step's for rows of 8192 and 8320 bytes (318 and 319 ns), and its time with
// eight stages instead of four or half the LDS reads (each wave one of a step's
// instructions for the whole tile: 21.0 against 20.7 us); fewer lines of scales
// are all that made it faster. Rows that start inside a cache line touch two
// lines a step: the 29.8 us above.
template <int BM, int BN, int WM, int WN, int STAGES, bool GROUPED, int PATH, int Q>
__global__ void __launch_bounds__(WM * WN * 64)
mx_tile_kernel(MxGemmProblem p, int tiles_m, int tiles_n) {
    constexpr int NW = WM * WN;
    constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
    static_assert(FM * 32 * WM == BM && FN * 32 * WN == BN, "whole instructions per wave");
    // A group of scales is loaded with the codes of its first step, STAGES steps
    // ahead, and read last with those of its last: so many groups are there at once.
    constexpr int GROUPS = (STAGES + Q - 2) / Q + 1;
    constexpr int STAGE = (BM + BN) * 128, SCALES = ScaleStager<BM, BN, NW, PATH, Q>::BYTES;
    constexpr int RING = STAGES * STAGE + GROUPS * SCALES, OUT = BM * BN * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > OUT ? RING : OUT];
    uint8_t* const scale_mem = smem + STAGES * STAGE;
    using StA = MxStager<BM, NW>;
    using StB = MxStager<BN, NW>;
    using StS = ScaleStager<BM, BN, NW, PATH, Q>;
    // loads a wave has in flight, at least, when only those of the STAGES - 1
    // or STAGES - 2 youngest steps are
    constexpr int L = StA::PER + StB::PER;
    constexpr int AHEAD1 = (STAGES - 1) * L + (STAGES - 1) / Q * StS::PER;
    constexpr int AHEAD2 = (STAGES - 2) * L + (STAGES - 2) / Q * StS::PER;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    TileRows t;
    if constexpr (GROUPED) {
        const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
        tm = 0;
        tn = j % tiles_n;
        t = group_tile(p.offsets, (int)p.E, (int)p.M, BM, x, j / tiles_n, lane);
        t.e = __builtin_amdgcn_readfirstlane(t.e);
        t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
        t.rows = __builtin_amdgcn_readfirstlane(t.rows);
        if (t.rows <= 0) return;
    } else {
        tile_of<ORDER_GEMM>((int)blockIdx.x, tiles_m, tiles_n, tm, tn);
        t = TileRows{0, tm * BM, min(BM, (int)p.M - tm * BM)};
    }
    const int n0 = tn * BN;
    const uint32_t blocks = p.K / 32;
    const int nsteps = (int)((blocks + STEP - 1) / STEP);
    const int64_t rb = (int64_t)t.e * p.N + n0;
    const int last_a = t.rows - 1, last_b = min(BN, (int)p.N - n0) - 1;

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};

    if (nsteps > 0) {
        StA sa;
        StB sb;
        StS ss;
        const int64_t rows_a = (int64_t)p.M - t.row0, rows_b = (int64_t)p.E * p.N - rb;     // of the operands, from here on
        sa.init(p.A + (int64_t)t.row0 * blocks * 16, last_a, rows_a * blocks * 16, blocks, wave, lane);
        sb.init(p.B + rb * blocks * 16, last_b, rows_b * blocks * 16, blocks, wave, lane);
        const uint8_t *scales_a = p.SFA + (int64_t)t.row0 * blocks, *scales_b = p.SFB + rb * blocks;
        ss.init(scales_a, scales_b, last_a, last_b, rows_a * blocks, rows_b * blocks, blocks, wave, lane);

        // a stage: A's codes, B's codes; before those of a group's first step, its scales
        auto group_mem = [&](int step) { return scale_mem + (uint32_t)step / Q % GROUPS * SCALES; };
        auto issue = [&](int step, uint8_t* st) {
            const int s = min(step, nsteps - 1);       // past the end: the last one again
            if constexpr (PATH != SHORT)
                if (step % Q == 0) ss.issue(StS::group_start(s, blocks), group_mem(step), wave);
            sa.template issue<PATH != WHOLE>((uint32_t)s * STEP, st, wave);
            sb.template issue<PATH != WHOLE>((uint32_t)s * STEP, st + BM * 128, wave);
        };
        auto fetch = [&](int step) {
            if constexpr (PATH == SHORT) ss.fetch(step, blocks, wave, lane);
        };
        auto store = [&](int step) {
            if constexpr (PATH == SHORT) ss.store(step, blocks, group_mem(step), wave, lane);
        };
        // Fragment addresses: block 4h + s of row 32 i + l % 32 of the wave's
        // rows; every second fragment's swizzle differs in bit 2 (64 bytes).
        const int row = lane & 31, h = lane >> 5;
        uint32_t va[4], vb[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            va[s] = (uint32_t)((wm * TM + row) * 128 + block_slot(wm * TM + row, 4 * h + s) * 16);
            vb[s] = (uint32_t)((BM + wn * TN + row) * 128 + block_slot(wn * TN + row, 4 * h + s) * 16);
        }
        auto frags = [&](const uint8_t* st, int s, u32x4 (&a)[FM], u32x4 (&b)[FN]) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
                a[i] = *reinterpret_cast<const u32x4*>(st + (va[s] ^ (64u * (i & 1))) + 4096 * i);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[j] = *reinterpret_cast<const u32x4*>(st + (vb[s] ^ (64u * (j & 1))) + 4096 * j);
        };
        // rows 32 apart start at the same byte of a word
        const uint32_t odd_a = (uint32_t)reinterpret_cast<uintptr_t>(scales_a) + (uint32_t)(wm * TM + row) * blocks;
        const uint32_t odd_b = (uint32_t)reinterpret_cast<uintptr_t>(scales_b) + (uint32_t)(wn * TN + row) * blocks;
        auto exps = [&](int step, int (&a)[FM], int (&b)[FN]) {
            const uint8_t* q = group_mem(step);
            const uint32_t ps = StS::group_start(step, blocks), at = (uint32_t)step * STEP - ps + 4 * h;
            StS::read(q, wm * TM + row, at, (odd_a + ps) & 3, a);
            StS::read(q, StS::PAD + wn * TN + row, at, (odd_b + ps) & 3, b);
            if constexpr (PATH == SHIFTED) {
                // past the row's end: zero
                const int left = (int)blocks - step * STEP - 4 * h;
                const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : ~0u >> (32 - 8 * left);
#pragma unroll
                for (int i = 0; i < FM; ++i) a[i] &= (int)keep;
#pragma unroll
                for (int j = 0; j < FN; ++j) b[j] &= (int)keep;
            }
        };
        // A's block s of the last step: zero past the row's end
        auto cut = [&](int s, u32x4 (&a)[FM]) {
            if constexpr (PATH != WHOLE) {
                const uint32_t keep = 4 * h + s < (int)(blocks - (uint32_t)(nsteps - 1) * STEP) ? ~0u : 0u;
#pragma unroll
                for (int i = 0; i < FM; ++i) a[i] &= u32x4{keep, keep, keep, keep};
            }
        };
        auto mfma = [&](auto sc, const u32x4 (&a)[FM], const u32x4 (&b)[FN], const int (&xa)[FM], const int (&xb)[FN]) {
            constexpr int s = decltype(sc)::value;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const i32x8 A = {(int)a[i].x, (int)a[i].y, (int)a[i].z, (int)a[i].w, 0, 0, 0, 0};
                    const i32x8 B = {(int)b[j].x, (int)b[j].y, (int)b[j].z, (int)b[j].w, 0, 0, 0, 0};
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(B, A, acc[i][j], 4, 4, s, xb[j], s, xa[i]);
                }
        };

        fetch(0);
        issue(0, smem);
        store(0);
#pragma unroll
        for (int st = 1; st < STAGES; ++st) issue(st, smem + st * STAGE);
        wait_vmcnt<AHEAD1>();
        lds_barrier();
        fetch(1);

        // the next step's stage, landed for every wave; this step's is free and refilled
        int cur = 0;
        auto advance = [&](int k) {
            uint8_t* st = smem + cur * STAGE;
            cur = cur + 1 == STAGES ? 0 : cur + 1;
            uint8_t* sn = smem + cur * STAGE;
            wait_vmcnt<AHEAD2>();                  // step k + 1 has landed for this wave ...
            store(k + 1);
            lds_barrier();                         // ... and for all, and all have read step k
            __builtin_amdgcn_sched_barrier(0);
            issue(k + STAGES, st);
            fetch(k + 2);
            return sn;
        };
        if constexpr (FM * FN <= 4) {
            // Small wave tiles: an instruction's worth of products is shorter
            // than an LDS read takes, so a whole step's fragments are read
            // while the step before is multiplied.
            u32x4 fa[2][4][FM], fb[2][4][FN];
            int ea[2][FM], eb[2][FN];
            auto read = [&](int k, const uint8_t* st, auto q) {
                constexpr int B = decltype(q)::value;
                exps(k, ea[B], eb[B]);
#pragma unroll
                for (int s = 0; s < 4; ++s) frags(st, s, fa[B][s], fb[B][s]);
            };
            auto last = [&](auto q) {
                constexpr int B = decltype(q)::value;
                static_for<4>([&](auto s) { cut(decltype(s)::value, fa[B][decltype(s)::value]); });
            };
            auto multiply = [&](auto q) {
                constexpr int B = decltype(q)::value;
                static_for<4>([&](auto s) { mfma(s, fa[B][decltype(s)::value], fb[B][decltype(s)::value], ea[B], eb[B]); });
            };
            constexpr std::integral_constant<int, 0> EVEN{};
            constexpr std::integral_constant<int, 1> ODD{};
            read(0, smem, EVEN);
            auto step = [&](int k, auto q, auto other) {
                const uint8_t* sn = advance(k);
                read(k + 1, sn, other);
                multiply(q);
                __builtin_amdgcn_sched_barrier(0);
            };
            int k = 0;
            for (; k + 2 < nsteps; k += 2) {
                step(k, EVEN, ODD);
                step(k + 1, ODD, EVEN);
            }
            if (k + 1 < nsteps) {
                step(k, EVEN, ODD);
                last(ODD);
                multiply(ODD);
            } else {
                last(EVEN);
                multiply(EVEN);
            }
        } else {
            // Instruction s of a step multiplies what was read during s - 1.
            // The barrier that retires a step comes before its last
            // instructions, whose operands are in registers, so the matrix
            // cores have work while the freed stage is refilled and the next
            // one's first fragments are read.
            u32x4 fa[2][FM], fb[2][FN];
            int ea[FM], eb[FN];
            frags(smem, 0, fa[0], fb[0]);
            exps(0, ea, eb);
            auto leading = [&](const uint8_t* st, auto last) {
                static_for<3>([&](auto s) {
                    constexpr int S = decltype(s)::value;
                    frags(st, S + 1, fa[(S + 1) & 1], fb[(S + 1) & 1]);
                    if constexpr (decltype(last)::value) cut(S, fa[S & 1]);
                    mfma(s, fa[S & 1], fb[S & 1], ea, eb);
                    interleave<FM * FN, FM + FN>();
                    __builtin_amdgcn_sched_barrier(0);
                });
            };
            for (int k = 0; k + 1 < nsteps; ++k) {
                leading(smem + cur * STAGE, std::false_type{});
                const uint8_t* sn = advance(k);
                int xa[FM], xb[FN];
                frags(sn, 0, fa[0], fb[0]);
                exps(k + 1, xa, xb);
                mfma(std::integral_constant<int, 3>{}, fa[1], fb[1], ea, eb);
                interleave<FM * FN, 2 * (FM + FN)>();
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < FM; ++i) ea[i] = xa[i];
#pragma unroll
                for (int j = 0; j < FN; ++j) eb[j] = xb[j];
            }
            leading(smem + cur * STAGE, std::true_type{});
            cut(3, fa[1]);
            mfma(std::integral_constant<int, 3>{}, fa[1], fb[1], ea, eb);
        }
        wait_vmcnt<0>();       // what was loaded past the end lands before LDS is used again
    }

    // Epilogue: each wave turns its own part of the tile through LDS, so that
    // rows leave in 16-byte pieces. Pieces rotate by row over the row's slots.
    lds_barrier();
    constexpr int OUTB = TN * 2, SLOTS = OUTB / 16;
    uint8_t* mine = smem + wave * (TM * OUTB);
    auto slot = [](int row, int c) { return row * OUTB + ((c + row) % SLOTS) * 16; };
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int r = i * 32 + (lane & 31), n = j * 32 + g * 8 + (lane >> 5) * 4;
                *reinterpret_cast<u32x2*>(mine + slot(r, n >> 3) + (lane >> 5) * 8) =
                    u32x2{pack_bf16x2(acc[i][j][4 * g], acc[i][j][4 * g + 1]),
                          pack_bf16x2(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3])};
            }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const bool vec = p.N % 8 == 0;
    constexpr int RPI = 64 / SLOTS;            // rows per store instruction
#pragma unroll 4
    for (int r0 = 0; r0 < TM; r0 += RPI) {
        const int r = r0 + lane / SLOTS, c = lane % SLOTS;
        const int m = wm * TM + r, n = n0 + wn * TN + c * 8;
        if (m >= t.rows || n >= (int)p.N) continue;
        const u32x4 w = *reinterpret_cast<const u32x4*>(mine + slot(r, c));
        uint16_t* out = p.C + (int64_t)(t.row0 + m) * p.N + n;
        if (n + 8 <= (int)p.N) {
            if (vec)
                __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(out));
            else
                *reinterpret_cast<u32x4_any*>(out) = w;
        } else {
            const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
            for (int e = 0; e < 8 && n + e < (int)p.N; ++e) out[e] = (uint16_t)(w4[e >> 1] >> ((e & 1) * 16));
        }
    }
}

// Few rows and few columns: the weights' bytes are the time, so they go
// straight from memory into the registers of the one wave that multiplies
// them, and K is shared out so that enough of them are in flight at once. A
// workgroup owns 16 columns and up to 16 rows; its NW waves take K in turns of
// 512 elements (16 blocks), and the sums meet in LDS, added in the waves'
// order. The matrix instruction is 16 x 16 x 128: lane l of instruction s of a
// turn holds block 4s + l / 16 of row l % 16, so a load of the wave covers 64
// consecutive bytes of 16 rows, and its scale is byte l / 16 of word s of the
// row's 16 scale bytes of the turn.
template <int NW>
__global__ void __launch_bounds__(NW * 64)
mx_skinny_kernel(MxGemmProblem p, int tiles_n) {
    constexpr int TURN = 16;                       // blocks per turn
    __shared__ f32x4 part[NW][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (int)blockIdx.x / tiles_n * 16, n0 = (int)blockIdx.x % tiles_n * 16;
    const int r = lane & 15, g = lane >> 4;
    const uint32_t blocks = p.K / 32;
    const int64_t ra = min(m0 + r, (int)p.M - 1), rb = min(n0 + r, (int)p.N - 1);
    const uint8_t *a = p.A + ra * blocks * 16, *sa = p.SFA + ra * blocks;
    const uint8_t *b = p.B + rb * blocks * 16, *sb = p.SFB + rb * blocks;
    f32x4 acc = {};
    auto mfma = [&](const u32x4& x, const u32x4& y, int ex, int ey) {
        const i32x8 X = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
        const i32x8 Y = {(int)y.x, (int)y.y, (int)y.z, (int)y.w, 0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(Y, X, acc, 4, 4, 0, ey, 0, ex);
    };
    // whole turns, the next one's loads in flight during a turn's products
    u32x4 wa[2][4], wb[2][4], ea[2], eb[2];
    auto load = [&](uint32_t turn, int q) {
        const uint32_t c0 = turn * TURN;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            wb[q][s] = *reinterpret_cast<const u32x4*>(b + (uint64_t)(c0 + 4 * s + g) * 16);
            wa[q][s] = *reinterpret_cast<const u32x4*>(a + (uint64_t)(c0 + 4 * s + g) * 16);
        }
        eb[q] = *reinterpret_cast<const u32x4_any*>(sb + c0);
        ea[q] = *reinterpret_cast<const u32x4_any*>(sa + c0);
    };
    auto multiply = [&](int q) {
#pragma unroll
        for (int s = 0; s < 4; ++s) mfma(wa[q][s], wb[q][s], (int)(ea[q][s] >> (8 * g)), (int)(eb[q][s] >> (8 * g)));
    };
    const uint32_t turns = blocks / TURN;
    uint32_t u = wave;
    if (u < turns) load(u, 0);
    for (; u + NW < turns; u += 2 * NW) {
        load(u + NW, 1);
        multiply(0);
        if (u + 2 * NW < turns) load(u + 2 * NW, 0);
        multiply(1);
    }
    if (u < turns) multiply(0);
    // the rest of K, by the next wave in turn: A's blocks past the end are zero
    if (blocks % TURN != 0 && wave == (int)(turns % NW)) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t c = turns * TURN + 4 * s + g, cc = min(c, blocks - 1);
            const u32x4 y = *reinterpret_cast<const u32x4*>(b + (uint64_t)cc * 16);
            u32x4 x = *reinterpret_cast<const u32x4*>(a + (uint64_t)cc * 16);
            if (c >= blocks) x = u32x4{0u, 0u, 0u, 0u};
            mfma(x, y, sa[cc], sb[cc]);
        }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    // lane l of the result holds columns 4 (l / 16) .. + 3 of row l % 16
#pragma unroll
    for (int w = 1; w < NW; ++w) acc += part[w][lane];
    const int m = m0 + r, n = n0 + 4 * g;
    if (m >= (int)p.M) return;
    uint16_t* out = p.C + (int64_t)m * p.N + n;
    const u32x2 w = {pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w)};
    if (n + 4 <= (int)p.N)
        *reinterpret_cast<u32x2_any*>(out) = w;
    else
        for (int e = 0; n + e < (int)p.N; ++e) out[e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
}

template <int NW>
hipError_t launch_skinny(const MxGemmProblem& p, hipStream_t stream) {
    const uint64_t tiles_n = (p.N + 15) / 16, tiles_m = (p.M + 15) / 16;
    mx_skinny_kernel<NW><<<dim3((uint32_t)(tiles_m * tiles_n)), NW * 64, 0, stream>>>(p, (int)tiles_n);
    return hipGetLastError();
}

// Tile I of its table. WM x WN waves and scales Q steps at a time where K is
// whole steps, WM2 x WN2 and pairs otherwise (more registers: fewer, larger
// waves keep two workgroups on a compute unit, or avoid spills). One instance
// spills: 256 x 256 of whole steps needs two registers more than the 256 a lane
// has; they are stored once before the K loop and loaded once behind it.
template <int I, bool GROUPED, int WM, int WN, int STAGES, int Q = 2, int WM2 = WM, int WN2 = WN>
hipError_t launch_tile(const MxGemmProblem& p, hipStream_t stream) {
    constexpr MxTile T = GROUPED ? kMxGrouped[I] : kMxDense[I];
    constexpr int BM = T.bm, BN = T.bn;
    static_assert(T.whole == WM * WN * 64 && T.other == WM2 * WN2 * 64, "threads of the grid's limit");
    const uint32_t tiles_n = (uint32_t)mx_ceil(p.N, BN);
    const uint32_t tiles_m = (uint32_t)(GROUPED ? mx_tiles_m_grouped(T, p.M, p.E) : mx_tiles_m(T, p.M));
    const dim3 grid(tiles_m * tiles_n);
    const ScalePath path = scale_path<Q>(p.K);
    if (path == WHOLE)
        mx_tile_kernel<BM, BN, WM, WN, STAGES, GROUPED, WHOLE, Q><<<grid, WM * WN * 64, 0, stream>>>(p, (int)tiles_m, (int)tiles_n);
    else if (path == SHIFTED)
        mx_tile_kernel<BM, BN, WM2, WN2, STAGES, GROUPED, SHIFTED, 2><<<grid, WM2 * WN2 * 64, 0, stream>>>(p, (int)tiles_m, (int)tiles_n);
    else
        mx_tile_kernel<BM, BN, WM2, WN2, STAGES, GROUPED, SHORT, 2><<<grid, WM2 * WN2 * 64, 0, stream>>>(p, (int)tiles_m, (int)tiles_n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_quantize(const MxQuantProblem& p, hipStream_t stream) {
    const uint32_t segs = mx_quant_pieces(p.K);
    const uint64_t waves = (uint64_t)p.R * segs;               // < 2^32: checked
    const uint32_t per_seg = segs == 1 ? 0xFFFFFFFFu : (uint32_t)(((uint64_t)1 << 32) / segs) + ((((uint64_t)1 << 32) % segs) != 0);
    const dim3 grid(grid_of((waves + 7) / 8));
    const bool f32 = p.type == BG_F32;
    const bool vec = (uint64_t)p.ldx * (f32 ? 4 : 2) % 16 == 0;
    auto k = f32 ? (vec ? mxfp4_quantize_kernel<true, true> : mxfp4_quantize_kernel<true, false>)
                 : (vec ? mxfp4_quantize_kernel<false, true> : mxfp4_quantize_kernel<false, false>);
    k<<<grid, 256, 0, stream>>>(p, segs, per_seg, (uint32_t)waves);
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
    if (p.offsets != nullptr) {
        switch (mx_grouped_tile(p.M, p.N, p.K, p.E)) {
            case MX_G32x128: return launch_tile<MX_G32x128, true, 1, 4, 2, 4>(p, stream);
            case MX_G64x128: return launch_tile<MX_G64x128, true, 2, 2, 3>(p, stream);
            case MX_G128x128: return launch_tile<MX_G128x128, true, 4, 2, 2, 4, 2, 2>(p, stream);
        }
        return hipErrorInvalidValue;
    }
    // Up to 16 rows, where 64-column tiles would fill under a third of the
    // compute units: 1 x 4096 x 7168 5.0 us against 8.0 us with the smallest
    // tile, 16 x 4096 x 7168 6.3 / 8.1 us (16 x 7168 x 16384: 20 / 15 us).
    // Eight waves from K = 4096 on, four below: 1 x 4096 x 7168 5.15 us against
    // 5.79, x 4096 3.62 / 3.72, x 2048 2.93 / 2.81, x 1024 2.55 / 2.42; 16 x 4096 x
    // 7168 6.51 / 6.77, x 2048 3.33 / 3.21.
    if (p.M <= 16 && (uint64_t)p.N * 3 <= (uint64_t)p.cus * 64)
        return p.K >= 8 * 512 ? launch_skinny<8>(p, stream) : launch_skinny<4>(p, stream);
    switch (mx_dense_tile(p.M, p.N, p.K, p.cus)) {
        case MX_256x256: return launch_tile<MX_256x256, false, 2, 4, 2, 2, 2, 2>(p, stream);
        case MX_256x128: return launch_tile<MX_256x128, false, 4, 2, 3>(p, stream);
        case MX_128x128:
            // one to a compute unit: LDS for four stages (512 x 7168 x 16384: 41 us, 50 with two)
            if (mx_ceil(p.M, 128) * mx_ceil(p.N, 128) <= p.cus)
                return launch_tile<MX_128x128, false, 4, 2, 4, 2, 2, 2>(p, stream);
            return launch_tile<MX_128x128, false, 4, 2, 2, 4, 2, 2>(p, stream);
        case MX_64x64: return launch_tile<MX_64x64, false, 2, 2, 4, 4>(p, stream);
        case MX_32x64: return launch_tile<MX_32x64, false, 1, 2, 4>(p, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace bg
