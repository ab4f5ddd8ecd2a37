// The gated MLP block and the gradients of dense products on the BF16 matrix
// cores:
//   gated  H = act(A B0^T) * (A B1^T), both products in one pass over A, the
//          activation and the product on the FP32 accumulators;
//   nn     C = A B           (A [M, K], B [K, N]; a linear layer's dX = dY W);
//   tn     C = A^T B         (A [K, M], B [K, N]; its dW = dY^T X);
//   the gated block's gradient: dG and dU elementwise, then one nn chain over
//   both (dA = dG B0 + dU B1) and one tn launch for dB0 and dB1.
//
// One main loop serves the three. A workgroup owns a BM x BN tile and walks the
// reduction in steps of 64 through a ring of LDS stages filled by direct loads
// (buffer_load_dwordx4 ... lds), completion counted by hand (s_waitcnt vmcnt).
// An operand lies in one of two ways:
//   KC  the reduction index is contiguous (rows of A, weights [N, K]): LDS rows
//       of 64, 16-byte chunks swizzled by row, a fragment is one 16-byte read;
//   MC  the output index is contiguous (B of nn, both of tn): LDS rows are the
//       64 reduction steps, as they lie in memory, and the matrix core's
//       k-contiguous fragments come out of ds_read_b64_tr_b16, which transposes
//       4 x 16 blocks on the way to the registers. No transposed copy of an
//       operand is ever written. 64-byte blocks are XORed by the row, so that
//       the 32 lanes served together touch every bank once.
// What is left of the reduction by 64, and operands whose rows do not start at
// multiples of 16 bytes, take guarded steps: element-wise checked loads
// through registers, no pipeline (nn and tn copy such operands to aligned rows
// first where that is faster).
//
// Bound by the matrix cores and the power they draw where there are tiles for
// every compute unit: 5120 x 11008 x 2048 gated 386 us (462 GFLOP, 1196 TFLOP/s;
// cores busy in 54% of the cycles), the nn chain of its gradient 5120 x 2048 x
// 22016 404 us (160 x 256 tiles, one round; 585 us with 256 x 256), the tn pair
// 22016 x 2048 x 5120 413 us. Where 256 x 256 tiles leave a round mostly empty the
// last columns go in 256 x 128 (gated_tiles.hpp): 5120 x 11008 x 2048 as nn 226 us
// instead of 241. Reading transposed costs nothing there: 4096^3 takes 129 us as nn
// and as tn. Steps of 32 in four or five stages (twice the time for a load to
// land) cost 3 and 11% more there, so it is not the loads' latency that bounds a
// step. These calls draw all the power there is: cards, and one card warm or
// rested, differ by 10 to 15%. Small products are bound by a fixed 5 us
// and 0.4 - 0.6 us a step, operands coming from the L2s at 50 - 80 bytes a ns
// and compute unit.
#include <type_traits>

#include "bg_internal.hpp"
#include "gate.hpp"
#include "gated_tiles.hpp"
#include "mma_common.hpp"
#include "tile_order.hpp"

#pragma clang fp contract(off)

namespace bg {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
// the same at any address: global memory takes unaligned accesses
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

enum Mode : int { MODE_GATED = 0, MODE_NN = 1, MODE_TN = 2 };
enum Layout : int { KC = 0, MC = 1 };

constexpr int STEP = 64;   // reduction per pipeline step

struct GatedParams {
    // gated: A0, B0, B1. nn: A0 B0 (+ A1 B1 where parts == 2). tn: A0^T B0 -> C0
    // (and A1^T B0 -> C1 where parts == 2).
    const uint16_t *A0, *A1, *B0, *B1;
    void *C0, *C1;          // bf16, or FP32 planes in C0 (splits > 1)
    void *G, *U;            // gated: the products themselves, or NULL
    int kept;               // bg_type of G and U
    int M, N, K;            // of one product
    int lda, ldb;           // elements between rows as they lie in memory
    int tiles_m, tiles_n;   // of one product
    int start;              // the first tile's column
    int parts;
    int64_t low;            // tn: 0, or from A to a second A, whose product with the same B is added
    int splits;             // of the reduction's whole steps
    int direct;             // rows start at multiples of 16 bytes: direct loads
};

// XOR of a 16-byte chunk's index in row k of an MC stage of COLS columns: its
// 64-byte blocks by the row (128 columns or more), or by every second row where
// two rows share the banks (64 columns).
template <int COLS>
__device__ __forceinline__ int mc_swizzle(int k) {
    static_assert(COLS == 64 || COLS % 128 == 0, "whole bank windows");
    return COLS == 64 ? ((k >> 1) & 1) << 2 : (k & 3) << 2;
}

// Row r of a gated tile's B stage: 32 rows of B0, 32 of B1, and so on, so that
// a wave holds g and u of the same outputs in neighbouring fragments.
__device__ __forceinline__ int pair_row(int r) { return (r >> 6) * 32 + (r & 31); }

// Direct loads of one operand's steps. Instruction j of a wave fills 1 KB of
// LDS (lane i at byte 16 i); every wave issues PER of them a step.
template <int ROWS, int NT, int LAYOUT, bool PAIR>
struct Direct {
    static constexpr int CPR = LAYOUT == KC ? STEP / 8 : ROWS / 8;    // chunks per LDS row
    static constexpr int RPS = 64 / CPR;                              // LDS rows per 1 KB
    static constexpr int NW = NT / 64;
    static constexpr int SEGS = ROWS * STEP * 2 / 1024;
    static constexpr int PER = SEGS / NW;
    static_assert(SEGS % NW == 0 && CPR <= 64 && 64 % CPR == 0, "whole 1 KB segments, alike for every wave");

    // A pair's 1 KB segments (8 rows) alternate between its matrices every four:
    // with eight waves a wave always loads from one of them, with four its
    // instructions alternate.
    static constexpr int SOURCES = PAIR && NW == 4 ? 2 : 1;
    static_assert(!PAIR || NW == 4 || NW == 8, "segments of a wave");

    uint32_t voff[PER];
    __amdgpu_buffer_rsrc_t rsrc[SOURCES];

    // row0: the tile's first row (KC) or column (MC) of nrows; ld: elements
    // between rows in memory. Rows and columns past the matrix re-read its
    // last ones: they belong to outputs that are never stored.
    __device__ __forceinline__ void init(int row0, int nrows, int ld, int wave, int lane) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int seg = wave + j * NW;
            const int r = seg * RPS + lane / CPR, slot = lane % CPR;
            if constexpr (LAYOUT == KC) {
                const int row = PAIR ? pair_row(r) : r;
                voff[j] = (uint32_t)((min(row0 + row, nrows - 1) - row0) * ld + chunk_slot<8>(r, slot) * 8) * 2u;
            } else {
                // rows are a multiple of 8 elements apart, so a last chunk of fewer columns exists whole
                const int col = min(row0 + (slot ^ mc_swizzle<ROWS>(r)) * 8, (nrows + 7) / 8 * 8 - 8) - row0;
                voff[j] = (uint32_t)(r * ld + col) * 2u;
            }
        }
    }

    // base (and base1 of a pair): the tile's first element of the step
    __device__ __forceinline__ void seek(const uint16_t* base, const uint16_t* base1, int wave) {
        if (PAIR && NW == 8 && (wave & 4)) base = base1;
        rsrc[0] = resource(base);
        if constexpr (SOURCES == 2) rsrc[1] = resource(base1);
    }

    // The wait: where the address comes out of a vector register, the loads,
    // which the compiler cannot see into, must keep five states' distance.
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t resource(const uint16_t* base) {
        __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(base), (short)0, 0x7FFFFFFF, 0x00020000);
        asm volatile("s_nop 4" : "+s"(r));
        return r;
    }

    __device__ __forceinline__ void issue(uint16_t* lds, int wave, int lo, int hi) const {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (j < lo || j >= hi) continue;
            const uint32_t l = (uint32_t)(uintptr_t)(
                (__attribute__((address_space(3))) uint16_t*)(lds + (wave + j * NW) * 512));
            // inline assembly: the compiler would make every later LDS read wait for these
            asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff[j]), "s"(rsrc[SOURCES == 2 ? j & 1 : 0]), "{m0}"(l));
        }
    }
};

// Eight elements p[0 .. 7] of which those below n exist.
__device__ __forceinline__ u32x4 guarded8(const uint16_t* p, int n) {
    if (n >= 8) return *reinterpret_cast<const u32x4_any*>(p);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}

// One step of len <= 64 with checked loads: zeros past the reduction's end.
// base as for Direct::seek.
template <int ROWS, int NT, int LAYOUT, bool PAIR>
__device__ __forceinline__ void guarded_stage(const uint16_t* base, const uint16_t* base1, int row0, int nrows, int ld,
                                              int len, uint16_t* lds, int tid) {
    constexpr int CPR = LAYOUT == KC ? STEP / 8 : ROWS / 8;
    constexpr int CHUNKS = ROWS * STEP / 8;
#pragma unroll 2
    for (int q = tid; q < CHUNKS; q += NT) {
        const int r = q / CPR, c = q % CPR;
        if constexpr (LAYOUT == KC) {
            const int row = min(row0 + (PAIR ? pair_row(r) : r), nrows - 1) - row0;
            const uint16_t* b = PAIR && (r & 32) ? base1 : base;
            *reinterpret_cast<u32x4*>(lds + r * STEP + chunk_slot<8>(r, c) * 8) =
                guarded8(b + (int64_t)row * ld + c * 8, len - c * 8);
        } else {
            *reinterpret_cast<u32x4*>(lds + r * ROWS + (c ^ mc_swizzle<ROWS>(r)) * 8) =
                guarded8(base + (int64_t)r * ld + c * 8, r < len ? nrows - row0 - c * 8 : 0);
        }
    }
}

// Per-lane byte offsets of one operand's fragments in a stage. KC: the chunk of
// fragment i at sub-step kk is (2 kk + h) ^ s(row), and fragments start on
// 32-row boundaries, so four offsets serve all (see FragAddr64's derivation in
// gemm_mfma.hip). MC: row and swizzle depend on the lane alone (sub-steps and
// the two halves of a fragment are multiples of four rows), so one offset per
// fragment.
template <int ROWS, int FRAGS, int LAYOUT>
struct Frags {
    static constexpr int N = LAYOUT == KC ? 4 : FRAGS;
    uint32_t v[N];

    __device__ __forceinline__ void init(int first, int lane, uint32_t base) {
        if constexpr (LAYOUT == KC) {
            const int row = first + (lane & 31), h = lane >> 5;
            const int s0 = (row ^ (row >> 3)) & 7;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = base + (uint32_t)(row * 128 + 16 * (h ^ (s0 & 1)) + 32 * (j ^ (s0 >> 1)));
        } else {
            const int r = 8 * (lane >> 5) + ((lane >> 2) & 3);
#pragma unroll
            for (int i = 0; i < FRAGS; ++i) {
                const int chunk = (first / 8 + 4 * i) ^ mc_swizzle<ROWS>(r);
                v[i] = base + (uint32_t)(r * ROWS * 2 + chunk * 16 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8);
            }
        }
    }

    __device__ __forceinline__ void read(const uint16_t* stage, int kk, bf16x8 (&f)[FRAGS]) const {
        const char* base = reinterpret_cast<const char*>(stage);
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) {
            if constexpr (LAYOUT == KC) {
                f[i] = *reinterpret_cast<const bf16x8*>(base + v[kk ^ (2 * (i & 1))] + 4096 * i);
            } else {
                typedef __attribute__((address_space(3))) s16x4* Ptr;
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(base + v[i] + kk * 16 * ROWS * 2));
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(base + v[i] + (kk * 16 + 4) * ROWS * 2));
                f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        }
    }
};

template <int FM, int FN>
__device__ __forceinline__ void mma(const bf16x8 (&fa)[FM], const bf16x8 (&fb)[FN], f32x16 (&acc)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
}

// Writes rows of bf16 (or FP32) results from the accumulators through LDS:
// whole rows, 16 contiguous bytes per lane. value(i, j, e) is element e of
// 16 of fragment (i, j), JN fragments a wave, TNO columns a wave. g and u of 5120 x
// 11008 in FP32 (450 MB) add 55 us to the call this way; straight from the
// accumulators, 32 bytes of a row at a time, 75 us, and 325 us past the caches.
template <typename OUT, bool STREAM, int BM, int BNO, int WM, int WN, int FM, int JN, int NT, int CAP, class Value>
__device__ __forceinline__ void store_tile(OUT* C, int64_t ldc, int M, int N, int m0, int n0, uint8_t* lds, int wm,
                                           int wn, int lane, int tid, Value&& value) {
    constexpr int ELEM = sizeof(OUT), ROWB = BNO * ELEM, CPR = ROWB / 16, EPC = 16 / ELEM;
    constexpr int TM = BM / WM, TNO = BNO / WN;
    constexpr int FIT = CAP / ROWB, RP = FIT >= BM ? BM : FIT / 32 * 32;
    static_assert(RP >= 32 && JN * 32 == TNO, "a pass holds a fragment's rows");
    constexpr int PASSES = (BM + RP - 1) / RP;
    // chunks rotate by the row: the 32 rows of one LDS write spread over the banks
    auto slot = [](int row, int chunk) { return row * ROWB + (((chunk + row) % CPR) << 4); };
    const bool aligned = ((uint64_t)ldc * ELEM) % 16 == 0;
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
        lds_barrier();
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int blk = wm * TM + i * 32;
            if (blk < pass * RP || blk >= (pass + 1) * RP) continue;
            const int row = blk + (lane & 31) - pass * RP;
#pragma unroll
            for (int j = 0; j < JN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = wn * TNO + j * 32 + g * 8 + (lane >> 5) * 4;
                    const float v0 = value(i, j, 4 * g), v1 = value(i, j, 4 * g + 1);
                    const float v2 = value(i, j, 4 * g + 2), v3 = value(i, j, 4 * g + 3);
                    if constexpr (ELEM == 4)
                        *reinterpret_cast<f32x4*>(lds + slot(row, n >> 2)) = f32x4{v0, v1, v2, v3};
                    else
                        *reinterpret_cast<u32x2*>(lds + slot(row, n >> 3) + (lane >> 5) * 8) =
                            u32x2{pack_bf16x2(v0, v1), pack_bf16x2(v2, v3)};
                }
        }
        lds_barrier();
        const int rows = min(RP, BM - pass * RP);
#pragma unroll 4
        for (int q = tid; q < rows * CPR; q += NT) {
            const int row = q / CPR, chunk = q % CPR;
            const int m = m0 + pass * RP + row, n = n0 + chunk * EPC;
            if (m >= M || n >= N) continue;
            const u32x4 w = *reinterpret_cast<const u32x4*>(lds + slot(row, chunk));
            OUT* dst = C + (int64_t)m * ldc + n;
            if (n + EPC <= N) {
                // results are not read again by this launch; planes are, by the next
                if (aligned && STREAM)
                    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(dst));
                else
                    *reinterpret_cast<u32x4_any*>(dst) = w;
            } else {
                for (int e = 0; n + e < N; ++e) {
                    if constexpr (ELEM == 4)
                        dst[e] = __builtin_bit_cast(float, (uint32_t)w[e]);
                    else
                        dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    }
}

// STAGES == 1: every step guarded, for rows that do not start at multiples of 16 bytes.
template <int MODE, int ACT, int BM, int BN, int WM, int WN, int STAGES, bool PLANES>
__device__ __forceinline__ void gated_body(const GatedParams& p, uint16_t* smem, int tile, int split) {
    constexpr bool PAIR = MODE == MODE_GATED;
    constexpr int LA = MODE == MODE_TN ? MC : KC, LB = MODE == MODE_GATED ? KC : MC;
    constexpr int NT = WM * WN * 64, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
    static_assert(FM * 32 * WM == BM && FN * 32 * WN == BN && (!PAIR || FN % 2 == 0), "whole fragments, pairs of them");
    constexpr int STAGE = (BM + BN) * STEP;
    constexpr int BNO = PAIR ? BN / 2 : BN;       // output columns

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    int tm, tn;
    tile_of<ORDER_GEMM>(tile, MODE == MODE_TN ? p.tiles_m * p.parts : p.tiles_m, p.tiles_n, tm, tn);
    const uint16_t* A0 = p.A0;
    void* C = p.C0;
    if (MODE == MODE_TN && tm >= p.tiles_m) {     // the second product
        tm -= p.tiles_m;
        A0 = p.A1;
        C = p.C1;
    }
    const int m0 = tm * BM, n0 = p.start + tn * BNO;

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    // the tile's first element of part `part` at reduction index k
    auto a_at = [&](int part, int k) {
        const uint16_t* a = MODE == MODE_NN && part ? p.A1 : MODE == MODE_TN && part ? A0 + p.low : A0;
        return LA == KC ? a + ((int64_t)m0 * p.lda + k) : a + ((int64_t)k * p.lda + m0);
    };
    auto b_at = [&](int part, int k) {
        const uint16_t* b = MODE == MODE_NN && part ? p.B1 : p.B0;
        return LB == KC ? b + ((int64_t)n0 * p.ldb + k) : b + ((int64_t)k * p.ldb + n0);
    };
    auto b1_at = [&](int k) { return PAIR ? p.B1 + ((int64_t)n0 * p.ldb + k) : nullptr; };

    Frags<BM, FM, LA> fra;
    Frags<BN, FN, LB> frb;
    fra.init(wm * TM, lane, 0u);
    frb.init(wn * TN, lane, (uint32_t)BM * STEP * 2u);

    constexpr int KK = STEP / 16;
    bf16x8 fa[2][FM], fb[2][FN];

    // Steps: the rest of each part by 64 first (guarded), then the whole steps of
    // all parts; the splits take consecutive ones. At most two are guarded, so
    // that they are among the stages that are filled ahead of the loop.
    const int parts = MODE == MODE_NN ? p.parts : MODE == MODE_TN && p.low ? 2 : 1;
    const int whole = p.K / STEP, rest = p.K % STEP, guarded = rest ? parts : 0;
    const int each = whole + (rest ? 1 : 0);     // steps of a part
    int first = 0, last = each * parts;
    if constexpr (PLANES) {
        const int per = (last + p.splits - 1) / p.splits;
        first = min(split * per, last);
        last = min(first + per, last);
    }
    const int nsteps = last - first;
    if constexpr (STAGES == 1) {
        for (int t = first; t < last; ++t) {
            const int part = t >= each ? 1 : 0, k = (t - part * each) * STEP, len = min(p.K - k, STEP);
            lds_barrier();
            guarded_stage<BM, NT, LA, false>(a_at(part, k), nullptr, m0, p.M, p.lda, len, smem, tid);
            guarded_stage<BN, NT, LB, PAIR>(b_at(part, k), b1_at(k), n0, p.N, p.ldb, len, smem + BM * STEP, tid);
            lds_barrier();
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                fra.read(smem, kk, fa[0]);
                frb.read(smem, kk, fb[0]);
                mma<FM, FN>(fa[0], fb[0], acc);
            }
        }
    } else if (nsteps > 0) {
        typedef Direct<BM, NT, LA, false> DA;
        typedef Direct<BN, NT, LB, PAIR> DB;
        constexpr int PA = DA::PER, L = PA + DB::PER;
        DA da;
        DB db;
        da.init(m0, p.M, p.lda, wave, lane);
        db.init(n0, p.N, p.ldb, wave, lane);
        // Direct loads are issued at a uniform rate, so that the waits can count
        // them: steps past the end re-load the last one, into a stage that is
        // not read again.
        const bool direct = last > guarded;
        auto seek = [&](int s) {
            s = min(s, last - 1) - guarded;
            const int part = s >= whole ? 1 : 0, k = (s - part * whole) * STEP;
            da.seek(a_at(part, k), nullptr, wave);
            db.seek(b_at(part, k), b1_at(k), wave);
        };
        auto issue = [&](uint16_t* buf, int lo, int hi) {
            da.issue(buf, wave, lo, min(hi, PA));
            db.issue(buf + BM * STEP, wave, max(lo - PA, 0), hi - PA);
        };
#pragma unroll
        for (int st = 0; st < STAGES; ++st) {
            uint16_t* buf = smem + st * STAGE;
            if (first + st < guarded) {
                if (first + st < last) {
                    const int k = whole * STEP;
                    guarded_stage<BM, NT, LA, false>(a_at(first + st, k), nullptr, m0, p.M, p.lda, rest, buf, tid);
                    guarded_stage<BN, NT, LB, PAIR>(b_at(first + st, k), b1_at(k), n0, p.N, p.ldb, rest, buf + BM * STEP, tid);
                }
            } else if (direct) {
                seek(first + st);
                issue(buf, 0, L);
            }
        }
        wait_vmcnt<(STAGES - 1) * L>();
        lds_barrier();
        fra.read(smem, 0, fa[0]);
        frb.read(smem, 0, fb[0]);

        // Sub-step kk multiplies what was read during kk - 1. The barrier that
        // retires a step stands before its last sub-step's products; the freed
        // stage is refilled in four parts, over that sub-step and the next
        // step's first three.
        constexpr int ND = FM * (LA == KC ? 1 : 2) + FN * (LB == KC ? 1 : 2);
        uint16_t* refill = smem;
        auto leading = [&](const uint16_t* stage, bool refilling) {
#pragma unroll
            for (int kk = 0; kk + 1 < KK; ++kk) {
                const int cur = kk & 1;
                if (refilling) issue(refill, L * (kk + 1) / KK, L * (kk + 2) / KK);
                fra.read(stage, kk + 1, fa[cur ^ 1]);
                frb.read(stage, kk + 1, fb[cur ^ 1]);
                mma<FM, FN>(fa[cur], fb[cur], acc);
                interleave_mfma<FM * FN, ND, 0>();
            }
        };
        for (int t = 0; t + 1 < nsteps; ++t) {
            leading(smem + (t % STAGES) * STAGE, direct && t > 0);
            wait_vmcnt<(STAGES - 2) * L>();      // step t + 1 has landed for this wave
            lds_barrier();                        // and for all; step t's stage is free
            refill = smem + (t % STAGES) * STAGE;
            if (direct) {
                seek(first + t + STAGES);
                issue(refill, 0, L / KK);
            }
            const uint16_t* next = smem + ((t + 1) % STAGES) * STAGE;
            fra.read(next, 0, fa[0]);
            frb.read(next, 0, fb[0]);
            mma<FM, FN>(fa[1], fb[1], acc);
            interleave_mfma<FM * FN, ND, 0>();
        }
        leading(smem + ((nsteps - 1) % STAGES) * STAGE, false);
        mma<FM, FN>(fa[1], fb[1], acc);
        wait_vmcnt<0>();      // no load may land in LDS behind this point
    }

    // Opaque to the compiler from here on: the addresses of the results are not
    // computed ahead of the main loop, where every register is taken.
    int etid = tid;
    asm volatile("" : "+v"(etid));
    const int elane = etid & 63;
    uint8_t* lds = reinterpret_cast<uint8_t*>(smem);
    constexpr int CAP = STAGES * STAGE * 2;
    if constexpr (PAIR) {
        auto out = [&](auto* dst, auto&& value) {
            store_tile<std::remove_reference_t<decltype(*dst)>, true, BM, BNO, WM, WN, FM, FN / 2, NT, CAP>(
                dst, p.N, p.M, p.N, m0, n0, lds, wm, wn, elane, etid, value);
        };
        if (p.G != nullptr) {
            auto g = [&](int i, int j, int e) { return acc[i][2 * j][e]; };
            auto u = [&](int i, int j, int e) { return acc[i][2 * j + 1][e]; };
            if (p.kept == BG_F32) {
                out(static_cast<float*>(p.G), g);
                out(static_cast<float*>(p.U), u);
            } else {
                out(static_cast<uint16_t*>(p.G), g);
                out(static_cast<uint16_t*>(p.U), u);
            }
        }
        out(static_cast<uint16_t*>(C), [&](int i, int j, int e) { return gate<ACT>(acc[i][2 * j][e]) * acc[i][2 * j + 1][e]; });
    } else {
        auto value = [&](int i, int j, int e) { return acc[i][j][e]; };
        if constexpr (PLANES) {
            const int64_t rows = MODE == MODE_TN ? (int64_t)p.M * p.parts : p.M;
            float* plane = static_cast<float*>(p.C0) + (int64_t)split * rows * p.N;
            if (MODE == MODE_TN && C != p.C0) plane += (int64_t)p.M * p.N;
            store_tile<float, false, BM, BNO, WM, WN, FM, FN, NT, CAP>(plane, p.N, p.M, p.N, m0, n0, lds, wm, wn, elane, etid, value);
        } else {
            store_tile<uint16_t, true, BM, BNO, WM, WN, FM, FN, NT, CAP>(static_cast<uint16_t*>(C), p.N, p.M, p.N, m0, n0, lds, wm,
                                                                  wn, elane, etid, value);
        }
    }
}

template <int MODE, int ACT, int BM, int BN, int WM, int WN, int STAGES, bool PLANES>
__global__ void __launch_bounds__(WM * WN * 64)
gated_kernel(GatedParams p) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[STAGES * (BM + BN) * STEP];
    gated_body<MODE, ACT, BM, BN, WM, WN, STAGES, PLANES>(p, smem, (int)blockIdx.x, (int)blockIdx.y);
}

// GT_MIXED: p's tiles of 256 x 256, then the columns from `start` on in 256 x 128.
template <int MODE, int ACT>
__global__ void __launch_bounds__(512)
mixed_kernel(GatedParams p, int wide, int start, int tiles_n) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[3 * (256 + 128) * STEP];
    const int i = (int)blockIdx.x;
    if (i < wide) {
        gated_body<MODE, ACT, 256, 256, 2, 4, 2, false>(p, smem, i, 0);
    } else {
        p.start = start;
        p.tiles_n = tiles_n;
        gated_body<MODE, ACT, 256, 128, 4, 2, 3, false>(p, smem, i - wide, 0);
    }
}

// An nn and a tn product that do not wait for each other, in one launch: the first
// workgroups take a's tiles (split by split), the others b's. Where neither fills
// the chip, both take the time of the longer: the gradient of 1015 x 1407 x 520
// 19 us instead of 16 + 15 us and a launch.
template <int BM, int BN, int WM, int WN, int STAGES, bool PLANES_A, bool PLANES_B>
__global__ void __launch_bounds__(WM * WN * 64)
pair_kernel(GatedParams a, GatedParams b, int tiles_a, int blocks_a, int tiles_b) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[STAGES * (BM + BN) * STEP];
    const int i = (int)blockIdx.x;
    if (i < blocks_a)
        gated_body<MODE_NN, 0, BM, BN, WM, WN, STAGES, PLANES_A>(a, smem, i % tiles_a, i / tiles_a);
    else
        gated_body<MODE_TN, 0, BM, BN, WM, WN, STAGES, PLANES_B>(b, smem, (i - blocks_a) % tiles_b, (i - blocks_a) / tiles_b);
}

// ---------------------------------------------------------------------------
// dG = dH U act'(G), dU = dH act(G), with act'(g) = s + g z'(g) s (1 - s).
// Rows of the results are ld elements apart (a multiple of 8); columns N .. ld-1
// are written as zeros. low != 0: what their rounding to BF16 leaves goes, rounded
// too, `low` elements behind them. Bound by memory: 10 bytes in, 4 out per
// element with G and U in FP32, 5120 x 11008 (789 MB) in 131 us (6.0 TB/s).
// ---------------------------------------------------------------------------
template <int ACT>
__device__ __forceinline__ void gate_grad(float dh, float g, float u, float& dg, float& du) {
    const float s = gate_sigmoid<ACT>(g);
    // past 10^4 s (1 - s) is 0, and must not meet an overflow
    const float c = __builtin_fminf(__builtin_fmaxf(g, -1e4f), 1e4f);
    const float slope = ACT == BG_SILU ? 1.0f : kGeluC * __builtin_fmaf(3.0f * kGeluK * c, c, 1.0f);
    du = dh * (g * s);
    dg = dh * u * __builtin_fmaf(c * slope, s * (1.0f - s), s);
}

// What rounding v to r left (nothing where that is no number: r says it all).
__device__ __forceinline__ float rest(float v, float r) {
    const float d = v - r;
    return __builtin_fabsf(d) < __builtin_inff() ? d : 0.0f;
}

// Eight values p[at ..] of which those below n exist.
template <bool F32>
__device__ __forceinline__ void kept8(const void* p, int64_t at, int n, float (&v)[8]) {
    if constexpr (F32) {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        const float* q = static_cast<const float*>(p) + at;
        if (n >= 8) {
            // read once, and more than the caches hold where it is long: past them the
            // gradient of 5120 x 11008 x 2048 takes 940 instead of 946 us
            const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(q));
            const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(q + 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = a[e], v[e + 4] = b[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? q[e] : 0.0f;
        }
    } else {
        const u32x4 w = guarded8(static_cast<const uint16_t*>(p) + at, n);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
    }
}

template <int ACT, bool F32>
__global__ void __launch_bounds__(256)
gate_grad_kernel(GateGradProblem p, int64_t chunks) {
    const int per = (int)(p.ld / 8);
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < chunks; q += (int64_t)gridDim.x * 256) {
        const int64_t row = q / per;
        const int n = (int)(q - row * per) * 8, left = (int)p.N - n;
        const int64_t at = row * p.N + n;
        float h[8], g[8], u[8];
        kept8<false>(p.dH, at, left, h);
        kept8<F32>(p.G, at, left, g);
        kept8<F32>(p.U, at, left, u);
        u32x4 og, ou, lg, lu;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float g0, g1, u0, u1;
            gate_grad<ACT>(h[2 * e], g[2 * e], u[2 * e], g0, u0);
            gate_grad<ACT>(h[2 * e + 1], g[2 * e + 1], u[2 * e + 1], g1, u1);
            og[e] = pack_bf16x2(g0, g1);
            ou[e] = pack_bf16x2(u0, u1);
            lg[e] = pack_bf16x2(rest(g0, bf16_lo(og[e])), rest(g1, bf16_hi(og[e])));
            lu[e] = pack_bf16x2(rest(u0, bf16_lo(ou[e])), rest(u1, bf16_hi(ou[e])));
        }
        uint16_t *dg = p.dG + row * p.ld + n, *du = p.dU + row * p.ld + n;
        *reinterpret_cast<u32x4*>(dg) = og;
        *reinterpret_cast<u32x4*>(du) = ou;
        if (p.low != 0) {
            *reinterpret_cast<u32x4*>(dg + p.low) = lg;
            *reinterpret_cast<u32x4*>(du + p.low) = lu;
        }
    }
}

// Rows to multiples of 16 bytes: 2048 x 11007 (90 MB moved) in 18.2 us, 4.9 TB/s.
__global__ void __launch_bounds__(256)
aligned_copy_kernel(AlignedCopy p) {
    const int i = blockIdx.y, per = (int)(p.ld[i] / 8);
    const int64_t chunks = (int64_t)p.rows[i] * per;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < chunks; q += (int64_t)gridDim.x * 256) {
        const int64_t row = chunks < (int64_t)1 << 32 ? (uint32_t)q / (uint32_t)per : q / per;
        const int n = (int)(q - row * per) * 8;
        *reinterpret_cast<u32x4*>(p.to[i] + q * 8) = guarded8(p.from[i] + row * p.cols[i] + n, (int)p.cols[i] - n);
    }
}

// C = bf16((P0 + P1) + ...), planes added in ascending order; blockIdx.y is the
// part (one output each), planes hold all parts' rows. Four planes of 512 x 2048
// from the caches: 4.2 us.
__global__ void __launch_bounds__(256)
planes_sum_kernel(const float* planes, uint16_t* C0, uint16_t* C1, int64_t count, int splits) {
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    const int64_t e0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e0 >= count) return;
    const int64_t stride = count * gridDim.y;
    const float* src = planes + blockIdx.y * count + e0;
    uint16_t* C = (blockIdx.y ? C1 : C0) + e0;
    if (e0 + 4 <= count) {
        f32x4 s = *reinterpret_cast<const f32x4_any*>(src);
        int i = 1;
        for (; i + 3 < splits; i += 4) {      // four loads in flight
            f32x4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const f32x4_any*>(src + (i + q) * stride);
#pragma unroll
            for (int q = 0; q < 4; ++q) s += v[q];
        }
        for (; i < splits; ++i) s += *reinterpret_cast<const f32x4_any*>(src + i * stride);
        *reinterpret_cast<u32x2*>(C) = u32x2{pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w)};
    } else {
        for (int e = 0; e0 + e < count; ++e) {
            float s = src[e];
            for (int i = 1; i < splits; ++i) s += src[i * stride + e];
            C[e] = (uint16_t)pack_bf16x2(s, 0.0f);
        }
    }
}

template <int MODE, int ACT, int BM, int BN, int WM, int WN, int STAGES, bool PLANES>
hipError_t launch_kernel(GatedParams p, hipStream_t stream) {
    p.tiles_m = (p.M + BM - 1) / BM;
    p.tiles_n = (p.N + tile_columns(BN, MODE == MODE_GATED) - 1) / tile_columns(BN, MODE == MODE_GATED);
    const unsigned n = (unsigned)p.tiles_m * (unsigned)p.tiles_n * (MODE == MODE_TN ? (unsigned)p.parts : 1u);
    hipLaunchKernelGGL((gated_kernel<MODE, ACT, BM, BN, WM, WN, STAGES, PLANES>), dim3(n, (unsigned)p.splits),
                       dim3(WM * WN * 64), 0, stream, p);
    return hipGetLastError();
}

template <int MODE, int ACT>
hipError_t launch_mixed(GatedParams p, int columns, hipStream_t stream) {
    constexpr bool GATED = MODE == MODE_GATED;
    p.tiles_m = (p.M + 255) / 256;
    p.tiles_n = columns;
    const int rows = p.tiles_m * (MODE == MODE_TN ? p.parts : 1), start = columns * tile_columns(256, GATED);
    const int tiles_n = start < p.N ? (p.N - start + tile_columns(128, GATED) - 1) / tile_columns(128, GATED) : 0;
    const int wide = rows * columns;
    mixed_kernel<MODE, ACT><<<dim3((unsigned)wide + (unsigned)rows * tiles_n), dim3(512), 0, stream>>>(p, wide, start, tiles_n);
    return hipGetLastError();
}

template <int MODE, int ACT, bool PLANES>
hipError_t launch_tile(const GatedParams& p, int tile, int wide, hipStream_t stream) {
    if (!p.direct) return launch_kernel<MODE, ACT, 128, 128, 2, 2, 1, PLANES>(p, stream);
    switch (tile) {
        //                                              BM   BN  WM WN ST
        case GT_160x256:
            if constexpr (MODE != MODE_TN) return launch_kernel<MODE, ACT, 160, 256, 1, 4, 3, PLANES>(p, stream);
            break;
        case GT_256x128: return launch_kernel<MODE, ACT, 256, 128, 4, 2, 3, PLANES>(p, stream);
        case GT_128x128: return launch_kernel<MODE, ACT, 128, 128, 2, 2, 2, PLANES>(p, stream);
        case GT_128x128_DEEP: return launch_kernel<MODE, ACT, 128, 128, 4, 2, 4, PLANES>(p, stream);
        case GT_64x128: return launch_kernel<MODE, ACT, 64, 128, 2, 2, 3, PLANES>(p, stream);
        case GT_MIXED:
            if constexpr (!PLANES) return launch_mixed<MODE, ACT>(p, wide, stream);
            break;
        default: break;
    }
    return launch_kernel<MODE, ACT, 256, 256, 2, 4, 2, PLANES>(p, stream);
}

}  // namespace

hipError_t launch_gated(const GatedProblem& p, hipStream_t stream) {
    GatedParams q{};
    q.A0 = p.A;
    q.B0 = p.B0;
    q.B1 = p.B1;
    q.C0 = p.H;
    q.G = p.G;
    q.U = p.U;
    q.kept = p.kept;
    q.M = (int)p.M;
    q.N = (int)p.N;
    q.K = (int)p.K;
    q.lda = q.ldb = (int)p.K;
    q.parts = q.splits = 1;
    q.direct = gated_direct(p.K);
    return p.act == BG_SILU ? launch_tile<MODE_GATED, BG_SILU, false>(q, p.tile, p.wide, stream)
                            : launch_tile<MODE_GATED, BG_GELU_TANH, false>(q, p.tile, p.wide, stream);
}

// Whether the product goes through planes, and its parameters.
static bool transposed_params(const TransposedProblem& p, GatedParams& q) {
    q = GatedParams{};
    q.A0 = p.A0;
    q.A1 = p.A1;
    q.B0 = p.B0;
    q.B1 = p.B1;
    q.M = (int)p.M;
    q.N = (int)p.N;
    q.K = (int)p.K;
    q.lda = (int)p.lda;
    q.ldb = (int)p.ldb;
    q.parts = (int)p.parts;
    q.splits = (int)p.splits;
    q.low = p.low;
    q.direct = gated_direct(p.lda) && gated_direct(p.ldb);
    const bool planes = p.splits > 1 || p.stacked > 1;
    q.C0 = planes ? static_cast<void*>(p.planes) : p.C0;
    q.C1 = planes ? static_cast<void*>(p.planes + (size_t)p.M * p.N) : p.C1;
    return planes;
}

static hipError_t launch_planes_sum(const TransposedProblem& p, hipStream_t stream) {
    // the rows of a plane that are one output's terms are planes of it themselves
    const int64_t count = (int64_t)(p.M / p.stacked) * p.N;
    hipLaunchKernelGGL(planes_sum_kernel, dim3((unsigned)((count + 1023) / 1024), p.tn ? (unsigned)p.parts : 1u), dim3(256), 0,
                       stream, p.planes, p.C0, p.C1, count, p.splits * (int)p.stacked);
    return hipGetLastError();
}

hipError_t launch_transposed(const TransposedProblem& p, hipStream_t stream) {
    GatedParams q;
    if (!transposed_params(p, q))
        return p.tn ? launch_tile<MODE_TN, 0, false>(q, p.tile, p.wide, stream) : launch_tile<MODE_NN, 0, false>(q, p.tile, p.wide, stream);
    const hipError_t e =
        p.tn ? launch_tile<MODE_TN, 0, true>(q, p.tile, p.wide, stream) : launch_tile<MODE_NN, 0, true>(q, p.tile, p.wide, stream);
    return e != hipSuccess ? e : launch_planes_sum(p, stream);
}

hipError_t launch_transposed_pair(const TransposedProblem& nn, const TransposedProblem& tn, hipStream_t stream) {
    GatedParams a, b;
    const bool pa = transposed_params(nn, a), pb = transposed_params(tn, b);
    constexpr int BM = 128, BN = 128;      // GT_128x128_DEEP
    for (GatedParams* q : {&a, &b}) {
        q->tiles_m = (q->M + BM - 1) / BM;
        q->tiles_n = (q->N + BN - 1) / BN;
    }
    const int ta = a.tiles_m * a.tiles_n, tb = b.tiles_m * b.tiles_n * b.parts, ba = ta * a.splits;
    auto k = pa ? (pb ? pair_kernel<BM, BN, 4, 2, 4, true, true> : pair_kernel<BM, BN, 4, 2, 4, true, false>)
                : (pb ? pair_kernel<BM, BN, 4, 2, 4, false, true> : pair_kernel<BM, BN, 4, 2, 4, false, false>);
    k<<<dim3((unsigned)(ba + tb * b.splits)), dim3(512), 0, stream>>>(a, b, ta, ba, tb);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && pa) e = launch_planes_sum(nn, stream);
    if (e == hipSuccess && pb) e = launch_planes_sum(tn, stream);
    return e;
}

hipError_t launch_aligned_copy(const AlignedCopy& p, hipStream_t stream) {
    int64_t chunks = 0;
    for (int i = 0; i < 2; ++i) {
        const int64_t c = (int64_t)p.rows[i] * (p.ld[i] / 8);
        chunks = c > chunks ? c : chunks;
    }
    const int64_t blocks = (chunks + 255) / 256;
    aligned_copy_kernel<<<dim3((unsigned)(blocks < 65536 ? blocks : 65536), 2), dim3(256), 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_gate_grad(const GateGradProblem& p, hipStream_t stream) {
    const int64_t chunks = (int64_t)p.M * (p.ld / 8);
    const int64_t blocks = (chunks + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    const bool f32 = p.kept == BG_F32;
    auto k = p.act == BG_SILU ? (f32 ? gate_grad_kernel<BG_SILU, true> : gate_grad_kernel<BG_SILU, false>)
                              : (f32 ? gate_grad_kernel<BG_GELU_TANH, true> : gate_grad_kernel<BG_GELU_TANH, false>);
    k<<<grid, dim3(256), 0, stream>>>(p, chunks);
    return hipGetLastError();
}

}  // namespace bg
