// Expert routing on gfx950: softmax, top-k, per-expert counts, the dispatch
// order and the balance loss of a batch of router logits, and the gradient.
//
// A token is held by G lanes (16, 32 or 64), VPL consecutive experts each, so
// a row's maximum, sum and top-k are exchanges within G lanes and a wave works
// on 64 / G tokens at once.
//
// Top-k without sorting: every logit becomes a key that orders as the values
// do, with the complement of the expert's index below it, so keys are distinct
// and ties go to the lowest index.
//  - BF16: 16 bits of value and 16 of index in an unsigned word. With v the
//    keys and P the last key taken, d = P - 1 - v (modulo 2^32) is below P
//    exactly for the keys below P, so the next key is P - 1 - min(d): one
//    subtraction and half a three-way minimum per logit and choice, and
//    nothing has to be marked as taken.
//  - FP32: 32 bits of value and 10 of index as the fraction of a double
//    between 1 and 2: one double-precision maximum per logit and choice, and
//    one comparison and one select to mark what was taken. (64-bit integers
//    by the first method: 65536 x 256 in 45 us.)
//
// The dispatch order is that of (expert, row). Workgroups own consecutive
// rows, at most 256 of them; the first kernel counts per workgroup and expert,
// the second sums the counts of the workgroups before its own, ranks the
// choices among its rows and writes the places; one more workgroup of it adds
// the statistics. All sums over rows are added in a fixed order.
#include <type_traits>

#include "bg_internal.hpp"

#pragma clang fp contract(off)

namespace bg {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float NEG_INF = -__builtin_inff();

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    bf16x2 v = {(__bf16)lo, (__bf16)hi};   // v_cvt_pk_bf16_f32: round to nearest even
    return __builtin_bit_cast(uint32_t, v);
}

// exp(x - top): the difference and its product with log2 e round once each, so
// the relative error is at most about 2^-23 of |x - top| plus the exponential
// instruction's own.
__device__ __forceinline__ float exp_below(float x, float top) {
    return __builtin_amdgcn_exp2f((x - top) * 0x1.715476p+0f);
}

// Lane exchanges within groups of G lanes: every lane gets the total.
template <int STEP>
__device__ __forceinline__ uint32_t exchange(uint32_t w) {
    if constexpr (STEP < 16)
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0x120 + STEP, 0xF, 0xF, true);   // rotate within 16 lanes
    else
        return (uint32_t)__shfl_xor((int)w, STEP);
}
template <int STEP>
__device__ __forceinline__ float exchange(float v) {
    return __builtin_bit_cast(float, exchange<STEP>(__builtin_bit_cast(uint32_t, v)));
}
template <int STEP>
__device__ __forceinline__ double exchange(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, u32x2{exchange<STEP>(w.x), exchange<STEP>(w.y)});
}
template <int G, class T, class F>
__device__ __forceinline__ T reduce(T v, F f) {
    if constexpr (G > 32) v = f(v, exchange<32>(v));
    if constexpr (G > 16) v = f(v, exchange<16>(v));
    v = f(v, exchange<8>(v));
    v = f(v, exchange<4>(v));
    v = f(v, exchange<2>(v));
    v = f(v, exchange<1>(v));
    return v;
}
template <int G>
__device__ __forceinline__ float sum(float v) {
    return reduce<G>(v, [](float a, float b) { return a + b; });
}

// The larger of two positive doubles: the instruction alone (the library
// function first quiets signalling NaNs, which these never are).
__device__ __forceinline__ double larger(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// A lane's VPL logits of row t; -infinity past E. VEC: rows start on whole
// loads and E is a multiple of a load's elements.
template <bool F32, int VPL, bool VEC>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int e0, float (&v)[VPL]) {
    if constexpr (VEC && F32) {
        const float* p = static_cast<const float*>(logits) + t * E;
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
            f32x4 w = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
            if (e0 + i < E) w = *reinterpret_cast<const f32x4*>(p + e0 + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + j] = w[j];
        }
    } else if constexpr (VEC) {
        using Load = std::conditional_t<VPL % 8 == 0, u32x4, u32x2>;
        constexpr int N = sizeof(Load) / 2;
        const uint16_t* p = static_cast<const uint16_t*>(logits) + t * E;
#pragma unroll
        for (int i = 0; i < VPL; i += N) {
            Load w = (Load)(0xFF80FF80u);
            if (e0 + i < E) w = *reinterpret_cast<const Load*>(p + e0 + i);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                v[i + 2 * j] = __builtin_bit_cast(float, w[j] << 16);
                v[i + 2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (e0 + i >= E)
                v[i] = NEG_INF;
            else if constexpr (F32)
                v[i] = static_cast<const float*>(logits)[t * E + e0 + i];
            else
                v[i] = __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(logits)[t * E + e0 + i] << 16);
        }
    }
}

// Bits that order as the values do. -0 + 0 = +0: equal values tie. NaN counts
// as -infinity, the lowest of all: not to be chosen.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, fmaxf(v + 0.0f, NEG_INF));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t b) {
    return __builtin_bit_cast(float, b ^ ((b & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t CHOOSABLE = 0x00800000u;      // ordered_bits of what lies above -infinity

// The lane's keys, and the largest key of the group below the last one taken.
template <bool F32, int G, int VPL>
struct TopK;

template <int G, int VPL>
struct TopK<false, G, VPL> {
    uint32_t key[VPL], prev = ~0u;               // prev: the last key taken, less 1
    __device__ __forceinline__ void init(const float (&v)[VPL], int e0) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = (ordered_bits(v[i]) & 0xFFFF0000u) | (uint32_t)(0xFFFF - e0 - i);
    }
    // bits (ordered) and expert of the next choice
    __device__ __forceinline__ void next(uint32_t& bits, int& expert) {
        uint32_t d = prev - key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) d = min(d, prev - key[i]);
        d = reduce<G>(d, [](uint32_t a, uint32_t b) { return min(a, b); });
        const uint32_t got = prev - d;
        prev = got - 1;
        // a negative value's complement fills the low half with ones
        bits = (got & 0x80000000u) ? (got & 0xFFFF0000u) : (got | 0xFFFFu);
        expert = 0xFFFF - (int)(got & 0xFFFFu);
    }
};

template <int G, int VPL>
struct TopK<true, G, VPL> {
    double key[VPL];
    __device__ __forceinline__ void init(const float (&v)[VPL], int e0) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const uint32_t b = ordered_bits(v[i]);
            key[i] = __builtin_bit_cast(double, u32x2{(b << 10) | (uint32_t)(1023 - e0 - i), 0x3FF00000u | (b >> 22)});
        }
    }
    __device__ __forceinline__ void next(uint32_t& bits, int& expert) {
        double m = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = larger(m, key[i]);
        m = reduce<G>(m, [](double a, double b) { return larger(a, b); });
        const u32x2 w = __builtin_bit_cast(u32x2, m);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            u32x2 k = __builtin_bit_cast(u32x2, key[i]);
            k.y = key[i] == m ? 0u : k.y;        // taken: below 1
            key[i] = __builtin_bit_cast(double, k);
        }
        bits = (w.y << 22) | (w.x >> 10);
        if (w.y < 0x3FF00000u) bits = 0;         // nothing left
        expert = 1023 - (int)(w.x & 1023u);
    }
};

// Workspace of the two-kernel form: [blocks][E] counts, [blocks][E] sums of
// probabilities, [blocks] live rows.
struct RouteWs {
    int32_t* hist;
    float* psum;
    int32_t* live;
};

__device__ inline RouteWs split_ws(void* ws, uint64_t blocks, uint32_t E) {
    RouteWs w;
    w.hist = static_cast<int32_t*>(ws);
    w.psum = reinterpret_cast<float*>(w.hist + blocks * E);
    w.live = reinterpret_cast<int32_t*>(w.psum + blocks * E);
    return w;
}

// Exclusive prefix over the E counts in LDS, in place: counts -> offsets
// (E + 1 values). At least 256 threads call it; E <= 1024, four per thread.
__device__ __forceinline__ void scan_counts(int32_t* c, int E, int tid) {
    __shared__ int32_t part[4];
    int v[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = tid * 4 + i < E ? c[tid * 4 + i] : 0;
        mine += v[i];
    }
    int upto = mine;
    const int lane = tid & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63 && tid < 256) part[tid >> 6] = upto;
    __syncthreads();
    if (tid < 256) {
        int base = upto - mine;
        for (int w = 0; w < (tid >> 6); ++w) base += part[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (tid * 4 + i <= E) c[tid * 4 + i] = base;
            base += v[i];
        }
        if (tid == 255 && E == 1024) c[E] = base;
    }
    __syncthreads();
}

// Writes the places of `slots` choices that start at slot0, in turns of one
// choice a thread. first[e] (LDS): the next place within expert e; cnt: LDS of
// NT / 64 times E words. Within a wave, the lanes of one expert find each
// other by a vote per bit of the index; the counts of the waves before give
// the rest of the rank.
template <int NT>
__device__ __forceinline__ void place(const int32_t* ids, int64_t slots, int64_t slot0, int32_t* first, int32_t* cnt,
                                      int E, uint32_t k, int32_t* rows, int32_t* pos, int tid) {
    const int lane = tid & 63, wave = tid >> 6;
    const int bits = 32 - __builtin_clz((uint32_t)(E - 1) | 1u);
    for (int64_t s0 = 0; s0 < slots; s0 += NT) {
        for (int i = tid; i < NT / 64 * E; i += NT) cnt[i] = 0;
        __syncthreads();
        const int64_t s = s0 + tid;
        const int id = s < slots ? ids[s] : -1;
        uint64_t same = __ballot(id >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint64_t ones = __ballot((id >> b) & 1);
            same &= ((id >> b) & 1) ? ones : ~ones;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        if (id >= 0 && rank == 0) cnt[wave * E + id] = __builtin_popcountll(same);
        __syncthreads();
        for (int e = tid; e < E; e += NT) {
            int at = first[e];
#pragma unroll
            for (int w = 0; w < NT / 64; ++w) {
                const int c = cnt[w * E + e];
                cnt[w * E + e] = at;
                at += c;
            }
            first[e] = at;
        }
        __syncthreads();
        if (s < slots) {
            int at = -1;
            if (id >= 0) {
                at = cnt[wave * E + id] + rank;
                rows[at] = (int32_t)((uint64_t)(slot0 + s) / k);
            }
            pos[slot0 + s] = at;
        }
        __syncthreads();
    }
}

// loss from the counts and mean probabilities (LDS), one wave, lanes in order
__device__ __forceinline__ float balance(const int32_t* counts, const float* mean, int E, uint32_t k, int n, int lane) {
    float s = 0.0f;
    for (int e = lane; e < E; e += 64) s += (float)counts[e] * mean[e];
    s = sum<64>(s);
    return n > 0 ? s * (float)E / ((float)k * (float)n) : 0.0f;
}

// ONE: the whole batch in one workgroup and launch.
template <bool F32, int G, int VPL, bool VEC, int NT, bool ONE>
__global__ void __launch_bounds__(NT)
route_kernel(RouteProblem p, int rows_per_block) {
    constexpr int TOK = NT / G;                  // tokens at once
    constexpr int W = NT / 64;
    __shared__ int32_t hist[kMaxExperts + 1];
    __shared__ float psum[W][G * VPL];
    __shared__ int32_t live_rows[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int gl = tid % G, tok = tid / G, e0 = gl * VPL;
    const int E = (int)p.E, k = (int)p.k;
    for (int e = tid; e < E; e += NT) hist[e] = 0;
    __syncthreads();

    float acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
    int live_count = 0;
    const int64_t t0 = (int64_t)blockIdx.x * rows_per_block;
    const int64_t t1 = min(t0 + rows_per_block, (int64_t)p.T);
    for (int64_t tb = t0; tb < t1; tb += TOK) {
        const int64_t t = tb + tok;
        const bool in = t < t1;
        float v[VPL];
        if (in && (p.valid == nullptr || p.valid[t] != 0)) {
            load_logits<F32, VPL, VEC>(p.logits, t, E, e0, v);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = NEG_INF;
        }
        TopK<F32, G, VPL> best;
        best.init(v, e0);
        uint32_t bits, mine = 0;
        int expert, my_expert = 0;
        best.next(bits, expert);
        const bool live = bits >= CHOOSABLE;
        const float top = live ? ordered_value(bits) : 0.0f;
        if (gl == 0) mine = bits, my_expert = expert;
        for (int j = 1; j < k; ++j) {
            best.next(bits, expert);
            if (gl == j) mine = bits, my_expert = expert;
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = exp_below(v[i], top);
            s += v[i];
        }
        s = sum<G>(s);
        const float inv = live ? 1.0f / s : 0.0f;
        if (!__all(live)) {                      // a row that is not live may hold NaN
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = live ? v[i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] = __builtin_fmaf(v[i], inv, acc[i]);
        live_count += live && gl == 0;

        const bool chosen = gl < k && mine >= CHOOSABLE;
        float w = chosen ? exp_below(ordered_value(mine), top) : 0.0f;
        const float ws = sum<G>(w);
        w = p.normalize ? w / ws : w * inv;
        if (s != s) w = s;                       // a NaN or an infinity in the row
        if (in && gl < k) {
            p.out.ids[t * k + gl] = chosen ? my_expert : -1;
            p.out.weights[t * k + gl] = chosen ? w : 0.0f;
            if (chosen) atomicAdd(&hist[my_expert], 1);      // whole numbers: any order, one sum
        }
    }

    // probabilities: over the tokens of a wave, then over the waves, in order
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float a = acc[i];
        if constexpr (G <= 16) a += exchange<16>(a);
        if constexpr (G <= 32) a += exchange<32>(a);
        if (lane < G) psum[wave][e0 + i] = a;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) live_count += __shfl_xor(live_count, d);
    if (lane == 0) live_rows[wave] = live_count;
    __syncthreads();
    int n = 0;
    for (int w = 0; w < W; ++w) n += live_rows[w];
    if constexpr (!ONE) {
        const RouteWs ws = split_ws(p.ws, gridDim.x, p.E);
        for (int e = tid; e < E; e += NT) {
            float a = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) a += psum[w][e];
            ws.hist[(int64_t)blockIdx.x * E + e] = hist[e];
            ws.psum[(int64_t)blockIdx.x * E + e] = a;
        }
        if (tid == 0) ws.live[blockIdx.x] = n;
    } else {
        __shared__ int32_t cnt[W * kMaxExperts];
        for (int e = tid; e < E; e += NT) {
            float a = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) a += psum[w][e];
            a = n > 0 ? a / (float)n : 0.0f;
            p.out.mean_probs[e] = a;
            p.out.counts[e] = hist[e];
            psum[0][e] = a;
        }
        __syncthreads();                         // the ids written above are visible to the workgroup too
        if (wave == 0) {
            const float l = balance(hist, psum[0], E, p.k, n, lane);
            if (lane == 0) {
                *p.out.loss = l;
                *p.out.n_valid = n;
            }
        }
        __syncthreads();
        scan_counts(hist, E, tid);
        for (int e = tid; e <= E; e += NT) p.out.offsets[e] = hist[e];
        const int slots = (int)p.T * k;
        for (int i = hist[E] + tid; i < slots; i += NT) p.out.rows[i] = -1;
        __syncthreads();
        place<NT>(p.out.ids, slots, 0, hist, cnt, E, p.k, p.out.rows, p.out.pos, tid);
    }
}

// Workgroup b < blocks: the places of the rows that workgroup b of the first
// kernel owned. The last workgroup: counts, offsets and statistics.
constexpr int PLACE_NT = 1024;
constexpr int STRETCHES = 16;
__global__ void __launch_bounds__(PLACE_NT)
route_place_kernel(RouteProblem p, int rows_per_block, int blocks) {
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ int32_t before[kMaxExperts];
    __shared__ float mean[kMaxExperts];
    __shared__ int32_t cnt[PLACE_NT / 64 * kMaxExperts];
    __shared__ float fsum[STRETCHES * 64];
    __shared__ int32_t live;
    const int tid = threadIdx.x, E = (int)p.E, b = (int)blockIdx.x;
    const RouteWs ws = split_ws(p.ws, (uint64_t)blocks, p.E);
    // Sums over the workgroups of the first kernel: thread (expert, stretch of
    // workgroups), 64 experts and 16 stretches at a time; the stretches'
    // sums meet in LDS and are added in order.
    const int el = tid & 63, seg = tid >> 6;
    const int per = (blocks + STRETCHES - 1) / STRETCHES, b0 = min(seg * per, blocks), b1 = min(b0 + per, blocks);
    if (tid == 0) live = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + el;
        int all = 0, mine = 0;
        float a = 0.0f;
        if (e < E) {
            if (b < blocks) {
#pragma unroll 8
                for (int q = b0; q < b1; ++q) {
                    const int c = ws.hist[(int64_t)q * E + e];
                    all += c;
                    mine += q < b ? c : 0;
                }
            } else {
#pragma unroll 8
                for (int q = b0; q < b1; ++q) {
                    all += ws.hist[(int64_t)q * E + e];
                    a += ws.psum[(int64_t)q * E + e];
                }
            }
        }
        cnt[seg * 64 + el] = all;
        cnt[(STRETCHES + seg) * 64 + el] = mine;
        fsum[seg * 64 + el] = a;
        __syncthreads();
        if (tid < 64 && e < E) {
            all = mine = 0;
            a = 0.0f;
#pragma unroll
            for (int q = 0; q < STRETCHES; ++q) {
                all += cnt[q * 64 + el];
                mine += cnt[(STRETCHES + q) * 64 + el];
                a += fsum[q * 64 + el];
            }
            off[e] = all;
            before[e] = mine;
            mean[e] = a;
        }
        __syncthreads();
    }
    if (b == blocks) {
        int n = 0;
        for (int q = tid; q < blocks; q += PLACE_NT) n += ws.live[q];
        if (n != 0) atomicAdd(&live, n);
        __syncthreads();
        n = live;
        for (int e = tid; e < E; e += PLACE_NT) {
            mean[e] = n > 0 ? mean[e] / (float)n : 0.0f;
            p.out.mean_probs[e] = mean[e];
            p.out.counts[e] = off[e];
        }
        __syncthreads();
        if (tid < 64) {
            const float l = balance(off, mean, E, p.k, n, tid);
            if (tid == 0) {
                *p.out.loss = l;
                *p.out.n_valid = n;
            }
        }
        __syncthreads();
        scan_counts(off, E, tid);
        for (int e = tid; e <= E; e += PLACE_NT) p.out.offsets[e] = off[e];
        return;
    }
    scan_counts(off, E, tid);
    // places behind the last choice, shared out over the workgroups
    const int64_t all = (int64_t)p.T * p.k;
    for (int64_t i = off[E] + (int64_t)b * PLACE_NT + tid; i < all; i += (int64_t)blocks * PLACE_NT) p.out.rows[i] = -1;
    for (int e = tid; e < E; e += PLACE_NT) off[e] += before[e];
    __syncthreads();
    const int64_t t0 = (int64_t)b * rows_per_block, t1 = min(t0 + rows_per_block, (int64_t)p.T);
    place<PLACE_NT>(p.out.ids + t0 * p.k, (t1 - t0) * p.k, t0 * p.k, off, cnt, E, p.k, p.out.rows, p.out.pos, tid);
}

// Gradient: the row's probabilities again from its logits, the loss's part in
// registers; the weights' part goes through a row of LDS that is zero but for
// the choices: the lanes that hold them write them, every lane reads its
// experts', and the choices are zeroed again. All within one wave, whose LDS
// operations stay in order.
template <bool F32, int G, int VPL, bool VEC>
__global__ void __launch_bounds__(256)
route_backward_kernel(RouteBackwardProblem p) {
    constexpr int NT = 256, TOK = NT / G, PITCH = VPL + 4;       // a lane's experts: 16-byte aligned, banks spread
    __shared__ __attribute__((aligned(16))) float extra[TOK][G * PITCH];
    const int tid = threadIdx.x, gl = tid % G, tok = tid / G, e0 = gl * VPL;
    const int E = (int)p.E, k = (int)p.k;
    const float n = (float)*p.n_valid;
    const float scale = p.dloss != nullptr && n > 0.0f ? *p.dloss * (float)E / ((float)k * n) / n : 0.0f;
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = e0 + i < E ? scale * (float)p.counts[e0 + i] : 0.0f;
    float* const row = extra[tok];
#pragma unroll
    for (int i = 0; i < PITCH; i += 4) *reinterpret_cast<f32x4*>(row + gl * PITCH + i) = f32x4{};
    for (int64_t tb = (int64_t)blockIdx.x * TOK; tb < (int64_t)p.T; tb += (int64_t)gridDim.x * TOK) {
        const int64_t t = tb + tok;
        if (t >= (int64_t)p.T) break;            // whole groups leave together
        // a live row has a first choice
        const bool live = p.ids[t * k] >= 0;
        float v[VPL], top = NEG_INF;
        if (live) {
            load_logits<F32, VPL, VEC>(p.logits, t, E, e0, v);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = NEG_INF;
        }
        int id = -1;
        float w = 0.0f, g = 0.0f;
        if (live && gl < k && p.dweights != nullptr) {
            id = p.ids[t * k + gl];
            if (id >= 0 && id < E) {
                w = p.weights[t * k + gl];
                g = w * p.dweights[t * k + gl];
            } else {
                id = -1;
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) top = fmaxf(top, v[i]);
        top = reduce<G>(top, [](float a, float b) { return fmaxf(a, b); });
        if (!live) top = 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = exp_below(v[i], top);
            s += v[i];
        }
        s = sum<G>(s);
        const float inv = live ? 1.0f / s : 0.0f;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] *= inv;
            dot = __builtin_fmaf(v[i], c[i], dot);
        }
        dot = sum<G>(dot);
        const float inner = sum<G>(g);
        if (p.normalize)
            g -= w * inner;
        else
            dot += inner;
        const int at = id / VPL * PITCH + id % VPL;
        if (id >= 0) row[at] = g;                // a row's choices are distinct
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(row + gl * PITCH + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + j] = __builtin_fmaf(v[i + j], c[i + j] - dot, x[j]);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        if (id >= 0) row[at] = 0.0f;
        if constexpr (VEC && F32) {
            float* o = static_cast<float*>(p.dlogits) + t * E + e0;
#pragma unroll
            for (int i = 0; i < VPL; i += 4)
                if (e0 + i < E) *reinterpret_cast<f32x4*>(o + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
        } else if constexpr (VEC) {
            using Store = std::conditional_t<VPL % 8 == 0, u32x4, u32x2>;
            constexpr int N = sizeof(Store) / 2;
            uint16_t* o = static_cast<uint16_t*>(p.dlogits) + t * E + e0;
#pragma unroll
            for (int i = 0; i < VPL; i += N) {
                Store x;
#pragma unroll
                for (int j = 0; j < N / 2; ++j) x[j] = pack_bf16x2(v[i + 2 * j], v[i + 2 * j + 1]);
                if (e0 + i < E) *reinterpret_cast<Store*>(o + i) = x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (e0 + i >= E) continue;
                if constexpr (F32)
                    static_cast<float*>(p.dlogits)[t * E + e0 + i] = v[i];
                else
                    static_cast<__bf16*>(p.dlogits)[t * E + e0 + i] = (__bf16)v[i];
            }
        }
    }
}

// Calls f with the smallest group that holds E experts (G, VPL), and whether
// rows start on whole loads and E is a multiple of them.
template <class F>
void by_experts(int type, uint32_t E, F&& f) {
    using std::integral_constant;
    auto vec = [&](auto g, auto v) {
        // a load's elements: 16 bytes, or 8 where a lane holds four BF16
        const uint32_t n = type == BG_F32 || decltype(v)::value == 4 ? 4 : 8;
        if (E % n == 0)
            f(g, v, std::true_type{});
        else
            f(g, v, std::false_type{});
    };
    if (E <= 64) vec(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (E <= 128) vec(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    else if (E <= 256) vec(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    else if (E <= 512) vec(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    else vec(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_moe_route(const RouteProblem& p, hipStream_t stream) {
    const uint32_t blocks = route_blocks(p.T);
    const bool one = p.T <= kRouteOneBlock, wide = p.T > kRouteWide;
    const int rows = one ? (int)kRouteOneBlock : (int)route_rows_per_block(p.T);
    by_experts(p.type, p.E, [&](auto g, auto v, auto vec) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        constexpr bool VEC = decltype(vec)::value;
        auto run = [&](auto f32) {
            constexpr bool F = decltype(f32)::value;
            if (one) route_kernel<F, G, V, VEC, 512, true><<<1, 512, 0, stream>>>(p, rows);
            else if (wide) route_kernel<F, G, V, VEC, 1024, false><<<blocks, 1024, 0, stream>>>(p, rows);
            else route_kernel<F, G, V, VEC, 256, false><<<blocks, 256, 0, stream>>>(p, rows);
        };
        if (p.type == BG_F32) run(std::true_type{});
        else run(std::false_type{});
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || one) return e;
    route_place_kernel<<<blocks + 1, PLACE_NT, 0, stream>>>(p, rows, (int)blocks);
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const RouteBackwardProblem& p, hipStream_t stream) {
    by_experts(p.type, p.E, [&](auto g, auto v, auto vec) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        constexpr bool VEC = decltype(vec)::value;
        const uint32_t passes = (p.T + 256 / G - 1) / (256 / G);
        const uint32_t blocks = passes < 2048 ? passes : 2048;
        if (p.type == BG_F32) route_backward_kernel<true, G, V, VEC><<<blocks, 256, 0, stream>>>(p);
        else route_backward_kernel<false, G, V, VEC><<<blocks, 256, 0, stream>>>(p);
    });
    return hipGetLastError();
}

}  // namespace bg
