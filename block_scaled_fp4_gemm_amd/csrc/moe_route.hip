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
// rows, at most 256 of them up to 16.7 million rows and one per 65472 beyond;
// the first kernel counts per workgroup and expert, the second sums the counts
// of the workgroups before its own (each of them reads all: the square of their
// number), ranks the choices among its rows and writes the places; one more
// workgroup of it adds the statistics. All sums over rows are added in a fixed
// order.
//
// Traced, 256 experts, k = 8, BF16 logits, 65536 / 4510 rows: the first kernel
// 22.6 / 6.6 us (about 16 of the 22.6 are the choices' vector operations, the
// rest the loads at the top of each pass: 1.5 TB/s), the second 15.6 / 10.0
// (latencies: the sums, then places scattered over 2 MB), the gradient 19.4 /
// 7.4 (3.5 TB/s of logits, gradients and choices). With FP32 logits the first
// takes 31.2 and the gradient 33.1 (4 TB/s). One launch does 16 rows in 8.4.
#include <type_traits>

#include "bg_internal.hpp"

#pragma clang fp contract(off)

namespace bg {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// the same at any element: global memory takes unaligned accesses
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
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

// The words of a load that starts `past` elements early, moved down by as many;
// -infinity behind them. BF16: two elements a word.
template <bool F32, int W>
__device__ __forceinline__ void move_down(uint32_t (&w)[W], int past) {
    constexpr uint32_t FILL = F32 ? 0xFF800000u : 0xFF80FF80u;
    constexpr int PER = F32 ? 1 : 2;
    auto by = [&](int words, bool is) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = is ? (i + words < W ? w[i + words] : FILL) : w[i];
    };
    by(W, past >= W * PER);
    if constexpr (W == 4) by(2, past & (2 * PER));
    by(1, past & PER);
    if constexpr (!F32) {
        const uint32_t half = past & 1 ? 2 : 0;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = __builtin_amdgcn_alignbyte(i + 1 < W ? w[i + 1] : FILL, w[i], half);
    }
}

// A lane's VPL logits of row t; -infinity past E. VEC: rows start on whole
// loads and E is a multiple of a load's elements. Otherwise loads start at any
// element, and one that would end past the row starts earlier, so that it ends
// with it (24670 x 470, BF16, k = 3, with its gradient: a call 114 us element
// by element; now the kernels' 17.7, 15.8 and 18.8 us).
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
        constexpr int W = F32 || VPL % 8 == 0 ? 4 : 2, N = F32 ? W : 2 * W;      // words and elements a load
        if (E >= N) {
            uint32_t w[VPL / N][W];
#pragma unroll
            for (int i = 0; i < VPL / N; ++i) {
                const int64_t at = t * E + min(e0 + i * N, E - N);
                const void* q = F32 ? (const void*)(static_cast<const float*>(logits) + at)
                                    : (const void*)(static_cast<const uint16_t*>(logits) + at);
                if constexpr (W == 4) {
                    const u32x4 x = *static_cast<const u32x4_any*>(q);
                    w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
                } else {
                    const u32x2 x = *static_cast<const u32x2_any*>(q);
                    w[i][0] = x.x, w[i][1] = x.y;
                }
            }
#pragma unroll
            for (int i = 0; i < VPL / N; ++i) {
                move_down<F32>(w[i], max(e0 + (i + 1) * N - E, 0));
#pragma unroll
                for (int j = 0; j < N; ++j)
                    v[i * N + j] = __builtin_bit_cast(float, F32       ? w[i][j % W]
                                                             : j % 2 == 0 ? w[i][j / 2 % W] << 16
                                                                          : w[i][j / 2 % W] & 0xFFFF0000u);
            }
        } else {
            // every lane loads (past E, the row's last logit again): a branch
            // around each load would wait for one after the other
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int64_t at = t * E + min(e0 + i, E - 1);
                if constexpr (F32)
                    v[i] = static_cast<const float*>(logits)[at];
                else
                    v[i] = __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(logits)[at] << 16);
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = e0 + i < E ? v[i] : NEG_INF;
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

// Workspace of the two-kernel form: [blocks][E] sums of probabilities, [blocks]
// live rows, [blocks][E] counts (16 bits: a workgroup has fewer than 2^16 rows).
struct RouteWs {
    uint16_t* hist;
    float* psum;
    int32_t* live;
};

__device__ inline RouteWs split_ws(void* ws, uint64_t blocks, uint32_t E) {
    RouteWs w;
    w.psum = static_cast<float*>(ws);
    w.live = reinterpret_cast<int32_t*>(w.psum + blocks * E);
    w.hist = reinterpret_cast<uint16_t*>(w.live + (blocks + 3) / 4 * 4);
    return w;
}

// A barrier that orders LDS only: nothing waits for stores to memory.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

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
    lds_barrier();
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
    lds_barrier();
}

// Writes the places of `slots` choices that start at slot0, in turns of one
// choice a thread; id: the thread's first choice (-1: none). first[e] (LDS):
// the next place within expert e; cnt: LDS of NT / 64 times E words. Within a
// wave, the lanes of one expert find each other by a vote per bit of the
// index; the counts of the waves before give the rest of the rank.
template <int NT>
__device__ __forceinline__ void place(const int32_t* ids, int id, int slots, int slot0, int32_t* first, int32_t* cnt,
                                      int E, uint32_t k, int32_t* rows, int32_t* pos, int tid) {
    constexpr int W = NT / 64;
    const int lane = tid & 63, wave = tid >> 6;
    const int bits = 32 - __builtin_clz((uint32_t)(E - 1) | 1u);
    for (int s0 = 0; s0 < slots; s0 += NT) {
        const int s = s0 + tid;
        const int next = slots - s > NT ? ids[s + NT] : -1;
        for (int i = tid; i < W * E; i += NT) cnt[i] = 0;
        uint64_t same = __ballot(id >= 0);
        for (int b = 0; b < bits; ++b) {
            const bool one = (id >> b) & 1;
            const uint64_t ones = __ballot(one);
            same &= one ? ones : ~ones;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        lds_barrier();
        if (id >= 0 && rank == 0) cnt[wave * E + id] = __builtin_popcountll(same);
        lds_barrier();
        for (int e = tid; e < E; e += NT) {
            int c[W], at = first[e];
#pragma unroll
            for (int w = 0; w < W; ++w) c[w] = cnt[w * E + e];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                cnt[w * E + e] = at;
                at += c[w];
            }
            first[e] = at;
        }
        lds_barrier();
        if (s < slots) {
            int at = -1;
            if (id >= 0) {
                at = cnt[wave * E + id] + rank;
                rows[at] = (int32_t)((uint32_t)(slot0 + s) / k);     // T * k < 2^31
            }
            pos[slot0 + s] = at;
        }
        id = next;
        lds_barrier();
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
            ws.hist[(int64_t)blockIdx.x * E + e] = (uint16_t)hist[e];
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
        place<NT>(p.out.ids, tid < slots ? p.out.ids[tid] : -1, slots, 0, hist, cnt, E, p.k, p.out.rows, p.out.pos, tid);
    }
}

constexpr int PLACE_NT = 1024;
constexpr int PARTS = 4096;                      // partial sums of experts in LDS

// Over the first kernel's workgroups: off[e], the counts of expert e; for
// b >= 0, before[e], those of the workgroups before b; for b < 0, mean[e], the
// sums of probabilities.
template <int N>
__device__ __forceinline__ void sum_blocks(const RouteWs& ws, int E, int blocks, int b, int32_t* cnt,
                                           int32_t* off, int32_t* before, float* mean, int tid) {
    typedef int32_t Ints __attribute__((ext_vector_type(N)));
    typedef float Floats __attribute__((ext_vector_type(N)));
    typedef uint16_t Shorts __attribute__((ext_vector_type(N)));
    const int groups = (E + N - 1) / N;          // of N experts
    int wide = 16;                               // threads side by side: a power of two that holds them
    while (wide < groups) wide *= 2;
    const int segs = min(PLACE_NT / wide, PARTS / (wide * N)), g = tid & (wide - 1), seg = tid / wide;
    const bool in = g < groups && seg < segs;
    Ints all = {}, mine = {};
    Floats a = {};
    if (in) {
        const uint16_t* h = ws.hist + g * N;
        const float* f = ws.psum + g * N;
        // Batches of loads in flight together (past the end the batch's first
        // again). For b < 0 half of the threads add the counts, half the
        // probabilities; a single part does both.
        const int part = b < 0 && segs > 1 ? segs / 2 : segs;
        const bool counts = seg < part, probs = b < 0 && (seg >= part || segs == 1);
        constexpr int BATCH = 8;
        for (int q0 = seg; counts && q0 < blocks; q0 += BATCH * part) {
            Shorts c[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                c[u] = *reinterpret_cast<const Shorts*>(h + (int64_t)(q0 + u * part < blocks ? q0 + u * part : q0) * E);
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int q = q0 + u * part;
                const Ints x = __builtin_convertvector(c[u], Ints);
                all += q < blocks ? x : Ints{};
                mine += q < b ? x : Ints{};
            }
        }
        for (int q0 = seg >= part ? seg - part : seg; probs && q0 < blocks; q0 += BATCH * part) {
            Floats d[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                d[u] = *reinterpret_cast<const Floats*>(f + (int64_t)(q0 + u * part < blocks ? q0 + u * part : q0) * E);
#pragma unroll
            for (int u = 0; u < BATCH; ++u) a += q0 + u * part < blocks ? d[u] : Floats{};
        }
        *reinterpret_cast<Ints*>(cnt + seg * wide * N + g * N) = all;
        *reinterpret_cast<Ints*>(cnt + PARTS + seg * wide * N + g * N) = mine;
        *reinterpret_cast<Ints*>(cnt + 2 * PARTS + seg * wide * N + g * N) = __builtin_bit_cast(Ints, a);
    }
    lds_barrier();
    for (int e = tid; e < E; e += PLACE_NT) {
        int x = 0, y = 0;
        float z = 0.0f;
        // four parts' loads at a time; past the last part, that one again, times nothing
        for (int q0 = 0; q0 < segs; q0 += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool is = q0 + u < segs;
                const int at = min(q0 + u, segs - 1) * wide * N + e;
                x += is ? cnt[at] : 0;
                y += is ? cnt[PARTS + at] : 0;
                z += is ? __builtin_bit_cast(float, cnt[2 * PARTS + at]) : 0.0f;
            }
        }
        off[e] = x;
        before[e] = y;
        mean[e] = z;
    }
    lds_barrier();
}

// Workgroup 0: counts, offsets and statistics. Workgroup b + 1: the places of
// the rows that workgroup b of the first kernel owned. Two of them have to fit
// one compute unit (80 KB of LDS, 64 registers): of 257 that fill one each, the
// last would start when another has ended.
__global__ void __launch_bounds__(PLACE_NT, 8)
route_place_kernel(RouteProblem p, int rows_per_block, int blocks) {
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ int32_t before[kMaxExperts];
    __shared__ float mean[kMaxExperts];
    __shared__ __attribute__((aligned(16))) int32_t cnt[PLACE_NT / 64 * kMaxExperts];
    __shared__ int32_t live;
    const int tid = threadIdx.x, E = (int)p.E, b = (int)blockIdx.x - 1;
    const RouteWs ws = split_ws(p.ws, (uint64_t)blocks, p.E);
    // Sums over the workgroups of the first kernel. A thread takes four experts
    // (two or one, where rows are not whole loads of four) and every `segs`-th
    // workgroup, with its loads in flight at once; the partial sums meet in
    // LDS and are added in order.
    if (tid == 0) live = 0;
    const int64_t t0 = (int64_t)max(b, 0) * rows_per_block, t1 = min(t0 + rows_per_block, (int64_t)p.T);
    const int slots = b >= 0 ? (int)(t1 - t0) * (int)p.k : 0, slot0 = (int)(t0 * p.k);
    const int id = tid < slots ? p.out.ids[slot0 + tid] : -1;    // in flight meanwhile
    int n = b < 0 && tid < blocks ? ws.live[tid] : 0;
    if (E % 4 == 0)
        sum_blocks<4>(ws, E, blocks, b, cnt, off, before, mean, tid);
    else if (E % 2 == 0)
        sum_blocks<2>(ws, E, blocks, b, cnt, off, before, mean, tid);
    else
        sum_blocks<1>(ws, E, blocks, b, cnt, off, before, mean, tid);
    if (b < 0) {
        for (int q = tid + PLACE_NT; q < blocks; q += PLACE_NT) n += ws.live[q];
        if (n != 0) atomicAdd(&live, n);
        lds_barrier();
        n = live;
        for (int e = tid; e < E; e += PLACE_NT) {
            mean[e] = n > 0 ? mean[e] / (float)n : 0.0f;
            p.out.mean_probs[e] = mean[e];
            p.out.counts[e] = off[e];
        }
        lds_barrier();
        if (tid < 64) {
            const float l = balance(off, mean, E, p.k, n, tid);
            if (tid == 0) {
                *p.out.loss = l;
                *p.out.n_valid = n;
            }
        }
        lds_barrier();
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
    place<PLACE_NT>(p.out.ids + slot0, id, slots, slot0, off, cnt, E, p.k, p.out.rows, p.out.pos, tid);
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
    for (int i = 0; i < VPL; ++i) c[i] = scale * (float)p.counts[min(e0 + i, E - 1)];     // past E: times a zero
    float* const row = extra[tok];
#pragma unroll
    for (int i = 0; i < PITCH; i += 4) *reinterpret_cast<f32x4*>(row + gl * PITCH + i) = f32x4{};
    for (int64_t t = (int64_t)blockIdx.x * TOK + tok; t < (int64_t)p.T; t += (int64_t)gridDim.x * TOK) {
        // whole groups leave the loop together; all of a row's loads go out at once
        float v[VPL], top = NEG_INF;
        load_logits<F32, VPL, VEC>(p.logits, t, E, e0, v);
        const int first = p.ids[t * k];          // a live row has a first choice
        int id = -1;
        float w = 0.0f, g = 0.0f;
        if (gl < k && p.dweights != nullptr) {
            id = p.ids[t * k + gl];
            w = p.weights[t * k + gl];
            g = w * p.dweights[t * k + gl];
        }
        const bool live = first >= 0;
        if (id < 0 || id >= E || !live) id = -1, w = 0.0f, g = 0.0f;
        if (!__all(live)) {                      // what a row that is not live holds is not used
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = live ? v[i] : NEG_INF;
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
            // whole pieces at any element, and what is left of the last one by itself
            constexpr int W = F32 || VPL % 8 == 0 ? 4 : 2, N = F32 ? W : 2 * W;
            const int64_t at = t * E + e0;
#pragma unroll
            for (int i = 0; i < VPL; i += N) {
                uint32_t w[W];
#pragma unroll
                for (int j = 0; j < W; ++j)
                    w[j] = F32 ? __builtin_bit_cast(uint32_t, v[i + j]) : pack_bf16x2(v[i + 2 * j % N], v[i + (2 * j + 1) % N]);
                if (e0 + i + N <= E) {
                    void* q = F32 ? (void*)(static_cast<float*>(p.dlogits) + at + i)
                                  : (void*)(static_cast<uint16_t*>(p.dlogits) + at + i);
                    if constexpr (W == 4)
                        *static_cast<u32x4_any*>(q) = u32x4{w[0], w[1], w[2], w[3]};
                    else
                        *static_cast<u32x2_any*>(q) = u32x2{w[0], w[1]};
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        if (e0 + i + j >= E) continue;
                        if constexpr (F32)
                            static_cast<float*>(p.dlogits)[at + i + j] = v[i + j];
                        else
                            static_cast<__bf16*>(p.dlogits)[at + i + j] = (__bf16)v[i + j];
                    }
                }
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
            else route_kernel<F, G, V, VEC, 512, false><<<blocks, 512, 0, stream>>>(p, rows);
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
        const uint32_t blocks = passes < 1024 ? passes : 1024;
        if (p.type == BG_F32) route_backward_kernel<true, G, V, VEC><<<blocks, 256, 0, stream>>>(p);
        else route_backward_kernel<false, G, V, VEC><<<blocks, 256, 0, stream>>>(p);
    });
    return hipGetLastError();
}

}  // namespace bg
