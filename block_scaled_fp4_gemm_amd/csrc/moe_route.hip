// Expert routing on gfx950: softmax, top-k, per-expert counts, the dispatch
// order and the balance loss of a batch of router logits, and the gradient.
//
// A token is held by G lanes (16, 32 or 64), VPL consecutive experts each, so
// a row's maximum, sum and top-k are exchanges within G lanes and a wave works
// on 64 / G tokens at once.
//
// Top-k without sorting: every logit becomes an unsigned key that orders as
// the values do, its low part the complement of the expert's index, so keys
// are distinct and ties go to the lowest index. With v the keys and P the last
// key taken, d = P - 1 - v (modulo 2^n) is below P exactly for the keys below
// P, so the next key is P - 1 - min(d): one subtraction and one minimum per
// logit and choice, and nothing has to be marked as taken. Key 0 stands for
// what may not be chosen (-infinity, NaN, positions past E).
//
// The dispatch order is that of (expert, row). Workgroups own consecutive
// rows; the first kernel counts per workgroup and expert, the second turns the
// counts into every workgroup's first place within each expert, the third
// ranks the choices inside its workgroup and writes the places. All sums over
// rows are added in a fixed order.
#include <type_traits>

#include "bg_internal.hpp"

#pragma clang fp contract(off)

namespace bg {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int NT = 256;
constexpr float NEG_INF = -__builtin_inff();

// exp(x) for x <= 0 (and NaN): 2^(x log2 e) with the product's rounding error
// carried, so the relative error stays near that of the exponential
// instruction itself for large |x| too. Below -104, exp is under half of the
// smallest FP32 subnormal.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float L = 0x1.715476p+0f, LL = 0x1.4ae0bep-26f;   // log2(e) in two parts
    const float t = x * L;
    const float r = __builtin_fmaf(x, LL, __builtin_fmaf(x, L, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    const float y = __builtin_fmaf(e, r * 0x1.62e43p-1f, e);
    return x < -104.0f ? 0.0f : y;
}

// Lane exchanges within groups of G lanes: every lane gets the total.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}
template <class T, int STEP>
__device__ __forceinline__ T exchange(T v) {
    auto one = [](uint32_t w) -> uint32_t {
        if constexpr (STEP < 16)
            return dpp<0x120 + STEP>(w);      // rotate by STEP within 16 lanes
        else
            return (uint32_t)__shfl_xor((int)w, STEP);
    };
    if constexpr (sizeof(T) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(T, ((uint64_t)one((uint32_t)(b >> 32)) << 32) | one((uint32_t)b));
    } else {
        return __builtin_bit_cast(T, one(__builtin_bit_cast(uint32_t, v)));
    }
}
template <int G, class T, class F>
__device__ __forceinline__ T reduce(T v, F f) {
    if constexpr (G > 32) v = f(v, exchange<T, 32>(v));
    if constexpr (G > 16) v = f(v, exchange<T, 16>(v));
    v = f(v, exchange<T, 8>(v));
    v = f(v, exchange<T, 4>(v));
    v = f(v, exchange<T, 2>(v));
    v = f(v, exchange<T, 1>(v));
    return v;
}
template <int G>
__device__ __forceinline__ float sum(float v) {
    return reduce<G>(v, [](float a, float b) { return a + b; });
}

// A lane's VPL logits of row t; -infinity past E.
template <bool F32, int VPL>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int e0, bool vec, float (&v)[VPL]) {
    if (vec) {   // rows start on 16 bytes and E is a multiple of a load's elements
        if constexpr (F32) {
            const float* p = static_cast<const float*>(logits) + t * E;
#pragma unroll
            for (int i = 0; i < VPL; i += 4) {
                f32x4 w = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
                if (e0 + i < E) w = *reinterpret_cast<const f32x4*>(p + e0 + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i + j] = w[j];
            }
        } else if constexpr (VPL % 8 == 0) {
            const uint16_t* p = static_cast<const uint16_t*>(logits) + t * E;
#pragma unroll
            for (int i = 0; i < VPL; i += 8) {
                u32x4 w = {0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
                if (e0 + i < E) w = *reinterpret_cast<const u32x4*>(p + e0 + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[i + 2 * j] = __builtin_bit_cast(float, w[j] << 16);
                    v[i + 2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
                }
            }
        }
        if (F32 || VPL % 8 == 0) return;
    }
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

// Keys. BF16: 16 bits of value, 16 of complemented index in 32 bits; FP32: 32 and 32.
template <bool F32>
using Key = std::conditional_t<F32, uint64_t, uint32_t>;

template <bool F32>
__device__ __forceinline__ Key<F32> key_of(float v, int e) {
    if (!(v > NEG_INF)) return 0;                       // -infinity, NaN
    uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);   // -0 + 0 = +0: equal values tie
    b ^= (uint32_t)((int32_t)b >> 31) | 0x80000000u;
    if constexpr (F32)
        return ((uint64_t)b << 32) | (uint32_t)~e;
    else
        return (b & 0xFFFF0000u) | (uint32_t)(0xFFFF - e);
}
template <bool F32>
__device__ __forceinline__ int key_expert(Key<F32> k) {
    if constexpr (F32)
        return (int)~(uint32_t)k;
    else
        return 0xFFFF - (int)(k & 0xFFFFu);
}
template <bool F32>
__device__ __forceinline__ float key_value(Key<F32> k) {
    uint32_t b;
    if constexpr (F32)
        b = (uint32_t)(k >> 32);
    else
        // a negative value's complement fills the low half with ones
        b = (k & 0x80000000u) ? (k & 0xFFFF0000u) : (k | 0xFFFFu);
    b ^= (b & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu;
    return __builtin_bit_cast(float, b);
}

// Workspace of the three-kernel form: [blocks][E] counts, [blocks][E] sums of
// probabilities, [blocks] live rows.
struct RouteWs {
    int32_t* hist;
    float* psum;
    int32_t* live;
};

__host__ __device__ inline RouteWs split_ws(void* ws, uint64_t blocks, uint32_t E) {
    RouteWs w;
    w.hist = static_cast<int32_t*>(ws);
    w.psum = reinterpret_cast<float*>(w.hist + blocks * E);
    w.live = reinterpret_cast<int32_t*>(w.psum + blocks * E);
    return w;
}

// Exclusive prefix over the E counts in LDS, in place: counts -> offsets
// (E + 1 values). All NT threads; E <= 1024, four per thread.
__device__ __forceinline__ void scan_counts(int32_t* c, int E, int tid) {
    __shared__ int32_t part[NT / 64];
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
    if (lane == 63) part[tid >> 6] = upto;
    __syncthreads();
    int base = upto - mine;
    for (int w = 0; w < (tid >> 6); ++w) base += part[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (tid * 4 + i <= E) c[tid * 4 + i] = base;
        base += v[i];
    }
    if (tid == NT - 1 && E == NT * 4) c[E] = base;
    __syncthreads();
}

// Writes the places of a workgroup's choices. ids: its slots in LDS (-1: none),
// first[e]: its first place within expert e (LDS).
__device__ __forceinline__ void place(const int32_t* ids, int slots, const int32_t* first, int64_t slot0, uint32_t k,
                                      int32_t* rows, int32_t* pos, int tid) {
    for (int s = tid; s < slots; s += NT) {
        const int id = ids[s];
        int at = -1;
        if (id >= 0) {
            int rank = 0;
            for (int q = 0; q < s; ++q) rank += ids[q] == id;
            at = first[id] + rank;
            rows[at] = (int32_t)((slot0 + s) / k);
        }
        pos[slot0 + s] = at;
    }
}

// loss from the counts (LDS) and mean probabilities, one wave, lanes in order.
__device__ __forceinline__ float balance(const int32_t* counts, const float* mean, int E, uint32_t k, int n, int lane) {
    float s = 0.0f;
    for (int e = lane; e < E; e += 64) s += (float)counts[e] * mean[e];
    s = sum<64>(s);
    return n > 0 ? s * (float)E / ((float)k * (float)n) : 0.0f;
}

template <bool F32, int G, int VPL, bool ONE>
__global__ void __launch_bounds__(NT)
route_kernel(RouteProblem p, int rows_per_block, bool vec) {
    constexpr int TOK = NT / G;                  // tokens at once
    constexpr int W = NT / 64;
    __shared__ int32_t hist[kMaxExperts + 1];
    __shared__ float psum[W][G * VPL];
    __shared__ int32_t slot_ids[ONE ? kRouteOneBlock * kMaxTopK : 1];
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
        bool live = in && (p.valid == nullptr || p.valid[t] != 0);
        float v[VPL];
        if (live) {
            load_logits<F32, VPL>(p.logits, t, E, e0, vec, v);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = NEG_INF;
        }
        Key<F32> key[VPL];
        float top = NEG_INF;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            key[i] = key_of<F32>(v[i], e0 + i);
            top = fmaxf(top, v[i]);
        }
        top = reduce<G>(top, [](float a, float b) { return fmaxf(a, b); });
        live = top > NEG_INF;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = live ? exp_neg(v[i] - top) : 0.0f;
            s += v[i];
        }
        s = sum<G>(s);
        const float inv = live ? 1.0f / s : 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += v[i] * inv;
        live_count += live && gl == 0;

        Key<F32> prev = ~(Key<F32>)0, mine = 0;      // the last key taken, less 1
        for (int j = 0; j < k; ++j) {
            Key<F32> d = prev - key[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) d = min(d, (Key<F32>)(prev - key[i]));
            d = reduce<G>(d, [](Key<F32> a, Key<F32> b) { return min(a, b); });
            const Key<F32> got = prev - d;
            if (gl == j) mine = got;
            prev = got != 0 ? got - 1 : 0;
        }
        const bool chosen = mine != 0 && gl < k;
        float w = chosen ? exp_neg(key_value<F32>(mine) - top) : 0.0f;
        const float ws = sum<G>(w);
        w = p.normalize ? w / ws : w * inv;
        if (s != s) w = s;                           // a NaN or an infinity in the row
        if (!chosen) w = 0.0f;
        const int id = chosen ? key_expert<F32>(mine) : -1;
        if (in && gl < k) {
            p.out.ids[t * k + gl] = id;
            p.out.weights[t * k + gl] = w;
            if constexpr (ONE) slot_ids[(t - t0) * k + gl] = id;
            if (id >= 0) atomicAdd(&hist[id], 1);    // whole numbers: any order, one sum
        }
    }

    // probabilities: over the tokens of a wave, then over the waves, in order
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float a = acc[i];
        if constexpr (G <= 16) a += exchange<float, 16>(a);
        if constexpr (G <= 32) a += exchange<float, 32>(a);
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
            for (int w = 0; w < W; ++w) a += psum[w][e];
            ws.hist[(int64_t)blockIdx.x * E + e] = hist[e];
            ws.psum[(int64_t)blockIdx.x * E + e] = a;
        }
        if (tid == 0) ws.live[blockIdx.x] = n;
    } else {
        for (int e = tid; e < E; e += NT) {
            float a = 0.0f;
            for (int w = 0; w < W; ++w) a += psum[w][e];
            a = n > 0 ? a / (float)n : 0.0f;
            p.out.mean_probs[e] = a;
            p.out.counts[e] = hist[e];
            psum[0][e] = a;
        }
        __syncthreads();
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
        place(slot_ids, slots, hist, 0, p.k, p.out.rows, p.out.pos, tid);
    }
}

// Sixteen experts per workgroup, sixteen stretches of workgroups each: totals
// and, in place, every workgroup's first place within the expert.
__global__ void __launch_bounds__(NT)
route_scan_kernel(RouteProblem p, int blocks) {
    __shared__ int32_t cs[16][17];
    __shared__ float ps[16][17];
    __shared__ int32_t live[NT / 64];
    const int tid = threadIdx.x, el = tid & 15, seg = tid >> 4;
    const int e = blockIdx.x * 16 + el;
    const RouteWs ws = split_ws(p.ws, (uint64_t)blocks, p.E);
    int n = 0;
    for (int b = tid; b < blocks; b += NT) n += ws.live[b];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
    if ((tid & 63) == 0) live[tid >> 6] = n;
    const int per = (blocks + 15) / 16, b0 = min(seg * per, blocks), b1 = min(b0 + per, blocks);
    int c = 0;
    float a = 0.0f;
    if (e < (int)p.E)
        for (int b = b0; b < b1; ++b) {
            c += ws.hist[(int64_t)b * p.E + e];
            a += ws.psum[(int64_t)b * p.E + e];
        }
    cs[seg][el] = c;
    ps[seg][el] = a;
    __syncthreads();
    n = live[0] + live[1] + live[2] + live[3];
    if (e < (int)p.E) {
        int base = 0;
        for (int s = 0; s < seg; ++s) base += cs[s][el];
        for (int b = b0; b < b1; ++b) {
            const int64_t at = (int64_t)b * p.E + e;
            const int h = ws.hist[at];
            ws.hist[at] = base;
            base += h;
        }
        if (seg == 15) p.out.counts[e] = base;
        if (seg == 0) {
            float t = 0.0f;
            for (int s = 0; s < 16; ++s) t += ps[s][el];
            p.out.mean_probs[e] = n > 0 ? t / (float)n : 0.0f;
        }
    }
    if (blockIdx.x == 0 && tid == 0) *p.out.n_valid = n;
}

__global__ void __launch_bounds__(NT)
route_place_kernel(RouteProblem p, int rows_per_block) {
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ int32_t slot_ids[128 * kMaxTopK];
    const int tid = threadIdx.x, E = (int)p.E, k = (int)p.k;
    for (int e = tid; e < E; e += NT) off[e] = p.out.counts[e];
    const int64_t t0 = (int64_t)blockIdx.x * rows_per_block, t1 = min(t0 + rows_per_block, (int64_t)p.T);
    const int64_t slot0 = t0 * k;
    const int slots = (int)(t1 - t0) * k;
    for (int s = tid; s < slots; s += NT) slot_ids[s] = p.out.ids[slot0 + s];
    __syncthreads();
    if (blockIdx.x == 0 && tid < 64) {
        const float l = balance(off, p.out.mean_probs, E, p.k, *p.out.n_valid, tid);
        if (tid == 0) *p.out.loss = l;
    }
    __syncthreads();
    scan_counts(off, E, tid);
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += NT) p.out.offsets[e] = off[e];
    const int64_t all = (int64_t)p.T * k;
    for (int64_t i = off[E] + (int64_t)blockIdx.x * NT + tid; i < all; i += (int64_t)gridDim.x * NT) p.out.rows[i] = -1;
    __syncthreads();
    const RouteWs ws = split_ws(p.ws, gridDim.x, p.E);
    for (int e = tid; e < E; e += NT) off[e] += ws.hist[(int64_t)blockIdx.x * E + e];
    __syncthreads();
    place(slot_ids, slots, off, slot0, p.k, p.out.rows, p.out.pos, tid);
}

// Gradient: the row's probabilities again from its logits, the loss's part in
// registers, the weights' part added to the row in LDS by the lanes that hold
// the choices.
template <bool F32, int G, int VPL>
__global__ void __launch_bounds__(NT)
route_backward_kernel(RouteBackwardProblem p, bool vec) {
    constexpr int TOK = NT / G;
    __shared__ __attribute__((aligned(16))) float row[TOK][G * VPL + 4];
    const int tid = threadIdx.x, gl = tid % G, tok = tid / G, e0 = gl * VPL;
    const int E = (int)p.E, k = (int)p.k;
    const float n = (float)*p.n_valid;
    const float scale = p.dloss != nullptr && n > 0.0f ? *p.dloss * (float)E / ((float)k * n) / n : 0.0f;
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = e0 + i < E ? scale * (float)p.counts[e0 + i] : 0.0f;
    for (int64_t tb = (int64_t)blockIdx.x * TOK; tb < (int64_t)p.T; tb += (int64_t)gridDim.x * TOK) {
        const int64_t t = tb + tok;
        const bool in = t < (int64_t)p.T;
        // a live row has a first choice
        const bool live = in && p.ids[t * k] >= 0;
        float v[VPL], top = NEG_INF;
        if (live) {
            load_logits<F32, VPL>(p.logits, t, E, e0, vec, v);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = NEG_INF;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) top = fmaxf(top, v[i]);
        top = reduce<G>(top, [](float a, float b) { return fmaxf(a, b); });
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] = live ? exp_neg(v[i] - top) : 0.0f;
            s += v[i];
        }
        s = sum<G>(s);
        const float inv = live ? 1.0f / s : 0.0f;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            v[i] *= inv;
            dot += v[i] * c[i];
        }
        int id = -1;
        float g = 0.0f;
        if (live && gl < k && p.dweights != nullptr) {
            id = p.ids[t * k + gl];
            if (id >= 0 && id < E) g = p.weights[t * k + gl] * p.dweights[t * k + gl];
        }
        const float inner = sum<G>(g);
        dot = sum<G>(dot);
        if (p.normalize) {
            if (id >= 0) g -= p.weights[t * k + gl] * inner;
        } else {
            dot += inner;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) row[tok][e0 + i] = v[i] * (c[i] - dot);
        __syncthreads();
        if (id >= 0 && id < E) row[tok][id] += g;       // a row's choices are distinct
        __syncthreads();
        if (in) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (e0 + i >= E) continue;
                const float d = row[tok][e0 + i];
                if constexpr (F32)
                    static_cast<float*>(p.dlogits)[t * E + e0 + i] = d;
                else
                    static_cast<__bf16*>(p.dlogits)[t * E + e0 + i] = (__bf16)d;
            }
        }
    }
}

bool vec_rows(int type, uint32_t E) { return E % (type == BG_F32 ? 4 : 8) == 0; }

// Calls f with the smallest group that holds E experts: (G, VPL).
template <class F>
void by_experts(uint32_t E, F&& f) {
    using std::integral_constant;
    if (E <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    else if (E <= 256) f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    else if (E <= 512) f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    else f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_moe_route(const RouteProblem& p, hipStream_t stream) {
    const uint32_t blocks = route_blocks(p.T);
    const bool one = p.T <= kRouteOneBlock, vec = vec_rows(p.type, p.E);
    const int rows = one ? (int)kRouteOneBlock : (int)route_rows_per_block(p.T);
    by_experts(p.E, [&](auto g, auto v) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        if (p.type == BG_F32) {
            if (one) route_kernel<true, G, V, true><<<1, NT, 0, stream>>>(p, rows, vec);
            else route_kernel<true, G, V, false><<<blocks, NT, 0, stream>>>(p, rows, vec);
        } else {
            if (one) route_kernel<false, G, V, true><<<1, NT, 0, stream>>>(p, rows, vec);
            else route_kernel<false, G, V, false><<<blocks, NT, 0, stream>>>(p, rows, vec);
        }
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || one) return e;
    route_scan_kernel<<<(p.E + 15) / 16, NT, 0, stream>>>(p, (int)blocks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_place_kernel<<<blocks, NT, 0, stream>>>(p, rows);
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const RouteBackwardProblem& p, hipStream_t stream) {
    const bool vec = vec_rows(p.type, p.E);
    by_experts(p.E, [&](auto g, auto v) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        const uint32_t passes = (p.T + NT / G - 1) / (NT / G);
        const uint32_t blocks = passes < 2048 ? passes : 2048;
        if (p.type == BG_F32) route_backward_kernel<true, G, V><<<blocks, NT, 0, stream>>>(p, vec);
        else route_backward_kernel<false, G, V><<<blocks, NT, 0, stream>>>(p, vec);
    });
    return hipGetLastError();
}

}  // namespace bg
