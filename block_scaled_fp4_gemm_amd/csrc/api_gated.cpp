// C ABI entry points of the gated MLP block and of the gradients of dense
// products: argument validation, device check, kernel dispatch. As in api.cpp,
// validation is plain host code and nothing is enqueued unless every check
// passes.
#include "api_checks.hpp"
#include "bg_internal.hpp"
#include "gated_tiles.hpp"

namespace {

using namespace bg;

uint64_t type_size(int type) { return type == BG_BF16 ? 2 : 4; }
bool type_ok(int type) { return type == BG_BF16 || type == BG_F32; }
bool act_ok(int act) { return act == BG_SILU || act == BG_GELU_TANH; }

// An operand of this size can exist: below 2^60 bytes, so that no byte count
// and no address range wraps.
bool fits(uint64_t rows, uint64_t cols, uint64_t size) {
    return (unsigned __int128)rows * cols * size < ((unsigned __int128)1 << 60);
}

struct Operand {
    const void* p;
    uint64_t bytes;
};

uint32_t pitch8(uint32_t n) { return (n + 7) / 8 * 8; }

// Pointers, alignment, and no output over an input or another output.
template <size_t NI, size_t NO>
bg_status check_operands(const Operand (&in)[NI], const Operand (&out)[NO]) {
    for (const Operand& o : in)
        if (missing(o.p, o.bytes)) return BG_ERR_NULL;
    for (const Operand& o : out)
        if (missing(o.p, o.bytes)) return BG_ERR_NULL;
    for (const Operand& o : in)
        if (misaligned(o.p, o.bytes)) return BG_ERR_ALIGN;
    for (const Operand& o : out)
        if (misaligned(o.p, o.bytes)) return BG_ERR_ALIGN;
    for (size_t i = 0; i < NO; ++i) {
        const Range r = range_of(out[i].p, out[i].bytes);
        for (const Operand& o : in)
            if (overlap(r, range_of(o.p, o.bytes))) return BG_ERR_ALIAS;
        for (size_t j = 0; j < i; ++j)
            if (overlap(r, range_of(out[j].p, out[j].bytes))) return BG_ERR_ALIAS;
    }
    return BG_OK;
}

// An nn (C [M, N] of K terms, parts of them) or tn (parts outputs) product, A's
// rows lda elements apart.
GatedPlan transposed_plan(bool tn, uint32_t M, uint32_t N, uint32_t K, uint32_t lda, uint32_t parts, uint32_t cus,
                          double* us = nullptr) {
    const bool direct = gated_direct(lda) && gated_direct(N);
    const uint32_t steps = direct ? K / 64 : K / 64 + (K % 64 != 0);
    return plan_of(false, tn, direct, M, N, tn ? steps : steps * parts, tn ? parts : 1, cus, tune(BG_TUNE_TILE), us);
}
uint64_t planes_bytes(const GatedPlan& p, uint32_t M, uint32_t N, uint32_t outputs) {
    return p.splits > 1 ? (uint64_t)p.splits * outputs * M * N * 4 : 0;
}

// A product that the caller gives whole: its plan, the rows of its operands (copied
// where lda or ldb is not their own), and the workspace: planes, A's copy, B's copy.
struct ProductPlan {
    GatedPlan plan;
    uint32_t lda, ldb;
    uint64_t planes, a, bytes;
};
ProductPlan product_plan(bool tn, uint32_t M, uint32_t N, uint32_t K, uint32_t cus) {
    const uint32_t cols = tn ? M : K, rows = tn ? K : M;
    ProductPlan p{{}, cols, N, 0, 0, 0};
    double us = 0;
    p.plan = transposed_plan(tn, M, N, K, cols, 1, cus, &us);
    // (a reduction below one step has no direct loads either way)
    if (K >= 64 && !(gated_direct(cols) && gated_direct(N)) && gated_direct(pitch8(cols)) && gated_direct(pitch8(N)) && tune(BG_TUNE_TILE) < 0) {
        double direct = 0;
        const GatedPlan plan = plan_of(false, tn, true, M, N, K / 64, 1, cus, -1, &direct);
        const uint64_t copied = (cols % 8 ? (uint64_t)rows * pitch8(cols) : 0) + (N % 8 ? (uint64_t)K * pitch8(N) : 0);
        if (direct + aligned_copy_us(copied) < us) {
            p.plan = plan;
            p.lda = pitch8(cols);
            p.ldb = pitch8(N);
        }
    }
    p.planes = (planes_bytes(p.plan, M, N, 1) + 15) / 16 * 16;
    p.a = p.lda != cols ? (uint64_t)rows * p.lda * 2 : 0;
    p.bytes = p.planes + p.a + (p.ldb != N ? (uint64_t)K * p.ldb * 2 : 0);
    return p;
}

bool transposed_shape_ok(bool tn, uint32_t M, uint32_t N, uint32_t K, uint32_t lda) {
    return dims_ok(M, N, K) && N <= kMaxDim - 7 && M <= kMaxDim - 7 && fits(M, K, 2) && fits(K, N, 2) &&
           fits(M, N, 64 * 4) && gated_fits(gated_direct(lda) && gated_direct(N), false, M, N, tn ? 2 : 1);
}

bg_status transposed_workspace(bool tn, uint32_t M, uint32_t N, uint32_t K, size_t* bytes) {
    if (bytes == nullptr) return BG_ERR_NULL;
    if (!transposed_shape_ok(tn, M, N, K, tn ? M : K)) return BG_ERR_SHAPE;
    uint32_t cus = 0;
    const bg_status s = check_device(&cus);
    if (s != BG_OK) return s;
    *bytes = M == 0 || N == 0 ? 0 : (size_t)product_plan(tn, M, N, K, cus).bytes;
    return BG_OK;
}

bg_status transposed(bool tn, const uint16_t* A, const uint16_t* B, uint16_t* C, void* ws, size_t ws_bytes, uint32_t M,
                     uint32_t N, uint32_t K, void* stream) {
    if (!transposed_shape_ok(tn, M, N, K, tn ? M : K)) return BG_ERR_SHAPE;
    if (M == 0 || N == 0) return BG_OK;
    const Operand in[] = {{A, (uint64_t)M * K * 2}, {B, (uint64_t)K * N * 2}};
    const Operand out[] = {{C, (uint64_t)M * N * 2}};
    bg_status s = check_operands(in, out);
    if (s != BG_OK) return s;
    uint32_t cus = 0;
    if ((s = check_device(&cus)) != BG_OK) return s;
    const ProductPlan plan = product_plan(tn, M, N, K, cus);
    if (plan.bytes != 0) {
        if (ws == nullptr || ws_bytes < plan.bytes) return BG_ERR_WORKSPACE;
        const Operand with[] = {in[0], in[1], out[0]}, space[] = {{ws, plan.bytes}};
        if ((s = check_operands(with, space)) != BG_OK) return s;
    }
    const hipStream_t st = (hipStream_t)stream;
    const uint32_t rows = tn ? K : M, cols = tn ? M : K;
    AlignedCopy copy{{A, B}, {}, {}, {cols, N}, {plan.lda, plan.ldb}};
    hipError_t e = hipSuccess;
    if (plan.lda != cols || plan.ldb != N) {
        uint16_t* to = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + plan.planes);
        if (plan.lda != cols) copy.rows[0] = rows, A = copy.to[0] = to;
        if (plan.ldb != N) copy.rows[1] = K, B = copy.to[1] = to + plan.a / 2;
        e = launch_aligned_copy(copy, st);
    }
    if (e == hipSuccess)
        e = launch_transposed(TransposedProblem{tn, A, nullptr, B, nullptr, C, nullptr, static_cast<float*>(ws), M, N, K, plan.lda,
                                                plan.ldb, 1, plan.plan.tile, plan.plan.splits, 0, 1, plan.plan.wide},
                              st);
    return launched(e);
}

bool gated_shape_ok(uint32_t M, uint32_t N, uint32_t K) {
    return dims_ok(M, N, K) && N <= kMaxDim - 7 && M <= kMaxDim - 7 && K <= kMaxDim - 7 && fits(M, K, 2) && fits(N, K, 2) &&
           fits(M, N, 4) && gated_fits(gated_direct(K), true, M, N, 1);
}

// The gradient's workspace: dG and dU, each followed by its low half where M is
// small, then the products' planes: both products' where one launch takes them
// (pair; a product that is wanted alone keeps its plan), else the larger of the two.
struct GradPlan {
    GatedPlan nn, tn;
    bool pair;
    uint32_t stacked;        // 2 with low halves: dA's product runs over both as 2 M rows
    uint64_t half, bytes;    // of dG (with its low half); of all
    uint64_t nn_planes;      // bytes, where both are kept
};
GradPlan grad_plan(uint32_t M, uint32_t N, uint32_t K, uint32_t cus) {
    GradPlan g;
    double us_nn = 0, us_tn = 0;
    g.stacked = M <= kFineRows ? 2 : 1;
    g.nn = transposed_plan(false, M * g.stacked, K, N, pitch8(N), 2, cus, &us_nn);
    g.tn = transposed_plan(true, N, K, M, pitch8(N), 2, cus, &us_tn);
    g.half = (uint64_t)M * pitch8(N) * 2 * g.stacked;
    g.pair = false;
    if (gated_direct(pitch8(N)) && gated_direct(K) && tune(BG_TUNE_TILE) < 0) {
        // a launch and the wait for the one before it take about 3 us
        const PairPlan p = pair_plan({M * g.stacked, N}, {K, K}, {N / 64 * 2, M / 64 * g.stacked}, {1, 2}, g.stacked, cus);
        if (p.nn != 0 && p.us < us_nn + us_tn + 3.0) {
            g.pair = true;
            g.nn = GatedPlan{GT_128x128_DEEP, p.nn};
            g.tn = GatedPlan{GT_128x128_DEEP, p.tn};
        }
    }
    const uint64_t rows = (uint64_t)M * g.stacked;
    const uint64_t a = g.nn.splits > 1 || g.stacked > 1 ? ((uint64_t)g.nn.splits * rows * K * 4 + 15) / 16 * 16 : 0;
    const uint64_t b = planes_bytes(g.tn, N, K, 2);
    g.nn_planes = g.pair ? a : 0;
    g.bytes = 2 * g.half + (g.pair ? a + b : a > b ? a : b);
    return g;
}

bool grad_shape_ok(uint32_t M, uint32_t N, uint32_t K) {
    // the sum of dA's planes: 1024 elements a workgroup in one launch
    if (M <= kFineRows && (uint64_t)M * K >= (uint64_t)1 << 33) return false;
    return gated_shape_ok(M, N, K) && transposed_shape_ok(false, M, K, N, pitch8(N)) && transposed_shape_ok(true, N, K, M, pitch8(N));
}

// One set of weights in 4 bits: its shape, and its operands in order.
bg_status check_w4(const bg_w4* w, uint32_t N, uint32_t K, Operand (&ops)[3]) {
    if (w == nullptr) return BG_ERR_NULL;
    uint64_t group = w->group, size = 1;
    if (w->format == BG_W4_INT4) {
        if (group == 0 || group % 32 != 0) return BG_ERR_SHAPE;
        size = 2;
    } else if (w->format == BG_W4_MXFP4 || w->format == BG_W4_NVFP4) {
        if (w->zeros != nullptr) return BG_ERR_SHAPE;
        if (group != (w->format == BG_W4_MXFP4 ? 32 : 16)) return BG_ERR_SHAPE;
    } else {
        return BG_ERR_SHAPE;
    }
    if (K % group != 0) return BG_ERR_SHAPE;
    const uint64_t groups = (uint64_t)N * (K / group);
    ops[0] = {w->codes, (uint64_t)N * (K / 2)};
    ops[1] = {w->scales, groups * size};
    ops[2] = {w->zeros, w->zeros != nullptr ? groups : 0};
    return BG_OK;
}

bg_status gemv(const uint16_t* x, const bg_w4* w0, const bg_w4* w1, uint16_t* y, bool gated, int act, uint32_t R, uint32_t N,
               uint32_t K, void* stream) {
    if (!dims_ok(R, N, K) || K % 32 != 0 || K > kMaxGemvK || R > kMaxGemvRows || !act_ok(act) || !fits(R, K, 2) || !fits(N, K, 2) ||
        !fits(R, N, 2))
        return BG_ERR_SHAPE;
    // a launch holds fewer than 2^32 threads: 1024 for 16 columns and 16 rows at most
    if (((uint64_t)N + 15) / 16 * (((uint64_t)R + 15) / 16) * 1024 >= ((uint64_t)1 << 32)) return BG_ERR_SHAPE;
    Operand a[3] = {}, b[3] = {};
    bg_status s = check_w4(w0, N, K, a);
    if (s == BG_OK && gated) s = check_w4(w1, N, K, b);
    if (s != BG_OK) return s;
    if (gated && (w0->format != w1->format || w0->group != w1->group || (w0->zeros == nullptr) != (w1->zeros == nullptr)))
        return BG_ERR_SHAPE;
    if (R == 0 || N == 0) return BG_OK;
    const Operand in[] = {{x, (uint64_t)R * K * 2}, a[0], a[1], a[2], b[0], b[1], b[2]};
    const Operand out[] = {{y, (uint64_t)R * N * 2}};
    if ((s = check_operands(in, out)) != BG_OK) return s;
    uint32_t cus = 0;
    if ((s = check_device(&cus)) != BG_OK) return s;
    auto operand = [](const bg_w4* w) {
        return W4Operand{w->codes, static_cast<const uint8_t*>(w->scales), w->zeros, w->scale_2};
    };
    return launched(launch_gemv_w4(GemvProblem{x, {operand(w0), gated ? operand(w1) : W4Operand{}}, y, R, N, K, w0->group,
                                               w0->format, gated, act, cus},
                                   (hipStream_t)stream));
}

}  // namespace

extern "C" {

bg_status gemv_w4(const uint16_t* X, const bg_w4* W, uint16_t* Y, uint32_t R, uint32_t N, uint32_t K, void* stream) {
    return gemv(X, W, nullptr, Y, false, BG_SILU, R, N, K, stream);
}

bg_status gemv_w4_gated(const uint16_t* X, const bg_w4* W0, const bg_w4* W1, uint16_t* H, int act, uint32_t R, uint32_t N,
                        uint32_t K, void* stream) {
    return gemv(X, W0, W1, H, true, act, R, N, K, stream);
}

bg_status gemm_bf16_gated(const uint16_t* A, const uint16_t* B0, const uint16_t* B1, uint16_t* H, void* G, void* U,
                          int kept_type, int act, uint32_t M, uint32_t N, uint32_t K, void* stream) {
    if (!gated_shape_ok(M, N, K) || !act_ok(act) || !type_ok(kept_type)) return BG_ERR_SHAPE;
    if (M == 0 || N == 0) return BG_OK;
    if ((G == nullptr) != (U == nullptr)) return BG_ERR_NULL;
    const uint64_t b = (uint64_t)N * K * 2, c = (uint64_t)M * N * 2, kept = G != nullptr ? (uint64_t)M * N * type_size(kept_type) : 0;
    const Operand in[] = {{A, (uint64_t)M * K * 2}, {B0, b}, {B1, b}};
    const Operand out[] = {{H, c}, {G, kept}, {U, kept}};
    bg_status s = check_operands(in, out);
    if (s != BG_OK) return s;
    uint32_t cus = 0;
    if ((s = check_device(&cus)) != BG_OK) return s;
    const GatedPlan plan = plan_of(true, false, gated_direct(K), M, N, K / 64, 1, cus, tune(BG_TUNE_TILE));
    return launched(launch_gated(GatedProblem{A, B0, B1, H, G, U, kept_type, M, N, K, act, plan.tile, plan.wide}, (hipStream_t)stream));
}

bg_status gemm_bf16_nn_workspace(uint32_t M, uint32_t N, uint32_t K, size_t* bytes) {
    return transposed_workspace(false, M, N, K, bytes);
}
bg_status gemm_bf16_tn_workspace(uint32_t M, uint32_t N, uint32_t K, size_t* bytes) {
    return transposed_workspace(true, M, N, K, bytes);
}

bg_status gemm_bf16_nn(const uint16_t* A, const uint16_t* B, uint16_t* C, void* workspace, size_t workspace_bytes, uint32_t M,
                       uint32_t N, uint32_t K, void* stream) {
    return transposed(false, A, B, C, workspace, workspace_bytes, M, N, K, stream);
}
bg_status gemm_bf16_tn(const uint16_t* A, const uint16_t* B, uint16_t* C, void* workspace, size_t workspace_bytes, uint32_t M,
                       uint32_t N, uint32_t K, void* stream) {
    return transposed(true, A, B, C, workspace, workspace_bytes, M, N, K, stream);
}

bg_status gemm_bf16_gated_backward_workspace(uint32_t M, uint32_t N, uint32_t K, size_t* bytes) {
    if (bytes == nullptr) return BG_ERR_NULL;
    if (!grad_shape_ok(M, N, K)) return BG_ERR_SHAPE;
    uint32_t cus = 0;
    const bg_status s = check_device(&cus);
    if (s != BG_OK) return s;
    *bytes = (size_t)grad_plan(M, N, K, cus).bytes;
    return BG_OK;
}

bg_status gemm_bf16_gated_backward(const uint16_t* dH, const uint16_t* A, const uint16_t* B0, const uint16_t* B1,
                                   const void* G, const void* U, int kept_type, uint16_t* dA, uint16_t* dB0, uint16_t* dB1,
                                   int act, void* workspace, size_t workspace_bytes, uint32_t M, uint32_t N, uint32_t K, void* stream) {
    if (!grad_shape_ok(M, N, K) || !act_ok(act) || !type_ok(kept_type)) return BG_ERR_SHAPE;
    if ((dB0 == nullptr) != (dB1 == nullptr)) return BG_ERR_NULL;
    const uint64_t a = (uint64_t)M * K * 2, b = (uint64_t)N * K * 2, c = (uint64_t)M * N * 2,
                   kept = (uint64_t)M * N * type_size(kept_type);
    const Operand in[] = {{dH, c}, {A, dB0 != nullptr ? a : 0}, {B0, dA != nullptr ? b : 0}, {B1, dA != nullptr ? b : 0},
                          {G, kept}, {U, kept}};
    const Operand out[] = {{dA, dA != nullptr ? a : 0}, {dB0, dB0 != nullptr ? b : 0}, {dB1, dB1 != nullptr ? b : 0}};
    bg_status s = check_operands(in, out);
    if (s != BG_OK) return s;
    uint32_t cus = 0;
    if ((s = check_device(&cus)) != BG_OK) return s;
    const bool want_a = dA != nullptr && M != 0 && K != 0, want_b = dB0 != nullptr && N != 0 && K != 0;
    const GradPlan plan = grad_plan(M, N, K, cus);
    if (plan.bytes != 0) {
        if (workspace == nullptr || workspace_bytes < plan.bytes) return BG_ERR_WORKSPACE;
        const Operand with[] = {in[0], in[1], in[2], in[3], in[4], in[5], out[0], out[1], out[2]}, ws[] = {{workspace, plan.bytes}};
        if ((s = check_operands(with, ws)) != BG_OK) return s;
    }
    const hipStream_t st = (hipStream_t)stream;
    uint16_t* dG = static_cast<uint16_t*>(workspace);
    uint16_t* dU = dG + plan.half / 2;
    float* planes = reinterpret_cast<float*>(dU + plan.half / 2);
    const uint32_t ld = pitch8(N);
    const int64_t low = plan.stacked > 1 ? (int64_t)M * ld : 0;
    if (!want_a && !want_b) return BG_OK;
    hipError_t e = hipSuccess;
    if (M != 0 && N != 0) e = launch_gate_grad(GateGradProblem{dH, G, U, kept_type, dG, dU, M, N, ld, act, low}, st);
    const TransposedProblem nn{false, dG, dU, B0, B1, dA, nullptr, planes, M * plan.stacked, K, N, ld, K, 2, plan.nn.tile,
                               plan.nn.splits, 0, plan.stacked, plan.nn.wide};
    const TransposedProblem tn{true, dG, dU, A, nullptr, dB0, dB1, planes + plan.nn_planes / 4, N, K, M, ld, K, 2, plan.tn.tile,
                               plan.tn.splits, low, 1, plan.tn.wide};
    if (plan.pair && want_a && want_b) {
        if (e == hipSuccess) e = launch_transposed_pair(nn, tn, st);
    } else {
        if (e == hipSuccess && want_a) e = launch_transposed(nn, st);
        if (e == hipSuccess && want_b) e = launch_transposed(tn, st);
    }
    return launched(e);
}

}  // extern "C"
