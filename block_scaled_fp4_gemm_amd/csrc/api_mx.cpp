// C ABI entry points of the MXFP4 operators and of the expert router: argument
// validation, device check, kernel dispatch. As in api.cpp, validation is
// plain host code and nothing is enqueued unless every check passes.
#include "api_checks.hpp"
#include "bg_internal.hpp"
#include "mx_tiles.hpp"

namespace {

using namespace bg;

uint64_t type_size(int type) { return type == BG_BF16 ? 2 : 4; }
bool type_ok(int type) { return type == BG_BF16 || type == BG_F32; }

// The small arrays (indices, counts, weights) need their elements' alignment only.
bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// An operand of this size can exist: below 2^60 bytes, so that no byte count
// and no address range wraps.
bool fits(uint64_t rows, uint64_t cols, uint64_t batch, uint64_t size) {
    const unsigned __int128 n = (unsigned __int128)rows * cols * batch * size;
    return n < ((unsigned __int128)1 << 60);
}

// C = A * B^T with B of E experts; every operand's pointer, alignment and overlap.
bg_status check_mx_gemm(const uint8_t* A, const uint8_t* SFA, const uint8_t* B, const uint8_t* SFB,
                        const int32_t* offsets, const uint16_t* C, uint32_t M, uint32_t N, uint32_t K,
                        uint32_t E) {
    const uint64_t a_bytes = (uint64_t)M * (K / 2), sa_bytes = (uint64_t)M * (K / 32);
    const uint64_t b_bytes = (uint64_t)E * N * (K / 2), sb_bytes = (uint64_t)E * N * (K / 32);
    const uint64_t c_bytes = (uint64_t)M * N * 2;
    const uint64_t o_bytes = offsets != nullptr ? ((uint64_t)E + 1) * 4 : 0;
    if (missing(A, a_bytes) || missing(SFA, sa_bytes) || missing(B, b_bytes) || missing(SFB, sb_bytes) ||
        missing(C, c_bytes))
        return BG_ERR_NULL;
    if (misaligned(A, a_bytes) || misaligned(SFA, sa_bytes) || misaligned(B, b_bytes) ||
        misaligned(SFB, sb_bytes) || misaligned(C, c_bytes) || misaligned4(offsets))
        return BG_ERR_ALIGN;
    const Range rc = range_of(C, c_bytes);
    if (overlap(rc, range_of(A, a_bytes)) || overlap(rc, range_of(SFA, sa_bytes)) ||
        overlap(rc, range_of(B, b_bytes)) || overlap(rc, range_of(SFB, sb_bytes)) ||
        overlap(rc, range_of(offsets, o_bytes)))
        return BG_ERR_ALIAS;
    return BG_OK;
}

bool route_shape_ok(uint32_t T, uint32_t E, uint32_t k) {
    return E >= 1 && E <= kMaxExperts && k >= 1 && k <= kMaxTopK && k <= E && (uint64_t)T * k <= kMaxDim;
}

}  // namespace

extern "C" {

bg_status mxfp4_quantize(const void* x, int x_type, uint32_t ldx, const int32_t* rows, uint8_t* codes,
                         uint8_t* scales, uint32_t M, uint32_t R, uint32_t K, void* stream) {
    if (!dims_ok(M, R, K) || ldx > kMaxDim || K % 32 != 0 || ldx < K || !type_ok(x_type)) return BG_ERR_SHAPE;
    if (rows == nullptr && R != M) return BG_ERR_SHAPE;
    if (!fits(M, ldx, 1, type_size(x_type)) || !fits(R, K, 1, 1)) return BG_ERR_SHAPE;
    if ((uint64_t)R * mx_quant_pieces(K) > 0xFFFFFFFFu) return BG_ERR_SHAPE;
    if (R == 0 || K == 0) return BG_OK;
    const uint64_t x_bytes = M == 0 ? 0 : ((uint64_t)(M - 1) * ldx + K) * type_size(x_type);
    const uint64_t c_bytes = (uint64_t)R * (K / 2), s_bytes = (uint64_t)R * (K / 32);
    if (missing(x, x_bytes) || missing(codes, c_bytes) || missing(scales, s_bytes)) return BG_ERR_NULL;
    if (misaligned(x, x_bytes) || misaligned(codes, c_bytes) || misaligned(scales, s_bytes) || misaligned4(rows))
        return BG_ERR_ALIGN;
    const Range rx = range_of(x, x_bytes), rc = range_of(codes, c_bytes), rs = range_of(scales, s_bytes);
    const Range rr = range_of(rows, rows != nullptr ? (uint64_t)R * 4 : 0);
    if (overlap(rc, rx) || overlap(rs, rx) || overlap(rc, rs) || overlap(rc, rr) || overlap(rs, rr))
        return BG_ERR_ALIAS;
    bg_status s = check_device();
    if (s != BG_OK) return s;
    return launched(launch_mxfp4_quantize(MxQuantProblem{x, rows, codes, scales, M, R, K, ldx, x_type},
                                          (hipStream_t)stream));
}

bg_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, void* out, int out_type, uint32_t M,
                           uint32_t K, void* stream) {
    if (!dims_ok(M, 0, K) || K % 32 != 0 || !type_ok(out_type) || !fits(M, K, 1, 4)) return BG_ERR_SHAPE;
    if (M == 0 || K == 0) return BG_OK;
    const uint64_t c_bytes = (uint64_t)M * (K / 2), s_bytes = (uint64_t)M * (K / 32);
    const uint64_t o_bytes = (uint64_t)M * K * type_size(out_type);
    if (missing(codes, c_bytes) || missing(scales, s_bytes) || missing(out, o_bytes)) return BG_ERR_NULL;
    if (misaligned(codes, c_bytes) || misaligned(scales, s_bytes) || misaligned(out, o_bytes)) return BG_ERR_ALIGN;
    const Range ro = range_of(out, o_bytes);
    if (overlap(ro, range_of(codes, c_bytes)) || overlap(ro, range_of(scales, s_bytes))) return BG_ERR_ALIAS;
    bg_status s = check_device();
    if (s != BG_OK) return s;
    return launched(launch_mxfp4_dequantize(codes, scales, out, out_type, M, K, (hipStream_t)stream));
}

bg_status gemm_mxfp4(const uint8_t* A, const uint8_t* SFA, const uint8_t* B, const uint8_t* SFB, uint16_t* C,
                     uint32_t M, uint32_t N, uint32_t K, void* stream) {
    if (!dims_ok(M, N, K) || K % 32 != 0 || K > kMaxMxK || !fits(M, K, 1, 1) || !fits(N, K, 1, 1) || !fits(M, N, 1, 2))
        return BG_ERR_SHAPE;
    if (M == 0 || N == 0) return BG_OK;
    if (!mx_dense_launches(M, N, K)) return BG_ERR_SHAPE;
    bg_status s = check_mx_gemm(A, SFA, B, SFB, nullptr, C, M, N, K, 1);
    if (s != BG_OK) return s;
    uint32_t cus = 0;
    if ((s = check_device(&cus)) != BG_OK) return s;
    return launched(launch_gemm_mxfp4(MxGemmProblem{A, SFA, B, SFB, C, M, N, K, nullptr, 1, cus},
                                      (hipStream_t)stream));
}

bg_status gemm_mxfp4_grouped(const uint8_t* A, const uint8_t* SFA, const uint8_t* B, const uint8_t* SFB,
                             const int32_t* offsets, uint16_t* C, uint32_t S, uint32_t N, uint32_t K, uint32_t E,
                             void* stream) {
    if (!dims_ok(S, N, K) || K % 32 != 0 || K > kMaxMxK || E > kMaxExperts || !fits(N, K, E, 1) || !fits(S, K, 1, 1) ||
        !fits(S, N, 1, 2))
        return BG_ERR_SHAPE;
    if (S == 0 || N == 0 || E == 0) return BG_OK;
    if (mx_grouped_tile(S, N, K, E) < 0) return BG_ERR_SHAPE;
    if (offsets == nullptr) return BG_ERR_NULL;
    bg_status s = check_mx_gemm(A, SFA, B, SFB, offsets, C, S, N, K, E);
    if (s != BG_OK) return s;
    uint32_t cus = 0;
    if ((s = check_device(&cus)) != BG_OK) return s;
    return launched(launch_gemm_mxfp4(MxGemmProblem{A, SFA, B, SFB, C, S, N, K, offsets, E, cus},
                                      (hipStream_t)stream));
}

size_t moe_route_workspace_bytes(uint32_t T, uint32_t E) { return route_workspace_bytes(T, E); }

bg_status moe_route(const void* logits, int logits_type, const uint8_t* valid, const bg_moe_routing* out,
                    void* workspace, size_t workspace_bytes, uint32_t T, uint32_t E, uint32_t k, int normalize,
                    void* stream) {
    if (!route_shape_ok(T, E, k) || !type_ok(logits_type)) return BG_ERR_SHAPE;
    const uint64_t l_bytes = (uint64_t)T * E * type_size(logits_type), tk = (uint64_t)T * k * 4;
    if (missing(logits, l_bytes) || out == nullptr) return BG_ERR_NULL;
    const bg_moe_routing& o = *out;
    // valid counts as one more input range: T bytes
    const Range outs[] = {range_of(o.ids, tk),           range_of(o.weights, tk),
                          range_of(o.counts, E * 4ull),  range_of(o.offsets, (E + 1) * 4ull),
                          range_of(o.rows, tk),          range_of(o.pos, tk),
                          range_of(o.mean_probs, E * 4ull), range_of(o.loss, 4),
                          range_of(o.n_valid, 4)};
    for (const Range& r : outs) {
        if (r.lo == 0 && r.hi != 0) return BG_ERR_NULL;
        if (r.hi != r.lo && (r.lo & 3u) != 0) return BG_ERR_ALIGN;
    }
    if (misaligned(logits, l_bytes)) return BG_ERR_ALIGN;
    const size_t need = route_workspace_bytes(T, E);
    if (need != 0 && (workspace == nullptr || workspace_bytes < need)) return BG_ERR_WORKSPACE;
    if (misaligned(workspace, need)) return BG_ERR_ALIGN;
    const Range rl = range_of(logits, l_bytes), rw = range_of(workspace, need);
    const Range rv = range_of(valid, valid != nullptr ? T : 0);
    if (overlap(rw, rl) || overlap(rw, rv)) return BG_ERR_ALIAS;
    for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
        if (overlap(outs[i], rl) || overlap(outs[i], rv) || overlap(outs[i], rw)) return BG_ERR_ALIAS;
        for (size_t j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return BG_ERR_ALIAS;
    }
    bg_status s = check_device();
    if (s != BG_OK) return s;
    return launched(launch_moe_route(RouteProblem{logits, logits_type, valid, o, workspace, T, E, k, normalize},
                                     (hipStream_t)stream));
}

bg_status moe_route_backward(const void* logits, int logits_type, const int32_t* ids, const float* weights,
                             const int32_t* counts, const int32_t* n_valid, const float* dweights,
                             const float* dloss, void* dlogits, uint32_t T, uint32_t E, uint32_t k, int normalize,
                             void* stream) {
    if (!route_shape_ok(T, E, k) || !type_ok(logits_type)) return BG_ERR_SHAPE;
    if (T == 0) return BG_OK;
    const uint64_t l_bytes = (uint64_t)T * E * type_size(logits_type), tk = (uint64_t)T * k * 4;
    if (logits == nullptr || ids == nullptr || weights == nullptr || counts == nullptr || n_valid == nullptr ||
        dlogits == nullptr)
        return BG_ERR_NULL;
    if (misaligned(logits, l_bytes) || misaligned(dlogits, l_bytes) || misaligned4(ids) || misaligned4(weights) ||
        misaligned4(counts) || misaligned4(n_valid) || misaligned4(dweights) || misaligned4(dloss))
        return BG_ERR_ALIGN;
    const Range ro = range_of(dlogits, l_bytes);
    // in place is fine; a shifted overlap is not
    if (dlogits != logits && overlap(ro, range_of(logits, l_bytes))) return BG_ERR_ALIAS;
    if (overlap(ro, range_of(ids, tk)) || overlap(ro, range_of(weights, tk)) ||
        overlap(ro, range_of(counts, E * 4ull)) || overlap(ro, range_of(n_valid, 4)) ||
        overlap(ro, range_of(dweights, dweights != nullptr ? tk : 0)) ||
        overlap(ro, range_of(dloss, dloss != nullptr ? 4 : 0)))
        return BG_ERR_ALIAS;
    bg_status s = check_device();
    if (s != BG_OK) return s;
    return launched(launch_moe_route_backward(
        RouteBackwardProblem{logits, logits_type, ids, weights, counts, n_valid, dweights, dloss, dlogits, T, E, k,
                             normalize},
        (hipStream_t)stream));
}

}  // extern "C"
