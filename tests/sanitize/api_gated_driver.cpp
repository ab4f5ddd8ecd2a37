// Sanitizer driver for the gated block's, the transposed products' and the 4-bit
// matrix-vector part of the C-ABI validation layer (api_gated.cpp) and for the
// tile choice (gated_tiles.hpp), built for the host with
// -fsanitize=address,undefined against hip_stub/. The launchers are replaced by
// recorders that check what validation hands them. Fake device addresses are
// never dereferenced.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "../../block_scaled_fp4_gemm_amd/csrc/bg_internal.hpp"
#include "../../block_scaled_fp4_gemm_amd/csrc/gated_tiles.hpp"

static int g_dev = 0, g_launches = 0, g_tune = -1;

hipError_t hipGetDevice(int* dev) {
    *dev = g_dev;
    return hipSuccess;
}

hipError_t hipGetDeviceProperties(hipDeviceProp_t* prop, int dev) {
    std::memset(prop, 0, sizeof(*prop));
    std::strcpy(prop->gcnArchName, dev == 0 ? "gfx950:sramecc+:xnack-" : "gfx942");
    prop->multiProcessorCount = 256;
    return hipSuccess;
}

#define CHECK(cond)                                                          \
    do {                                                                     \
        if (!(cond)) {                                                       \
            std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
            std::exit(1);                                                    \
        }                                                                    \
    } while (0)

static uintptr_t g_ws_lo = 0, g_ws_hi = 0;
static void inside(const void* p, uint64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    CHECK(a >= g_ws_lo && a + bytes <= g_ws_hi && a % 16 == 0);
}

namespace bg {
int tune(int) { return g_tune; }
hipError_t launch_gated(const GatedProblem& p, hipStream_t) {
    CHECK(p.tile != GT_MIXED || (uint64_t)p.wide * 128 < (uint64_t)p.N + 128);
    CHECK(p.M > 0 && p.N > 0 && p.tile >= 0 && p.tile < GT_TILES && (p.G == nullptr) == (p.U == nullptr));
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_transposed(const TransposedProblem& p, hipStream_t) {
    CHECK(p.M > 0 && p.N > 0 && p.tile >= 0 && p.tile < GT_TILES && p.splits >= 1);
    CHECK(p.tile != GT_MIXED || (p.splits == 1 && (uint64_t)p.wide * 256 < (uint64_t)p.N + 256));
    CHECK(!(p.tn && p.tile == GT_160x256) && p.stacked >= 1 && p.M % p.stacked == 0 && p.lda >= (p.tn ? p.M / p.stacked : p.K));
    CHECK(p.splits <= (int)(p.K / 64 + 1) * (p.tn ? (p.low ? 2 : 1) : (int)p.parts));
    if (p.splits > 1 || p.stacked > 1) inside(p.planes, (uint64_t)p.splits * (p.tn ? p.parts : 1) * p.M * p.N * 4);
    if (p.parts == 2) {
        inside(p.A0, (uint64_t)(p.tn ? p.K : p.M) * p.lda * 2 + (p.low ? 2 * p.low : 0));
        inside(p.A1, (uint64_t)(p.tn ? p.K : p.M) * p.lda * 2 + (p.low ? 2 * p.low : 0));
    }
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_aligned_copy(const AlignedCopy& p, hipStream_t) {
    for (int i = 0; i < 2; ++i) {
        if (p.rows[i] == 0) continue;
        CHECK(p.ld[i] % 8 == 0 && p.ld[i] >= p.cols[i] && p.ld[i] < p.cols[i] + 8);
        inside(p.to[i], (uint64_t)p.rows[i] * p.ld[i] * 2);
    }
    CHECK(p.rows[0] != 0 || p.rows[1] != 0);
    return hipSuccess;
}
hipError_t launch_transposed_pair(const TransposedProblem& nn, const TransposedProblem& tn, hipStream_t s) {
    CHECK(!nn.tn && tn.tn && nn.tile == GT_128x128_DEEP && tn.tile == GT_128x128_DEEP);
    // all workgroups at once, planes that do not meet
    CHECK(gated_tiles(nn.tile, false, nn.M, nn.N, 1) * nn.splits + gated_tiles(tn.tile, false, tn.M, tn.N, 2) * tn.splits <= 256);
    CHECK(tn.planes >= nn.planes + (nn.splits > 1 || nn.stacked > 1 ? (uint64_t)nn.splits * nn.M * nn.N : 0));
    (void)launch_transposed(nn, s);
    (void)launch_transposed(tn, s);
    return hipSuccess;
}
hipError_t launch_gate_grad(const GateGradProblem& p, hipStream_t) {
    CHECK(p.M > 0 && p.N > 0 && p.ld % 8 == 0 && p.ld >= p.N && p.ld < p.N + 8);
    inside(p.dG, (uint64_t)p.M * p.ld * 2 + 2 * p.low);
    inside(p.dU, (uint64_t)p.M * p.ld * 2 + 2 * p.low);
    CHECK(p.dU == p.dG + (uint64_t)p.M * p.ld + p.low);
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_gemv_w4(const GemvProblem& p, hipStream_t) {
    CHECK(p.R > 0 && p.N > 0 && p.K % 32 == 0 && p.K % p.group == 0 && p.cus == 256);
    ++g_launches;
    return hipSuccess;
}
}  // namespace bg

template <class T>
static T* at(uintptr_t a) {
    return reinterpret_cast<T*>(a);
}

int main() {
    using namespace bg;
    const uint16_t *A = at<uint16_t>(0x1000000000), *B = at<uint16_t>(0x2000000000), *B1 = at<uint16_t>(0x3000000000),
                   *dH = at<uint16_t>(0x4000000000);
    uint16_t *C = at<uint16_t>(0x5000000000), *D = at<uint16_t>(0x6000000000), *D1 = at<uint16_t>(0x7000000000);
    void *G = at<void>(0x8000000000), *U = at<void>(0x9000000000), *ws = at<void>(0xA000000000);

    // every tile choice over a grid of shapes: a launch holds it, and the workspace holds what it is given
    const uint32_t sizes[] = {1, 7, 64, 65, 200, 1015, 4096, 11008, 40000};
    for (uint32_t M : sizes)
        for (uint32_t N : sizes)
            for (uint32_t K : sizes) {
                for (g_tune = -1; g_tune < 16 * 4; g_tune += g_tune < 0 ? 17 : 5) {
                    CHECK(gemm_bf16_gated(A, B, B1, C, G, U, BG_F32, BG_SILU, M, N, K, nullptr) == BG_OK);
                    for (int tn = 0; tn < 2; ++tn) {
                        size_t need = 1;
                        CHECK((tn ? gemm_bf16_tn_workspace : gemm_bf16_nn_workspace)(M, N, K, &need) == BG_OK);
                        g_ws_lo = (uintptr_t)ws, g_ws_hi = g_ws_lo + need;
                        CHECK((tn ? gemm_bf16_tn : gemm_bf16_nn)(A, B, C, ws, need, M, N, K, nullptr) == BG_OK);
                        if (need != 0) {
                            CHECK((tn ? gemm_bf16_tn : gemm_bf16_nn)(A, B, C, ws, need - 1, M, N, K, nullptr) == BG_ERR_WORKSPACE);
                            CHECK((tn ? gemm_bf16_tn : gemm_bf16_nn)(A, B, C, nullptr, need, M, N, K, nullptr) == BG_ERR_WORKSPACE);
                            CHECK((tn ? gemm_bf16_tn : gemm_bf16_nn)(A, B, C, C, need, M, N, K, nullptr) == BG_ERR_ALIAS);
                            CHECK((tn ? gemm_bf16_tn : gemm_bf16_nn)(A, B, C, at<void>(0xA000000008), need, M, N, K, nullptr) ==
                                  BG_ERR_ALIGN);
                        }
                    }
                    size_t need = 0;
                    CHECK(gemm_bf16_gated_backward_workspace(M, N, K, &need) == BG_OK && need > 0);
                    g_ws_lo = (uintptr_t)ws, g_ws_hi = g_ws_lo + need;
                    const int before = g_launches;
                    CHECK(gemm_bf16_gated_backward(dH, A, B, B1, G, U, BG_BF16, C, D, D1, BG_GELU_TANH, ws, need, M, N, K,
                                                   nullptr) == BG_OK);
                    CHECK(g_launches == before + 3);
                    CHECK(gemm_bf16_gated_backward(dH, A, B, B1, G, U, BG_BF16, C, D, D1, BG_GELU_TANH, ws, need - 1, M, N, K,
                                                   nullptr) == BG_ERR_WORKSPACE);
                }
            }
    g_tune = -1;
    // empty dimensions: an empty sum is still written
    size_t need = 0;
    CHECK(gemm_bf16_gated_backward_workspace(0, 5, 8, &need) == BG_OK);
    g_ws_lo = (uintptr_t)ws, g_ws_hi = g_ws_lo + need + 16;
    int before = g_launches;
    CHECK(gemm_bf16_gated_backward(nullptr, nullptr, B, B1, nullptr, nullptr, BG_F32, nullptr, D, D1, BG_SILU, ws, need, 0, 5, 8,
                                   nullptr) == BG_OK);
    CHECK(g_launches == before + 1);
    CHECK(gemm_bf16_gated_backward_workspace(70, 0, 8, &need) == BG_OK);
    CHECK(gemm_bf16_gated_backward(nullptr, A, nullptr, nullptr, nullptr, nullptr, BG_F32, C, nullptr, nullptr, BG_SILU, ws, need,
                                   70, 0, 8, nullptr) == BG_OK);
    CHECK(g_launches == before + 2);
    CHECK(gemm_bf16_gated_backward(dH, nullptr, nullptr, nullptr, G, U, BG_F32, C, D, D1, BG_SILU, ws, 1 << 20, 70, 5, 0,
                                   nullptr) == BG_OK);
    CHECK(g_launches == before + 2);
    // operands that no memory holds are refused before their byte counts are used
    CHECK(gemm_bf16_gated(A, B, B1, C, nullptr, nullptr, BG_F32, BG_SILU, 0x7FFFFFF0u, 1, 0x7FFFFFF0u, nullptr) == BG_ERR_SHAPE);
    CHECK(gemm_bf16_nn(A, B, C, nullptr, 0, 0x7FFFFFF0u, 1, 0x7FFFFFF0u, nullptr) == BG_ERR_SHAPE);

    bg_w4 w{at<uint8_t>(0x2000000000), at<void>(0x3000000000), nullptr, BG_W4_INT4, 64, 1.0f}, w1 = w;
    w1.codes = at<uint8_t>(0x8000000000), w1.scales = at<void>(0x9000000000);
    for (uint32_t R : {1u, 16u, 17u, 65536u})
        for (uint32_t K : {0u, 64u, 1u << 20}) {
            CHECK(gemv_w4(A, &w, at<uint16_t>(0xF000000000), R, 100, K, nullptr) == BG_OK);
            CHECK(gemv_w4_gated(A, &w, &w1, at<uint16_t>(0xF000000000), BG_SILU, R, 100, K, nullptr) == BG_OK);
        }
    g_dev = 1;
    CHECK(gemv_w4(A, &w, at<uint16_t>(0xF000000000), 1, 100, 64, nullptr) == BG_ERR_DEVICE);
    CHECK(gemm_bf16_gated_backward_workspace(5, 5, 8, &need) == BG_ERR_DEVICE);
    std::printf("api_gated sanitizer driver: ok\n");
    return 0;
}
