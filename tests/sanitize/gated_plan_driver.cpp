// Sanitizer driver for the plans that the GPU tests' shapes of the gradient and of products
// with tiles of two sizes take: what the argument layer (api_gated.cpp) hands to the
// launchers, which are replaced by recorders. Fake addresses are never dereferenced.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../block_scaled_fp4_gemm_amd/csrc/bg_internal.hpp"
#include "../../block_scaled_fp4_gemm_amd/csrc/gated_tiles.hpp"

hipError_t hipGetDevice(int* dev) {
    *dev = 0;
    return hipSuccess;
}

hipError_t hipGetDeviceProperties(hipDeviceProp_t* prop, int) {
    std::memset(prop, 0, sizeof(*prop));
    std::strcpy(prop->gcnArchName, "gfx950");
    prop->multiProcessorCount = 256;
    return hipSuccess;
}

static uint32_t m, n, k;

#define CHECK(cond)                                                                                              \
    do {                                                                                                         \
        if (!(cond)) {                                                                                           \
            std::fprintf(stderr, "%s:%d: check failed: %s (%ux%ux%u)\n", __FILE__, __LINE__, #cond, m, n, k);    \
            std::exit(1);                                                                                        \
        }                                                                                                        \
    } while (0)

static bg::TransposedProblem g_nn, g_tn;
static int g_gated = -1, g_pairs = 0, g_singles = 0;

namespace bg {
int tune(int) { return -1; }
hipError_t launch_gated(const GatedProblem& p, hipStream_t) {
    g_gated = p.tile;
    return hipSuccess;
}
hipError_t launch_transposed(const TransposedProblem& p, hipStream_t) {
    (p.tn ? g_tn : g_nn) = p;
    ++g_singles;
    return hipSuccess;
}
hipError_t launch_transposed_pair(const TransposedProblem& nn, const TransposedProblem& tn, hipStream_t) {
    g_nn = nn, g_tn = tn;
    ++g_pairs;
    return hipSuccess;
}
hipError_t launch_aligned_copy(const AlignedCopy&, hipStream_t) { return hipSuccess; }
hipError_t launch_gate_grad(const GateGradProblem&, hipStream_t) { return hipSuccess; }
hipError_t launch_gemv_w4(const GemvProblem&, hipStream_t) { return hipSuccess; }
}  // namespace bg

template <class T>
static T* at(uintptr_t a) {
    return reinterpret_cast<T*>(a << 40);
}

using namespace bg;

static void backward(uint32_t M, uint32_t N, uint32_t K) {
    m = M, n = N, k = K;
    g_pairs = g_singles = 0;
    CHECK(gemm_bf16_gated_backward(at<uint16_t>(1), at<uint16_t>(2), at<uint16_t>(3), at<uint16_t>(4), at<void>(5), at<void>(6), BG_F32,
                                   at<uint16_t>(7), at<uint16_t>(8), at<uint16_t>(9), BG_SILU, at<void>(10), (size_t)1 << 39, M, N, K,
                                   nullptr) == BG_OK);
    CHECK(g_pairs + g_singles == (g_pairs ? 1 : 2));
}

// The gradient's launch: both products at once or not, and through planes or not.
struct Pin {
    uint32_t m, n, k;
    bool pair, nn_planes, tn_planes;
};

int main() {
    // the shapes of the GPU tests, so that a change of the cost table shows where a
    // variant would no longer run
    const Pin pins[] = {{2000, 1000, 128, true, true, true},  {1030, 72, 64, true, false, true}, {300, 200, 136, true, false, false},
                        {1015, 1407, 520, true, true, false}, {40, 264, 1032, true, true, false}, {2100, 4100, 1032, false, true, false}, {5120, 11008, 2048, false, false, false}};
    for (const Pin& p : pins) {
        backward(p.m, p.n, p.k);
        std::printf("%ux%ux%u pair %d nn %d x %d tn %d x %d\n", p.m, p.n, p.k, g_pairs, g_nn.tile, g_nn.splits, g_tn.tile, g_tn.splits);
        CHECK((g_pairs == 1) == p.pair && (g_nn.splits > 1 || g_nn.stacked > 1) == p.nn_planes && (g_tn.splits > 1) == p.tn_planes);
        if (p.nn_planes && p.tn_planes) CHECK(g_tn.planes >= g_nn.planes + (size_t)g_nn.splits * g_nn.M * g_nn.N);
    }
    const uint32_t two[][3] = {{1016, 22000, 1032}, {2944, 10792, 1744}};
    for (const auto& s : two) {
        m = s[0], n = s[1], k = s[2];
        CHECK(gemm_bf16_nn(at<uint16_t>(1), at<uint16_t>(2), at<uint16_t>(3), at<void>(4), (size_t)1 << 39, m, n, k, nullptr) == BG_OK);
        CHECK(gemm_bf16_tn(at<uint16_t>(1), at<uint16_t>(2), at<uint16_t>(3), at<void>(4), (size_t)1 << 39, m, n, k, nullptr) == BG_OK);
        CHECK(gemm_bf16_gated(at<uint16_t>(1), at<uint16_t>(2), at<uint16_t>(3), at<uint16_t>(4), nullptr, nullptr, BG_F32, BG_SILU, m, n / 2,
                              k, nullptr) == BG_OK);
        std::printf("%ux%ux%u nn %d tn %d gated %d\n", m, n, k, g_nn.tile, g_tn.tile, g_gated);
        CHECK(g_nn.tile == GT_MIXED && g_tn.tile == GT_MIXED && g_gated == GT_MIXED);
    }
    std::printf("gated plan driver: ok\n");
    return 0;
}
