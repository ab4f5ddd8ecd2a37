// Sanitizer driver for the MXFP4 and routing part of the C-ABI validation
// layer (api_mx.cpp), built for the host with -fsanitize=address,undefined
// against hip_stub/. The launchers are replaced by recorders that check what
// validation hands them. Fake device addresses are never dereferenced.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "../../block_scaled_fp4_gemm_amd/csrc/bg_internal.hpp"

static int g_dev = 0;
static int g_launches = 0;

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

namespace bg {
hipError_t launch_mxfp4_quantize(const MxQuantProblem& p, hipStream_t) {
    CHECK(p.R > 0 && p.K > 0 && p.K % 32 == 0 && p.ldx >= p.K);
    CHECK(p.rows != nullptr || p.R == p.M);
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_mxfp4_dequantize(const uint8_t*, const uint8_t*, void*, int, uint32_t M, uint32_t K, hipStream_t) {
    CHECK(M > 0 && K > 0 && K % 32 == 0);
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_gemm_mxfp4(const MxGemmProblem& p, hipStream_t) {
    CHECK(p.M > 0 && p.N > 0 && p.K % 32 == 0 && p.cus == 256);
    CHECK(p.E >= 1 && p.E <= kMaxExperts && (p.offsets != nullptr || p.E == 1));
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_moe_route(const RouteProblem& p, hipStream_t) {
    CHECK(p.E >= 1 && p.E <= kMaxExperts && p.k >= 1 && p.k <= kMaxTopK && p.k <= p.E);
    CHECK(p.T <= kRouteOneBlock || p.ws != nullptr);
    // every workgroup owns a row range, and the ranges cover the batch
    const uint64_t rows = route_rows_per_block(p.T), blocks = route_blocks(p.T);
    CHECK(p.T <= kRouteOneBlock || (rows * blocks >= p.T && rows * (blocks - 1) < p.T));
    CHECK(rows % 32 == 0 && rows < 65536 && (blocks <= 256 || p.T > 256 * 65000u));
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_moe_route_backward(const RouteBackwardProblem& p, hipStream_t) {
    CHECK(p.T > 0 && p.E >= 1 && p.k >= 1);
    ++g_launches;
    return hipSuccess;
}
}  // namespace bg

template <class T>
static T* at(uintptr_t a) {
    return reinterpret_cast<T*>(a);
}

int main() {
    const uint8_t *A = at<uint8_t>(0x10000000), *B = at<uint8_t>(0x20000000), *SA = at<uint8_t>(0x40000000),
                  *SB = at<uint8_t>(0x50000000);
    uint16_t* C = at<uint16_t>(0x30000000);
    int32_t* off = at<int32_t>(0x70000000);
    uint8_t *codes = at<uint8_t>(0x100000000), *scales = at<uint8_t>(0x200000000);

    CHECK(mxfp4_quantize(A, BG_BF16, 64, nullptr, codes, scales, 5, 5, 64, nullptr) == BG_OK);
    CHECK(mxfp4_quantize(A, BG_F32, 70, off, codes, scales, 5, 9, 64, nullptr) == BG_OK);
    CHECK(mxfp4_quantize(nullptr, BG_F32, 64, off, codes, scales, 0, 9, 64, nullptr) == BG_OK);
    // operands that no memory holds are refused before their byte counts are used
    CHECK(mxfp4_quantize(A, BG_F32, 0x7FFFFFE0u, nullptr, codes, scales, 0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFE0u,
                         nullptr) == BG_ERR_SHAPE);
    CHECK(gemm_mxfp4(A, SA, B, SB, C, 0x7FFFFFFFu, 0x7FFFFFFFu, 32, nullptr) == BG_ERR_SHAPE);
    CHECK(gemm_mxfp4_grouped(A, SA, B, SB, off, C, 4, 0x7FFFFFFFu, 0x7FFFFFE0u, 1024, nullptr) == BG_ERR_SHAPE);
    CHECK(mxfp4_dequantize(codes, scales, C, BG_F32, 3, 96, nullptr) == BG_OK);
    CHECK(gemm_mxfp4(A, SA, B, SB, C, 7, 9, 96, nullptr) == BG_OK);
    CHECK(gemm_mxfp4(nullptr, nullptr, nullptr, nullptr, C, 7, 9, 0, nullptr) == BG_OK);
    CHECK(gemm_mxfp4_grouped(A, SA, B, SB, off, C, 7, 9, 96, 3, nullptr) == BG_OK);
    CHECK(g_launches == 7);

    bg_moe_routing out{at<int32_t>(0x300000000), at<float>(0x400000000), at<int32_t>(0x500000000),
                       at<int32_t>(0x600000000), at<int32_t>(0x700000000), at<int32_t>(0x800000000),
                       at<float>(0x900000000),   at<float>(0xA00000000),   at<int32_t>(0xB00000000)};
    void* ws = at<void>(0xC00000000);
    for (uint32_t T : {0u, 1u, 64u, 65u, 100u, 16384u, 16385u, 4510u, 65536u, 1000003u, 100000000u}) {
        const size_t need = moe_route_workspace_bytes(T, 256);
        CHECK((need == 0) == (T <= bg::kRouteOneBlock));
        CHECK(moe_route(A, BG_BF16, nullptr, &out, ws, need, T, 256, 8, 1, nullptr) ==
              (T > 30000000u ? BG_ERR_ALIAS : BG_OK));   // the longest batch's arrays meet at these addresses
        if (need != 0) CHECK(moe_route(A, BG_BF16, nullptr, &out, ws, need - 1, T, 256, 8, 1, nullptr) == BG_ERR_WORKSPACE);
    }
    CHECK(moe_route_backward(A, BG_BF16, out.ids, out.weights, out.counts, out.n_valid, nullptr, nullptr, codes, 9,
                             8, 2, 0, nullptr) == BG_OK);
    g_dev = 1;
    CHECK(gemm_mxfp4(A, SA, B, SB, C, 7, 9, 96, nullptr) == BG_ERR_DEVICE);
    CHECK(moe_route(A, BG_F32, nullptr, &out, nullptr, 0, 4, 256, 8, 1, nullptr) == BG_ERR_DEVICE);
    std::printf("api_mx sanitizer driver: ok\n");
    return 0;
}
