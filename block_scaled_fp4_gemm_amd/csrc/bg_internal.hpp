// Internal host-side declarations shared by the C-ABI layer and the kernel
// translation units. Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/blockgemm.h"

namespace bg {

// Epilogue applied to the FP32 accumulator tile of the MFMA core.
enum Epilogue : int {
    EPI_STORE_BF16 = 0,   // C = bf16(acc)
    EPI_SCALED_ACC = 1,   // out = bf16(out + scale * bf16(acc)), in place
    EPI_STORE_F32 = 2,    // plane[blockIdx.z] = acc (split-K partials)
    EPI_SCALE_BF16 = 3,   // C = bf16(fl32(scale * acc))  (W4A16 per-tensor scale)
};

struct DenseProblem {
    const uint16_t* A;   // [M, K] bf16
    const uint16_t* B;   // [N, K] bf16
    void* C;             // [M, N] bf16, or [splits][M][N] f32 planes
    uint32_t M, N, K;
    uint32_t lda, ldb;   // elements between rows of A and of B (>= K)
    uint32_t ldc;        // elements between rows of C (>= N; N for split-K planes)
    uint32_t k_chunk;    // K elements per split (multiple of 64, or K)
    uint32_t splits;
    float scale;
    uint32_t cus;        // compute units of the current device (tile choice), 0 = unknown
};

struct Fp4Problem {
    const uint8_t* A;    // [batch][M, K/2]
    const uint8_t* SFA;  // [batch][M, K/16]
    const uint8_t* B;    // [batch][N, K/2]
    const uint8_t* SFB;  // [batch][N, K/16]
    void* C;             // [batch][M, N] bf16, or [splits][M][N] f32 planes
    uint32_t M, N, K;
    uint32_t k_chunk;    // K elements per split (multiple of 64, or K)
    uint32_t splits;     // > 1: FP32 planes (batch must be 1)
    uint32_t batch;
    uint32_t cus;        // compute units of the device (0: 256)
};

struct W4a16Problem {
    const uint16_t* A;   // [M, K] bf16 activations
    const uint8_t* B;    // [N, K/2] packed e2m1 weights
    const uint8_t* SFB;  // [N, K/16] e4m3fn
    uint16_t* C;         // [M, N] bf16
    uint32_t M, N, K;
    float scale_2;       // per-tensor weight scale
    uint32_t cus;        // compute units of the current device (tile choice)
    uint32_t ldbt;       // 0: B [N, K/2], SFB [N, K/16]; else B [K/2, ldbt], SFB [K/16, ldbt] (transposed)
};

struct MxQuantProblem {
    const void* x;         // [M, K] of type, rows ldx elements apart
    const int32_t* rows;   // [R] source rows, or NULL (row i is row i)
    uint8_t* codes;        // [R, K/2]
    uint8_t* scales;       // [R, K/32]
    uint32_t M, R, K, ldx;
    int type;              // bg_type of x
};

struct MxGemmProblem {
    const uint8_t* A;      // [M, K/2] packed e2m1
    const uint8_t* SFA;    // [M, K/32] e8m0
    const uint8_t* B;      // [E][N, K/2]
    const uint8_t* SFB;    // [E][N, K/32]
    uint16_t* C;           // [M, N] bf16
    uint32_t M, N, K;
    const int32_t* offsets;   // [E + 1] row ranges of the experts, or NULL (one product of all rows)
    uint32_t E;
    uint32_t cus;          // compute units of the device (tile choice)
};

struct RouteProblem {
    const void* logits;    // [T, E] of type
    int type;              // bg_type of the logits
    const uint8_t* valid;  // [T] or NULL
    bg_moe_routing out;
    void* ws;              // route_workspace_bytes(T, E)
    uint32_t T, E, k;
    int normalize;
};

struct RouteBackwardProblem {
    const void* logits;    // [T, E] of type
    int type;
    const int32_t* ids;
    const float* weights;
    const int32_t* counts;
    const int32_t* n_valid;
    const float* dweights;   // [T, k] or NULL
    const float* dloss;      // [1] or NULL
    void* dlogits;         // [T, E] of type
    uint32_t T, E, k;
    int normalize;
};

// Pieces of 512 elements (a wave's) of a row of mxfp4_quantize, which numbers those of all rows in 32 bits.
constexpr uint32_t mx_quant_pieces(uint32_t K) { return K / 512 + (K % 512 != 0); }
constexpr uint32_t kMaxMxK = 1u << 24;     // MXFP4 products: 256 rows of K / 2 bytes stay within 32-bit offsets
constexpr uint32_t kMaxExperts = 1024;   // routing and grouped products
constexpr uint32_t kMaxTopK = 16;

// Up to this many rows one workgroup routes alone, in one launch, without a
// workspace. 256 experts, k = 8, us alone and in two launches, BF16: 32 rows 7.8
// and 11.5, 64 rows 9.8 and 11.6, 96 rows 13.0 and 11.7; FP32: 9.2 and 12.7, 12.8
// and 12.9, 17.0 and 13.0.
constexpr uint32_t kRouteOneBlock = 64;
// Above this many rows the workgroups of moe_route have 1024 threads, else 512.
// 256 experts, k = 8, us of a call with 512 and 1024, BF16: 2048 rows 13.6 and
// 14.8, 4510 rows 16.1 and 16.3, 16384 rows 21.8 and 21.3, 65536 rows 38.9 and
// 36.4; FP32: 15.1 and 17.2, 18.0 and 19.0, 25.8 and 24.7, 50.0 and 45.1. (From
// 8192 rows on 1024 is level or ahead: 19.4 and 16.9 there, 18.3 and 18.0 at 12288.)
constexpr uint32_t kRouteWide = 16384;
// Rows per workgroup of moe_route: of whole passes (32 tokens per 512 threads
// where 16 lanes hold one), as many as leave at most 256 workgroups, so that each
// can sum the counts of all the others by itself; but fewer than 2^16 rows, so
// that counts fit 16 bits. Past 256 * 65472 rows there are more workgroups, and
// that sum grows as the square of the rows.
constexpr uint32_t kRouteMaxRows = 65472;
inline uint32_t route_rows_per_block(uint32_t T) {
    const uint32_t pass = T > kRouteWide ? 64 : 32;
    const uint32_t rows = (T / 256 + (T % 256 != 0) + pass - 1) / pass * pass;
    return rows < kRouteMaxRows ? rows : kRouteMaxRows;
}
inline uint32_t route_blocks(uint32_t T) {
    if (T <= kRouteOneBlock) return 1;
    const uint32_t r = route_rows_per_block(T);
    return T / r + (T % r != 0);
}
// Per workgroup: E sums of probabilities, the number of live rows (the whole
// rounded up to 16 bytes), E counts of 16 bits.
inline size_t route_workspace_bytes(uint32_t T, uint32_t E) {
    if (T <= kRouteOneBlock) return 0;
    const size_t n = route_blocks(T);
    return n * E * 4 + (n + 3) / 4 * 16 + n * E * 2;
}

// Size of the library-owned split-K scratch of gemm_bf16_splitk_noalloc, per
// device (noalloc.hip).
constexpr size_t kNoallocScratchBytes = BG_NOALLOC_SCRATCH_BYTES;
// Device address of the current device's scratch (taken once per device).
hipError_t noalloc_scratch(void** ptr);

// Current tuning override of a bg_tune_key (-1: automatic choice).
int tune(int key);

// Kernel launchers (defined in the .hip files). They enqueue on `stream` and
// return hipGetLastError() of the launch. Shapes are already validated and
// non-empty (M > 0, N > 0).
hipError_t launch_dense(const DenseProblem& p, Epilogue epi, hipStream_t stream);
// C0 = bf16(A * B^T) (the problem p, BF16 store) and C1 = bf16(A * B1^T) of the
// same shape, in one launch when the direct kernels apply.
hipError_t launch_dense_dual(const DenseProblem& p, const uint16_t* B1, uint16_t* C1, hipStream_t stream);
hipError_t launch_fp4(const Fp4Problem& p, hipStream_t stream);
// Stream-K (gemm_bf16_streamk; the plan and the tile choice are in
// streamk_plan.hpp): p.C is the BF16 output, ws the workspace of
// streamk_choose's size for configuration cfg.
hipError_t launch_streamk(const DenseProblem& p, void* ws, int cfg, uint64_t epoch, hipStream_t stream);
hipError_t launch_scales_from_blocked(const uint8_t* src, uint8_t* dst, uint32_t rows, uint32_t k_groups,
                                      uint32_t batch, hipStream_t stream);
hipError_t launch_w4a16(const W4a16Problem& p, hipStream_t stream);
hipError_t launch_ordered(const uint16_t* A, const uint16_t* B, void* C, bool f32_out,
                          uint32_t M, uint32_t N, uint32_t K, uint32_t cus, hipStream_t stream);
hipError_t launch_splitk_reduce(const float* ws, uint16_t* C, uint32_t M, uint32_t N,
                                uint32_t splits, hipStream_t stream);
hipError_t launch_scaled_add(uint16_t* out, const uint16_t* delta, size_t count, float scale,
                             hipStream_t stream);

hipError_t launch_mxfp4_quantize(const MxQuantProblem& p, hipStream_t stream);
hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, void* out, int type, uint32_t M,
                                   uint32_t K, hipStream_t stream);
// Dense (offsets NULL) and grouped MXFP4 products; K > 0 or K == 0 (zeros).
hipError_t launch_gemm_mxfp4(const MxGemmProblem& p, hipStream_t stream);
// T may be 0 (the sums of an empty batch are still written).
hipError_t launch_moe_route(const RouteProblem& p, hipStream_t stream);
hipError_t launch_moe_route_backward(const RouteBackwardProblem& p, hipStream_t stream);

}  // namespace bg
