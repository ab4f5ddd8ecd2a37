// Device helpers of the matrix-core kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Swizzled 16-byte chunk slot of logical chunk c in a tile row of CPR chunks
// (CPR = BK/8). The XOR keeps the eight (CPR = 8) or four (CPR = 4) chunks of a
// row in distinct slots, and gives one logical chunk distinct banks across the
// 8 consecutive rows (or the 16 rows, for 256-byte bank windows) that the
// lanes of one 16-byte LDS read touch. It is an involution in c.
template <int CPR>
__device__ __forceinline__ int chunk_slot(int row, int c) {
    if constexpr (CPR == 8)
        return c ^ ((row ^ (row >> 3)) & 7);
    else
        return c ^ (((row >> 1) ^ (row >> 3)) & 3);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup barrier that orders LDS only. __syncthreads() would also wait for
// every outstanding global load of the wave (its release fence covers global
// memory), which would drain the direct-load ring at every step. Before the
// barrier this wave's LDS reads and writes are complete; the direct loads
// the caller needs are covered by its own vmcnt wait.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    bf16x2 v = {(__bf16)lo, (__bf16)hi};   // v_cvt_pk_bf16_f32: round to nearest even
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

// A pointer every lane holds the same value of, stated as such so that a
// buffer resource built from it stays in scalar registers (the inline-asm
// loads need it there) whatever the compiler's divergence analysis concludes.
__device__ __forceinline__ void* uniform_ptr(const void* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
}

// Scheduling groups for one sub-step: NM MFMAs, ND LDS reads and NV direct
// (VMEM) loads, issued as MFMA, LDS read, VMEM, MFMA, ... until the memory
// instructions run out, then the remaining MFMAs.
template <int NM, int ND, int NV>
__device__ __forceinline__ void interleave_mfma() {
#pragma unroll
    for (int q = 0; q < NM; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                     // MFMA
        if (q < ND) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);         // LDS read
        if (q < NV) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);         // VMEM read
    }
    if (NV > NM) __builtin_amdgcn_sched_group_barrier(0x020, NV - NM, 0);
    if (ND > NM) __builtin_amdgcn_sched_group_barrier(0x100, ND - NM, 0);
}

}  // namespace bg
