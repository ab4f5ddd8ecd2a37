// The activations of the gated MLP block, on FP32 values in registers.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/blockgemm.h"

namespace bg {

// act(g) = g s(z(g)), s(z) = 1 / (1 + e^-z). Silu: z = g; gelu (tanh form): z =
// 2 sqrt(2 / pi) (g + 0.044715 g^3). e^-z is one exp2, whose argument rounds
// twice (2^-23 of |z|), so s is off by 2^-23 (|z| + 2) of its value: far below
// half a BF16 step, 2^-9. Past z = -88.7 e^-z overflows and s is 0, where act(g)
// is below 2^-121 and would be 0 or the smallest numbers of BF16.
constexpr float kLog2e = 1.44269504f;
constexpr float kGeluC = 1.59576912f;         // 2 sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;

template <int ACT>
__device__ __forceinline__ float gate_sigmoid(float g) {
    const float z = ACT == BG_SILU ? g : kGeluC * __builtin_fmaf(kGeluK * g * g, g, g);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -kLog2e));
}

template <int ACT>
__device__ __forceinline__ float gate(float g) {
    return g * gate_sigmoid<ACT>(g);
}

}  // namespace bg
