"""Helpers of the MXFP4 and routing GPU tests: operands, uploads, tolerances."""
import numpy as np
import torch

import oracle
import synthetic

U = 2.0 ** -24          # half a step of FP32, relative


def e8m0(rows, groups, lo, hi, seed, tid):
    """[rows, groups] scale bytes uniform over lo .. hi."""
    g = synthetic._rng(seed, tid)
    return g.integers(lo, hi + 1, size=(rows, groups), dtype=np.uint8)


def operand(rows, k, seed, tid, lo=122, hi=132):
    """Packed codes [rows, k/2] (all 16 codes alike) and scales 2^(lo-127) .. 2^(hi-127)."""
    return synthetic.fp4_packed(rows, k, seed, tid), e8m0(rows, k // 32, lo, hi, seed, tid + 50)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def check_product(got, a, sa, b, sb, what):
    """Against the FP64 product: half a BF16 step (2^-8 of the value), plus K
    roundings of FP32 (each at most 2^-24 of a partial sum, itself at most
    sum |a||b|), doubled for a sum inside the matrix instruction that keeps
    one bit less."""
    k = 2 * a.shape[-1]
    ref, size = oracle.gemm_mxfp4_ref(a, sa, b, sb), oracle.gemm_mxfp4_abs(a, sa, b, sb)
    got = f64(got)
    nan = np.isnan(ref)
    assert np.array_equal(nan, np.isnan(got)), f"{what}: NaN in other places"
    tol = 2.0 ** -8 * np.abs(ref) + 2 * (k + 1) * U * size
    bad = ~nan & ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def exact_bits(a, sa, b, sb):
    """BF16 bits of the product where every partial sum is exact in FP32."""
    return oracle.f32_to_bf16(oracle.gemm_mxfp4_ref(a, sa, b, sb).astype(np.float32))
