"""MXFP4 definitions (test infrastructure only), written out with numpy in FP64.

OCP Microscaling Formats v1.0: blocks of 32 consecutive elements of a row, one
E8M0 scale byte s per block (2^(s-127), 255 = NaN), E2M1 elements.
"""
from __future__ import annotations

import numpy as np

from .codecs import e2m1_to_f64, unpack_e2m1

BLOCK = 32


def e8m0_to_f64(b) -> np.ndarray:
    """2^(b - 127); 255 is NaN."""
    v = np.asarray(b, dtype=np.int64)
    return np.where(v == 255, np.nan, np.exp2((v - 127).astype(np.float64)))


def f64_to_e2m1(x) -> np.ndarray:
    """The nearest E2M1 code, by distance to every magnitude: ties to the even
    code, beyond 6 the code of 6; the sign bit of x is kept."""
    x = np.asarray(x, dtype=np.float64)
    mags = e2m1_to_f64(np.arange(8))
    dist = np.abs(np.minimum(np.abs(x), 8.0)[..., None] - mags)      # 8 and all above it are nearest to 6
    near = dist.min(-1, keepdims=True)
    tied = dist == near
    # among the (at most two) nearest codes an even one wins
    even = tied & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), tied.argmax(-1))
    return (pick + 8 * np.signbit(x)).astype(np.uint8)


def quantize_mxfp4(x):
    """(packed codes [R, K/2], scale bytes [R, K/32]) of values x [R, K].

    Shared exponent of a block: floor(log2(max |x|)) - 2, at least -127; blocks
    whose maximum is zero or below 2^-126 take scale byte 0; blocks with a NaN
    or an infinity take 255 and codes 0.
    """
    x = np.asarray(x, dtype=np.float64)
    r, k = x.shape
    assert k % BLOCK == 0
    b = x.reshape(r, k // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    top = np.abs(np.where(bad[..., None], 0.0, b)).max(-1, initial=0.0)
    # frexp: top = m * 2^e with 1/2 <= m < 1, so floor(log2 top) = e - 1
    e = np.frexp(top)[1] - 1 - 2
    s = np.where(top < 2.0 ** -126, 0, np.maximum(e + 127, 0))
    codes = f64_to_e2m1(np.where(bad[..., None], 0.0, b) * np.exp2(127.0 - s)[..., None])
    codes = np.where(bad[..., None], 0, codes).reshape(r, k).astype(np.uint8)
    scales = np.where(bad, 255, s).astype(np.uint8)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def dequant_mxfp4(packed, scales) -> np.ndarray:
    """Exact FP64 values [..., K] of packed codes [..., K/2] and scales [..., K/32]."""
    codes = unpack_e2m1(packed)
    return e2m1_to_f64(codes) * np.repeat(e8m0_to_f64(scales), BLOCK, axis=-1)


def gemm_mxfp4_ref(a, sfa, b, sfb) -> np.ndarray:
    """FP64 C = deq(A) @ deq(B)^T. NaN blocks make their row or column NaN."""
    with np.errstate(invalid="ignore"):
        return dequant_mxfp4(a, sfa) @ dequant_mxfp4(b, sfb).T


def gemm_mxfp4_abs(a, sfa, b, sfb) -> np.ndarray:
    """sum_k |a||b|: what the rounding errors of a sum are measured against."""
    with np.errstate(invalid="ignore"):
        return np.abs(dequant_mxfp4(a, sfa)) @ np.abs(dequant_mxfp4(b, sfb)).T


def gemm_mxfp4_grouped_ref(a, sfa, b, sfb, offsets) -> np.ndarray:
    """Rows offsets[e] .. offsets[e+1]-1 of A times B[e]^T; rows outside every range are NaN."""
    out = np.full((a.shape[0], b.shape[1]), np.nan)
    for e in range(b.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            out[lo:hi] = gemm_mxfp4_ref(a[lo:hi], sfa[lo:hi], b[e], sfb[e])
    return out
