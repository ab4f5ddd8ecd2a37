"""Values of weights in 4 bits with group scales, in FP64 (test infrastructure only)."""
from __future__ import annotations

import numpy as np

from .codecs import bf16_to_f64, e2m1_to_f64, e4m3fn_to_f64
from .mxfp4 import e8m0_to_f64


def _nibbles(codes):
    codes = np.asarray(codes, dtype=np.uint8)
    out = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), np.uint8)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def dequant_w4(codes, scales, fmt: str, group: int, zeros=None, scale_2: float = 1.0) -> np.ndarray:
    """[N, K] values: codes [N, K/2] bytes, scales [N, K/group] (BF16 bits for
    "int4", bytes otherwise), zeros [N, K/group] bytes or None (8)."""
    q = _nibbles(codes)
    per = lambda v: np.repeat(v, group, axis=1)  # noqa: E731
    if fmt == "int4":
        z = 8.0 if zeros is None else per(np.asarray(zeros).astype(np.float64))
        return (q.astype(np.float64) - z) * per(bf16_to_f64(scales))
    if fmt == "mxfp4":
        return e2m1_to_f64(q) * per(e8m0_to_f64(scales))
    return e2m1_to_f64(q) * per(e4m3fn_to_f64(scales)) * float(np.float32(scale_2))
