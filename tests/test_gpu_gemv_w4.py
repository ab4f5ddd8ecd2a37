"""Few rows times weights in 4 bits, and the gated block of few rows, against FP64."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
from gated_util import TINY, U16, U32, gate_error, normal, sum_error, within
from oracle import gated as og
from oracle.w4 import dequant_w4

pytestmark = pytest.mark.gpu

FORMATS = [("int4", 32, True), ("int4", 32, False), ("int4", 64, True), ("int4", 96, True), ("int4", 128, False),
           ("int4", 128, True), ("int4", 256, True), ("mxfp4", 32, False), ("nvfp4", 16, False)]


def weights(n, k, fmt, group, zeros, seed):
    """(W4Weights on the device, FP64 values): every code, scales over several
    binades, zero points over the whole byte now and then."""
    r = np.random.default_rng(seed)
    codes = r.integers(0, 256, (n, k // 2), dtype=np.uint8)
    z = None
    scale_2 = 1.0
    if fmt == "int4":
        s = (r.uniform(0.5, 2.0, (n, k // group)) * 2.0 ** r.integers(-4, 3, (n, k // group)) * r.choice([-1, 1], (n, k // group)))
        t = torch.from_numpy(s).bfloat16()
        raw, scales = t.view(torch.int16).numpy().view(np.uint16), t.cuda()
        if zeros:
            z = r.integers(0, 16, (n, k // group), dtype=np.uint8)
            z[r.random(z.shape) < 0.02] = 255
    elif fmt == "mxfp4":
        raw = r.integers(120, 131, (n, k // 32), dtype=np.uint8)
    else:
        raw = r.integers(0, 256, (n, k // 16), dtype=np.uint8)
        raw[(raw & 0x7F) == 0x7F] = 0x38
        scale_2 = 0.375
    if fmt != "int4":
        scales = torch.from_numpy(raw).cuda()
    w = bg.W4Weights(torch.from_numpy(codes).cuda(), scales, fmt, group=group, zeros=None if z is None else torch.from_numpy(z).cuda(),
                     scale_2=scale_2)
    return w, torch.from_numpy(dequant_w4(codes, raw, fmt, group, z, scale_2)).cuda()


def bound(x, v, w):
    """(value, error bound) of the FP32 sums. INT4 sums (16 + q) x and (16 + z) x
    instead of (q - z) x: codes at most 31, zero points at most 271, times |s|."""
    x = x.double()
    size = x.abs() @ v.abs().T
    if w.format == "int4":
        s = w.scales.double().abs().repeat_interleave(w.group, 1)
        z = 24.0 if w.zeros is None else 16.0 + w.zeros.double().repeat_interleave(w.group, 1)
        size = x.abs() @ (s * (31 + z)).T
    return x @ v.T, sum_error(size, 2 * x.shape[1]) + 4 * U32 * size


def check(y, x, w, v, what):
    want, err = bound(x, v, w)
    within(y, want, U16 * (want.abs() + err) + err + TINY, what)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("r,n,groups", [(1, 1, 1), (1, 64, 3), (2, 17, 5), (16, 100, 8), (17, 33, 9), (5, 300, 40), (40, 16, 2)])
def test_gemv(r, n, groups, fmt, group, zeros):
    k = groups * max(group, 32)
    x = normal((r, k), 1.0, 1)
    w, v = weights(n, k, fmt, group, zeros, 2)
    y = bg.gemv_w4(x, w)
    check(y, x, w, v, f"{r}x{n}x{k} {fmt} {group}")
    for i in (0, r - 1):       # whatever the other rows hold: the same bits
        other = torch.full_like(x, float("nan"))
        other[i] = x[i]
        assert torch.equal(bg.gemv_w4(other, w)[i], y[i])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("r,n,groups", [(1, 1, 1), (3, 70, 7), (16, 64, 16), (18, 33, 5)])
def test_gemv_gated(r, n, groups, fmt, group, zeros, act):
    k = groups * max(group, 32)
    x = normal((r, k), 0.05, 1)
    (w0, v0), (w1, v1) = (weights(n, k, fmt, group, zeros, seed) for seed in (2, 3))
    h = bg.gemv_w4_gated(x, w0, w1, act=act)
    (g, eg), (u, eu) = bound(x, v0, w0), bound(x, v1, w1)
    a = og.gate(g, act)[0].abs()
    want = og.gate(g, act)[0] * u
    err = 1.13 * eg * (u.abs() + eu) + a * eu + gate_error(g, act) * (a + 1.13 * eg) * (u.abs() + eu)
    within(h, want, U16 * (want.abs() + err) + err + TINY, f"{r}x{n}x{k} {fmt} {group} {act}")
