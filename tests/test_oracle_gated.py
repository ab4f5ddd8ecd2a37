"""The gated block's and the 4-bit weights' oracle, pinned against something
other than itself: torch's activations and their autograd in FP64, central
differences, and the codes written out one by one."""
import numpy as np
import pytest
import torch

from oracle import gated as og
from oracle.w4 import dequant_w4

G = np.concatenate((np.linspace(-30, 30, 601), [0.0, -0.0, 1e-8, -1e-8, 300.0, -300.0]))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activation_and_slope(act):
    t = torch.from_numpy(G).requires_grad_()
    want = torch.nn.functional.silu(t) if act == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    (slope,) = torch.autograd.grad(want.sum(), t)
    v, s = og.gate(G, act)
    assert np.allclose(v, want.detach().numpy(), rtol=1e-12, atol=1e-15)
    assert np.allclose(s, slope.numpy(), rtol=1e-9, atol=1e-12)
    v, s = og.gate(torch.from_numpy(G), act)
    assert np.allclose(v.numpy(), want.detach().numpy(), rtol=1e-12, atol=1e-15)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradient_against_differences(act):
    r = np.random.default_rng(1)
    a, b0, b1, dh = r.normal(size=(5, 7)), r.normal(size=(6, 7)), r.normal(size=(6, 7)), r.normal(size=(5, 6))
    _, g, u = og.gated(a, b0, b1, act)
    grads = og.gated_backward(dh, a, b0, b1, g, u, act)
    for i, x in enumerate((a, b0, b1)):
        d, eps = r.normal(size=x.shape), 1e-5
        ends = []
        for s in (eps, -eps):
            args = [a, b0, b1]
            args[i] = x + s * d
            ends.append((dh * og.gated(*args, act)[0]).sum())
        # a central difference is off by eps^2 / 6 times a third derivative of order one
        assert abs((ends[0] - ends[1]) / (2 * eps) - (grads[i] * d).sum()) < 1e-7


E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_dequant_w4_code_by_code():
    r = np.random.default_rng(2)
    n, k = 3, 128
    q = r.integers(0, 16, (n, k))
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)
    s = torch.from_numpy(r.normal(size=(n, k // 32))).bfloat16()
    z = r.integers(0, 256, (n, k // 32), dtype=np.uint8)
    bits = s.view(torch.int16).numpy().view(np.uint16)
    got, sym = dequant_w4(codes, bits, "int4", 32, z), dequant_w4(codes, bits, "int4", 32)
    e8, e4 = r.integers(100, 150, (n, k // 32), dtype=np.uint8), r.integers(0, 0x7F, (n, k // 16), dtype=np.uint8)
    gm, gn = dequant_w4(codes, e8, "mxfp4", 32), dequant_w4(codes, e4, "nvfp4", 16, scale_2=0.75)
    e4v = torch.from_numpy(e4).view(torch.float8_e4m3fn).double().numpy()
    for i in range(n):
        for j in range(k):
            sv = s[i, j // 32].item()
            assert got[i, j] == sv * (q[i, j] - float(z[i, j // 32])) and sym[i, j] == sv * (q[i, j] - 8.0)
            assert gm[i, j] == E2M1[q[i, j]] * 2.0 ** (int(e8[i, j // 32]) - 127)
            assert gn[i, j] == E2M1[q[i, j]] * e4v[i, j // 16] * 0.75
