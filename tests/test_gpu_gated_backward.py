"""The gated block's gradient in the launch variants and sizes where it could go
wrong: both products through planes of their own in one launch, drawn shapes,
operands past 32-bit offsets."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
from gated_util import U32, check_backward, normal, sum_error, within

pytestmark = pytest.mark.gpu


def operands(m, n, k):
    return (normal((m, n), 0.01, 4), normal((m, k), 1.0, 1), normal((n, k), 1.5 / k ** 0.5, 2), normal((n, k), 1.0 / k ** 0.5, 3))


def guarded_backward(dh, a, b0, b1, g, u, act):
    """In a workspace of just the size, full of NaN."""
    nbytes = bg.gemm_bf16_gated_backward_workspace(*g.shape, a.shape[1])
    buf = torch.full((nbytes + 512,), 0xFF, device="cuda", dtype=torch.uint8)
    grads = bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, act=act, workspace=buf[256:256 + nbytes])
    assert (buf[:256] == 0xFF).all() and (buf[256 + nbytes:] == 0xFF).all()
    return grads


# planes of: both, tn alone, nn alone, neither; two launches; K % 8 != 0
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,n,k", [(2000, 1000, 128), (1030, 72, 64), (1015, 1407, 520), (300, 200, 136), (2100, 4100, 1032),
                                   (40, 264, 1032), (64, 3000, 72), (1, 24, 11008), (700, 520, 1003), (50, 520, 1003), (33, 265, 27)])
def test_workspace_of_just_the_size(m, n, k, act):
    dh, a, b0, b1 = operands(m, n, k)
    _, g, u = bg.gemm_bf16_gated(a, b0, b1, act=act, save=True)
    grads = guarded_backward(dh, a, b0, b1, g, u, act)
    check_backward(*grads, dh, a, b0, b1, g, u, act, f"{m}x{n}x{k} {act}")
    for again in range(2):
        assert all(torch.equal(p, q) for p, q in zip(bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, act=act), grads))


@pytest.mark.parametrize("seed", range(24))
def test_drawn_shapes(seed):
    r = np.random.default_rng(300 + seed)
    m, n, k = (int(v) for v in np.exp(r.uniform(0, np.log([2500, 1500, 1500]))))
    if seed % 2:
        k = (k + 7) // 8 * 8
    act, kept = ("silu", "gelu_tanh")[seed // 2 % 2], (torch.float32, torch.bfloat16)[seed // 4 % 2]
    dh, a, b0, b1 = operands(m, n, k)
    _, g, u = bg.gemm_bf16_gated(a, b0, b1, act=act, save=kept)
    check_backward(*guarded_backward(dh, a, b0, b1, g, u, act), dh, a, b0, b1, g, u, act, f"{m}x{n}x{k} {act}")


def test_offsets_past_32_bits():
    """dH, dG and dU of more than 2^32 bytes, G and U of twice as many, checked at
    rows and columns up to the last."""
    m, n, k = (1 << 16) + 77, 33_000, 64
    dh, a, b0, b1 = operands(m, n, k)
    _, g, u = bg.gemm_bf16_gated(a, b0, b1, save=True)
    rows = torch.cat([torch.arange(35), torch.arange(m - 35, m)]).cuda()
    cols = torch.cat([torch.arange(3), torch.arange(n - 35, n)]).cuda()
    for kept, b in ((g, b0), (u, b1)):
        x, w = a[rows].double(), b.double()
        want = x @ w.T
        within(kept[rows], want, U32 * want.abs() + sum_error(x.abs() @ w.abs().T, k), "kept")
    da, db0, db1 = bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u)
    check_backward(da[rows], None, None, dh[rows], a[rows], b0, b1, g[rows], u[rows], "silu", "rows")
    check_backward(None, db0[cols], db1[cols], dh[:, cols], a, b0[cols], b1[cols], g[:, cols], u[:, cols], "silu", "columns")
