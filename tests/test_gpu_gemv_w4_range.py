"""MXFP4 weights over the whole range of their scale bytes: 6 * 2^127 is past
BF16, 0.5 * 2^-127 among its smallest numbers."""
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
from gated_util import TINY, U16, gate_error, normal, within
from oracle import gated as og
from oracle.w4 import dequant_w4
from test_gpu_gemv_w4 import bound, check

pytestmark = pytest.mark.gpu

ENDS = (0, 1, 2, 127, 251, 252, 253, 254)


def held(codes, scales):
    """(W4Weights, FP64 values) of host tensors."""
    v = torch.from_numpy(dequant_w4(codes.numpy(), scales.numpy(), "mxfp4", 32)).cuda()
    return bg.W4Weights(codes.cuda(), scales.cuda(), "mxfp4"), v


def far_weights(n, blocks, seed):
    """Random codes; a block's byte is at an end of the range, one more or one less by
    the row, and 127 in every fifth row. Also 2^(127 - byte), as BF16 holds it."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, 16 * blocks), generator=g, dtype=torch.uint8)
    base = torch.tensor(ENDS)[torch.randint(0, len(ENDS), (blocks,), generator=g)]
    scales = (base + torch.randint(-1, 2, (n, blocks), generator=g)).clamp(0, 254)
    scales[::5] = 127
    size = torch.exp2((127 - base).clamp(-120, 100).double()).repeat_interleave(32)
    return codes, scales.to(torch.uint8), size.cuda()


@pytest.mark.parametrize("others", [(), (254, 1, 253)])
@pytest.mark.parametrize("byte", ENDS)
def test_every_code_exactly(byte, others):
    scales = torch.tensor([byte, *others], dtype=torch.uint8).repeat(16, 1)
    codes = torch.arange(16, dtype=torch.uint8).view(16, 1).repeat(1, 16 * scales.shape[1])
    k = 2 * codes.shape[1]
    w, v = held(codes, scales)
    x = torch.zeros(3, k, device="cuda", dtype=torch.bfloat16)
    size = 2.0 ** max(-100, min(100, 127 - byte))
    x[0, 4], x[1, 10], x[2, 30] = size, -size, 1.5 * size
    assert torch.equal(bg.gemv_w4(x, w).double(), x.double() @ v.T)
    inf = torch.full((1, k), float("inf"), device="cuda", dtype=torch.bfloat16)
    inf[0, 1:] = 0
    want = (inf.double()[:, :1] * v[:, :1].T).float()        # 0 * inf and the zeros: NaN
    got = bg.gemv_w4(inf, w).float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7), want.nan_to_num(7))


@pytest.mark.parametrize("r,n,blocks", [(1, 5, 1), (1, 70, 23), (3, 33, 130), (8, 100, 65), (16, 64, 67), (18, 33, 16)])
def test_far_scales(r, n, blocks):
    codes, scales, size = far_weights(n, blocks, n)
    w, v = held(codes, scales)
    x = (normal((r, 32 * blocks), 1.0, 1).double() * size).bfloat16()
    y = bg.gemv_w4(x, w)
    check(y, x, w, v, f"{r}x{n}x{32 * blocks}")
    # a row of weights without such bytes: the same bits whatever its neighbours hold
    near = scales.clone()
    near[torch.arange(n) % 5 != 0] = 120
    assert torch.equal(bg.gemv_w4(x, held(codes, near)[0])[:, ::5], y[:, ::5])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("r,n,blocks", [(1, 40, 20), (5, 33, 40), (16, 17, 9)])
def test_far_scales_gated(r, n, blocks, act):
    codes, scales, size = far_weights(n, blocks, 3)
    size = size.clamp(max=1)               # or the rows of 127 pass the range
    (w0, v0), (w1, v1) = held(codes, scales), held(codes.flip(0).contiguous(), scales)
    x = (normal((r, 32 * blocks), 0.05, 1).double() * size).bfloat16()
    (g, eg), (u, eu) = bound(x, v0, w0), bound(x, v1, w1)
    gate = og.gate(g, act)[0]
    err = 1.13 * eg * (u.abs() + eu) + gate.abs() * eu + gate_error(g, act) * (gate.abs() + 1.13 * eg) * (u.abs() + eu)
    within(bg.gemv_w4_gated(x, w0, w1, act=act), gate * u, U16 * ((gate * u).abs() + err) + err + TINY, f"{r}x{n}x{32 * blocks} {act}")
