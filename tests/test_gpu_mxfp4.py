"""GPU parity of MXFP4 quantisation and reading back: bit for bit."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
import oracle
import synthetic
from mx_util import dev, f64

pytestmark = pytest.mark.gpu


def _x(rows, k, dtype, seed):
    """N(0, 1) rows with a wide spread of block sizes, zeros of both signs and empty blocks."""
    g = synthetic._rng(seed, 7)
    x = g.standard_normal((rows, k)) * np.repeat(np.exp2(g.integers(-40, 40, (rows, k // 32))), 32, 1)
    x[g.random((rows, k)) < 0.1] = 0.0
    x[g.random((rows, k)) < 0.05] = -0.0
    x[np.repeat(g.random((rows, k // 32)) < 0.1, 32, 1)] = 0.0
    return torch.from_numpy(x).to(dtype)


def _check(x, codes, scales, what, rows=None):
    v = f64(x)
    if rows is not None:
        ok = (rows >= 0) & (rows < v.shape[0])
        v = np.where(ok[:, None], v[np.where(ok, rows, 0)], 0.0)
    want, ws = oracle.quantize_mxfp4(v)
    assert np.array_equal(scales.cpu().numpy(), ws), f"{what}: scales"
    assert np.array_equal(codes.cpu().numpy(), want), f"{what}: codes"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 7168), (3, 96), (17, 544), (5, 512), (130, 1056), (300, 2080), (2, 32768)])
def test_quantize_bit_exact(rows, k, dtype):
    print(f"quantize {rows}x{k} {dtype}", flush=True)
    x = _x(rows, k, dtype, rows + k)
    codes, scales = bg.mxfp4_quantize(x.cuda())
    _check(x, codes, scales, f"{rows}x{k}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_code_boundary_and_its_neighbours(dtype):
    """Each value and midpoint of E2M1 (and the next numbers beside it) under
    every scale byte that a value of the type can give, both signs."""
    mags = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9375])
    t = torch.tensor(np.concatenate([mags, -mags]), dtype=torch.float32).to(dtype)
    up, down = torch.nextafter(t, torch.full_like(t, 100.0)), torch.nextafter(t, torch.full_like(t, -100.0))
    v = torch.cat([t, up, down]).double().numpy()
    v = v[np.abs(v) < 8]
    blocks = -(-len(v) // 31)
    v = np.resize(v, (blocks, 31))
    rows = []
    for e in range(-126, 126):
        rows.append(np.concatenate([np.full((blocks, 1), 4.0), v], 1) * 2.0 ** e)      # the 4 fixes the scale
    x = torch.from_numpy(np.stack(rows).reshape(252, -1)).to(dtype)
    codes, scales = bg.mxfp4_quantize(x.cuda())
    _check(x, codes, scales, "boundaries")
    assert set(np.unique(scales.cpu().numpy())) == set(range(1, 253))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_values(dtype):
    info = torch.finfo(dtype)
    vals = [float("nan"), float("inf"), -float("inf"), info.max, info.min, info.tiny, -info.tiny, info.smallest_normal / 2,
            info.smallest_normal * info.eps, 2.0 ** -124, 2.0 ** -125, 1.0]
    x = torch.zeros(len(vals), 128, dtype=dtype)
    for i, v in enumerate(vals):
        x[i, 40] = v
        x[i, 64:96] = v
    codes, scales = bg.mxfp4_quantize(x.cuda())
    _check(x, codes, scales, "special")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pitch", [1, 4, 8, 64])
def test_row_strides(dtype, pitch):
    k = 160
    base = _x(33, 2048, dtype, 3).cuda()
    view = base[:, :k + pitch].clone()[:, :k]
    assert view.stride(0) == k + pitch
    codes, scales = bg.mxfp4_quantize(view)
    _check(view, codes, scales, f"pitch {pitch}")
    codes, scales = bg.mxfp4_quantize(base[:, :k])
    _check(base[:, :k], codes, scales, "wide pitch")


@pytest.mark.parametrize("k", [32, 544, 2048])
def test_row_list(k):
    x = _x(50, k, torch.bfloat16, 4)
    rows = np.array([49, 0, 0, 7, -1, 50, 7, 2 ** 31 - 1, -2 ** 31, 13], np.int32)
    codes, scales = bg.mxfp4_quantize(x.cuda(), rows=dev(rows))
    _check(x, codes, scales, "row list", rows=rows.astype(np.int64))
    none = bg.mxfp4_quantize(x.cuda(), rows=dev(rows[:0]))
    assert none[0].shape == (0, k // 2)
    # a source without rows: everything is zero
    c, s = bg.mxfp4_quantize(x[:0].cuda(), rows=dev(rows[:3]))
    assert not c.any() and not s.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequantize_every_code_under_every_scale(dtype):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))          # K = 512, 16 blocks
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    got = bg.mxfp4_dequantize(dev(codes), dev(scales), dtype=dtype)
    want = torch.from_numpy(oracle.dequant_mxfp4(codes, scales)).to(dtype)      # exact, or infinite
    g, w = got.cpu().double(), want.double()
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    assert torch.equal(g[~torch.isnan(w)], w[~torch.isnan(w)])
    assert torch.equal(torch.signbit(g[:255]), torch.signbit(w[:255]))


def test_round_trip_is_idempotent_and_within_half_a_step():
    x = _x(64, 4096, torch.bfloat16, 5).cuda()
    codes, scales = bg.mxfp4_quantize(x)
    v = bg.mxfp4_dequantize(codes, scales, dtype=torch.float32)
    c2, s2 = bg.mxfp4_quantize(v)
    assert torch.equal(bg.mxfp4_dequantize(c2, s2, dtype=torch.float32), v)
    # a step of the top binade is 2 (in units of the scale): off by 1, and by 2 where 8 saturates at 6
    unit = torch.exp2(scales.float() - 127).repeat_interleave(32, 1)
    assert ((v - x.float()).abs() <= 2 * unit).all()


def test_quantize_past_32_bit_offsets():
    """More than 2^32 elements, sampled rows."""
    rows, k = 140000, 32768
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 20000):
        x[i:i + 20000].normal_()
    codes, scales = bg.mxfp4_quantize(x)
    back = bg.mxfp4_dequantize(codes, scales)
    for i in (0, 1, 65535, 65536, 131071, 131072, rows - 1):
        xi = x[i:i + 1].cpu()
        _check(xi, codes[i:i + 1], scales[i:i + 1], f"row {i}")
        want = oracle.dequant_mxfp4(codes[i:i + 1].cpu().numpy(), scales[i:i + 1].cpu().numpy())
        assert np.array_equal(f64(back[i:i + 1]), want)
    # the same rows by a row list
    pick = torch.tensor([rows - 1, 131073, 5], dtype=torch.int32, device="cuda")
    c, s = bg.mxfp4_quantize(x, rows=pick)
    assert torch.equal(c, codes[pick.long()]) and torch.equal(s, scales[pick.long()])
