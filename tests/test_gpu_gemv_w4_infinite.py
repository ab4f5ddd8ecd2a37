"""Weights in 4 bits beside infinities and values next to FP32's range: what the
definition gives, sum of s (q - z) x, not what its rearrangement gives."""
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
from gated_util import U16, normal, sum_error
from oracle import gated as og
from test_gpu_gemv_w4 import bound, weights

pytestmark = pytest.mark.gpu

INF = float("inf")
GROUPS = [(32, True), (64, False), (96, True), (128, True), (256, False)]


def same(got, want, tol, what):
    """Finite where want is, within tol; elsewhere the same infinity, or NaN."""
    got = got.double()
    finite = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: {got} {want}"
    assert torch.equal(got[~finite].nan_to_num(7), want[~finite].nan_to_num(7)), what
    assert ((got - want).abs()[finite] <= tol[finite]).all(), what


def terms(x, v):
    """Sum of the products one by one: 0 inf is NaN there, whatever a library's product does."""
    return (x.double().unsqueeze(1) * v.unsqueeze(0)).sum(-1)


@pytest.mark.parametrize("group,zeros", GROUPS)
@pytest.mark.parametrize("r", [1, 3, 16, 18])
def test_infinite_activations(r, group, zeros):
    n, k = 37, 5 * group
    w, v = weights(n, k, "int4", group, zeros, 2)
    w.codes[0], v[0] = 0x88, 0
    if zeros:
        w.zeros[0] = 8
    x = normal((r, k), 1.0, 1)
    clean = bg.gemv_w4(x, w)
    x[0, 7] = INF
    if r > 2:
        x[2, k - 1] = -INF
        x[1, 3], x[1, k - 2] = INF, -INF
    size = terms(x.nan_to_num(0, 0, 0).abs(), (w.scales.double().abs() * 300).repeat_interleave(group, 1))
    want = terms(x, v)
    assert want[0, 0].isnan() and want[0].isinf().any()         # q = z, and others
    same(bg.gemv_w4(x, w), want, U16 * want.abs() + sum_error(size, 2 * k), f"{r} {group}")
    keep = [i for i in range(r) if i > 2 or (i and r < 3)]
    assert torch.equal(bg.gemv_w4(x, w)[keep], clean[keep])
    if r > 2:
        h = bg.gemv_w4_gated(x, w, w)
        g = want[[0, 2]]
        ref = og.gate(g, "silu")[0] * g
        assert torch.equal(h[[0, 2]].isnan(), ref.isnan()) and torch.equal(h[[0, 2]].double().nan_to_num(7, 8, 9), ref.nan_to_num(7, 8, 9))


@pytest.mark.parametrize("group,zeros", GROUPS)
def test_sums_next_to_the_range(group, zeros):
    """(16 + q) x and (16 + z) sum x pass 2^128, s (q - z) x does not."""
    n, k = 20, 3 * group
    w, v = weights(n, k, "int4", group, zeros, 3)
    w = w._replace(scales=(w.scales.double() * 2.0 ** -20).bfloat16())
    v = v * 2.0 ** -20
    x = (normal((2, k), 1.0, 1).double() * 2.0 ** 124).clamp(-3e38, 3e38).bfloat16()
    size = terms(x.abs(), v.abs())
    assert size.max() < 2.0 ** 126
    want, err = bound(x, v, w)           # of the rearranged sum, where it stays in the range
    same(bg.gemv_w4(x, w), want, U16 * (want.abs() + err) + err, f"{group}")


@pytest.mark.parametrize("group,zeros", GROUPS)
def test_infinite_scales(group, zeros):
    """An infinite scale is its column's; K ends inside a stretch, behind which
    the column's first scale must not be used."""
    r, n, k = 3, 20, 3 * group
    w, v = weights(n, k, "int4", group, zeros, 4)
    x = normal((r, k), 1.0, 1).abs() + 1
    clean = bg.gemv_w4(x, w)
    s, codes, z = w.scales.clone(), w.codes.clone(), w.zeros
    s[3, 0], s[5, 1], s[6, 0] = INF, -INF, INF
    codes[3], codes[5], codes[6, 0] = 0x99, 0x99, 0x88
    if zeros:
        z = z.clone()
        z[3], z[5], z[6] = 8, 8, 8
    y = bg.gemv_w4(x, w._replace(scales=s, codes=codes, zeros=z))
    assert (y[:, 3] == INF).all() and (y[:, 5] == -INF).all() and y[:, 6].isnan().all()
    cols = [i for i in range(n) if i not in (3, 5, 6)]
    assert torch.equal(y[:, cols], clean[:, cols])


def test_nvfp4_sums_past_the_range_before_the_second_scale():
    n, k = 20, 96
    w, v = weights(n, k, "nvfp4", 16, False, 5)
    w, v = w._replace(scale_2=2.0 ** -30), v / 0.375 * 2.0 ** -30
    x = (normal((2, k), 1.0, 1).double() * 2.0 ** 125).clamp(-3e38, 3e38).bfloat16()
    size = terms(x.abs(), v.abs())
    assert size.max() < 2.0 ** 126 and (size.min() * 2.0 ** 30).item() > 2.0 ** 128
    want = terms(x, v)
    same(bg.gemv_w4(x, w), want, U16 * want.abs() + sum_error(size, 2 * k), "nvfp4")
    x[1, 40] = -INF
    want = terms(x, v)
    same(bg.gemv_w4(x, w), want, U16 * want.abs() + sum_error(size, 2 * k), "nvfp4, infinite")
