"""The gated block, its gradient and the transposed products against FP64."""
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
from gated_util import check_backward, check_gated, check_product, grid, normal
from oracle import gated as og

pytestmark = pytest.mark.gpu

TILES = range(7)
# one element, one row, less than a step, whole steps, odd everything, several
# tiles of every size with ragged edges
SHAPES = [(1, 1, 1), (1, 8, 8), (3, 130, 64), (64, 64, 64), (65, 127, 72), (128, 136, 128), (300, 200, 136),
          (257, 513, 1000), (70, 1000, 251), (5, 2048, 2056)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gated(m, n, k, act):
    a, b0, b1 = normal((m, k), 1.0, 1), normal((n, k), 1.5 / k ** 0.5, 2), normal((n, k), 1.0 / k ** 0.5, 3)
    h = bg.gemm_bf16_gated(a, b0, b1, act=act)
    check_gated(h, a, b0, b1, act, f"{m}x{n}x{k} {act}")
    h2, g, u = bg.gemm_bf16_gated(a, b0, b1, act=act, save=torch.bfloat16)
    h3, g32, u32 = bg.gemm_bf16_gated(a, b0, b1, act=act, save=True)
    assert torch.equal(h, h2) and torch.equal(h, h3)
    check_product(g, a, b0.t(), "G")
    check_product(u, a, b1.t(), "U")
    assert g32.dtype == torch.float32 and torch.equal(g32.bfloat16(), g) and torch.equal(u32.bfloat16(), u)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n,k", [(3, 130, 64), (257, 300, 1000), (513, 261, 72), (300, 200, 131)])
def test_every_tile_gives_the_same_bits(m, n, k, tile, force):
    a, b0, b1 = normal((m, k), 1.0, 1), normal((n, k), 1.0 / k ** 0.5, 2), normal((n, k), 1.0 / k ** 0.5, 3)
    bt = b0.t().contiguous()
    at = a.t().contiguous()
    want = bg.gemm_bf16_gated(a, b0, b1, save=True)
    force(bg.TUNE_TILE, 16 + 0)
    nn, tn = bg.gemm_bf16_nn(a, bt), bg.gemm_bf16_tn(at, bt)
    force(bg.TUNE_TILE, 16 + tile)
    for got, w in zip(bg.gemm_bf16_gated(a, b0, b1, save=True), want):
        assert torch.equal(got, w)
    assert torch.equal(bg.gemm_bf16_nn(a, bt), nn)
    assert torch.equal(bg.gemm_bf16_tn(at, bt), tn)
    check_product(nn, a, bt, "nn")
    check_product(tn, a, bt, "tn")


# 1.3 and 3.9 rounds of the widest tiles: the last columns go in narrower ones
@pytest.mark.parametrize("m,n,k", [(1016, 22000, 1032), (2944, 10792, 1744)])
def test_tiles_of_two_sizes_in_one_launch(m, n, k, force):
    a, b = normal((m, k), 1.0, 1), normal((k, n), 1.0 / k ** 0.5, 2)
    at, b0, b1 = a.t().contiguous(), b[:, :n // 2].t().contiguous(), b[:, n // 2:].t().contiguous()
    run = lambda: (bg.gemm_bf16_nn(a, b), bg.gemm_bf16_tn(at, b), *bg.gemm_bf16_gated(a, b0, b1, save=True))
    got = run()
    force(bg.TUNE_TILE, 16 + 0)
    for g, w in zip(got, run()):
        assert torch.equal(g, w)
    check_product(got[0], a, b, "nn")
    check_gated(got[2], a, b0, b1, "silu", "gated")


@pytest.mark.parametrize("m,n,k", SHAPES + [(512, 264, 5000), (16, 64, 4096), (2048, 520, 64)])
def test_transposed_products(m, n, k):
    a, b = normal((m, k), 1.0, 1), normal((k, n), 1.0, 2)
    check_product(bg.gemm_bf16_nn(a, b), a, b, f"nn {m}x{n}x{k}")
    at = a.t().contiguous()
    check_product(bg.gemm_bf16_tn(at, b), a, b, f"tn {m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1015, 2087, 1001), (513, 1000, 1291), (2056, 777, 264), (77, 2047, 640), (1, 5461, 2049), (130, 71, 4097)])
def test_rows_copied_to_aligned_ones(m, n, k):
    """In a workspace of just the size, full of NaN."""
    a, b = normal((m, k), 1.0, 1), normal((k, n), 1.0, 2)
    for f, need, x in ((bg.gemm_bf16_nn, bg.gemm_bf16_nn_workspace, a), (bg.gemm_bf16_tn, bg.gemm_bf16_tn_workspace, a.t().contiguous())):
        size = need(m, n, k)
        copies = sum(t.shape[0] * ((t.shape[1] + 7) // 8 * 16) for t in (x, b) if t.shape[1] % 8)
        assert size >= copies
        buf = torch.full((size + 256,), 0xFF, device="cuda", dtype=torch.uint8)
        got = f(x, b, workspace=buf[:size])
        check_product(got, a, b, f"{f.__name__} {m}x{n}x{k}")
        assert (buf[size:] == 0xFF).all() and torch.equal(f(x, b), got)


@pytest.mark.parametrize("splits", [2, 3, 7])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n,k", [(130, 264, 1000), (64, 121, 448), (72, 128, 40)])
def test_split_reduction_is_exact_on_whole_numbers(m, n, k, tile, splits, force):
    a, b = grid((m, k), 1), grid((k, n), 2)
    want = (a.double() @ b.double()).float().bfloat16()
    force(bg.TUNE_TILE, 16 * splits + tile)
    for _ in range(2):
        assert torch.equal(bg.gemm_bf16_nn(a, b), want)
        assert torch.equal(bg.gemm_bf16_tn(a.t().contiguous(), b), want)


@pytest.mark.parametrize("kept", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,n,k", SHAPES + [(1030, 72, 64), (40, 3000, 136), (33, 1029, 264), (63, 520, 1000)])
def test_backward(m, n, k, act, kept):
    a, b0, b1 = normal((m, k), 1.0, 1), normal((n, k), 1.5 / k ** 0.5, 2), normal((n, k), 1.0 / k ** 0.5, 3)
    dh = normal((m, n), 0.01, 4)
    _, g, u = bg.gemm_bf16_gated(a, b0, b1, act=act, save=kept)
    grads = bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, act=act)
    check_backward(*grads, dh, a, b0, b1, g, u, act, f"{m}x{n}x{k} {act}")
    da, n0, n1 = bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, act=act, need_b=False)
    assert n0 is None and n1 is None and torch.equal(da, grads[0])
    na, db0, db1 = bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, act=act, need_a=False)
    assert na is None and torch.equal(db0, grads[1]) and torch.equal(db1, grads[2])


@pytest.mark.parametrize("parts", [0, 3])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n,k", [(40, 300, 600), (300, 515, 264)])
def test_backward_of_every_tile(m, n, k, tile, parts, force):
    a, b0, b1 = normal((m, k), 1.0, 1), normal((n, k), 1.5 / k ** 0.5, 2), normal((n, k), 1.0 / k ** 0.5, 3)
    dh = normal((m, n), 0.01, 4)
    _, g, u = bg.gemm_bf16_gated(a, b0, b1, save=True)
    force(bg.TUNE_TILE, 16 * parts + tile)
    grads = bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u)
    check_backward(*grads, dh, a, b0, b1, g, u, "silu", f"{m}x{n}x{k} tile {tile}")
