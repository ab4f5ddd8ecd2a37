"""Size limits of the MXFP4 entry points (CPU only): the tile choice under
sanitizers, and the C ABI's answers at the limits, with fake addresses that
are never dereferenced."""
import os

import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
from test_sanitizers_cpu import GXX, SAN, _build_and_run

L = bg.lib
BIG = (1 << 31) - 1
A, SA, B, SB, C, O = (i << 50 for i in range(1, 7))
BF16, F32 = 0, 1


@pytest.mark.skipif(GXX is None, reason="g++ not found")
def test_tile_choice_under_sanitizers(tmp_path):
    out = _build_and_run(tmp_path, "mx_tiles_san", [os.path.join(SAN, "mx_tiles_driver.cpp")])
    assert "mx_tiles sanitizer driver: ok" in out


def test_products_that_no_launch_holds_are_refused_as_shapes():
    assert L.gemm_mxfp4(A, SA, B, SB, C, BIG, 100000, 32, None) == bg.BG_ERR_SHAPE
    assert L.gemm_mxfp4(A, SA, B, SB, C, BIG, 1, 512, None) == bg.BG_ERR_SHAPE
    assert L.gemm_mxfp4_grouped(A, SA, B, SB, O, C, BIG, 1, 32, 1024, None) == bg.BG_ERR_SHAPE
    # empty products have no size to refuse
    assert L.gemm_mxfp4(None, None, None, None, None, BIG, 0, 512, None) == bg.BG_OK
    assert L.gemm_mxfp4_grouped(None, None, None, None, None, None, BIG, 0, 32, 1024, None) == bg.BG_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="a device is present")
def test_sizes_within_the_limits_pass_the_checks():
    for m, n, k in [(1 << 29, 64, 32), ((1 << 29) + 5, 3, 32), (BIG, 1, 32), (64, 1 << 29, 32), ((1 << 31) - 256, 1, 512)]:
        assert L.gemm_mxfp4(A, SA, B, SB, C, m, n, k, None) == bg.BG_ERR_DEVICE, (m, n, k)
    for s, n, k, e in [((1 << 29) + 5, 3, 32, 2), (1 << 24, 4096, 2048, 256), ((1 << 30) - (1 << 18), 1, 1024, 1024)]:
        assert L.gemm_mxfp4_grouped(A, SA, B, SB, O, C, s, n, k, e, None) == bg.BG_ERR_DEVICE, (s, n, k, e)
    assert L.mxfp4_quantize(A, BF16, 544, None, B, SB, BIG, BIG, 544, None) == bg.BG_ERR_DEVICE


def test_quantisation_of_more_pieces_than_it_numbers_is_refused_as_a_shape():
    q = L.mxfp4_quantize
    assert q(A, BF16, 1056, None, B, SB, BIG, BIG, 1056, None) == bg.BG_ERR_SHAPE
    assert q(A, F32, 1 << 20, O, B, SB, 4, 1 << 21, 1 << 20, None) == bg.BG_ERR_SHAPE
