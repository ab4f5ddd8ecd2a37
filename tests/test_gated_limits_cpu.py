"""Sizes whose tiles a launch does not hold are refused as shapes, for operands
whose rows do not start at multiples of 16 bytes too: those go in smaller tiles
(CPU only; addresses are fake and never dereferenced)."""
import ctypes

import pytest
import torch

import block_scaled_fp4_gemm_amd as bg

L = bg.lib
A, B, B1, C = 0x10_0000_0000_0000, 0x20_0000_0000_0000, 0x30_0000_0000_0000, 0x40_0000_0000_0000
G, U, D, D1, W = (0x50_0000_0000_0000 + 0x8_0000_0000_0000 * i for i in range(5))


def gated(m, n, k):
    return L.gemm_bf16_gated(A, B, B1, C, None, None, 0, 0, m, n, k, None)


def nn(m, n, k):
    return L.gemm_bf16_nn_workspace(m, n, k, ctypes.byref(ctypes.c_size_t()))


def tn(m, n, k):
    return L.gemm_bf16_tn_workspace(m, n, k, ctypes.byref(ctypes.c_size_t()))


def grad(m, n, k):
    return L.gemm_bf16_gated_backward_workspace(m, n, k, ctypes.byref(ctypes.c_size_t()))


# 2^24 tiles of 128 x 128 and more, 256 threads each: 2^32 threads
REFUSED = [
    (gated, 1 << 30, 65, 1),                       # 2^23 x 2 tiles of 128 rows and 64 columns
    (gated, 129, (1 << 29) + 192, 7),
    (gated, 129, (1 << 29) + 192, 129),
    (nn, 1 << 30, 129, 1), (nn, 129, (1 << 30) + 1, 8), (nn, 1 << 30, 136, 7),
    (tn, 1 << 29, 129, 1), (tn, (1 << 29) + 1, 136, 1),
    (tn, 1 << 29, 136, 8),                         # A's rows hold M elements, past 32-bit offsets of a tile's rows
    (grad, 1 << 30, 65, 1),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_too_many_small_tiles(i):
    call, *size = REFUSED[i]
    assert call(*size) == bg.BG_ERR_SHAPE


HELD = [
    (gated, 1 << 30, 65, 8),                       # tiles of 256 rows and 128 columns
    (gated, (1 << 30) - 128, 65, 1), (gated, 129, (1 << 29) - 64, 1), (gated, 128, (1 << 30) - 128, 1),
    (nn, 1 << 30, 136, 8), (nn, (1 << 30) - 128, 129, 1), (nn, 128, (1 << 31) - 256, 1), (nn, 1 << 30, 128, 1),
    (tn, (1 << 29) - 128, 129, 1),
    (grad, 1 << 30, 64, 1),
]


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the gated calls would launch on fake pointers")
@pytest.mark.parametrize("i", range(len(HELD)))
def test_the_largest_sizes_reach_the_device_check(i):
    call, *size = HELD[i]
    assert call(*size) == bg.BG_ERR_DEVICE
