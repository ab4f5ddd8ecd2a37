"""Argument checks of the MXFP4 and routing entry points (CPU only): the
binding's, with the library replaced by a stub that fails if reached, and the
C ABI's, with fake addresses that are never dereferenced."""
import ctypes

import pytest
import torch

import block_scaled_fp4_gemm_amd as bg


class _NoLib:
    def __getattr__(self, name):
        if name == "moe_route_workspace_bytes":
            return lambda t, e: 0

        def called(*a, **k):
            raise AssertionError(f"library entry point {name} was called")
        return called


@pytest.fixture
def nolib(monkeypatch):
    monkeypatch.setattr(bg, "lib", _NoLib())


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def f32(*s):
    return torch.zeros(s)


def routing(t, e, k, **other):
    r = bg.MoeRouting(i32(t, k), f32(t, k), i32(e), i32(e + 1), i32(t * k), i32(t, k), f32(e), f32(1)[0], i32(1)[0], k, True)
    return r._replace(**other)


BAD = [
    (lambda: bg.mxfp4_quantize(bf(4, 48)), ValueError),                              # K % 32
    (lambda: bg.mxfp4_quantize(bf(4, 32, 1)), ValueError),
    (lambda: bg.mxfp4_quantize(torch.zeros(4, 32, dtype=torch.float16)), TypeError),
    (lambda: bg.mxfp4_quantize([1.0]), TypeError),
    (lambda: bg.mxfp4_quantize(bf(32, 4).t()), ValueError),                          # columns apart
    (lambda: bg.mxfp4_quantize(bf(4, 32), rows=torch.zeros(4, dtype=torch.int64)), TypeError),
    (lambda: bg.mxfp4_quantize(bf(4, 32), rows=i32(4, 1)), ValueError),
    (lambda: bg.mxfp4_quantize(bf(4, 32), rows=i32(3), out=u8(4, 16)), ValueError),
    (lambda: bg.mxfp4_quantize(bf(4, 32), scales=u8(4, 2)), ValueError),
    (lambda: bg.mxfp4_quantize(bf(4, 32), out=bf(4, 16)), TypeError),
    (lambda: bg.mxfp4_dequantize(u8(4, 8), u8(4, 1)), ValueError),                   # K = 16
    (lambda: bg.mxfp4_dequantize(u8(4, 16), u8(4, 2)), ValueError),
    (lambda: bg.mxfp4_dequantize(u8(4, 16), u8(4, 1), dtype=torch.float16), TypeError),
    (lambda: bg.mxfp4_dequantize(u8(4, 16), u8(4, 1), out=bf(4, 31)), ValueError),
    (lambda: bg.gemm_mxfp4(u8(4, 16), u8(4, 2), u8(5, 16), u8(5, 1)), ValueError),   # SFA
    (lambda: bg.gemm_mxfp4(u8(4, 16), u8(4, 1), u8(5, 16), u8(5, 2)), ValueError),   # SFB
    (lambda: bg.gemm_mxfp4(u8(4, 16), u8(4, 1), u8(5, 32), u8(5, 2)), ValueError),   # K
    (lambda: bg.gemm_mxfp4(u8(4, 24), u8(4, 1), u8(5, 24), u8(5, 1)), ValueError),   # K = 48
    (lambda: bg.gemm_mxfp4(bf(4, 16), u8(4, 1), u8(5, 16), u8(5, 1)), TypeError),
    (lambda: bg.gemm_mxfp4(u8(4, 16), u8(4, 1), u8(5, 16), u8(5, 1), out=bf(5, 4)), ValueError),
    (lambda: bg.gemm_mxfp4(u8(4, 16), u8(4, 1), u8(5, 16), u8(5, 1), out=f32(4, 5)), TypeError),
    (lambda: bg.gemm_mxfp4_grouped(u8(4, 16), u8(4, 1), u8(5, 16), u8(5, 1), i32(2)), ValueError),      # B without experts
    (lambda: bg.gemm_mxfp4_grouped(u8(4, 16), u8(4, 1), u8(2, 5, 16), u8(2, 5, 1), i32(2)), ValueError),
    (lambda: bg.gemm_mxfp4_grouped(u8(4, 16), u8(4, 1), u8(2, 5, 16), u8(2, 5, 1), f32(3)), TypeError),
    (lambda: bg.gemm_mxfp4_grouped(u8(4, 16), u8(4, 1), u8(2, 5, 16), u8(5, 1), i32(3)), ValueError),
    (lambda: bg.moe_route(f32(4, 8), 0), ValueError),
    (lambda: bg.moe_route(f32(4, 8), 9), ValueError),
    (lambda: bg.moe_route(f32(4, 64), 17), ValueError),
    (lambda: bg.moe_route(torch.zeros(4, 8, dtype=torch.float64), 2), TypeError),
    (lambda: bg.moe_route(f32(8), 2), ValueError),
    (lambda: bg.moe_route(f32(4, 8), 2, valid=i32(4)), TypeError),
    (lambda: bg.moe_route(f32(4, 8), 2, valid=u8(5)), ValueError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(5, 8, 2)), ValueError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 9, 2)), ValueError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2), dweights=f32(4, 3)), ValueError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2), dweights=bf(4, 2)), TypeError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2), dloss=f32(2)), ValueError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2), out=bf(4, 8)), TypeError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2), out=f32(4, 9)), ValueError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2, ids=f32(4, 2))), TypeError),
    (lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2, n_valid=i32(2))), ValueError),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_bad_arguments_raise_before_the_library(i, nolib):
    call, exc = BAD[i]
    with pytest.raises(exc):
        call()


HOST = [
    lambda: bg.mxfp4_quantize(bf(4, 32)),
    lambda: bg.mxfp4_quantize(f32(4, 64), rows=i32(3)),
    lambda: bg.mxfp4_dequantize(u8(4, 16), u8(4, 1)),
    lambda: bg.gemm_mxfp4(u8(4, 16), u8(4, 1), u8(5, 16), u8(5, 1)),
    lambda: bg.gemm_mxfp4_grouped(u8(4, 16), u8(4, 1), u8(2, 5, 16), u8(2, 5, 1), i32(3)),
    lambda: bg.moe_route(f32(4, 8), 2),
    lambda: bg.moe_route_backward(f32(4, 8), routing(4, 8, 2)),
]


@pytest.mark.parametrize("i", range(len(HOST)))
def test_host_tensors_are_rejected(i, nolib):
    with pytest.raises(ValueError, match="device"):
        HOST[i]()


# --- the C ABI ---------------------------------------------------------------

A, B, C, S1, S2, W, O = (0x10000000 * i for i in range(1, 8))
L = bg.lib
BF16, F32 = 0, 1


def test_quantize_checks():
    q = L.mxfp4_quantize
    assert q(None, BF16, 32, None, None, None, 0, 0, 32, None) == bg.BG_OK
    assert q(None, BF16, 0, None, None, None, 4, 4, 0, None) == bg.BG_OK
    assert q(A, BF16, 48, None, C, S1, 4, 4, 48, None) == bg.BG_ERR_SHAPE
    assert q(A, BF16, 31, None, C, S1, 4, 4, 32, None) == bg.BG_ERR_SHAPE
    assert q(A, BF16, 32, None, C, S1, 4, 5, 32, None) == bg.BG_ERR_SHAPE
    assert q(A, 2, 32, None, C, S1, 4, 4, 32, None) == bg.BG_ERR_SHAPE
    assert q(A, BF16, 1 << 31, None, C, S1, 4, 4, 32, None) == bg.BG_ERR_SHAPE
    assert q(None, BF16, 32, None, C, S1, 4, 4, 32, None) == bg.BG_ERR_NULL
    assert q(A, BF16, 32, None, None, S1, 4, 4, 32, None) == bg.BG_ERR_NULL
    assert q(A, BF16, 32, None, C, None, 4, 4, 32, None) == bg.BG_ERR_NULL
    assert q(A + 8, BF16, 32, None, C, S1, 4, 4, 32, None) == bg.BG_ERR_ALIGN
    assert q(A, BF16, 32, W + 2, C, S1, 4, 4, 32, None) == bg.BG_ERR_ALIGN
    assert q(A, BF16, 32, None, A, S1, 4, 4, 32, None) == bg.BG_ERR_ALIAS
    assert q(A, F32, 64, None, A + 4 * (3 * 64 + 32) - 16, S1, 4, 4, 32, None) == bg.BG_ERR_ALIAS
    assert q(A, BF16, 32, W, C, C + 32, 4, 4, 32, None) == bg.BG_ERR_ALIAS
    assert q(A, BF16, 32, C + 16, C, S1, 4, 4, 32, None) == bg.BG_ERR_ALIAS


def test_dequantize_checks():
    q = L.mxfp4_dequantize
    assert q(None, None, None, BF16, 0, 32, None) == bg.BG_OK
    assert q(A, S1, C, BF16, 4, 16, None) == bg.BG_ERR_SHAPE
    assert q(A, S1, C, 7, 4, 32, None) == bg.BG_ERR_SHAPE
    assert q(A, None, C, BF16, 4, 32, None) == bg.BG_ERR_NULL
    assert q(A, S1, C + 4, F32, 4, 32, None) == bg.BG_ERR_ALIGN
    assert q(A, S1, A + 32, F32, 4, 32, None) == bg.BG_ERR_ALIAS


def test_product_checks():
    g, e = L.gemm_mxfp4, L.gemm_mxfp4_grouped
    assert g(None, None, None, None, None, 0, 4, 32, None) == bg.BG_OK
    assert g(A, S1, B, S2, C, 4, 4, 16, None) == bg.BG_ERR_SHAPE
    assert g(A, S1, B, S2, C, 1 << 31, 4, 32, None) == bg.BG_ERR_SHAPE
    assert g(A, None, B, S2, C, 4, 4, 32, None) == bg.BG_ERR_NULL
    assert g(A, S1, B, S2 + 1, C, 4, 4, 32, None) == bg.BG_ERR_ALIGN
    assert g(A, S1, B, S2, B, 4, 4, 32, None) == bg.BG_ERR_ALIAS
    assert e(None, None, None, None, None, None, 0, 4, 32, 3, None) == bg.BG_OK
    assert e(A, S1, B, S2, O, C, 4, 4, 32, 0, None) == bg.BG_OK
    assert e(A, S1, B, S2, O, C, 4, 4, 32, 1025, None) == bg.BG_ERR_SHAPE
    assert e(A, S1, B, S2, O, C, 4, (1 << 31) - 1, (1 << 31) - 32, 1024, None) == bg.BG_ERR_SHAPE
    assert e(A, S1, B, S2, None, C, 4, 4, 32, 2, None) == bg.BG_ERR_NULL
    assert e(A, S1, B, S2, O + 2, C, 4, 4, 32, 2, None) == bg.BG_ERR_ALIGN
    assert e(A, S1, B, S2, O, O - 16, 4, 4, 32, 2, None) == bg.BG_ERR_ALIAS
    # C inside the second expert's weights
    assert e(A, S1, B, S2, O, B + 64 + 16, 2, 4, 32, 2, None) == bg.BG_ERR_ALIAS


def outs(**other):
    p = bg._RoutingPointers(*[0x100000000 + 0x1000000 * i for i in range(9)])
    for f, v in other.items():
        setattr(p, f, v)
    return ctypes.byref(p)


def test_route_checks():
    r = L.moe_route
    ws = bg.moe_route_workspace_bytes(4000, 64)
    assert ws > 0 and bg.moe_route_workspace_bytes(1, 64) == 0
    ok = (4000, 64, 4, 1, None)
    assert r(A, BF16, None, outs(), W, ws, 4000, 0, 1, 1, None) == bg.BG_ERR_SHAPE
    assert r(A, BF16, None, outs(), W, ws, 4000, 1025, 1, 1, None) == bg.BG_ERR_SHAPE
    assert r(A, BF16, None, outs(), W, ws, 4000, 64, 0, 1, None) == bg.BG_ERR_SHAPE
    assert r(A, BF16, None, outs(), W, ws, 4000, 64, 17, 1, None) == bg.BG_ERR_SHAPE
    assert r(A, BF16, None, outs(), W, ws, 4000, 3, 4, 1, None) == bg.BG_ERR_SHAPE
    assert r(A, BF16, None, outs(), W, 1 << 40, 1 << 28, 64, 8, 1, None) == bg.BG_ERR_SHAPE
    assert r(A, 3, None, outs(), W, ws, *ok) == bg.BG_ERR_SHAPE
    assert r(None, BF16, None, outs(), W, ws, *ok) == bg.BG_ERR_NULL
    assert r(A, BF16, None, None, W, ws, *ok) == bg.BG_ERR_NULL
    assert r(A, BF16, None, outs(loss=None), W, ws, *ok) == bg.BG_ERR_NULL
    assert r(A + 2, BF16, None, outs(), W, ws, *ok) == bg.BG_ERR_ALIGN
    assert r(A, BF16, None, outs(pos=A * 8 + 2), W, ws, *ok) == bg.BG_ERR_ALIGN
    assert r(A, BF16, None, outs(), W + 4, ws, *ok) == bg.BG_ERR_ALIGN
    assert r(A, BF16, None, outs(), None, ws, *ok) == bg.BG_ERR_WORKSPACE
    assert r(A, BF16, None, outs(), W, ws - 1, *ok) == bg.BG_ERR_WORKSPACE
    assert r(A, BF16, None, outs(ids=A), W, ws, *ok) == bg.BG_ERR_ALIAS
    assert r(A, BF16, S1, outs(rows=S1), W, ws, *ok) == bg.BG_ERR_ALIAS
    assert r(A, BF16, None, outs(counts=W + 64), W, ws, *ok) == bg.BG_ERR_ALIAS
    assert r(A, BF16, None, outs(loss=0x100000000), W, ws, *ok) == bg.BG_ERR_ALIAS
    assert r(A, BF16, None, outs(), A + 16, ws, *ok) == bg.BG_ERR_ALIAS


def test_route_backward_checks():
    b = L.moe_route_backward
    ok = (40, 64, 4, 1, None)
    assert b(None, F32, None, None, None, None, None, None, None, 0, 64, 4, 1, None) == bg.BG_OK
    assert b(A, F32, B, C, S1, S2, None, None, O, 40, 64, 65, 1, None) == bg.BG_ERR_SHAPE
    assert b(A, F32, None, C, S1, S2, None, None, O, *ok) == bg.BG_ERR_NULL
    assert b(A, F32, B, C, S1, S2, W + 1, None, O, *ok) == bg.BG_ERR_ALIGN
    assert b(A, F32, B, C, S1, S2, None, None, O + 4, *ok) == bg.BG_ERR_ALIGN
    assert b(A, F32, B, C, S1, S2, None, None, A + 16, *ok) == bg.BG_ERR_ALIAS
    assert b(A, F32, B, C, S1, S2, W, None, W, *ok) == bg.BG_ERR_ALIAS
    assert b(A, F32, B, C, S1, S2, None, O + 32, O, *ok) == bg.BG_ERR_ALIAS


@pytest.mark.skipif(torch.cuda.is_available(), reason="a device is present")
def test_valid_arguments_report_the_missing_device():
    assert L.mxfp4_quantize(A, BF16, 32, None, C, S1, 4, 4, 32, None) == bg.BG_ERR_DEVICE
    assert L.gemm_mxfp4(A, S1, B, S2, C, 4, 4, 32, None) == bg.BG_ERR_DEVICE
    assert L.gemm_mxfp4_grouped(A, S1, B, S2, O, C, 4, 4, 32, 2, None) == bg.BG_ERR_DEVICE
    assert L.moe_route(A, BF16, None, outs(), None, 0, 4, 64, 4, 1, None) == bg.BG_ERR_DEVICE
    # in place, without gradients, is a valid call
    assert L.moe_route_backward(A, F32, B, C, S1, S2, None, None, A, 40, 64, 4, 1, None) == bg.BG_ERR_DEVICE
