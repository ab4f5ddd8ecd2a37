"""Argument checks of the gated block's, the transposed products' and the 4-bit
matrix-vector entry points (CPU only): the binding's, with the library replaced
by a stub that fails if reached, and the C ABI's, with fake addresses that are
never dereferenced."""
import ctypes

import pytest
import torch

import block_scaled_fp4_gemm_amd as bg


class _NoLib:
    def __getattr__(self, name):
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


def f32(*s):
    return torch.zeros(s)


def int4(n=5, k=64, group=32, **other):
    return bg.W4Weights(u8(n, k // 2), bf(n, k // group), "int4", group=group)._replace(**other)


def mx(n=5, k=64, **other):
    return bg.W4Weights(u8(n, k // 2), u8(n, k // 32), "mxfp4")._replace(**other)


def nv(n=5, k=64, **other):
    return bg.W4Weights(u8(n, k // 2), u8(n, k // 16), "nvfp4")._replace(**other)


def backward(**other):
    a = dict(dh=bf(4, 5), a=bf(4, 8), b0=bf(5, 8), b1=bf(5, 8), g=f32(4, 5), u=f32(4, 5)) | other
    return bg.gemm_bf16_gated_backward(**a)


BAD = [
    (lambda: bg.gemm_bf16_nn(bf(4, 8), bf(9, 5)), ValueError),
    (lambda: bg.gemm_bf16_nn(bf(4, 8), bf(8)), ValueError),
    (lambda: bg.gemm_bf16_nn(f32(4, 8), bf(8, 5)), TypeError),
    (lambda: bg.gemm_bf16_nn(bf(4, 8), bf(8, 5), workspace=[0]), TypeError),
    (lambda: bg.gemm_bf16_tn(bf(8, 4), bf(9, 5)), ValueError),
    (lambda: bg.gemm_bf16_tn(bf(8, 4), u8(8, 5)), TypeError),
    (lambda: bg.gemm_bf16_gated(bf(4, 8), bf(5, 8), bf(5, 8), act="relu"), ValueError),
    (lambda: bg.gemm_bf16_gated(bf(4, 8), bf(5, 8), bf(6, 8)), ValueError),
    (lambda: bg.gemm_bf16_gated(bf(4, 8), bf(5, 9), bf(5, 9)), ValueError),
    (lambda: bg.gemm_bf16_gated(bf(4, 8, 1), bf(5, 8), bf(5, 8)), ValueError),
    (lambda: bg.gemm_bf16_gated(bf(4, 8), f32(5, 8), bf(5, 8)), TypeError),
    (lambda: backward(act="tanh"), ValueError),
    (lambda: backward(dh=bf(4, 6)), ValueError),
    (lambda: backward(dh=f32(4, 5)), TypeError),
    (lambda: backward(g=f32(5, 4)), ValueError),
    (lambda: backward(u=f32(4, 6)), ValueError),
    (lambda: backward(u=bf(4, 5)), TypeError),                    # g and u of one type
    (lambda: backward(g=torch.zeros(4, 5, dtype=torch.float16)), TypeError),
    (lambda: backward(b1=bf(5, 9)), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), int4(k=96)), ValueError),
    (lambda: bg.gemv_w4(bf(2, 48), int4(k=48, group=16)), ValueError),          # group
    (lambda: bg.gemv_w4(bf(2, 64), int4(group=48)), ValueError),
    (lambda: bg.gemv_w4(bf(2, 96), int4(k=96, group=64)), ValueError),          # K % group
    (lambda: bg.gemv_w4(bf(2, 64), int4()._replace(group=None)), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), int4()._replace(group=0)), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), int4(scales=u8(5, 2))), TypeError),
    (lambda: bg.gemv_w4(bf(2, 64), int4(scales=bf(5, 3))), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), int4(zeros=u8(5, 1))), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), int4(zeros=bf(5, 2))), TypeError),
    (lambda: bg.gemv_w4(bf(2, 64), int4(format="int8")), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), mx(group=16)), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), mx(zeros=u8(5, 2))), ValueError),
    (lambda: bg.gemv_w4(bf(2, 64), mx(scales=bf(5, 2))), TypeError),
    (lambda: bg.gemv_w4(bf(2, 64), nv(scales=u8(5, 2))), ValueError),
    (lambda: bg.gemv_w4(bf(2, 48), nv(k=48)), ValueError),                      # K % 32
    (lambda: bg.gemv_w4(bf(64), mx()), ValueError),
    (lambda: bg.gemv_w4(f32(2, 64), mx()), TypeError),
    (lambda: bg.gemv_w4_gated(bf(2, 64), mx(), mx(n=6)), ValueError),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_bad_arguments_raise_before_the_library(i, nolib):
    call, exc = BAD[i]
    with pytest.raises(exc):
        call()


HOST = [
    lambda: bg.gemm_bf16_nn(bf(4, 8), bf(8, 5)),
    lambda: bg.gemm_bf16_tn(bf(8, 4), bf(8, 5)),
    lambda: bg.gemm_bf16_gated(bf(4, 8), bf(5, 8), bf(5, 8), save=True),
    lambda: backward(),
    lambda: backward(g=bf(4, 5), u=bf(4, 5)),
    lambda: bg.gemv_w4(bf(2, 64), int4(zeros=u8(5, 2))),
    lambda: bg.gemv_w4(bf(2, 64), mx(group=32)),
    lambda: bg.gemv_w4_gated(bf(2, 64), nv(), nv()),
]


@pytest.mark.parametrize("i", range(len(HOST)))
def test_host_tensors_are_rejected(i, nolib):
    with pytest.raises(ValueError, match="device"):
        HOST[i]()


# --- the C ABI ---------------------------------------------------------------

A, B, B1, C, G, U, W, D, D1 = (0x10000000 * i for i in range(1, 10))
L = bg.lib
F32, BF16 = 1, 0
OK, NULL, SHAPE, ALIGN, WORKSPACE, ALIAS, DEVICE = (bg.BG_OK, bg.BG_ERR_NULL, bg.BG_ERR_SHAPE, bg.BG_ERR_ALIGN,
                                                    bg.BG_ERR_WORKSPACE, bg.BG_ERR_ALIAS, bg.BG_ERR_DEVICE)
BIG = (1 << 31) - 1


def gated(a=A, b0=B, b1=B1, h=C, g=G, u=U, kept=F32, act=0, m=4, n=5, k=8):
    return L.gemm_bf16_gated(a, b0, b1, h, g, u, kept, act, m, n, k, None)


def grad(dh=C, a=A, b0=B, b1=B1, g=G, u=U, kept=F32, da=D, db0=D1, db1=D1 + 0x1000, act=0, ws=W, nbytes=1 << 20, m=4,
         n=5, k=8):
    return L.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, kept, da, db0, db1, act, ws, nbytes, m, n, k, None)


def w4(fmt=0, codes=B, scales=G, zeros=None, group=32):
    return bg._W4(codes, scales, zeros, fmt, group, 1.0)


def gemv(x=A, w=None, y=C, r=2, n=5, k=64):
    w = w4() if w is None else w
    return L.gemv_w4(x, ctypes.byref(w) if w != 0 else None, y, r, n, k, None)


def gemv_gated(x=A, w0=None, w1=None, y=C, act=0, r=2, n=5, k=64):
    w0, w1 = w0 or w4(), w1 or w4(codes=B1, scales=U)
    return L.gemv_w4_gated(x, ctypes.byref(w0), ctypes.byref(w1), y, act, r, n, k, None)


STATUS = [
    (lambda: gated(m=0), OK), (lambda: gated(n=0), OK),
    (lambda: gated(a=None), NULL), (lambda: gated(b0=None), NULL), (lambda: gated(b1=None), NULL),
    (lambda: gated(h=None), NULL), (lambda: gated(g=None), NULL), (lambda: gated(u=None), NULL),
    (lambda: gated(a=A + 2), ALIGN), (lambda: gated(b1=B1 + 8), ALIGN), (lambda: gated(h=C + 2), ALIGN),
    (lambda: gated(g=G + 4), ALIGN), (lambda: gated(u=U + 4), ALIGN),
    (lambda: gated(act=2), SHAPE), (lambda: gated(act=-1), SHAPE), (lambda: gated(kept=2), SHAPE),
    (lambda: gated(m=1 << 31), SHAPE), (lambda: gated(n=BIG, k=1), SHAPE), (lambda: gated(m=1 << 30, n=1 << 10), SHAPE),
    (lambda: gated(h=A), ALIAS), (lambda: gated(h=B + 16), ALIAS), (lambda: gated(g=C + 16), ALIAS),
    (lambda: gated(u=G + 64), ALIAS), (lambda: gated(u=B1), ALIAS),
    (lambda: grad(db0=None), NULL), (lambda: grad(db1=None), NULL), (lambda: grad(dh=None), NULL),
    (lambda: grad(g=None), NULL), (lambda: grad(a=None), NULL), (lambda: grad(b0=None), NULL),
    (lambda: grad(act=3), SHAPE), (lambda: grad(kept=-1), SHAPE), (lambda: grad(k=BIG), SHAPE),
    (lambda: grad(m=64, n=1, k=1 << 27), SHAPE), (lambda: grad(m=8, n=1, k=1 << 30), SHAPE),
    (lambda: grad(da=D + 2), ALIGN), (lambda: grad(g=G + 8), ALIGN),
    (lambda: grad(da=C), ALIAS), (lambda: grad(db0=A), ALIAS), (lambda: grad(db1=D1 + 16), ALIAS),
    (lambda: grad(da=G + 16), ALIAS),
    (lambda: L.gemm_bf16_nn(None, None, None, None, 0, 0, 5, 8, None), OK),
    (lambda: L.gemm_bf16_tn(None, None, None, None, 0, 5, 0, 8, None), OK),
    (lambda: L.gemm_bf16_nn(A, None, C, None, 0, 4, 5, 8, None), NULL),
    (lambda: L.gemm_bf16_tn(A, B, None, None, 0, 4, 5, 8, None), NULL),
    (lambda: L.gemm_bf16_nn(A, B + 2, C, None, 0, 4, 5, 8, None), ALIGN),
    (lambda: L.gemm_bf16_tn(A, B, A + 16, None, 0, 4, 5, 8, None), ALIAS),
    (lambda: L.gemm_bf16_nn(A, B, C, None, 0, 1 << 31, 5, 8, None), SHAPE),
    (lambda: L.gemm_bf16_tn(A, B, C, None, 0, 1 << 22, 1 << 18, 1, None), SHAPE),
    (lambda: L.gemm_bf16_nn_workspace(4, 5, 8, None), NULL),
    (lambda: L.gemm_bf16_tn_workspace(4, 5, 8, None), NULL),
    (lambda: L.gemm_bf16_gated_backward_workspace(4, 5, 8, None), NULL),
    (lambda: L.gemm_bf16_nn_workspace(BIG, 5, 8, ctypes.byref(ctypes.c_size_t())), SHAPE),
    (lambda: gemv(r=0), OK), (lambda: gemv(n=0), OK),
    (lambda: gemv(w=0), NULL), (lambda: gemv(x=None), NULL), (lambda: gemv(y=None), NULL),
    (lambda: gemv(w=w4(codes=None)), NULL), (lambda: gemv(w=w4(scales=None)), NULL),
    (lambda: gemv(x=A + 8), ALIGN), (lambda: gemv(w=w4(codes=B + 4)), ALIGN), (lambda: gemv(w=w4(scales=G + 2)), ALIGN),
    (lambda: gemv(w=w4(zeros=U + 1)), ALIGN),
    (lambda: gemv(w=w4(fmt=3)), SHAPE), (lambda: gemv(w=w4(fmt=-1)), SHAPE), (lambda: gemv(w=w4(group=0)), SHAPE),
    (lambda: gemv(w=w4(group=48), k=96), SHAPE), (lambda: gemv(w=w4(group=64), k=96), SHAPE),
    (lambda: gemv(w=w4(fmt=1, group=16)), SHAPE), (lambda: gemv(w=w4(fmt=2, group=32)), SHAPE),
    (lambda: gemv(w=w4(fmt=1, zeros=U)), SHAPE), (lambda: gemv(k=48), SHAPE), (lambda: gemv(k=(1 << 20) + 32), SHAPE),
    (lambda: gemv(r=(1 << 16) + 1), SHAPE), (lambda: gemv(n=1 << 26), SHAPE), (lambda: gemv(r=1 << 16, n=1 << 15), SHAPE),
    (lambda: gemv(y=A), ALIAS), (lambda: gemv(y=B), ALIAS), (lambda: gemv(w=w4(zeros=U), y=U), ALIAS),
    (lambda: gemv_gated(act=5), SHAPE), (lambda: gemv_gated(w1=w4(fmt=1)), SHAPE),
    (lambda: gemv_gated(w1=w4(group=64)), SHAPE), (lambda: gemv_gated(w1=w4(codes=B1, scales=U, zeros=D)), SHAPE),
    (lambda: gemv_gated(w1=w4(codes=None)), NULL), (lambda: gemv_gated(y=B1 + 16), ALIAS),
]


@pytest.mark.parametrize("i", range(len(STATUS)))
def test_status(i):
    call, want = STATUS[i]
    assert call() == want


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="valid call would launch on fake pointers")
@pytest.mark.parametrize("i", range(11))
def test_valid_arguments_reach_the_device_check(i):
    n = ctypes.c_size_t(0)
    call = [gated, lambda: gated(g=None, u=None), lambda: gated(kept=BF16, act=1, k=7), grad, lambda: grad(da=None, b0=None, b1=None),
            lambda: grad(db0=None, db1=None, a=None), lambda: L.gemm_bf16_nn(A, B, C, None, 0, 4, 5, 8, None),
            lambda: L.gemm_bf16_tn_workspace(4, 5, 8, ctypes.byref(n)), lambda: gemv(w=w4(zeros=U)),
            lambda: gemv(w=w4(fmt=2, group=16), k=0), lambda: gemv_gated(act=1)][i]
    assert call() == DEVICE
