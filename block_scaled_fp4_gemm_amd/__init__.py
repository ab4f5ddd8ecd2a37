"""Python binding of libblockgemm (MI355X / gfx950 GEMM library).

Argument marshalling only: every function here forwards device pointers,
sizes and the current HIP stream to the C ABI declared in include/blockgemm.h
and raises BlockGemmError on a non-OK status. All arithmetic runs in the HIP
kernels of the shared library; there is no fallback path. PyTorch provides
device memory and streams.

Importing this module fails if the library has not been built, or was built
from older sources (`python block_scaled_fp4_gemm_amd/build.py`, or
__graft_entry__.build()).
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libblockgemm.so")

_REBUILD = "python block_scaled_fp4_gemm_amd/build.py"

if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with `{_REBUILD}`")

lib = ctypes.CDLL(_LIB_PATH)

_p, _u32, _f32, _sz = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "gemm_bf16": [_p, _p, _p, _u32, _u32, _u32, _p],
    "gemm_bf16_strided": [_p, _u32, _p, _u32, _p, _u32, _u32, _u32, _u32, _p],
    "gemm_bf16_dual": [_p, _p, _p, _p, _p, _u32, _u32, _u32, _p],
    "gemm_bf16_scaled_acc": [_p, _p, _p, _u32, _u32, _u32, _f32, _p],
    "gemm_bf16_splitk": [_p, _p, _p, _p, _sz, _u32, _u32, _u32, _u32, _p],
    "gemm_bf16_splitk_noalloc": [_p, _p, _p, _u32, _u32, _u32, _u32, _p],
    "gemm_bf16_streamk": [_p, _p, _p, _p, _sz, _u32, _u32, _u32, _p],
    "gemm_bf16_streamk_workspace": [_u32, _u32, _u32, _p],
    "bg_streamk_plan": [_u32, _u32, _u32, _p, _sz, _p],
    "gemm_bf16_ordered": [_p, _p, _p, _u32, _u32, _u32, _p],
    "gemm_bf16_ordered_f32": [_p, _p, _p, _u32, _u32, _u32, _p],
    "gemm_fp4_blockscaled": [_p, _p, _p, _p, _p, _u32, _u32, _u32, _p],
    "gemm_w4a16": [_p, _p, _p, _f32, _p, _u32, _u32, _u32, _p],
    "gemm_w4a16_t": [_p, _p, _p, _u32, _f32, _p, _u32, _u32, _u32, _p],
    "gemm_fp4_blockscaled_batched": [_p, _p, _p, _p, _p, _u32, _u32, _u32, _u32, _p],
    "gemm_fp4_blockscaled_splitk": [_p, _p, _p, _p, _p, _p, _sz, _u32, _u32, _u32, _u32, _p],
    "fp4_scales_from_blocked": [_p, _p, _u32, _u32, _u32, _p],
    "bf16_scaled_add": [_p, _p, _sz, _f32, _p],
    "mxfp4_quantize": [_p, ctypes.c_int, _u32, _p, _p, _p, _u32, _u32, _u32, _p],
    "mxfp4_dequantize": [_p, _p, _p, ctypes.c_int, _u32, _u32, _p],
    "gemm_mxfp4": [_p, _p, _p, _p, _p, _u32, _u32, _u32, _p],
    "gemm_mxfp4_grouped": [_p, _p, _p, _p, _p, _p, _u32, _u32, _u32, _u32, _p],
    "moe_route": [_p, ctypes.c_int, _p, _p, _p, _sz, _u32, _u32, _u32, ctypes.c_int, _p],
    "moe_route_backward": [_p, ctypes.c_int, _p, _p, _p, _p, _p, _p, _p, _u32, _u32, _u32, ctypes.c_int, _p],
    "gemm_bf16_gated": [_p, _p, _p, _p, _p, _p, ctypes.c_int, ctypes.c_int, _u32, _u32, _u32, _p],
    "gemm_bf16_gated_backward": [_p, _p, _p, _p, _p, _p, ctypes.c_int, _p, _p, _p, ctypes.c_int, _p, _sz, _u32, _u32, _u32,
                                 _p],
    "gemm_bf16_gated_backward_workspace": [_u32, _u32, _u32, _p],
    "gemm_bf16_nn": [_p, _p, _p, _p, _sz, _u32, _u32, _u32, _p],
    "gemm_bf16_tn": [_p, _p, _p, _p, _sz, _u32, _u32, _u32, _p],
    "gemm_bf16_nn_workspace": [_u32, _u32, _u32, _p],
    "gemm_bf16_tn_workspace": [_u32, _u32, _u32, _p],
    "gemv_w4": [_p, _p, _p, _u32, _u32, _u32, _p],
    "gemv_w4_gated": [_p, _p, _p, _p, ctypes.c_int, _u32, _u32, _u32, _p],
}
for _name, _args in _SIGS.items():
    try:
        _fn = getattr(lib, _name)
    except AttributeError as _e:
        raise ImportError(f"{_LIB_PATH} lacks {_name} (built from older sources): rebuild it with "
                          f"`{_REBUILD}`") from _e
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
lib.gemm_bf16_splitk_workspace_bytes.argtypes = [_u32, _u32, _u32]
lib.gemm_bf16_splitk_workspace_bytes.restype = ctypes.c_size_t
lib.moe_route_workspace_bytes.argtypes = [_u32, _u32]
lib.moe_route_workspace_bytes.restype = ctypes.c_size_t
lib.bg_status_string.argtypes = [ctypes.c_int]
lib.bg_status_string.restype = ctypes.c_char_p
lib.bg_tune_set.argtypes = [ctypes.c_int, ctypes.c_int]
lib.bg_tune_set.restype = ctypes.c_int
lib.bg_tune_get.argtypes = [ctypes.c_int]
lib.bg_tune_get.restype = ctypes.c_int
lib.bg_tile_map.argtypes = [ctypes.c_int, _u32, _u32, _p, _p]
lib.bg_tile_map.restype = ctypes.c_int

EXPORTS = tuple(_SIGS) + ("gemm_bf16_splitk_workspace_bytes", "bg_status_string", "bg_tune_set", "bg_tune_get",
                          "bg_tile_map", "moe_route_workspace_bytes")

BG_OK, BG_ERR_NULL, BG_ERR_SHAPE, BG_ERR_ALIGN, BG_ERR_WORKSPACE, BG_ERR_ALIAS, BG_ERR_DEVICE, \
    BG_ERR_LAUNCH = range(8)


class BlockGemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bg_status_string(status)} (status {status})")


def bg_status_string(status: int) -> str:
    return lib.bg_status_string(int(status)).decode()


def gemm_bf16_splitk_workspace_bytes(m: int, n: int, k_splits: int) -> int:
    return int(lib.gemm_bf16_splitk_workspace_bytes(m, n, k_splits))


def _check(status: int, where: str) -> None:
    if status != BG_OK:
        raise BlockGemmError(status, where)


# ---------------------------------------------------------------------------
# Argument checks. The C ABI sees only pointers and sizes, so everything it
# cannot see is checked here, before the library is called: tensor kind,
# element size, shape (including outputs the caller supplies), contiguity and
# that every tensor lives on the current HIP device. A failed check raises and
# launches nothing.
# ---------------------------------------------------------------------------

def _tensor(t, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor, got {type(t).__name__}")
    return t


def _bits16(t: torch.Tensor, what: str = "tensor") -> torch.Tensor:
    _tensor(t, what)
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{what}: expected bfloat16 (or its 16-bit pattern), got {t.dtype}")
    return t


def _bytes(t: torch.Tensor, what: str) -> torch.Tensor:
    _tensor(t, what)
    if t.element_size() != 1 or t.dtype == torch.bool:
        raise TypeError(f"{what}: expected a byte tensor (uint8, int8 or an FP8 dtype), got {t.dtype}")
    return t


def _f32(t: torch.Tensor, what: str) -> torch.Tensor:
    _tensor(t, what)
    if t.dtype != torch.float32:
        raise TypeError(f"{what}: expected float32, got {t.dtype}")
    return t


def _shape(t: torch.Tensor, shape, what: str) -> None:
    if t.shape != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dims(t: torch.Tensor, n: int, what: str):
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{what} must be {n}-D, got shape {tuple(shape)}")
    return shape


# torch's raw accessors for the current device and stream (the public
# torch.cuda.current_stream() builds a Stream object per call: about 3 us of a
# 10 us call on MI355X), with the public API as the fallback
_raw_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_device() -> int:
    return _raw_device() if _raw_device is not None else torch.cuda.current_device()


def _on_device(*ts) -> None:
    """Every tensor (None skipped) is on the current HIP device (contiguity is
    checked where its pointer is taken, in _ptr)."""
    cur = None
    for t in ts:
        if t is not None:
            d = t.get_device()
            if d != cur or d < 0:
                if cur is None and d >= 0:
                    cur = _current_device()
                if d != cur:
                    _wrong_device(ts)


def _wrong_device(ts) -> None:
    ts = [t for t in ts if t is not None]
    for t in ts:
        if not t.is_cuda:
            raise ValueError(f"tensors must be on a HIP device, got one on {t.device}")
    cur = _current_device()
    for t in ts:
        if t.get_device() != cur:
            raise ValueError(f"tensors must be on the current device cuda:{cur}, got one on {t.device}")


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous (row-major)")
    return t.data_ptr()


def _out16(out, shape, like: torch.Tensor, what: str = "out") -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)
    _shape(_bits16(out, what), shape, what)
    return out


def _workspace(ws, k_splits: int, m: int, n: int):
    if ws is None:
        return None
    _f32(ws, "workspace")
    if ws.numel() < k_splits * m * n:
        raise ValueError(f"workspace holds {ws.numel()} floats, {k_splits * m * n} needed")
    return ws


def _fp4_operands(a, sfa, b, sfb, batched: bool = False):
    """Shapes of packed FP4 operands: A [(L,) M, K/2], SFA [(L,) M, K/16], B and SFB likewise."""
    nd = 3 if batched else 2
    for t, w in ((a, "A"), (sfa, "SFA"), (b, "B"), (sfb, "SFB")):
        _dims(_bytes(t, w), nd, w)
    lead = a.shape[:-2]
    m, kh = a.shape[-2:]
    n = b.shape[-2]
    k = 2 * kh
    if k % 16 != 0:
        raise ValueError(f"K = {k} must be a multiple of 16 (one scale per 16 elements)")
    _shape(b, (*lead, n, kh), "B")
    _shape(sfa, (*lead, m, k // 16), "SFA")
    _shape(sfb, (*lead, n, k // 16), "SFB")
    return lead, m, n, k


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------

def gemm_bf16(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """C[M,N] = bf16(A[M,K] @ B[N,K]^T), FP32 accumulation."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (n, k), "B")
    out = _out16(out, (m, n), a)
    _on_device(a, b, out)
    _check(lib.gemm_bf16(_ptr(a), _ptr(b), _ptr(out), m, n, k, _stream(stream)), "gemm_bf16")
    return out


def gemm_bf16_dual(a: torch.Tensor, b0: torch.Tensor, b1: torch.Tensor, out0: torch.Tensor | None = None,
                   out1: torch.Tensor | None = None, stream=None):
    """C0 = bf16(A @ B0^T) and C1 = bf16(A @ B1^T) (same shapes) in one launch."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b0, "B0"), 2, "B0")
    _shape(b0, (n, k), "B0")
    _shape(_bits16(b1, "B1"), (n, k), "B1")
    out0 = _out16(out0, (m, n), a, "out0")
    out1 = _out16(out1, (m, n), a, "out1")
    _on_device(a, b0, b1, out0, out1)
    _check(lib.gemm_bf16_dual(_ptr(a), _ptr(b0), _ptr(b1), _ptr(out0), _ptr(out1), m, n, k, _stream(stream)),
           "gemm_bf16_dual")
    return out0, out1


def _rows(t: torch.Tensor, what: str):
    """(rows, cols, row stride) of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be 2-D with contiguous rows")
    return t.shape[0], t.shape[1], t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def gemm_bf16_strided(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor, stream=None):
    """C = bf16(A @ B^T) on row-strided views (each row contiguous, any row stride)."""
    for t, w in ((a, "A"), (b, "B"), (out, "C")):
        _bits16(t, w)
    m, k, lda = _rows(a, "A")
    n, kb, ldb = _rows(b, "B")
    mc, nc, ldc = _rows(out, "C")
    if kb != k or (mc, nc) != (m, n):
        raise ValueError("shapes must be A [M,K], B [N,K], C [M,N]")
    _on_device(a, b, out)
    _check(lib.gemm_bf16_strided(a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldc, m, n, k,
                                 _stream(stream)), "gemm_bf16_strided")
    return out


def gemm_bf16_scaled_acc(x: torch.Tensor, b: torch.Tensor, out: torch.Tensor, scale: float,
                         stream=None):
    """out[M,N] = bf16(out + scale * bf16(X[M,K] @ B[N,K]^T)), in place."""
    m, k = _dims(_bits16(x, "X"), 2, "X")
    n, _ = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (n, k), "B")
    _shape(_bits16(out, "out"), (m, n), "out")
    _on_device(x, b, out)
    _check(lib.gemm_bf16_scaled_acc(_ptr(x), _ptr(b), _ptr(out), m, n, k, float(scale),
                                    _stream(stream)), "gemm_bf16_scaled_acc")
    return out


def gemm_bf16_splitk(a: torch.Tensor, b: torch.Tensor, k_splits: int,
                     workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     stream=None):
    """Split-K GEMM with an FP32 workspace of k_splits*M*N floats (allocated if None)."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (n, k), "B")
    out = _out16(out, (m, n), a)
    workspace = _workspace(workspace, k_splits, m, n)
    _on_device(a, b, out, workspace)
    if workspace is None and k_splits > 1:
        workspace = torch.empty((k_splits, m, n), dtype=torch.float32, device=a.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * 4
    _check(lib.gemm_bf16_splitk(_ptr(a), _ptr(b), _ptr(out), _ptr(workspace), ws_bytes, m, n, k,
                                k_splits, _stream(stream)), "gemm_bf16_splitk")
    return out


NOALLOC_SCRATCH_BYTES = 32 << 20   # BG_NOALLOC_SCRATCH_BYTES


def gemm_bf16_splitk_noalloc(a: torch.Tensor, b: torch.Tensor, k_splits: int, out: torch.Tensor,
                             stream=None):
    """Split-K GEMM whose FP32 planes live in the library's static per-device
    scratch (k_splits*M*N*4 <= NOALLOC_SCRATCH_BYTES); allocates nothing, so
    `out` must be supplied. Calls that may overlap on one device race."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (n, k), "B")
    if out is None:
        raise ValueError("gemm_bf16_splitk_noalloc allocates nothing: pass `out`")
    _shape(_bits16(out, "out"), (m, n), "out")
    _on_device(a, b, out)
    _check(lib.gemm_bf16_splitk_noalloc(_ptr(a), _ptr(b), _ptr(out), m, n, k, k_splits, _stream(stream)),
           "gemm_bf16_splitk_noalloc")
    return out


def gemm_bf16_streamk_workspace(m: int, n: int, k: int) -> int:
    """Bytes of workspace gemm_bf16_streamk needs for (M, N, K) on the current device."""
    nbytes = ctypes.c_size_t(0)
    _check(lib.gemm_bf16_streamk_workspace(m, n, k, ctypes.byref(nbytes)), "gemm_bf16_streamk_workspace")
    return int(nbytes.value)


def gemm_bf16_streamk(a: torch.Tensor, b: torch.Tensor, workspace: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None):
    """C = bf16(A @ B^T) with the stream-K schedule. `workspace` is a byte
    tensor of at least gemm_bf16_streamk_workspace(M, N, K) bytes (allocated
    if None); it needs no initialization."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (n, k), "B")
    out = _out16(out, (m, n), a)
    _on_device(a, b, out, workspace)
    if workspace is None:
        need = gemm_bf16_streamk_workspace(m, n, k) if m and n else 0
        workspace = torch.empty(need, dtype=torch.uint8, device=a.device) if need else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gemm_bf16_streamk(_ptr(a), _ptr(b), _ptr(out), _ptr(workspace), ws_bytes, m, n, k,
                                 _stream(stream)), "gemm_bf16_streamk")
    return out


def streamk_plan(tiles: int, steps: int, wgs_per_xcd: int):
    """The stream-K plan (host only): an int32 array of rows (workgroup, grid
    tile, first step, end step, partial, lowest source or -1), one per piece
    of work, in the order the kernel runs them."""
    import numpy as np
    count = ctypes.c_size_t(0)
    _check(lib.bg_streamk_plan(tiles, steps, wgs_per_xcd, None, 0, ctypes.byref(count)), "bg_streamk_plan")
    rows = np.zeros((count.value, 6), np.int32)
    _check(lib.bg_streamk_plan(tiles, steps, wgs_per_xcd, rows.ctypes.data if count.value else None,
                               count.value, ctypes.byref(count)), "bg_streamk_plan")
    return rows


def gemm_bf16_ordered(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
                      stream=None):
    """Strict k = 0..K-1 FP32 recurrence per output (no FMA), BF16 out."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (n, k), "B")
    out = _out16(out, (m, n), a)
    _on_device(a, b, out)
    _check(lib.gemm_bf16_ordered(_ptr(a), _ptr(b), _ptr(out), m, n, k, _stream(stream)),
           "gemm_bf16_ordered")
    return out


def gemm_bf16_ordered_f32(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
                          stream=None):
    """As gemm_bf16_ordered, storing the FP32 sums."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (n, k), "B")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=a.device)
    _shape(_f32(out, "out"), (m, n), "out")
    _on_device(a, b, out)
    _check(lib.gemm_bf16_ordered_f32(_ptr(a), _ptr(b), _ptr(out), m, n, k, _stream(stream)),
           "gemm_bf16_ordered_f32")
    return out


def gemm_fp4_blockscaled(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                         out: torch.Tensor | None = None, stream=None):
    """C = bf16(deq(A) @ deq(B)^T): A [M,K/2] packed e2m1, SFA [M,K/16] e4m3fn, same for B."""
    _, m, n, k = _fp4_operands(a, sfa, b, sfb)
    out = _out16(out, (m, n), a)
    _on_device(a, sfa, b, sfb, out)
    _check(lib.gemm_fp4_blockscaled(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), m, n, k,
                                    _stream(stream)), "gemm_fp4_blockscaled")
    return out


def gemm_fp4_blockscaled_batched(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                                 out: torch.Tensor | None = None, stream=None):
    """C[l] = bf16(deq(A[l]) @ deq(B[l])^T) for A [L,M,K/2], SFA [L,M,K/16], B [L,N,K/2], SFB [L,N,K/16]."""
    (l,), m, n, k = _fp4_operands(a, sfa, b, sfb, batched=True)
    out = _out16(out, (l, m, n), a)
    _on_device(a, sfa, b, sfb, out)
    _check(lib.gemm_fp4_blockscaled_batched(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), m, n, k, l,
                                            _stream(stream)), "gemm_fp4_blockscaled_batched")
    return out


def gemm_fp4_blockscaled_splitk(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                                k_splits: int, workspace: torch.Tensor | None = None,
                                out: torch.Tensor | None = None, stream=None):
    """FP4 GEMM through k_splits FP32 planes (workspace of k_splits*M*N floats, allocated if None)."""
    _, m, n, k = _fp4_operands(a, sfa, b, sfb)
    out = _out16(out, (m, n), a)
    workspace = _workspace(workspace, k_splits, m, n)
    _on_device(a, sfa, b, sfb, out, workspace)
    if workspace is None and k_splits > 1:
        workspace = torch.empty((k_splits, m, n), dtype=torch.float32, device=a.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * 4
    _check(lib.gemm_fp4_blockscaled_splitk(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), _ptr(workspace),
                                           ws_bytes, m, n, k, k_splits, _stream(stream)),
           "gemm_fp4_blockscaled_splitk")
    return out


def fp4_scales_from_blocked(blocked: torch.Tensor, rows: int, k_groups: int, batch: int = 1,
                            out: torch.Tensor | None = None, stream=None):
    """Plain [batch, rows, k_groups] scale bytes from the blocked (l, tile_m, tile_k, 32, 4, 4) layout."""
    _bytes(blocked, "blocked")
    if blocked.numel() != batch * rows * k_groups:
        raise ValueError(f"blocked holds {blocked.numel()} bytes, {batch * rows * k_groups} expected")
    if out is None:
        out = torch.empty((batch, rows, k_groups), dtype=torch.uint8, device=blocked.device)
    _shape(_bytes(out, "out"), (batch, rows, k_groups), "out")
    _on_device(blocked, out)
    _check(lib.fp4_scales_from_blocked(_ptr(blocked), _ptr(out), rows, k_groups, batch, _stream(stream)),
           "fp4_scales_from_blocked")
    return out


def gemm_w4a16(a: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor, scale_2: float,
               out: torch.Tensor | None = None, stream=None):
    """C = bf16(scale_2 * (A @ deq(B)^T)): A [M,K] bf16, B [N,K/2] packed e2m1, SFB [N,K/16] e4m3fn. Made for many
    rows: up to about 100 of them gemv_w4 takes the same weights ("nvfp4", K a multiple of 32) faster."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bytes(b, "B"), 2, "B")
    if k % 16 != 0:
        raise ValueError(f"K = {k} must be a multiple of 16 (one scale per 16 elements)")
    _shape(b, (n, k // 2), "B")
    _shape(_bytes(sfb, "SFB"), (n, k // 16), "SFB")
    out = _out16(out, (m, n), a)
    _on_device(a, b, sfb, out)
    _check(lib.gemm_w4a16(_ptr(a), _ptr(b), _ptr(sfb), float(scale_2), _ptr(out), m, n, k, _stream(stream)),
           "gemm_w4a16")
    return out


def gemm_w4a16_t(a: torch.Tensor, bt: torch.Tensor, sfbt: torch.Tensor, n: int, scale_2: float,
                 out: torch.Tensor | None = None, stream=None):
    """gemm_w4a16 with transposed weights: Bt [K/2, ldb] bytes (k pairs as rows), SFBt [K/16, ldb],
    ldb >= n taken from Bt's row length (pad columns n..ldb-1 unused)."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    if k % 16 != 0:
        raise ValueError(f"K = {k} must be a multiple of 16 (one scale per 16 elements)")
    rows, ldb = _dims(_bytes(bt, "Bt"), 2, "Bt")
    if rows != k // 2 or ldb < n or n < 0:
        raise ValueError(f"Bt must be [K/2, ldb] = [{k // 2}, >= {n}], got {tuple(bt.shape)}")
    _shape(_bytes(sfbt, "SFBt"), (k // 16, ldb), "SFBt")
    out = _out16(out, (m, n), a)
    _on_device(a, bt, sfbt, out)
    _check(lib.gemm_w4a16_t(_ptr(a), _ptr(bt), _ptr(sfbt), ldb, float(scale_2), _ptr(out), m, n, k,
                            _stream(stream)), "gemm_w4a16_t")
    return out


def bf16_scaled_add(out: torch.Tensor, delta: torch.Tensor, scale: float, stream=None):
    """out = bf16(out + fl32(scale * delta)) elementwise, in place."""
    _bits16(out, "out")
    _bits16(delta, "delta")
    if out.numel() != delta.numel():
        raise ValueError("out and delta must have the same number of elements")
    _on_device(out, delta)
    _check(lib.bf16_scaled_add(_ptr(out), _ptr(delta), out.numel(), float(scale), _stream(stream)),
           "bf16_scaled_add")
    return out


class _on_stream:
    """Context in which new tensors are taken for a call on `stream` (None: the
    current one). Memory of torch's pool belongs to the stream it was taken on:
    taken on another one, it could still be in use there, or be handed out
    there again while the call runs."""

    def __new__(cls, stream, device):
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream), device=device)
        return torch.cuda.stream(stream)


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    if stream is None or not like.is_cuda:
        return like.new_empty(shape, dtype=dtype)
    with _on_stream(stream, like.device):
        return like.new_empty(shape, dtype=dtype)


# ---------------------------------------------------------------------------
# MXFP4: E2M1 elements, one E8M0 scale per 32 of them
# ---------------------------------------------------------------------------

_BG_TYPES = {torch.bfloat16: 0, torch.float32: 1}   # bg_type


def _type(t: torch.Tensor, what: str) -> int:
    kind = _BG_TYPES.get(_tensor(t, what).dtype)
    if kind is None:
        raise TypeError(f"{what}: expected bfloat16 or float32, got {t.dtype}")
    return kind


def _i32(t: torch.Tensor, what: str) -> torch.Tensor:
    if _tensor(t, what).dtype != torch.int32:
        raise TypeError(f"{what}: expected int32, got {t.dtype}")
    return t


def _blocks32(k: int) -> None:
    if k % 32 != 0:
        raise ValueError(f"K = {k} must be a multiple of 32 (one scale per 32 elements)")


def _mx_operands(a, sfa, b, sfb, nd: int):
    """Shapes of MXFP4 operands: A [M, K/2], SFA [M, K/32], B [(E,) N, K/2], SFB [(E,) N, K/32]."""
    m, kh = _dims(_bytes(a, "A"), 2, "A")
    *lead, _ = _dims(_bytes(b, "B"), nd, "B")
    k = 2 * kh
    _blocks32(k)
    _shape(b, (*lead, kh), "B")
    _shape(_bytes(sfa, "SFA"), (m, k // 32), "SFA")
    _shape(_bytes(sfb, "SFB"), (*lead, k // 32), "SFB")
    return lead, m, k


def mxfp4_quantize(x: torch.Tensor, rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   scales: torch.Tensor | None = None, stream=None):
    """(codes [R, K/2], scales [R, K/32]) of x [M, K] (bfloat16 or float32, contiguous rows at any row
    stride). With `rows` (int32 [R]), row i of the result is x[rows[i]], all zero where rows[i] is not a
    row of x; without, R = M."""
    kind = _type(x, "x")
    r, k = _dims(x, 2, "x")
    m, k, ldx = (r, k, k) if x.is_contiguous() else _rows(x, "x")
    _blocks32(k)
    if rows is not None:
        (r,) = _dims(_i32(rows, "rows"), 1, "rows")
    if out is None:
        out = _new(x, (r, k // 2), torch.uint8, stream)
    else:
        _shape(_bytes(out, "out"), (r, k // 2), "out")
    if scales is None:
        scales = _new(x, (r, k // 32), torch.uint8, stream)
    else:
        _shape(_bytes(scales, "scales"), (r, k // 32), "scales")
    _on_device(x, rows, out, scales)
    if r == 0:      # an empty row list has no address, which the library would take for no list
        return out, scales
    _check(lib.mxfp4_quantize(x.data_ptr(), kind, ldx, _ptr(rows), _ptr(out), _ptr(scales), m, r, k,
                              _stream(stream)), "mxfp4_quantize")
    return out, scales


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                     out: torch.Tensor | None = None, stream=None):
    """The values [M, K] of MXFP4 codes [M, K/2] and scales [M, K/32], as bfloat16 or float32."""
    m, kh = _dims(_bytes(codes, "codes"), 2, "codes")
    k = 2 * kh
    _blocks32(k)
    _shape(_bytes(scales, "scales"), (m, k // 32), "scales")
    if out is None:
        out = _new(codes, (m, k), dtype, stream)
    else:
        _shape(out, (m, k), "out")
    kind = _type(out, "out")
    _on_device(codes, scales, out)
    _check(lib.mxfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(out), kind, m, k, _stream(stream)),
           "mxfp4_dequantize")
    return out


def gemm_mxfp4(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
               out: torch.Tensor | None = None, stream=None):
    """C = bf16(deq(A) @ deq(B)^T): A [M, K/2] packed e2m1, SFA [M, K/32] e8m0, B [N, K/2], SFB [N, K/32]."""
    (n,), m, k = _mx_operands(a, sfa, b, sfb, 2)
    if out is None:
        out = _new(a, (m, n), torch.bfloat16, stream)
    else:
        _shape(_bits16(out, "out"), (m, n), "out")
    _on_device(a, sfa, b, sfb, out)
    _check(lib.gemm_mxfp4(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), m, n, k, _stream(stream)),
           "gemm_mxfp4")
    return out


def gemm_mxfp4_grouped(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                       offsets: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """Rows offsets[e] .. offsets[e+1]-1 of A [S, K/2] times expert e of B [E, N, K/2] (scales SFA [S, K/32],
    SFB [E, N, K/32], offsets int32 [E + 1] on the device) -> bf16 [S, N]. Rows before offsets[0] and from
    offsets[E] on are not written."""
    (e, n), s, k = _mx_operands(a, sfa, b, sfb, 3)
    _shape(_i32(offsets, "offsets"), (e + 1,), "offsets")
    if out is None:
        out = _new(a, (s, n), torch.bfloat16, stream)
    else:
        _shape(_bits16(out, "out"), (s, n), "out")
    _on_device(a, sfa, b, sfb, offsets, out)
    _check(lib.gemm_mxfp4_grouped(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(offsets), _ptr(out), s, n, k, e,
                                  _stream(stream)), "gemm_mxfp4_grouped")
    return out


# ---------------------------------------------------------------------------
# Expert routing
# ---------------------------------------------------------------------------

class MoeRouting(NamedTuple):
    """What moe_route decides (see include/blockgemm.h): device tensors, and the two arguments that
    moe_route_backward needs again."""
    ids: torch.Tensor          # int32 [T, k], -1: no choice
    weights: torch.Tensor      # float32 [T, k]
    counts: torch.Tensor       # int32 [E]
    offsets: torch.Tensor      # int32 [E + 1]
    rows: torch.Tensor         # int32 [T * k]: the row at every place, -1 behind the last
    pos: torch.Tensor          # int32 [T, k]: the place of every choice, -1: none
    mean_probs: torch.Tensor   # float32 [E]
    loss: torch.Tensor         # float32 scalar
    n_valid: torch.Tensor      # int32 scalar
    k: int
    normalize: bool


class _RoutingPointers(ctypes.Structure):
    _fields_ = [(f, _p) for f in MoeRouting._fields[:9]]


def moe_route_workspace_bytes(t: int, e: int) -> int:
    return int(lib.moe_route_workspace_bytes(t, e))


def _new_routing(logits: torch.Tensor, t: int, e: int, k: int):
    """The tensors of a MoeRouting, and their addresses. Arrays of a kind share one allocation (a
    caching allocation costs the host more than a view)."""
    i32, f32 = torch.int32, torch.float32
    choices, whole = logits.new_empty((3, t, k), dtype=i32), logits.new_empty(2 * e + 2, dtype=i32)
    weights, real = logits.new_empty((t, k), dtype=f32), logits.new_empty(e + 1, dtype=f32)
    ids, pos, rows = choices.unbind(0)
    counts, offsets, n_valid = whole.split_with_sizes((e, e + 1, 1))
    mean_probs, loss = real.split_with_sizes((e, 1))
    c, w, r = choices.data_ptr(), whole.data_ptr(), real.data_ptr()
    n = 4 * t * k
    return ((ids, weights, counts, offsets, rows.view(-1), pos, mean_probs, loss.view(()), n_valid.view(())),
            _RoutingPointers(c, weights.data_ptr(), w, w + 4 * e, c + 2 * n, c + n, r, r + 4 * e, w + 8 * e + 4))


def moe_route(logits: torch.Tensor, k: int, valid: torch.Tensor | None = None, normalize: bool = True,
              workspace: torch.Tensor | None = None, stream=None) -> MoeRouting:
    """Top-k routing of router logits [T, E] (bfloat16 or float32): choices, weights, per-expert counts, the
    dispatch order and the balance loss. `valid` (bool or byte [T]) leaves rows out. `workspace` is a byte
    tensor of moe_route_workspace_bytes(T, E) bytes (allocated if None)."""
    kind = _type(logits, "logits")
    t, e = _dims(logits, 2, "logits")
    if not 1 <= k <= min(e, 16):
        raise ValueError(f"k = {k} must lie in 1 .. min(E, 16) = {min(e, 16)}")
    if valid is not None:
        _tensor(valid, "valid")
        if valid.element_size() != 1 or valid.is_floating_point():
            raise TypeError(f"valid: expected bool or bytes, got {valid.dtype}")
        _shape(valid, (t,), "valid")
    _on_device(logits, valid, workspace)
    if workspace is None:
        need = moe_route_workspace_bytes(t, e)
        workspace = _new(logits, need, torch.uint8, stream) if need else None
    if stream is None:
        tensors, ptrs = _new_routing(logits, t, e, k)
    else:
        with _on_stream(stream, logits.device):
            tensors, ptrs = _new_routing(logits, t, e, k)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.moe_route(_ptr(logits), kind, _ptr(valid), ctypes.byref(ptrs), _ptr(workspace), ws_bytes, t, e, k,
                         1 if normalize else 0, _stream(stream)), "moe_route")
    return MoeRouting(*tensors, k, bool(normalize))


def moe_route_backward(logits: torch.Tensor, routing: MoeRouting, dweights: torch.Tensor | None = None,
                       dloss: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """The gradient of the logits, for gradients of routing.weights (float32 [T, k]) and of routing.loss (one
    float32); None is zero. `out` may be the logits."""
    kind = _type(logits, "logits")
    t, e = _dims(logits, 2, "logits")
    _shape(_i32(routing.ids, "ids"), (t, routing.k), "ids")
    _shape(_f32(routing.weights, "weights"), (t, routing.k), "weights")
    _shape(_i32(routing.counts, "counts"), (e,), "counts")
    if _i32(routing.n_valid, "n_valid").numel() != 1:
        raise ValueError(f"n_valid must hold one value, got shape {tuple(routing.n_valid.shape)}")
    if dweights is not None:
        _shape(_f32(dweights, "dweights"), (t, routing.k), "dweights")
    if dloss is not None and _f32(dloss, "dloss").numel() != 1:
        raise ValueError(f"dloss must hold one value, got shape {tuple(dloss.shape)}")
    if out is None:
        out = _new(logits, (t, e), logits.dtype, stream)
    elif _type(out, "out") != kind:
        raise TypeError(f"out: expected {logits.dtype}, got {out.dtype}")
    else:
        _shape(out, (t, e), "out")
    _on_device(logits, routing.ids, routing.weights, routing.counts, routing.n_valid, dweights, dloss, out)
    _check(lib.moe_route_backward(_ptr(logits), kind, _ptr(routing.ids), _ptr(routing.weights), _ptr(routing.counts),
                                  _ptr(routing.n_valid), _ptr(dweights), _ptr(dloss), _ptr(out), t, e, routing.k,
                                  1 if routing.normalize else 0, _stream(stream)), "moe_route_backward")
    return out


# ---------------------------------------------------------------------------
# The gated MLP block, and the gradients of dense products
# ---------------------------------------------------------------------------

_ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}   # bg_activation


def _activation(act: str) -> int:
    kind = _ACTIVATIONS.get(act)
    if kind is None:
        raise ValueError(f"act must be one of {', '.join(map(repr, _ACTIVATIONS))}, got {act!r}")
    return kind


def _bytes_of(query, name: str, m: int, n: int, k: int) -> int:
    nbytes = ctypes.c_size_t(0)
    _check(query(m, n, k, ctypes.byref(nbytes)), name)
    return nbytes.value


def gemm_bf16_nn_workspace(m: int, n: int, k: int) -> int:
    """Bytes of workspace gemm_bf16_nn needs on the current device."""
    return _bytes_of(lib.gemm_bf16_nn_workspace, "gemm_bf16_nn_workspace", m, n, k)


def gemm_bf16_tn_workspace(m: int, n: int, k: int) -> int:
    """Bytes of workspace gemm_bf16_tn needs on the current device."""
    return _bytes_of(lib.gemm_bf16_tn_workspace, "gemm_bf16_tn_workspace", m, n, k)


def gemm_bf16_gated_backward_workspace(m: int, n: int, k: int) -> int:
    """Bytes of workspace gemm_bf16_gated_backward needs on the current device."""
    return _bytes_of(lib.gemm_bf16_gated_backward_workspace, "gemm_bf16_gated_backward_workspace", m, n, k)


def _given(out, shape, what: str = "out"):
    """An output that the caller may supply: None, or checked."""
    if out is not None:
        _shape(_bits16(out, what), shape, what)
    return out


def _scratch(workspace, need, like: torch.Tensor, stream):
    """(workspace, its bytes): the caller's, or a new one of need() bytes."""
    if workspace is None:
        nbytes = need()
        if nbytes == 0:
            return None, 0
        return _new(like, nbytes, torch.uint8, stream), nbytes
    return workspace, workspace.numel() * workspace.element_size()


def gemm_bf16_nn(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """C[M,N] = bf16(A[M,K] @ B[K,N]), FP32 accumulation: dX = dY @ W for weights W [out, in]. `workspace` is a
    byte tensor of gemm_bf16_nn_workspace(M, N, K) bytes (allocated if None)."""
    m, k = _dims(_bits16(a, "A"), 2, "A")
    _, n = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (k, n), "B")
    _given(out, (m, n))
    if workspace is not None:
        _tensor(workspace, "workspace")
    _on_device(a, b, out, workspace)
    if out is None:
        out = _new(a, (m, n), torch.bfloat16, stream)
    workspace, ws_bytes = _scratch(workspace, lambda: gemm_bf16_nn_workspace(m, n, k), a, stream)
    _check(lib.gemm_bf16_nn(_ptr(a), _ptr(b), _ptr(out), _ptr(workspace), ws_bytes, m, n, k, _stream(stream)),
           "gemm_bf16_nn")
    return out


def gemm_bf16_tn(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """C[M,N] = bf16(A[K,M]^T @ B[K,N]), FP32 accumulation: dW = dY^T @ X, the sum over the rows of both.
    `workspace` is a byte tensor of gemm_bf16_tn_workspace(M, N, K) bytes (allocated if None)."""
    k, m = _dims(_bits16(a, "A"), 2, "A")
    _, n = _dims(_bits16(b, "B"), 2, "B")
    _shape(b, (k, n), "B")
    _given(out, (m, n))
    if workspace is not None:
        _tensor(workspace, "workspace")
    _on_device(a, b, out, workspace)
    if out is None:
        out = _new(a, (m, n), torch.bfloat16, stream)
    workspace, ws_bytes = _scratch(workspace, lambda: gemm_bf16_tn_workspace(m, n, k), a, stream)
    _check(lib.gemm_bf16_tn(_ptr(a), _ptr(b), _ptr(out), _ptr(workspace), ws_bytes, m, n, k, _stream(stream)),
           "gemm_bf16_tn")
    return out


def gemm_bf16_gated(a: torch.Tensor, b0: torch.Tensor, b1: torch.Tensor, act: str = "silu",
                    save: bool | torch.dtype = False, out: torch.Tensor | None = None, stream=None):
    """H = bf16(act(A @ B0^T) * (A @ B1^T)) for A [M,K], B0 and B1 [N,K]; act is "silu" or "gelu_tanh". With
    `save`, (H, G, U): G = A @ B0^T and U = A @ B1^T too, for gemm_bf16_gated_backward, in float32 (True) or in
    the dtype given (torch.bfloat16: half the memory, the gradient a little less exact). K % 8 != 0 is slow: pad
    such a K with zeros where that matters."""
    kind = _activation(act)
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b0, "B0"), 2, "B0")
    _shape(b0, (n, k), "B0")
    _shape(_bits16(b1, "B1"), (n, k), "B1")
    _given(out, (m, n))
    _on_device(a, b0, b1, out)
    if out is None:
        out = _new(a, (m, n), torch.bfloat16, stream)
    kept = torch.float32 if save is True else save
    g, u = (_new(a, (m, n), kept, stream) for _ in range(2)) if save else (None, None)
    _check(lib.gemm_bf16_gated(_ptr(a), _ptr(b0), _ptr(b1), _ptr(out), _ptr(g), _ptr(u), _type(g, "save") if save else 0,
                               kind, m, n, k,
                               _stream(stream)), "gemm_bf16_gated")
    return (out, g, u) if save else out


def gemm_bf16_gated_backward(dh: torch.Tensor, a: torch.Tensor, b0: torch.Tensor, b1: torch.Tensor, g: torch.Tensor,
                             u: torch.Tensor, act: str = "silu", need_a: bool = True, need_b: bool = True,
                             workspace: torch.Tensor | None = None, stream=None):
    """(dA, dB0, dB1) for a gradient dH [M,N] of gemm_bf16_gated's H, with the G and U it saved; None where need_a
    or need_b is false. `workspace` is a byte tensor of gemm_bf16_gated_backward_workspace(M, N, K) bytes (allocated
    if None). K % 8 != 0 is slow (any N is not): pad such a K with zeros where that matters."""
    kind = _activation(act)
    m, k = _dims(_bits16(a, "A"), 2, "A")
    n, _ = _dims(_bits16(b0, "B0"), 2, "B0")
    _shape(b0, (n, k), "B0")
    _shape(_bits16(b1, "B1"), (n, k), "B1")
    _shape(_bits16(dh, "dH"), (m, n), "dH")
    kept = _type(g, "G")
    _shape(g, (m, n), "G")
    if _type(u, "U") != kept:
        raise TypeError(f"U: expected {g.dtype}, got {u.dtype}")
    _shape(u, (m, n), "U")
    if workspace is not None:
        _tensor(workspace, "workspace")
    _on_device(dh, a, b0, b1, g, u, workspace)
    da = _new(a, (m, k), torch.bfloat16, stream) if need_a else None
    db0, db1 = (_new(a, (n, k), torch.bfloat16, stream) for _ in range(2)) if need_b else (None, None)
    workspace, ws_bytes = _scratch(workspace, lambda: gemm_bf16_gated_backward_workspace(m, n, k), a, stream)
    _check(lib.gemm_bf16_gated_backward(_ptr(dh), _ptr(a), _ptr(b0), _ptr(b1), _ptr(g), _ptr(u), kept, _ptr(da),
                                        _ptr(db0), _ptr(db1), kind, _ptr(workspace), ws_bytes, m, n, k, _stream(stream)),
           "gemm_bf16_gated_backward")
    return da, db0, db1


# ---------------------------------------------------------------------------
# Few rows times weights in 4 bits
# ---------------------------------------------------------------------------

_W4_FORMATS = {"int4": 0, "mxfp4": 1, "nvfp4": 2}   # bg_w4_format
_W4_GROUPS = {"mxfp4": 32, "nvfp4": 16}


class W4Weights(NamedTuple):
    """Weights [N, K] in 4 bits for gemv_w4 and gemv_w4_gated (see bg_w4 in include/blockgemm.h)."""
    codes: torch.Tensor                    # bytes [N, K/2]
    scales: torch.Tensor                   # [N, K/group]: bfloat16 for "int4", else bytes
    format: str                            # "int4", "mxfp4" or "nvfp4"
    group: int | None = None               # elements under a scale (None: the format's own)
    zeros: torch.Tensor | None = None      # "int4": bytes [N, K/group], or None (8)
    scale_2: float = 1.0                   # "nvfp4"


class _W4(ctypes.Structure):
    _fields_ = [("codes", _p), ("scales", _p), ("zeros", _p), ("format", ctypes.c_int), ("group", _u32), ("scale_2", ctypes.c_float)]


def _w4(w: W4Weights, k: int, what: str):
    """(struct, N) of weights with K = k."""
    codes, scales, fmt, group, zeros, scale_2 = w
    kind = _W4_FORMATS.get(fmt)
    if kind is None:
        raise ValueError(f"{what}: format must be one of {', '.join(map(repr, _W4_FORMATS))}, got {fmt!r}")
    own = _W4_GROUPS.get(fmt)
    if group is None:
        group = own
    if group is None or group <= 0 or (group != own if own else group % 32 != 0):
        raise ValueError(f"{what}: group of {fmt} weights must be {own or 'a multiple of 32'}, got {w.group}")
    _blocks32(k)
    if k % group != 0:
        raise ValueError(f"{what}: K = {k} must be a multiple of the group, {group}")
    shape = _dims(_bytes(codes, what), 2, what)
    n = shape[0]
    if shape[1] != k // 2:
        raise ValueError(f"{what}: codes must have shape {(n, k // 2)}, got {tuple(shape)}")
    if own is None:
        _bits16(scales, what)
    else:
        _bytes(scales, what)
    _shape(scales, (n, k // group), what)
    if zeros is not None:
        if own is not None:
            raise ValueError(f"{what}: {fmt} weights have no zeros")
        _shape(_bytes(zeros, what), (n, k // group), what)
    _on_device(codes, scales, zeros)
    return _W4(_ptr(codes), _ptr(scales), _ptr(zeros), kind, group, scale_2), n


def gemv_w4(x: torch.Tensor, w: W4Weights, out: torch.Tensor | None = None, stream=None):
    """Y[R,N] = bf16(x[R,K] @ deq(W)^T) for few rows of bfloat16 activations (16 at a time; from about 128 rows
    gemm_w4a16 is faster for "nvfp4"). K is a multiple of 32."""
    r, k = _dims(_bits16(x, "x"), 2, "x")
    held, n = _w4(w, k, "W")
    _given(out, (r, n))
    _on_device(x, out)
    if out is None:
        out = _new(x, (r, n), torch.bfloat16, stream)
    _check(lib.gemv_w4(_ptr(x), ctypes.byref(held), _ptr(out), r, n, k, _stream(stream)), "gemv_w4")
    return out


def gemv_w4_gated(x: torch.Tensor, w0: W4Weights, w1: W4Weights, act: str = "silu", out: torch.Tensor | None = None,
                  stream=None):
    """H[R,N] = bf16(act(x @ deq(W0)^T) * (x @ deq(W1)^T)) for few rows; both weights of one format and group."""
    kind = _activation(act)
    r, k = _dims(_bits16(x, "x"), 2, "x")
    held0, n = _w4(w0, k, "W0")
    held1, n1 = _w4(w1, k, "W1")
    if n1 != n or held1.format != held0.format or held1.group != held0.group or (w0.zeros is None) != (w1.zeros is None):
        raise ValueError("W0 and W1 must have the same shape, format and group, both or neither zeros")
    _given(out, (r, n))
    _on_device(x, out)
    if out is None:
        out = _new(x, (r, n), torch.bfloat16, stream)
    _check(lib.gemv_w4_gated(_ptr(x), ctypes.byref(held0), ctypes.byref(held1), _ptr(out), kind, r, n, k,
                             _stream(stream)), "gemv_w4_gated")
    return out


# ---------------------------------------------------------------------------
# Tuning overrides and the tile-order helper (host only)
# ---------------------------------------------------------------------------

TUNE_TILE, TUNE_COLSPLIT, TUNE_ORDERED, TUNE_FP4_TILE, TUNE_FP4_SPLITK_TILE, TUNE_W4A16_TILE, \
    TUNE_STREAMK_TILE = range(7)


def tune_set(key: int, value: int) -> None:
    """Force one automatic choice of the library (value -1 restores it)."""
    _check(lib.bg_tune_set(int(key), int(value)), "bg_tune_set")


def tune_get(key: int) -> int:
    return int(lib.bg_tune_get(int(key)))


class tuned:
    """Context manager: `with tuned(TUNE_TILE, 3): ...` forces a choice and restores the previous one."""

    def __init__(self, key: int, value: int):
        self.key, self.value, self.prev = key, value, None

    def __enter__(self):
        self.prev = tune_get(self.key)
        tune_set(self.key, self.value)
        return self

    def __exit__(self, *exc):
        tune_set(self.key, self.prev)
        return False


def tile_map(order: int, tiles_m: int, tiles_n: int):
    """(tm, tn) int32 arrays: the tile each workgroup of a tiles_m x tiles_n grid computes."""
    import numpy as np
    n = tiles_m * tiles_n
    tm = np.zeros(n, np.int32)
    tn = np.zeros(n, np.int32)
    _check(lib.bg_tile_map(int(order), tiles_m, tiles_n, tm.ctypes.data, tn.ctypes.data), "bg_tile_map")
    return tm, tn
