"""The gated block and the 4-bit products as a program uses them: a whole MLP
training step against differences, graphs, streams, given outputs and
workspaces, special values, empty dimensions, offsets past 32 bits."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
from gated_util import U16, check_gated, check_product, grid, normal
from oracle import gated as og
from test_gpu_gemv_w4 import check, weights

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu_tanh"]


def mlp_step(x, w0, w1, wd, dy, act):
    """(y, dx, dw0, dw1, dwd) of y = gated(x) wd^T."""
    h, g, u = bg.gemm_bf16_gated(x, w0, w1, act=act, save=True)
    y = bg.gemm_bf16(h, wd)
    dh, dwd = bg.gemm_bf16_nn(dy, wd), bg.gemm_bf16_tn(dy, h)
    return y, *bg.gemm_bf16_gated_backward(dh, x, w0, w1, g, u, act=act), dwd


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(2, 72, 64), (150, 208, 136), (70, 129, 96)])
def test_mlp_step_against_differences(m, n, k, act):
    """sum dy y, whose exact gradients are the step's, along random directions.
    Every product's operands are rounded to BF16 at most three times on the way
    to a gradient (h, dh, dg), and the gradient once: 4 U16 of each element's
    terms, which with independent signs stay below 4 U16 of the norms."""
    x, w0, w1, wd = normal((m, k), 1.0, 1), normal((n, k), 1.2 / k ** 0.5, 2), normal((n, k), 1.0 / k ** 0.5, 3), normal((k, n), 1.0 / n ** 0.5, 4)
    dy = normal((m, k), 1.0, 5)
    y, *grads = mlp_step(x, w0, w1, wd, dy, act)
    args = [t.double() for t in (x, w0, w1, wd)]

    def loss(a, b0, b1, d):
        return (dy.double() * (og.gated(a, b0, b1, act)[0] @ d.T)).sum().item()

    gen = torch.Generator(device="cuda").manual_seed(6)
    for i, got in enumerate(grads):
        for _ in range(3):
            d = torch.randn(args[i].shape, generator=gen, device="cuda", dtype=torch.float64)
            eps = 1e-5
            ends = [loss(*(a + s * d if i == j else a for j, a in enumerate(args))) for s in (eps, -eps)]
            want = (ends[0] - ends[1]) / (2 * eps)
            # d is normal: the error's sum over it is a normal of the error's norm (five deviations)
            tol = 5 * 4 * U16 * got.double().norm().item() + 1e-4
            assert abs((got.double() * d).sum().item() - want) <= tol, (i, want)


def test_step_captured_and_replayed():
    m, n, k = 96, 264, 128
    w0, w1, wd = normal((n, k), 0.1, 2), normal((n, k), 0.1, 3), normal((k, n), 0.1, 4)
    x, dy = torch.empty(m, k, device="cuda", dtype=torch.bfloat16), torch.empty(m, k, device="cuda", dtype=torch.bfloat16)
    q, _ = weights(n, k, "int4", 32, True, 7)
    q1, _ = weights(n, k, "int4", 32, True, 8)

    def step():
        return *mlp_step(x, w0, w1, wd, dy, "silu"), bg.gemv_w4_gated(x[:3], q, q1), bg.gemv_w4(x[:1], q)

    def fill(seed):
        x.copy_(normal((m, k), 1.0, 10 + seed))
        dy.copy_(normal((m, k), 1.0, 20 + seed))

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(5):
        fill(seed)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), seed


def test_on_another_stream():
    """Given as an argument and as the current stream, behind work on it."""
    m, n, k = 200, 136, 512
    a, b0, b1, dh = normal((m, k), 1.0, 1), normal((n, k), 0.1, 2), normal((n, k), 0.1, 3), normal((m, n), 0.1, 4)
    bt = b0.t().contiguous()
    w, _ = weights(n, k, "mxfp4", 32, False, 5)

    def calls(a, **on):
        h, g, u = bg.gemm_bf16_gated(a, b0, b1, save=True, **on)
        return (h, *bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, **on), bg.gemm_bf16_nn(a, bt, **on),
                bg.gemm_bf16_tn(a, dh, **on), bg.gemv_w4(a[:2], w, **on))

    want = calls(a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for arg in (True, False):
        late = torch.empty_like(a)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
            late.copy_(a)
            got = None if arg else calls(late)
        if arg:
            got = calls(late, stream=s)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        del got


def test_given_outputs_and_workspaces_keep_their_surroundings():
    """Outputs inside a larger buffer, exact workspaces full of NaN: the same
    bits, and nothing written outside."""
    m, n, k = 67, 77, 392
    a, b0, b1, dh = normal((m, k), 1.0, 1), normal((n, k), 0.1, 2), normal((n, k), 0.1, 3), normal((m, n), 0.1, 4)
    at, bt = a.t().contiguous(), b0.t().contiguous()
    w, _ = weights(n, k // 32 * 32, "nvfp4", 16, False, 5)
    xw = a[:5, :k // 32 * 32].contiguous()

    def inside(rows, cols):
        buf = torch.full((rows * cols + 512,), 7.0, device="cuda", dtype=torch.bfloat16)
        return buf, buf[256:256 + rows * cols].view(rows, cols)

    def scratch(nbytes):
        buf = torch.full((nbytes + 512,), 0xFF, device="cuda", dtype=torch.uint8)
        return buf, buf[256:256 + nbytes]

    def kept(buf, size):
        return (buf[:256] == buf[0]).all() and (buf[256 + size:] == buf[0]).all()

    for call, want in ((lambda o: bg.gemm_bf16_gated(a, b0, b1, out=o), bg.gemm_bf16_gated(a, b0, b1)),
                       (lambda o: bg.gemv_w4(xw, w, out=o), bg.gemv_w4(xw, w)),
                       (lambda o: bg.gemv_w4_gated(xw, w, w, out=o), bg.gemv_w4_gated(xw, w, w))):
        buf, out = inside(*want.shape)
        assert call(out) is out and torch.equal(out, want) and kept(buf, out.numel())
    for f, need, x, y in ((bg.gemm_bf16_nn, bg.gemm_bf16_nn_workspace, a, bt), (bg.gemm_bf16_tn, bg.gemm_bf16_tn_workspace, at, bt)):
        want = f(x, y)
        nbytes = need(m, n, k)
        buf, out = inside(m, n)
        wbuf, ws = scratch(nbytes)
        assert torch.equal(f(x, y, out=out, workspace=ws), want) and kept(buf, m * n) and kept(wbuf, nbytes)
        if nbytes:
            with pytest.raises(bg.BlockGemmError):
                f(x, y, workspace=ws[:-1])
    for rows in (m, 30):
        _, g, u = bg.gemm_bf16_gated(a[:rows], b0, b1, save=True)
        want = bg.gemm_bf16_gated_backward(dh[:rows], a[:rows], b0, b1, g, u)
        nbytes = bg.gemm_bf16_gated_backward_workspace(rows, n, k)
        wbuf, ws = scratch(nbytes)
        got = bg.gemm_bf16_gated_backward(dh[:rows], a[:rows], b0, b1, g, u, workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip(got, want)) and kept(wbuf, nbytes)
        with pytest.raises(bg.BlockGemmError) as e:
            bg.gemm_bf16_gated_backward(dh[:rows], a[:rows], b0, b1, g, u, workspace=ws[:-1])
        assert e.value.status == bg.BG_ERR_WORKSPACE


@pytest.mark.parametrize("act", ACTS)
def test_special_values_stay_in_their_rows(act):
    """NaN and infinities reach what depends on them, and nothing else; far
    pre-activations give act's limits."""
    m, n, k = 70, 130, 72
    a, b0, b1, dh = normal((m, k), 1.0, 1), normal((n, k), 0.1, 2), normal((n, k), 0.1, 3), normal((m, n), 0.1, 4)
    h, g, u = bg.gemm_bf16_gated(a, b0, b1, act=act, save=True)
    clean = bg.gemm_bf16_gated_backward(dh, a, b0, b1, g, u, act=act)
    bad = a.clone()
    bad[5, 7], bad[69, 0] = float("nan"), float("inf")
    h2, g2, u2 = bg.gemm_bf16_gated(bad, b0, b1, act=act, save=True)
    same = torch.ones(m, dtype=torch.bool, device="cuda")
    same[5] = same[69] = False
    assert torch.equal(h2[same], h[same]) and h2[5].isnan().all() and not h2[69].isfinite().any()
    dh2 = dh.clone()
    dh2[3, 4] = float("nan")
    da, db0, db1 = bg.gemm_bf16_gated_backward(dh2, a, b0, b1, g, u, act=act)
    rows = torch.arange(m, device="cuda") != 3
    cols = torch.arange(n, device="cuda") != 4
    assert torch.equal(da[rows], clean[0][rows]) and da[3].isnan().all()
    assert torch.equal(db0[cols], clean[1][cols]) and db0[4].isnan().all() and torch.equal(db1[cols], clean[2][cols])
    # one term per sum: g as given
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 88.0, -88.0, -89.0, 200.0, -200.0, 3e38, -3e38, 1e30, -1e30,
                         float("inf"), float("-inf"), float("nan")], device="cuda").bfloat16()
    x = torch.zeros(len(vals), 8, device="cuda", dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = vals, 1.0
    e0, e1 = torch.zeros(1, 8, device="cuda").bfloat16(), torch.zeros(1, 8, device="cuda").bfloat16()
    e0[0, 0], e1[0, 1] = 1.0, 1.0
    finite = vals.isfinite()
    h, g, u = bg.gemm_bf16_gated(x[finite], e0, e1, act=act, save=True)
    want = og.gate(vals[finite].double(), act)
    ref = want[0].clamp(-3.4e38, 3.4e38)
    # past e^88 the sigmoid is 0 where act is below 2^-120
    assert ((h[:, 0].double() - ref).abs() <= 2 * U16 * ref.abs() + 2.0 ** -120).all()
    one = torch.ones_like(h)
    da = bg.gemm_bf16_gated_backward(one, x[finite], e0, e1, g, u, act=act)[0]
    dg = da[:, 0]
    slope = og.gate(vals[finite].double().clamp(-1e18, 1e18), act)[1]      # the slope's limits: 0 and 1
    assert ((dg.double() - slope).abs() <= 2 * U16 * slope.abs() + 2.0 ** -100).all()


@pytest.mark.parametrize("fmt,group", [("int4", 32), ("int4", 128), ("mxfp4", 32), ("nvfp4", 16)])
def test_gemv_special_values(fmt, group):
    """A row with a NaN is NaN and leaves the others; a NaN or infinite scale is
    one column's; scale bytes at their ends."""
    r, n, k = 5, 40, 256
    x = normal((r, k), 1.0, 1)
    w, v = weights(n, k, fmt, group, False, 2)
    y = bg.gemv_w4(x, w)
    bad = x.clone()
    bad[2, 100] = float("nan")
    y2 = bg.gemv_w4(bad, w)
    keep = torch.arange(r, device="cuda") != 2
    assert torch.equal(y2[keep], y[keep]) and y2[2].isnan().all()
    s = w.scales.clone()
    s[3, -1] = float("nan") if fmt == "int4" else 255 if fmt == "mxfp4" else 0x7F
    y3 = bg.gemv_w4(x, w._replace(scales=s))
    cols = torch.arange(n, device="cuda") != 3
    assert torch.equal(y3[:, cols], y[:, cols]) and y3[:, 3].isnan().all()
    if fmt == "mxfp4":         # 2^-127, 2^-126 and 2^127 exactly
        for byte in (0, 1, 254):
            one = bg.W4Weights(torch.full((16, 16), 0x22, device="cuda", dtype=torch.uint8),
                               torch.full((16, 1), byte, device="cuda", dtype=torch.uint8), "mxfp4")
            e = torch.zeros(1, 32, device="cuda", dtype=torch.bfloat16)
            e[0, 9] = 1.0
            assert (bg.gemv_w4(e, one).double() == 2.0 ** (byte - 127)).all()


def test_empty_dimensions():
    dev = dict(device="cuda", dtype=torch.bfloat16)
    e = lambda *s: torch.empty(s, **dev)  # noqa: E731
    assert bg.gemm_bf16_gated(e(0, 8), e(5, 8), e(5, 8)).shape == (0, 5)
    assert bg.gemm_bf16_gated(e(4, 8), e(0, 8), e(0, 8)).shape == (4, 0)
    assert (bg.gemm_bf16_gated(e(70, 0), e(5, 0), e(5, 0)) == 0).all()
    for m, n in ((70, 40), (300, 200)):
        assert (bg.gemm_bf16_nn(e(m, 0), e(0, n)) == 0).all() and (bg.gemm_bf16_tn(e(0, m), e(0, n)) == 0).all()
    b0, b1 = normal((40, 72), 1.0, 1), normal((40, 72), 1.0, 2)
    f = torch.empty((0, 40), device="cuda")
    da, db0, db1 = bg.gemm_bf16_gated_backward(e(0, 40), e(0, 72), b0, b1, f, f)
    assert da.shape == (0, 72) and (db0 == 0).all() and (db1 == 0).all()
    for m in (5, 100):
        f = torch.empty((m, 0), device="cuda")
        da, db0, db1 = bg.gemm_bf16_gated_backward(e(m, 0), normal((m, 72), 1.0, 3), e(0, 72), e(0, 72), f, f)
        assert (da == 0).all() and da.shape == (m, 72) and db0.shape == db1.shape == (0, 72)
    w = bg.W4Weights(torch.empty((6, 0), device="cuda", dtype=torch.uint8), torch.empty((6, 0), device="cuda", dtype=torch.uint8), "nvfp4")
    assert (bg.gemv_w4(e(3, 0), w) == 0).all() and (bg.gemv_w4_gated(e(20, 0), w, w) == 0).all()
    w, _ = weights(6, 64, "int4", 64, True, 1)
    assert bg.gemv_w4(e(0, 64), w).shape == (0, 6)


def test_offsets_past_32_bits():
    """Operands and outputs of more than 2^32 bytes, checked where they end."""
    m, n, k = (1 << 20) + 77, 40, 2304
    a = torch.randint(-2, 3, (m, k), device="cuda", dtype=torch.int8).bfloat16()     # 4.8 GB
    b0, b1 = grid((n, k), 2), grid((n, k), 3)
    rows = torch.tensor([0, 1, 900_001, 1_000_000, m - 2, m - 1], device="cuda")
    h = bg.gemm_bf16_gated(a, b0 * 2.0 ** -7, b1)
    check_gated(h[rows], a[rows], b0 * 2.0 ** -7, b1, "silu", "gated")
    nn = bg.gemm_bf16_nn(a, b0.t().contiguous())
    check_product(nn[rows], a[rows], b0.t(), "nn")
    dy = torch.zeros(m, n, device="cuda", dtype=torch.bfloat16)
    dy[rows] = grid((len(rows), n), 4)
    want = dy[rows].double().T @ a[rows].double()
    assert torch.equal(bg.gemm_bf16_tn(dy, a).double(), want.bfloat16().double())
    wide = bg.gemm_bf16_nn(dy[:70_000], torch.ones(n, 40_000, device="cuda", dtype=torch.bfloat16))     # 5.6 GB out
    for i in (0, 1, 69_999):
        assert (wide[i].double() == dy[i].double().sum().bfloat16().double()).all()
    del wide, a, h, nn, dy
    n, k = 70_001, 131_072
    codes = torch.randint(0, 256, (n, k // 2), device="cuda", dtype=torch.uint8)       # 4.6 GB
    scales = torch.randint(120, 130, (n, k // 32), device="cuda", dtype=torch.uint8)
    x = normal((2, k), 1.0, 5)
    y = bg.gemv_w4(x, bg.W4Weights(codes, scales, "mxfp4"))
    pick = torch.tensor([0, 40_000, n - 1], device="cuda")
    part = bg.W4Weights(codes[pick].contiguous(), scales[pick].contiguous(), "mxfp4")
    from oracle.w4 import dequant_w4
    v = torch.from_numpy(dequant_w4(part.codes.cpu().numpy(), part.scales.cpu().numpy(), "mxfp4", 32)).cuda()
    check(y[:, pick], x, part, v, "gemv")


def test_scales_at_the_end_of_their_memory():
    """Odd numbers of scale bytes, read up to the end of the array's last word."""
    for fmt, k in (("mxfp4", 32), ("mxfp4", 160), ("nvfp4", 32), ("nvfp4", 96)):
        for n in (1, 3, 17):
            w, v = weights(n, k, fmt, 32 if fmt == "mxfp4" else 16, False, n)
            x = normal((2, k), 1.0, k)
            check(bg.gemv_w4(x, w), x, w, v, f"{fmt} {n}x{k}")


@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(seed):
    r = np.random.default_rng(100 + seed)
    m, n, k = (int(v) for v in np.exp(r.uniform(0, np.log([700, 900, 900]))))
    act = ACTS[seed % 2]
    a, b0, b1 = normal((m, k), 1.0, 1), normal((n, k), 1.0 / k ** 0.5, 2), normal((n, k), 1.0 / k ** 0.5, 3)
    check_gated(bg.gemm_bf16_gated(a, b0, b1, act=act), a, b0, b1, act, f"{m}x{n}x{k}")
    bt = b0.t().contiguous()
    check_product(bg.gemm_bf16_nn(a, bt), a, bt, f"nn {m}x{n}x{k}")
    check_product(bg.gemm_bf16_tn(a.t().contiguous(), bt), a, bt, f"tn {m}x{n}x{k}")
    fmt, group = (("int4", 32), ("int4", 64), ("int4", 160), ("mxfp4", 32), ("nvfp4", 16))[seed % 5]
    kk = max(1, k // max(group, 32)) * max(group, 32) * (4 if seed % 3 == 0 else 1)
    rows = int(r.integers(1, 20))
    x = normal((rows, kk), 1.0, 4)
    w, v = weights(n, kk, fmt, group, bool(seed % 2) and fmt == "int4", 5)
    check(bg.gemv_w4(x, w), x, w, v, f"gemv {rows}x{n}x{kk} {fmt}")
