"""GPU parity of the dense and grouped MXFP4 products."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
import oracle
import synthetic
from gpu_util import assert_bits_equal, bits_of
from mx_util import check_product, dev, e8m0, exact_bits, operand

pytestmark = pytest.mark.gpu

# one row to many, N and M around the tiles' edges, K of one block, of odd
# numbers of blocks, and around the steps of 256 and 512 elements
SHAPES = [(1, 1, 32), (1, 300, 64), (2, 17, 96), (1, 4096, 512), (3, 129, 544), (5, 64, 1024), (15, 33, 2080), (16, 256, 256), (17, 257, 288),
          (31, 70, 736), (32, 512, 1056), (33, 31, 512), (47, 200, 4128), (64, 130, 768), (65, 129, 160), (100, 1000, 320), (127, 255, 2080), (128, 256, 2048),
          (129, 65, 480), (200, 384, 1536), (255, 257, 1056), (256, 256, 256), (257, 513, 224), (300, 520, 2048), (513, 300, 992), (700, 1100, 544)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k):
    print(f"mxfp4 {m}x{n}x{k}", flush=True)
    a, sa = operand(m, k, 200 + m, 0)
    b, sb = operand(n, k, 200 + n, 1)
    c = bg.gemm_mxfp4(dev(a), dev(sa), dev(b), dev(sb))
    check_product(c, a, sa, b, sb, f"{m}x{n}x{k}")
    # scales of 1 and 2: products are multiples of 1/4 up to 144, sums of 4128 of them exact in FP32
    ea, eb = e8m0(m, k // 32, 127, 128, 3, 4), e8m0(n, k // 32, 127, 128, 3, 5)
    c = bg.gemm_mxfp4(dev(a), dev(ea), dev(b), dev(eb))
    assert_bits_equal(bits_of(c), exact_bits(a, ea, b, eb), f"exact {m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1, 4096, 7168), (128, 7168, 16384), (1015, 12287, 2080), (5120, 11008, 2048), (4096, 4096, 8192)])
def test_product_at_full_size(m, n, k):
    """Exact sums (scales of 1 and 2, at most 16384 products of at most 144,
    in quarters: below 2^24 quarters), sampled rows, every column."""
    print(f"mxfp4 full {m}x{n}x{k}", flush=True)
    a, b = synthetic.fp4_packed(m, k, 7, 0), synthetic.fp4_packed(n, k, 7, 1)
    ea, eb = e8m0(m, k // 32, 127, 128, 7, 4), e8m0(n, k // 32, 127, 128, 7, 5)
    got = bits_of(bg.gemm_mxfp4(dev(a), dev(ea), dev(b), dev(eb)))
    rows = synthetic.sample_rows(m, 96, 7)
    assert_bits_equal(got[rows], exact_bits(a[rows], ea[rows], b, eb), f"full {m}x{n}x{k}")


# Every tile of the dense product with K below 512, of whole steps, and of any
# other length; few rows with K that ends inside a turn of the eight waves.
TILES = [(9, 500, 4128), (16, 60, 8192), (100, 4100, 32), (100, 4099, 480), (2812, 1430, 288), (100, 9000, 4096), (100, 9000, 4128),
         (129, 12000, 512), (129, 12001, 544), (129, 12002, 160), (2000, 4100, 512), (2001, 4100, 480), (300, 12000, 1056),
         (300, 12004, 352), (3000, 4100, 2080), (3001, 4097, 416), (1000, 4100, 4096), (1001, 4099, 4128), (2000, 4104, 1280), (130, 12000, 1792), (5000, 3000, 1024)]


@pytest.mark.parametrize("m,n,k", TILES)
def test_product_of_every_tile(m, n, k):
    """Exact sums as above; every row of few columns and every column of few rows."""
    print(f"mxfp4 tiles {m}x{n}x{k}", flush=True)
    a, b = synthetic.fp4_packed(m, k, 21, 0), synthetic.fp4_packed(n, k, 21, 1)
    ea, eb = e8m0(m, k // 32, 127, 128, 21, 4), e8m0(n, k // 32, 127, 128, 21, 5)
    got = bits_of(bg.gemm_mxfp4(dev(a), dev(ea), dev(b), dev(eb)))
    rows, cols = synthetic.sample_rows(m, min(m, 64), 21), synthetic.sample_rows(n, min(n, 64), 22)
    assert_bits_equal(got[rows], exact_bits(a[rows], ea[rows], b, eb), f"rows of {m}x{n}x{k}")
    assert_bits_equal(got[:, cols], exact_bits(a, ea, b[cols], eb[cols]), f"columns of {m}x{n}x{k}")


def test_scales_over_the_whole_range():
    """Scale bytes from 0 to 254: products from 2^-254 (zero in FP32) past FP32's largest."""
    a, _ = operand(40, 256, 11, 0)
    b, _ = operand(50, 256, 11, 1)
    sa, sb = np.tile(np.linspace(0, 254, 40).astype(np.uint8)[:, None], (1, 8)), np.full((50, 8), 127, np.uint8)
    c = bg.gemm_mxfp4(dev(a), dev(sa), dev(b), dev(sb)).double().cpu().numpy()
    ref = oracle.gemm_mxfp4_ref(a, sa, b, sb)
    size = oracle.gemm_mxfp4_abs(a, sa, b, sb)
    fine = size < 2.0 ** 127
    # BF16's smallest step is 2^-133; FP32 sums may flush what lies below its normal range
    tol = 2.0 ** -8 * np.abs(ref) + 2 * 257 * 2.0 ** -24 * size + 2.0 ** -126
    assert (np.abs(c - ref)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("m,n,k", [(1, 40, 64), (20, 100, 1056), (130, 300, 512), (300, 300, 800)])
def test_nan_blocks_make_their_row_or_column_nan(m, n, k):
    a, sa = operand(m, k, 12, 0)
    b, sb = operand(n, k, 12, 1)
    sa[m // 2, k // 32 - 1] = 255
    sb[n - 1, 0] = 255
    a[m // 2] = 0                          # zero codes under a NaN scale are NaN too
    c = bg.gemm_mxfp4(dev(a), dev(sa), dev(b), dev(sb))
    check_product(c, a, sa, b, sb, "nan blocks")


@pytest.mark.parametrize("m,n,k", [(1, 33, 96), (20, 70, 288), (150, 200, 608), (300, 260, 1056)])
def test_nothing_behind_the_operands_is_used(m, n, k):
    """Operands inside larger buffers whose other bytes are NaN scales and large codes."""
    a, sa = operand(m, k, 13, 0)
    b, sb = operand(n, k, 13, 1)

    def inside(x):
        buf = np.full(x.size + 4096, 255, np.uint8)
        buf[1024:1024 + x.size] = x.reshape(-1)
        return dev(buf)[1024:1024 + x.size].view(x.shape)

    c = torch.full((m * n + 2048,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = c[1024:1024 + m * n].view(m, n)
    bg.gemm_mxfp4(inside(a), inside(sa), inside(b), inside(sb), out=out)
    check_product(out, a, sa, b, sb, "inside")
    assert (c[:1024] == 3).all() and (c[1024 + m * n:] == 3).all()


def test_empty_k_is_zero():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    out = torch.full((3, 5), 7.0, dtype=torch.bfloat16, device="cuda")
    bg.gemm_mxfp4(z(3, 0), z(3, 0), z(5, 0), z(5, 0), out=out)
    assert (out == 0).all()
    out.fill_(7.0)
    bg.gemm_mxfp4_grouped(z(3, 0), z(3, 0), z(2, 5, 0), z(2, 5, 0), dev(np.array([0, 1, 2], np.int32)), out=out)
    assert (out[:2] == 0).all() and (out[2] == 7).all()


def test_weights_past_32_bit_offsets():
    n, k = 300000, 32768                    # 4.9 GB of codes
    b = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    sb = torch.randint(127, 129, (n, k // 32), dtype=torch.uint8, device="cuda")
    for m in (1, 40, 200):
        a, sa = synthetic.fp4_packed(m, k, 14, 0), e8m0(m, k // 32, 127, 127, 14, 4)
        c = bg.gemm_mxfp4(dev(a), dev(sa), b, sb)
        cols = torch.tensor([0, 1, 131071, 131072, 262143, 262144, 262145, n - 1], device="cuda")
        # quarters below 2^24: sums of 32768 products of at most 72 may pass it, so compare within the bound
        check_product(c[:, cols], a, sa, b[cols].cpu().numpy(), sb[cols].cpu().numpy(), f"far columns, {m} rows")


# --- grouped -----------------------------------------------------------------

GROUPS = {
    "even": [0, 20, 40, 60, 80],
    "some empty": [0, 0, 33, 33, 33, 97, 97],
    "all on one": [0, 0, 0, 150, 150, 150],
    "one row each": list(range(0, 41)),
    "first starts late, last ends early": [5, 9, 60, 61],
    "large and small": [0, 1, 258, 259, 259, 523, 530],
    "single expert": [0, 70],
    "nothing": [0, 0, 0, 0],
}


@pytest.mark.parametrize("name", sorted(GROUPS))
@pytest.mark.parametrize("n,k", [(40, 96), (200, 544), (256, 2048), (513, 1056)])
def test_grouped(name, n, k):
    print(f"grouped {name} n={n} k={k}", flush=True)
    off = np.array(GROUPS[name], np.int32)
    s, e = int(off[-1]) + 3, len(off) - 1
    a, sa = operand(s, k, 300 + e, 0)
    b, sb = operand(e * n, k, 300 + e, 1)
    b, sb = b.reshape(e, n, -1), sb.reshape(e, n, -1)
    out = torch.full((s, n), 9.0, dtype=torch.bfloat16, device="cuda")
    bg.gemm_mxfp4_grouped(dev(a), dev(sa), dev(b), dev(sb), dev(off), out=out)
    for i in range(e):
        lo, hi = off[i], off[i + 1]
        if hi > lo:
            check_product(out[lo:hi], a[lo:hi], sa[lo:hi], b[i], sb[i], f"{name}, expert {i}")
    assert (out[:off[0]] == 9).all() and (out[off[-1]:] == 9).all()


def test_grouped_many_experts_and_exact_bits():
    """1024 experts, up to 40 rows each, exact sums; equal to the dense product of each."""
    rng = np.random.default_rng(15)
    counts = rng.integers(0, 41, 1024)
    counts[rng.random(1024) < 0.4] = 0
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    s, n, k, e = int(off[-1]), 48, 128, 1024
    a, b = synthetic.fp4_packed(s, k, 15, 0), synthetic.fp4_packed(e * n, k, 15, 1).reshape(e, n, -1)
    sa, sb = e8m0(s, k // 32, 127, 128, 15, 4), e8m0(e * n, k // 32, 127, 128, 15, 5).reshape(e, n, -1)
    got = bits_of(bg.gemm_mxfp4_grouped(dev(a), dev(sa), dev(b), dev(sb), dev(off)))
    for i in range(e):
        lo, hi = off[i], off[i + 1]
        if hi > lo:
            assert_bits_equal(got[lo:hi], exact_bits(a[lo:hi], sa[lo:hi], b[i], sb[i]), f"expert {i}")


@pytest.mark.parametrize("off", [[-5, 3, 400, 10 ** 9], [50, 20, 60, 10], [2 ** 31 - 1, -2 ** 31, 7, 30], [90, 95, 99, 120]])
def test_grouped_offsets_out_of_order_or_range_stay_inside(off):
    """Offsets the documentation does not allow: the results are unspecified,
    but nothing outside the output is written."""
    s, n, k, e = 80, 96, 160, 3
    a, sa = operand(s, k, 16, 0)
    b, sb = operand(e * n, k, 16, 1)
    buf = torch.full((s * n + 8192,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[4096:4096 + s * n].view(s, n)
    bg.gemm_mxfp4_grouped(dev(a), dev(sa), dev(b.reshape(e, n, -1)), dev(sb.reshape(e, n, -1)),
                          dev(np.array(off, np.int64).astype(np.int32)), out=out)
    torch.cuda.synchronize()
    assert (buf[:4096] == 5).all() and (buf[4096 + s * n:] == 5).all()


def test_same_bits_every_time_also_captured_and_on_two_streams():
    cases = []
    for m, n, k in [(1, 520, 2080), (64, 300, 1024), (300, 512, 1056)]:
        a, sa = operand(m, k, 17, 0)
        b, sb = operand(n, k, 17, 1)
        cases.append([dev(x) for x in (a, sa, b, sb)])
    want = [bg.gemm_mxfp4(*c).clone() for c in cases]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o in zip(cases, outs):
            bg.gemm_mxfp4(*c, out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [[bg.gemm_mxfp4(*c, stream=s) for c in cases] for s in streams]
        torch.cuda.synchronize()
        for g in got:
            for o, w in zip(g, want):
                assert torch.equal(o, w)
