"""MXFP4 products under extreme scales, on every path the scales take; grouped
products whose last group of scales starts early; grouped weights past 32-bit
offsets."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
import oracle
import synthetic
from gpu_util import assert_bits_equal, bits_of
from mx_util import check_product, dev, e8m0, exact_bits

pytestmark = pytest.mark.gpu

# few rows (whole turns, and K that ends inside one); then tiles small and
# large with K below 512, of whole steps (an odd number of them too), and of
# any other length
PATHS = [(9, 60, 4128), (16, 60, 8192), (1, 33, 96), (40, 50, 480), (40, 50, 1056), (40, 50, 2048), (40, 50, 1280), (100, 9000, 4096),
         (300, 300, 1536), (2001, 4100, 480), (2000, 4104, 1280), (3000, 4100, 2080), (5000, 3000, 1024), (300, 12000, 1056), (130, 12000, 1792)]


def _sampled(m, n, seed):
    return synthetic.sample_rows(m, min(m, 48), seed), synthetic.sample_rows(n, min(n, 48), seed + 1)


@pytest.mark.parametrize("shift", [-100, 0, 100])
@pytest.mark.parametrize("m,n,k", PATHS)
def test_far_scales_that_cancel(m, n, k, shift):
    """Block c of A is scaled by 2^(s_c - 127 + u_i), of B by 2^(127 - s_c + shift
    - v_j), with s_c over everything that keeps both bytes in 0 .. 254 and u, v
    in {0, 1}: products are multiples of 2^(shift - 3), of at most 72 * 2^shift,
    so sums of 8192 of them are below 2^23 of these steps: exact in FP32."""
    print(f"far scales {m}x{n}x{k} shift {shift}", flush=True)
    g = synthetic._rng(91, m + k)
    lo, hi = max(0, shift), min(253, 253 + shift)
    s = g.integers(lo, hi + 1, k // 32)
    s[0], s[-1] = lo, hi
    u, v = g.integers(0, 2, (m, 1)), g.integers(0, 2, (n, 1))
    sa, sb = (s + u).astype(np.uint8), (254 - s + shift - v).astype(np.uint8)
    assert (s + u).max() <= 254 and (254 - s + shift - v).min() >= 0 and (254 - s + shift - v).max() <= 254
    a, b = synthetic.fp4_packed(m, k, 91, 0), synthetic.fp4_packed(n, k, 91, 1)
    got = bits_of(bg.gemm_mxfp4(dev(a), dev(sa), dev(b), dev(sb)))
    rows, cols = _sampled(m, n, 91)
    assert_bits_equal(got[rows], exact_bits(a[rows], sa[rows], b, sb), f"rows of {m}x{n}x{k}")
    assert_bits_equal(got[:, cols], exact_bits(a, sa, b[cols], sb[cols]), f"columns of {m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", PATHS)
def test_overflow_is_a_signed_infinity_and_underflow_zero(m, n, k):
    """Products of ones, with a sign for every column, so partial sums have one
    sign: 2^254 each, and 2^127 each (the first is finite, the sum of two is
    not); a single 2^127 stays finite; products of 2^-254 sum to zero."""
    print(f"overflow {m}x{n}x{k}", flush=True)
    ones = np.full((m, k // 2), 0x22, np.uint8)              # 1.0, 1.0
    sign = synthetic._rng(92, n).integers(0, 2, (n, 1)).astype(np.uint8)
    b = np.repeat(0x22 | sign * 0x88, k // 2, 1).astype(np.uint8)
    want = torch.from_numpy(np.where(sign[:, 0] == 1, -1.0, 1.0)).cuda()

    def product(x, s_a, s_b):
        full = lambda r, s: torch.full((r, k // 32), s, dtype=torch.uint8, device="cuda")  # noqa: E731
        return bg.gemm_mxfp4(dev(x), full(m, s_a), dev(b), full(n, s_b)).double()

    assert (product(ones, 254, 254) == want * float("inf")).all()
    assert (product(ones, 254, 127) == want * float("inf")).all()
    assert (product(ones, 127, 254) == want * float("inf")).all()
    single = np.zeros_like(ones)
    at = synthetic._rng(92, m).integers(0, k // 2, m)
    single[np.arange(m), at] = 0x20                          # 0, 1.0
    assert (product(single, 254, 127) == want * 2.0 ** 127).all()
    assert (product(single, 100, 154) == want).all()
    assert (product(ones, 0, 0) == 0).all()


# rows of every expert: 32-, 64- and 128-row tiles by their mean
COUNTS = {"few": [3, 0, 20, 1, 0, 9], "some": [33, 0, 65, 17, 40], "many": [128, 0, 257, 100, 1]}


@pytest.mark.parametrize("rows", sorted(COUNTS))
@pytest.mark.parametrize("n,k", [(200, 512), (130, 768), (256, 1024), (129, 1280), (300, 1536), (200, 1792), (64, 2304)])
def test_grouped_groups_of_scales_that_start_early(rows, n, k):
    """K of whole steps whose number is no multiple of a group of scales: the
    last group starts early. Exact sums."""
    print(f"grouped groups {rows} n={n} k={k}", flush=True)
    off = np.concatenate([[0], np.cumsum(COUNTS[rows])]).astype(np.int32)
    s, e = int(off[-1]), len(off) - 1
    a, b = synthetic.fp4_packed(s, k, 93, 0), synthetic.fp4_packed(e * n, k, 93, 1).reshape(e, n, -1)
    sa, sb = e8m0(s, k // 32, 127, 128, 93, 4), e8m0(e * n, k // 32, 127, 128, 93, 5).reshape(e, n, -1)
    got = bits_of(bg.gemm_mxfp4_grouped(dev(a), dev(sa), dev(b), dev(sb), dev(off)))
    for i in range(e):
        lo, hi = off[i], off[i + 1]
        if hi > lo:
            assert_bits_equal(got[lo:hi], exact_bits(a[lo:hi], sa[lo:hi], b[i], sb[i]), f"{rows}, expert {i}")


@pytest.mark.parametrize("rows", [3, 30, 90])
@pytest.mark.parametrize("k", [32768, 32800])
def test_grouped_weights_past_32_bit_offsets(rows, k):
    """6.6 GB of codes and 410 MB of scales; an expert's own are 330 MB."""
    print(f"far experts, {rows} rows each, k={k}", flush=True)
    e, n = 20, 20000
    b = torch.empty((e, n, k // 2), dtype=torch.uint8, device="cuda").random_(0, 256)
    sb = torch.empty((e, n, k // 32), dtype=torch.uint8, device="cuda").random_(127, 129)
    a, sa = synthetic.fp4_packed(e * rows, k, 94, 0), e8m0(e * rows, k // 32, 127, 127, 94, 4)
    off = torch.arange(0, (e + 1) * rows, rows, dtype=torch.int32, device="cuda")
    c = bg.gemm_mxfp4_grouped(dev(a), dev(sa), b, sb, off)
    cols = torch.tensor([0, 1, 6143, 6144, 13107, 13108, n - 2, n - 1], device="cuda")
    for i in (0, 1, 12, 13, 14, e - 1):
        lo, hi = i * rows, (i + 1) * rows
        # sums of 32800 products of at most 72 may pass 2^24 quarters: within the bound of a sum
        check_product(c[lo:hi][:, cols], a[lo:hi], sa[lo:hi], b[i][cols].cpu().numpy(), sb[i][cols].cpu().numpy(), f"expert {i}")


def test_oracle_of_far_scales_is_exact():
    """The FP64 reference itself: scales of 2^127 and 2^-127 cancel."""
    a = np.full((1, 16), 0x22, np.uint8)
    ref = oracle.gemm_mxfp4_ref(a, np.array([[254]], np.uint8), a, np.array([[0]], np.uint8))
    assert ref[0, 0] == 32.0
