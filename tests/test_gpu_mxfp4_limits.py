"""MXFP4 products of more rows than 2^22 small tiles hold."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
import synthetic
from mx_util import dev, e8m0, exact_bits

pytestmark = pytest.mark.gpu


def test_product_of_half_a_thousand_million_rows():
    """2^29 + 5 rows, every one compared: they repeat 4099 different ones (no
    tile height divides it). Exact sums."""
    m, n, k, period = (1 << 29) + 5, 3, 32, 4099
    a, sa = synthetic.fp4_packed(period, k, 31, 0), e8m0(period, 1, 127, 128, 31, 4)
    b, sb = synthetic.fp4_packed(2 * n, k, 31, 1).reshape(2, n, -1), e8m0(2 * n, 1, 127, 128, 31, 5).reshape(2, n, -1)
    want = [dev(exact_bits(a, sa, b[i], sb[i]).view(np.int16)) for i in (0, 1)]
    times = -(-m // period)
    ad, sad = dev(a).repeat(times, 1)[:m], dev(sa).repeat(times, 1)[:m]

    def check(got, first, last, w, what):
        """Rows first .. last - 1 against the repeated rows of w, many periods at a time."""
        got = got.view(torch.int16)
        lo = -(-first // period) * period
        assert torch.equal(got[first:lo], w[first % period:][:lo - first]), what
        per = 20000 * period
        for at in range(lo, last, per):
            hi = min(at + per, last)
            whole = (hi - at) // period
            assert (got[at:at + whole * period].view(whole, period, n) == w).all(), (what, at)
            assert torch.equal(got[at + whole * period:hi], w[:hi - at - whole * period]), (what, at)

    out = bg.gemm_mxfp4(ad, sad, dev(b[0]), dev(sb[0]))
    check(out, 0, m, want[0], "dense")
    out.fill_(7.0)
    cut = (1 << 28) + 77
    off = torch.tensor([0, cut, m - 1], dtype=torch.int32, device="cuda")
    bg.gemm_mxfp4_grouped(ad, sad, dev(b), dev(sb), off, out=out)
    check(out, 0, cut, want[0], "expert 0")
    check(out, cut, m - 1, want[1], "expert 1")
    assert (out[m - 1] == 7.0).all()
