"""Pins of the MXFP4 and routing oracle (CPU only) against things other than itself."""
import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle import routing


def test_e8m0_is_a_power_of_two_for_every_byte():
    v = oracle.e8m0_to_f64(np.arange(256))
    assert np.isnan(v[255])
    for s in range(255):
        want = Fraction(2) ** (s - 127)
        assert Fraction(float(v[s])) == want
    # torch's own E8M0 type, where this build has one
    if hasattr(torch, "float8_e8m0fnu"):
        t = torch.arange(255, dtype=torch.uint8).view(torch.float8_e8m0fnu).to(torch.float32).double().numpy()
        assert np.array_equal(t, v[:255])


def test_e2m1_rounding_on_every_value_midpoint_and_its_neighbours():
    mags = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]
    tiny = Fraction(1, 1 << 40)
    for c in range(8):
        assert oracle.f64_to_e2m1(float(mags[c])) == c
        assert oracle.f64_to_e2m1(-float(mags[c])) == c + 8
    for c in range(7):
        mid = (mags[c] + mags[c + 1]) / 2
        assert oracle.f64_to_e2m1(float(mid)) == (c if c % 2 == 0 else c + 1)
        assert oracle.f64_to_e2m1(float(mid - tiny)) == c
        assert oracle.f64_to_e2m1(float(mid + tiny)) == c + 1
    assert oracle.f64_to_e2m1(1e300) == 7 and oracle.f64_to_e2m1(-7.99) == 15
    assert oracle.f64_to_e2m1(-0.0) == 8 and oracle.f64_to_e2m1(-0.25) == 8


@pytest.mark.parametrize("top,scale", [(1.0, 125), (1.999, 125), (2.0, 126), (6.0, 127), (4.0, 127), (7.99, 127), (8.0, 128),
                                       (2.0 ** -126, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (2.0 ** -140, 0), (0.0, 0),
                                       (3.3895e38, 252)])
def test_shared_exponent(top, scale):
    x = np.zeros((1, 32))
    x[0, 17] = -top
    codes, s = oracle.quantize_mxfp4(x)
    assert s[0, 0] == scale
    back = oracle.dequant_mxfp4(codes, s)
    # nearest, or saturated at 6: within a quarter of the value, or half a step of the subnormal range
    assert abs(back[0, 17] + top) <= max(top / 4, 0.25 * 2.0 ** (scale - 127))


def test_blocks_with_nan_or_infinity_are_nan():
    x = np.ones((3, 64))
    x[0, 5], x[1, 40], x[2, 0] = np.nan, np.inf, -np.inf
    codes, s = oracle.quantize_mxfp4(x)
    assert s.tolist() == [[255, 125], [125, 255], [255, 125]]
    back = oracle.dequant_mxfp4(codes, s)
    assert np.isnan(back).sum() == 3 * 32
    assert (back[~np.isnan(back)] == 1.0).all()


def test_values_of_the_format_come_back_unchanged():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (40, 32), dtype=np.uint8)
    codes[:, ::16] |= 0x07                     # every block holds a 6 (or -6): the scale is determined
    s = rng.integers(3, 250, (40, 2), dtype=np.uint8)
    v = oracle.dequant_mxfp4(codes, s)
    c2, s2 = oracle.quantize_mxfp4(v)
    assert np.array_equal(s2, s) and np.array_equal(c2, codes)


def test_product_by_exact_rationals():
    rng = np.random.default_rng(2)
    a, b = rng.integers(0, 256, (3, 32), dtype=np.uint8), rng.integers(0, 256, (4, 32), dtype=np.uint8)
    sa, sb = rng.integers(120, 134, (3, 2), dtype=np.uint8), rng.integers(120, 134, (4, 2), dtype=np.uint8)
    mags = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4), Fraction(6)]

    def val(p, s, i, k):
        c = (int(p[i, k // 2]) >> (4 * (k % 2))) & 15
        return (-1) ** (c >> 3) * mags[c & 7] * Fraction(2) ** (int(s[i, k // 32]) - 127)

    got = oracle.gemm_mxfp4_ref(a, sa, b, sb)
    for i, j in itertools.product(range(3), range(4)):
        assert Fraction(float(got[i, j])) == sum(val(a, sa, i, k) * val(b, sb, j, k) for k in range(64))


def test_grouped_is_the_product_of_every_range():
    rng = np.random.default_rng(3)
    a, sa = rng.integers(0, 256, (9, 16), dtype=np.uint8), rng.integers(120, 130, (9, 1), dtype=np.uint8)
    b, sb = rng.integers(0, 256, (3, 5, 16), dtype=np.uint8), rng.integers(120, 130, (3, 5, 1), dtype=np.uint8)
    got = oracle.gemm_mxfp4_grouped_ref(a, sa, b, sb, [1, 4, 4, 8])
    assert np.isnan(got[0]).all() and np.isnan(got[8]).all()
    for i in range(1, 8):
        e = 0 if i < 4 else 2
        assert np.array_equal(got[i], oracle.dequant_mxfp4(a[i:i + 1], sa[i:i + 1])[0] @ oracle.dequant_mxfp4(b[e], sb[e]).T)


def test_route_against_torch():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(50, 12, generator=g, dtype=torch.float64)
    r = routing.route(x.numpy(), 3)
    p = torch.softmax(x, 1)
    top = torch.topk(p, 3, dim=1)
    assert np.array_equal(r["ids"], top.indices.numpy())
    assert np.allclose(r["weights"], (top.values / top.values.sum(1, keepdim=True)).numpy(), rtol=1e-13)
    assert np.array_equal(r["counts"], torch.bincount(top.indices.flatten(), minlength=12).numpy())
    assert np.allclose(r["mean_probs"], p.mean(0).numpy(), rtol=1e-13)
    # places: sorted by expert, rows ascending within one, and pos is their inverse
    flat = r["ids"].reshape(-1)
    by = np.argsort(flat, kind="stable")
    assert np.array_equal(r["rows"], by // 3)
    assert np.array_equal(r["pos"].reshape(-1)[by], np.arange(150))


def test_route_balanced_batch_has_loss_one():
    x = np.zeros((8, 8))
    for i in range(8):
        x[i, i] = 30.0
    r = routing.route(x, 1)
    assert abs(r["loss"] - 1.0) < 1e-9
    # everything on one expert: E
    assert abs(routing.route(np.tile(x[:1], (8, 1)), 1)["loss"] - 8.0) < 1e-9


def test_route_ties_masks_and_empty_rows():
    x = np.array([[1.0, 1.0, 1.0, 0.5], [-np.inf, -np.inf, -np.inf, -np.inf], [-np.inf, 2.0, -np.inf, -np.inf],
                  [0.0, -0.0, 0.0, -0.0], [9.0, 9.0, 9.0, 9.0]])
    r = routing.route(x, 2, valid=[1, 1, 1, 1, 0])
    assert r["ids"].tolist() == [[0, 1], [-1, -1], [1, -1], [0, 1], [-1, -1]]
    assert r["n_valid"] == 3
    assert r["weights"][2].tolist() == [1.0, 0.0]
    assert r["rows"].tolist() == [0, 3, 0, 2, 3] + [-1] * 5
    e = routing.route(x, 2, valid=np.zeros(5))
    assert e["loss"] == 0.0 and e["n_valid"] == 0 and (e["rows"] == -1).all()


@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_against_differences_and_autograd(normalize):
    rng = np.random.default_rng(5)
    t, e, k = 7, 6, 2
    x = rng.normal(size=(t, e))
    x[2, :] = -np.inf
    x[3, 1:] = -np.inf
    valid = np.array([1, 1, 1, 1, 1, 0, 1])
    dw, dl = rng.normal(size=(t, k)), 1.7
    r = routing.route(x, k, valid, normalize)
    d, mag = routing.route_backward(r, k, normalize, dw, dl)
    assert (np.abs(d) <= mag + 1e-15).all()

    def value(y):
        q = routing.route(y, k, valid, normalize)
        assert np.array_equal(q["ids"], r["ids"])
        return (q["weights"] * dw).sum() + dl * q["loss"]

    h = 1e-6
    for i, f in itertools.product(range(t), range(e)):
        if not np.isfinite(x[i, f]):
            assert d[i, f] == 0.0
            continue
        up, down = x.copy(), x.copy()
        up[i, f] += h
        down[i, f] -= h
        assert abs((value(up) - value(down)) / (2 * h) - d[i, f]) < 1e-8
    # autograd on the live rows with all logits finite
    y = torch.tensor(x[[0, 1, 4, 6]], requires_grad=True)
    p = torch.softmax(y, 1)
    ids = torch.tensor(r["ids"][[0, 1, 4, 6]]).long()
    w = torch.gather(p, 1, ids)
    w = w / w.sum(1, keepdim=True) if normalize else w
    n = r["n_valid"]
    loss = e / (k * n) * (torch.tensor(r["counts"]) * p.sum(0) / n).sum()
    ((w * torch.tensor(dw[[0, 1, 4, 6]])).sum() + dl * loss).backward()
    assert np.allclose(y.grad.numpy(), d[[0, 1, 4, 6]], rtol=1e-10, atol=1e-14)
