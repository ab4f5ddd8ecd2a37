"""Helpers of the gated block's GPU tests: operands and error bounds."""
import torch

from oracle import gated as og

U32 = 2.0 ** -24       # half a step of FP32, relative
U16 = 2.0 ** -8        # half a step of BF16, relative
TINY = 2.0 ** -130     # below it BF16's steps no longer shrink with the value


def normal(shape, scale, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


def grid(shape, seed):
    """Small whole numbers: every partial sum of a product is exact in FP32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=g, device="cuda").bfloat16()


def within(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()!r}, "
                             f"want {want[i].item()!r}, tolerance {tol[i].item()!r}")


def sum_error(size, k):
    """Bound of an FP32 sum of k exact products: each addition is off by at most
    U32 of a partial sum, itself at most size = sum |a||b|; doubled for a sum
    inside the matrix instruction that keeps one bit less."""
    return 2 * (k + 1) * U32 * size


def check_product(got, a, b, what):
    """got = bf16(a b), a and b BF16 tensors in the shapes of a plain product."""
    a, b = a.double(), b.double()
    want, size = a @ b, a.abs() @ b.abs()
    within(got, want, U16 * want.abs() + sum_error(size, a.shape[1]) + TINY, what)


def gate_error(g, act):
    """Relative error of act(g) in FP32: the exponent's argument rounds four
    times (gelu) or twice, each at most U32 of |z|, and shifts e^-z by as much;
    exp2, the addition, the reciprocal and the product add a unit or less each."""
    z = g.abs() if act == "silu" else 1.6 * (g.abs() + 0.044715 * g.abs() ** 3)
    return U32 * (8 * z + 16)


def check_gated(h, a, b0, b1, act, what):
    a, b0, b1 = a.double(), b0.double(), b1.double()
    want, g, u = og.gated(a, b0, b1, act)
    eg = sum_error(a.abs() @ b0.abs().T, a.shape[1])
    eu = sum_error(a.abs() @ b1.abs().T, a.shape[1])
    v = og.gate(g, act)[0].abs()
    # |act'| <= 1.13
    err = 1.13 * eg * (u.abs() + eu) + v * eu + gate_error(g, act) * (v + 1.13 * eg) * (u.abs() + eu)
    within(h, want, U16 * (want.abs() + err) + err + TINY, what)


def check_backward(da, db0, db1, dh, a, b0, b1, g, u, act, what):
    """Against the formula on g and u as they were kept. dG and dU are rounded
    to BF16 before the products (U16 of their value, or U16 squared up to 64
    rows, besides FP32's few units and the slope's, of which |g| z' s (1 - s) +
    s <= 3 is the size)."""
    low = U16 * U16 if g.shape[0] <= 64 else U16
    dh, a, b0, b1, g, u = (t.double() for t in (dh, a, b0, b1, g, u))
    dg, du = og.gate_grad(dh, g, u, act)
    rel = gate_error(g, act)
    eg = low * dg.abs() + (1 + U16) * rel * 3 * (dh * u).abs() + TINY
    eu = low * du.abs() + (1 + U16) * rel * du.abs() + TINY
    want = og.gated_backward(dh, a, b0, b1, g, u, act)
    sizes = (dg.abs() @ b0.abs() + du.abs() @ b1.abs(), dg.abs().T @ a.abs(), du.abs().T @ a.abs())
    errs = (eg @ b0.abs() + eu @ b1.abs(), eg.T @ a.abs(), eu.T @ a.abs())
    terms = (4 * g.shape[1], 2 * g.shape[0], 2 * g.shape[0])
    for got, w, size, err, k, name in zip((da, db0, db1), want, sizes, errs, terms, ("dA", "dB0", "dB1")):
        if got is None:
            continue
        err = err + sum_error(size + err, k)
        within(got, w, U16 * (w.abs() + err) + err + TINY, f"{what} {name}")
        # rounding errors are independent: together far below their linear sum
        if w.numel() >= 4096:
            rms = ((got.double() - w).square().mean() / w.square().mean()).sqrt().item()
            assert rms <= U16, f"{what} {name}: rms error {rms}"
