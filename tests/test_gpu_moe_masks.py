"""The routing gradient where rows are short, masked or not live, beside rows
that are live, and the order of logits below the types' normal range."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
import synthetic
from mx_util import U, dev, f64
from oracle import routing
from test_gpu_moe_route import WHOLE, _logits, _p_err

pytestmark = pytest.mark.gpu


def _masked(t, e, dtype, seed):
    """Logits masked by -infinity (half of them; whole rows; all but one, all
    but fewer than k) and by the type's lowest value; rows full of NaN that
    `valid` leaves out, beside live ones. Returns them, the mask, and what the
    oracle reads (the rows left out as zeros)."""
    x = _logits(t, e, dtype, seed)
    g = synthetic._rng(seed, 5)
    x[torch.from_numpy(g.random((t, e)) < 0.5)] = -float("inf")
    x[1] = -float("inf")
    x[2, 1:] = -float("inf")
    x[2, 0] = 3.0
    x[3, 2:] = -float("inf")
    x[3, :2] = torch.tensor([-1.0, 2.0], dtype=dtype)
    x[4, 2:] = torch.finfo(dtype).min
    x[4, :2] = torch.tensor([1.0, 2.0], dtype=dtype)
    x[5] = torch.finfo(dtype).min
    valid = g.random(t) < 0.8
    valid[:6], valid[[0, 7, t - 1]] = True, False
    x[torch.from_numpy(~valid)] = float("nan")
    seen = x.clone()
    seen[torch.from_numpy(~valid)] = 0.0
    return x, valid, seen


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("t,e,k", [(20, 6, 4), (33, 96, 6), (64, 257, 8), (333, 96, 6), (700, 200, 5), (150, 513, 16)])
def test_gradient_of_masked_and_short_rows(t, e, k, normalize, dtype):
    print(f"masked gradient {t}x{e} k={k} {dtype} normalize={normalize}", flush=True)
    x, valid, seen = _masked(t, e, dtype, 71 + t)
    r = bg.moe_route(x.cuda(), k, valid=dev(valid), normalize=normalize)
    q = routing.route(seen.double().numpy(), k, valid, normalize)
    for f in WHOLE:
        assert np.array_equal(getattr(r, f).cpu().numpy(), q[f]), f
    # gradients of choices that do not exist are not used, whatever they hold
    dw = synthetic._rng(t, 6).standard_normal((t, k)).astype(np.float32)
    missing = q["ids"] < 0
    assert missing[2, 1:].all() and missing[1].all() and missing[~valid].all() and (k < 4 or missing[3, 2:].all())
    dw[missing] = np.nan
    dl = np.float32(1.75)
    # the span of the logits that have a probability: the others' are exactly 0
    low = torch.finfo(dtype).min / 2
    rel = _p_err(torch.where(seen > low, seen, torch.full_like(seen, -float("inf"))))
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        d = bg.moe_route_backward(x.cuda(), r, dweights=dev(dw) if use_w else None,
                                  dloss=torch.tensor(float(dl), device="cuda") if use_l else None)
        ref, mag = routing.route_backward(q, k, normalize, dw if use_w else None, dl if use_l else None)
        # as for whole rows: three factors a term, sums over E and k, the output's half step
        tol = (3 * rel + U * (2 * e + 4 * k + 16)) * mag + torch.finfo(dtype).eps / 2 * np.abs(ref) + 2.0 ** -120
        bad = ~(np.abs(f64(d) - ref) <= tol)
        assert not bad.any(), f"{bad.sum()} off, first at {np.argwhere(bad)[0]}"
        assert (d[~dev(valid)] == 0).all() and (d[1] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_below_the_normal_range_keep_their_order(dtype):
    """Subnormal logits of both signs differ, and are chosen in their order."""
    t, e, k = 70, 40, 12
    step = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    g = synthetic._rng(81, 7)
    n = torch.from_numpy(np.stack([g.permutation(e) - e // 2 for _ in range(t)]))
    x = (n.double() * step).to(dtype)
    assert torch.equal(x.double(), n.double() * step)
    r = bg.moe_route(x.cuda(), k)
    want = torch.sort(n, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.cpu().long(), want)
