"""GPU parity of expert routing, its balance loss and its gradient."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
import synthetic
from mx_util import U, dev, f64
from oracle import routing

pytestmark = pytest.mark.gpu

WHOLE = ("ids", "counts", "offsets", "rows", "pos")


def _logits(t, e, dtype, seed, spread=1.5):
    g = synthetic._rng(seed, 9)
    x = g.standard_normal((t, e)) * spread + 0.5 * g.standard_normal(e)
    return torch.from_numpy(x).to(dtype)


def _span(x):
    """The largest |logit - row maximum| of the finite logits."""
    v = x.double().numpy()
    v = np.where(np.isfinite(v), v, np.nan)
    if not np.isfinite(v).any():
        return 0.0
    return float(np.nanmax(v) - np.nanmin(v))


def _p_err(x):
    """Relative error of a probability: the difference of two logits rounds
    once (2^-24 of at most the span) and its product with log2 e once more,
    both in the exponent; the exponential is off by two steps of 2^-23, the
    sum of E of them by E roundings, the quotient by three."""
    return U * (x.shape[1] + 2 * _span(x) + 16)


def _check(x, k, got, valid=None, normalize=True, what=""):
    """got: moe_route's answer for logits x (a CPU tensor)."""
    r = routing.route(x.double().numpy(), k, valid, normalize)
    for f in WHOLE:
        assert np.array_equal(getattr(got, f).cpu().numpy(), r[f]), f"{what}: {f}"
    assert int(got.n_valid) == r["n_valid"], what
    rel = _p_err(x)
    # FP32 flushes what lies below its normal range: 2^-126 of slack
    for f, extra in (("weights", 2 * U * k), ("mean_probs", U * (x.shape[0] + 2)), ("loss", U * (x.shape[0] + 2 * x.shape[1] + 8))):
        w, g = np.asarray(r[f]), f64(getattr(got, f))
        # a mean takes every row's absolute error: the flushed parts of rows too
        assert (np.abs(g - w) <= (2 * rel + extra) * np.abs(w) + 2.0 ** -120).all(), f"{what}: {f}"
    return r


SIZES = [(1, 1, 1), (1, 4, 2), (3, 5, 5), (16, 256, 8), (17, 256, 8), (31, 64, 6), (32, 128, 4), (33, 8, 2), (50, 65, 3), (100, 160, 6), (257, 16, 16),
         (300, 257, 7), (70, 512, 8), (40, 513, 10), (1000, 256, 8), (90, 1000, 16), (64, 1024, 16), (2255, 60, 1), (20000, 24, 4),
         (64, 300, 5), (65, 33, 4), (16385, 100, 3), (17000, 256, 8), (600, 1024, 9), (700, 470, 3), (100, 6, 2), (3000, 1022, 9), (90, 2, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,e,k", SIZES)
def test_route(t, e, k, dtype):
    print(f"route {t}x{e} k={k} {dtype}", flush=True)
    x = _logits(t, e, dtype, t + e)
    _check(x, k, bg.moe_route(x.cuda(), k), what="all rows")
    valid = synthetic._rng(t, 3).random(t) < 0.7
    got = bg.moe_route(x.cuda(), k, valid=dev(valid), normalize=False)
    _check(x, k, got, valid, False, "masked")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,e,k", [(5, 8, 3), (40, 64, 8), (700, 256, 8), (60, 600, 16)])
def test_ties_go_to_the_lowest_index(t, e, k, dtype):
    g = synthetic._rng(t, 4)
    x = torch.from_numpy(g.integers(-2, 3, (t, e)).astype(np.float64)).to(dtype)
    x[g.integers(0, t)] = 0.0
    x[0, ::2] = -0.0                        # equal to +0
    _check(x, k, bg.moe_route(x.cuda(), k), what="ties")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t", [20, 333])
def test_masked_logits_and_empty_rows(t, dtype):
    """Experts masked by -infinity or by the type's lowest value, rows with
    fewer than k choices, rows with none, masked rows full of NaN."""
    e, k = 96, 6
    x = _logits(t, e, dtype, 21)
    g = synthetic._rng(21, 5)
    x[torch.from_numpy(g.random((t, e)) < 0.5)] = -float("inf")
    x[1] = -float("inf")
    x[2, 1:] = -float("inf")
    x[3, 4:] = -float("inf")
    x[4, 3:] = torch.finfo(dtype).min       # finite: may be chosen, with weight 0
    x[4, :3] = torch.tensor([1.0, 2.0, 3.0], dtype=dtype)
    x[5] = torch.finfo(dtype).min
    valid = np.ones(t, bool)
    valid[[0, 7]] = False
    x[7] = float("nan")
    seen = x.clone()
    seen[7] = 0.0                           # what the oracle reads of a masked row
    got = bg.moe_route(x.cuda(), k, valid=dev(valid))
    r = routing.route(seen.double().numpy(), k, valid)
    for f in WHOLE:
        assert np.array_equal(getattr(got, f).cpu().numpy(), r[f]), f
    assert int(got.n_valid) == r["n_valid"]
    tol = 2 * U * (e + 2 * 20 + 16 + t)     # the masked values' exponentials are exactly 0
    for f in ("weights", "mean_probs", "loss"):
        assert (np.abs(f64(getattr(got, f)) - r[f]) <= tol * np.abs(r[f]) + 2.0 ** -120).all(), f
    none = bg.moe_route(x.cuda(), k, valid=torch.zeros(t, dtype=torch.bool, device="cuda"))
    assert (none.ids == -1).all() and (none.rows == -1).all() and (none.pos == -1).all() and not none.counts.any()
    assert float(none.loss) == 0 and not none.mean_probs.any() and int(none.n_valid) == 0
    d = bg.moe_route_backward(x.cuda(), none, dloss=torch.ones((), device="cuda"), dweights=torch.ones(t, k, device="cuda"))
    assert (d == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("normalize", [True, False])
def test_nan_and_infinite_logits_keep_the_choices_valid(dtype, normalize):
    t, e, k = 40, 20, 4
    x = _logits(t, e, dtype, 22)
    x[3, 5] = float("nan")
    x[9, 2] = float("inf")
    x[11] = float("nan")                    # nothing to choose: not live
    r = bg.moe_route(x.cuda(), k, normalize=normalize)
    want = routing.route(x.double().numpy(), k, None, normalize)
    for f in WHOLE:
        assert np.array_equal(getattr(r, f).cpu().numpy(), want[f]), f
    w = r.weights.cpu()
    assert torch.isnan(w[[3, 9]]).all() and torch.isnan(r.loss).item()
    keep = [i for i in range(t) if i not in (3, 9)]
    assert torch.isfinite(w[keep]).all() and (w[11] == 0).all()


def test_empty_batch():
    r = bg.moe_route(torch.zeros(0, 8, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and r.rows.numel() == 0 and not r.counts.any() and not r.offsets.any()
    assert float(r.loss) == 0 and int(r.n_valid) == 0
    assert bg.moe_route_backward(torch.zeros(0, 8, device="cuda"), r).shape == (0, 8)


def _check_backward(x, k, valid, normalize, use, in_place=False):
    g = synthetic._rng(31, 6)
    t, e = x.shape
    dw = g.standard_normal((t, k)).astype(np.float32) if "w" in use else None
    dl = np.float32(1.25) if "l" in use else None
    xd = x.cuda()
    r = bg.moe_route(xd, k, valid=None if valid is None else dev(valid), normalize=normalize)
    d = bg.moe_route_backward(xd, r, dweights=None if dw is None else dev(dw), dloss=None if dl is None else torch.tensor(1.25, device="cuda"),
                              out=xd if in_place else None)
    ref, mag = routing.route_backward(routing.route(x.double().numpy(), k, valid, normalize), k, normalize, dw, dl)
    # every term's factors (p, w: _p_err; sums over E and k; counts, scale) and the output's half step
    tol = (3 * _p_err(x) + U * (2 * e + 4 * k + 16)) * mag + torch.finfo(x.dtype).eps / 2 * np.abs(ref) + 2.0 ** -120
    bad = ~(np.abs(f64(d) - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} off, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (5, 7, 3), (40, 64, 8), (33, 100, 1), (130, 256, 8), (50, 500, 6), (20, 1024, 16), (5000, 60, 4)])
def test_backward(t, e, k, normalize, dtype):
    print(f"route backward {t}x{e} k={k} {dtype}", flush=True)
    x = _logits(t, e, dtype, 3 * t + e)
    valid = synthetic._rng(t, 8).random(t) < 0.8
    valid[0] = True
    _check_backward(x, k, valid, normalize, "wl")
    _check_backward(x, k, None, normalize, "l")
    _check_backward(x, k, None, normalize, "w", in_place=True)


def test_backward_against_differences():
    """FP32 gradient against central differences of the kernel's own forward.
    With step h the difference is off by the forward's error over h (2^-24 of
    the value, times the number of summed terms) and by h^2."""
    t, e, k, h = 24, 16, 3, 2.0 ** -6
    x = _logits(t, e, torch.float32, 41).cuda()
    dw = torch.randn(t, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    r = bg.moe_route(x, k)
    d = bg.moe_route_backward(x, r, dweights=dw, dloss=torch.tensor(2.0, device="cuda"))

    def value(y):
        q = bg.moe_route(y, k)
        return q, (q.weights.double() * dw.double()).sum() + 2.0 * q.loss.double()

    tried = 0
    for i, f in [(0, 0), (1, 5), (7, 15), (13, 2), (23, 8), (10, 10)]:
        up, down = x.clone(), x.clone()
        up[i, f] += h
        down[i, f] -= h
        (qu, vu), (qd, vd) = value(up), value(down)
        if not (torch.equal(qu.ids, r.ids) and torch.equal(qd.ids, r.ids)):
            continue                        # another choice: no derivative there
        tried += 1
        assert abs(float((vu - vd) / (2 * h)) - float(d[i, f])) < 2e-3
    assert tried >= 3


def test_two_graphs_streams_and_repeats_give_the_same_bits():
    x1, x2 = _logits(3000, 128, torch.bfloat16, 51).cuda(), _logits(3000, 128, torch.bfloat16, 52).cuda()
    dw, dl = torch.randn(3000, 4, device="cuda"), torch.tensor(0.5, device="cuda")

    def step(x, stream=None):
        r = bg.moe_route(x, 4, stream=stream)
        return list(r[:9]) + [bg.moe_route_backward(x, r, dw, dl, stream=stream)]

    want = [[v.clone() for v in step(x)] for x in (x1, x2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (x1, x2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        step(x2)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [step(x, st) for x, st in zip((x1, x2), s)]
        torch.cuda.synchronize()
        for o, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_large_batch_counts_and_places():
    """A batch past 2^24 choices: whole numbers checked against torch."""
    t, e, k = 2200000, 32, 8
    x = torch.randn(t, e, device="cuda").bfloat16()
    r = bg.moe_route(x, k)
    ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids.long(), ids)
    assert torch.equal(r.counts.long(), torch.bincount(ids.flatten(), minlength=e))
    by = torch.sort(ids.flatten(), stable=True).indices
    assert torch.equal(r.rows.long(), by // k)
    assert torch.equal(r.pos.flatten().long()[by], torch.arange(t * k, device="cuda"))
    p = torch.softmax(x.double(), 1).mean(0)
    assert ((r.mean_probs.double() - p).abs() <= 2.0 ** -24 * (e + 2 * 20 + 16 + 300) * p).all()


def test_more_rows_than_256_workgroups_count():
    """Workgroups count at most 65472 rows each (16 bits): a batch of 260 of
    them, an odd number of experts, a mask that starts at an odd address."""
    t, e = 17000000, 3
    x = torch.randn(t, e, device="cuda").bfloat16()
    valid = (torch.rand(t + 1, device="cuda") < 0.9)[1:]
    r = bg.moe_route(x, 1, valid=valid)
    ids = torch.where(valid, torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, 0], -1)
    assert torch.equal(r.ids[:, 0].long(), ids)
    live = valid.nonzero().flatten()
    by = live[torch.sort(ids[live], stable=True).indices]
    n = int(by.numel())
    assert int(r.n_valid) == n
    assert torch.equal(r.counts.long(), torch.bincount(ids[live], minlength=e))
    assert torch.equal(r.rows[:n].long(), by) and (r.rows[n:] == -1).all()
    assert torch.equal(r.pos[by, 0].long(), torch.arange(n, device="cuda")) and (r.pos[~valid] == -1).all()
    p = torch.softmax(x[valid].double(), 1).mean(0)
    # 65472 rows of a workgroup 64 at a time: 1023 additions in a lane, 4 over lanes, 16 over waves, 260 over workgroups
    assert ((r.mean_probs.double() - p).abs() <= 2.0 ** -24 * (e + 2 * 12 + 16 + 1400) * p).all()
    d = bg.moe_route_backward(x, r, dloss=torch.tensor(1e6, device="cuda"))
    assert (d[~valid] == 0).all()
    c = 1e6 * e * r.counts.double() / float(n) ** 2
    at = torch.cat((live[:1000], live[-1000:]))
    pr = torch.softmax(x[at].double(), 1)
    want = pr * (c - (pr * c).sum(1, keepdim=True))
    size = pr * (c + (pr * c).sum(1, keepdim=True))
    assert ((d[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -24 * 3 * (e + 2 * 12 + 32) * size).all()
