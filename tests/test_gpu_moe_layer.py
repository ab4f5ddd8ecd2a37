"""The operators together, as a mixture-of-experts layer uses them: router
GEMM, routing, gather and quantisation, the experts' products, and the rows
brought back to their tokens."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_gemm_amd as bg
import oracle
import synthetic
from gpu_util import to_dev_bf16
from mx_util import U, dev, f64
from oracle import routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,e,k,d,n", [(1, 16, 4, 256, 200), (40, 16, 4, 512, 300), (200, 8, 2, 544, 130)])
def test_expert_layer(t, e, k, d, n):
    x = synthetic.normal_bf16((t, d), 1.0, 61, 0)
    wr = synthetic.normal_bf16((e, d), 0.05, 61, 1)
    we = synthetic.normal_bf16((e * n, d), 0.05, 61, 2)
    valid = np.ones(t, bool)
    valid[t // 2 + 1:t // 2 + 9] = False

    xd = to_dev_bf16(x)
    logits = bg.gemm_bf16_ordered_f32(xd, to_dev_bf16(wr))
    r = bg.moe_route(logits, k, valid=dev(valid))
    wq, ws = bg.mxfp4_quantize(to_dev_bf16(we))
    a, sa = bg.mxfp4_quantize(xd, rows=r.rows)
    y = bg.gemm_mxfp4_grouped(a, sa, wq.view(e, n, -1), ws.view(e, n, -1), r.offsets)
    place = r.pos.long()
    chosen = torch.where((place >= 0)[..., None], y[place.clamp(min=0)].float(), 0.0)
    out = (chosen * r.weights[..., None]).sum(1)

    # the same, from the oracle
    q = routing.route(f64(logits), k, valid)
    assert np.array_equal(r.ids.cpu().numpy(), q["ids"]) and np.array_equal(r.rows.cpu().numpy(), q["rows"])
    xv = oracle.dequant_mxfp4(*oracle.quantize_mxfp4(oracle.bf16_to_f64(x)))
    wv = oracle.dequant_mxfp4(*oracle.quantize_mxfp4(oracle.bf16_to_f64(we))).reshape(e, n, d)
    want, size = np.zeros((t, n)), np.zeros((t, n))
    for i in range(t):
        for j in range(k):
            if q["ids"][i, j] >= 0:
                want[i] += q["weights"][i, j] * (wv[q["ids"][i, j]] @ xv[i])
                size[i] += q["weights"][i, j] * (np.abs(wv[q["ids"][i, j]]) @ np.abs(xv[i]))
    # BF16 rounding of each expert's row (2^-8 of it, at most of size), the sums in FP32, the weights
    tol = (2.0 ** -8 + 2 * (d + 1) * U + U * (e + k + 80)) * size
    assert (np.abs(f64(out) - want) <= tol).all()
    assert (out[~dev(valid)] == 0).all()
    # the gradient reaches the logits of live rows only
    g = bg.moe_route_backward(logits, r, dloss=torch.ones((), device="cuda"))
    assert (g[~dev(valid)] == 0).all() and torch.isfinite(g).all()
    assert (g.double().sum(1).abs() <= 1e-6).all()          # softmax gradients of a row add up to zero
    # a row at a time gives the row of the batch
    one = bg.mxfp4_quantize(xd[:1])
    assert torch.equal(one[0][0], a[int(r.pos[0, 0])])


def test_quantised_linear_close_to_the_unquantised_product():
    """gemm_mxfp4 of quantised operands against the FP64 product of the same
    quantised values, through mxfp4_dequantize and gemm_bf16 (exact operands
    in BF16): the two agree to their summation orders."""
    m, n, k = 77, 190, 1056
    x, w = to_dev_bf16(synthetic.normal_bf16((m, k), 1.0, 62, 0)), to_dev_bf16(synthetic.normal_bf16((n, k), 0.05, 62, 1))
    a, sa = bg.mxfp4_quantize(x)
    b, sb = bg.mxfp4_quantize(w)
    got = bg.gemm_mxfp4(a, sa, b, sb)
    av, bv = bg.mxfp4_dequantize(a, sa), bg.mxfp4_dequantize(b, sb)
    dense = bg.gemm_bf16(av, bv)
    size = f64(av.abs()) @ f64(bv.abs()).T
    ref = f64(av) @ f64(bv).T
    tol = 2.0 ** -7 * np.abs(ref) + 4 * (k + 1) * U * size
    assert (np.abs(f64(got) - f64(dense)) <= tol).all()


@pytest.mark.parametrize("t", [1, 200])
def test_layer_captured_and_replayed(t):
    """The whole chain in one graph, replayed over changing inputs with eager
    calls between, gives the eager bits; places behind the last keep what the
    output held."""
    e, k, d, n = 16, 4, 512, 264
    w, ws = bg.mxfp4_quantize(torch.randn(e * n, d, device="cuda").bfloat16())
    w, ws = w.view(e, n, -1), ws.view(e, n, -1)
    router = torch.randn(e, d, device="cuda").bfloat16()
    x, valid = torch.empty(t, d, device="cuda", dtype=torch.bfloat16), torch.empty(t, device="cuda", dtype=torch.bool)
    y = torch.empty(t * k, n, device="cuda", dtype=torch.bfloat16)
    dw, dl = torch.randn(t, k, device="cuda"), torch.tensor(0.3, device="cuda")

    def layer():
        logits = bg.gemm_bf16_ordered_f32(x, router)
        r = bg.moe_route(logits, k, valid=valid)
        a, sa = bg.mxfp4_quantize(x, rows=r.rows)
        bg.gemm_mxfp4_grouped(a, sa, w, ws, r.offsets, out=y)
        return *r[:9], a, sa, bg.moe_route_backward(logits, r, dw, dl)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(t, d, device="cuda", generator=g))
        valid.copy_(torch.rand(t, device="cuda", generator=g) < (0.7 if seed % 2 else 2.0))
        y.fill_(5.0)

    fill(0)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for seed in range(5):
        fill(seed)
        want = [v.clone() for v in (*layer(), y)]
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*held, y), want)), seed
        assert (y[int(held[3][-1]):] == 5.0).all()
