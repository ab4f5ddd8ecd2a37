"""Measured cases of the microscaled FP4 (MXFP4) operators and of the expert router.

Four operators, each through the calls a user makes:
  quantise   mxfp4_quantize, then mxfp4_dequantize (the fake quantisation of a
             tensor: its values after the trip through 4 bits, and its scales);
  linear     activations quantised per call, times weights held in MXFP4
             (mxfp4_quantize + gemm_mxfp4);
  experts    tokens gathered by expert while they are quantised, times every
             expert's weights (mxfp4_quantize with a row list +
             gemm_mxfp4_grouped);
  route      top-k routing with per-expert counts, the dispatch order and the
             balance loss (moe_route), and its gradient (moe_route_backward).

With `own` false the same results come from elementary torch operations in 32
bits. MXFP4 (OCP Microscaling Formats v1.0): 32 consecutive elements share the
scale 2^(s-127), s one E8M0 byte; the elements are E2M1.
"""
import numpy as np
import torch

own = False

BLOCK = 32          # elements under one scale
EMAX = 2            # exponent of the largest E2M1 binade (4 and 6)
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token's hidden vector
        {"name": "quantise one token", "kind": "quantise", "rows": 1, "k": 7168, "dtype": "bf16"},
        # the activations of an MLP's down projection at prefill
        {"name": "quantise prefill", "kind": "quantise", "rows": 5120, "k": 11008, "dtype": "bf16"},
        # one token through a projection: the weights' bytes are the time
        {"name": "linear one token", "kind": "linear", "rows": 1, "n": 4096, "k": 7168, "dtype": "bf16"},
        # a batch of 128 sequences in decode
        {"name": "linear decode batch", "kind": "linear", "rows": 128, "n": 7168, "k": 16384, "dtype": "bf16"},
        # a ragged prompt, an output width that no tile divides and a K that ends inside a step
        {"name": "linear ragged", "kind": "linear", "rows": 1015, "n": 12287, "k": 2080, "dtype": "f32"},
        # the gate projection of an MLP at prefill
        {"name": "linear gate", "kind": "linear", "rows": 5120, "n": 11008, "k": 2048, "dtype": "bf16"},
        # a square, deep product: the matrix cores are the time
        {"name": "linear deep", "kind": "linear", "rows": 4096, "n": 4096, "k": 8192, "dtype": "bf16"},
        # a small decode batch: most chosen experts see one token
        {"name": "experts decode", "kind": "experts", "tokens": 16, "experts": 256, "top": 8, "n": 2048, "k": 2048},
        # a prompt: about 140 tokens an expert, unevenly
        {"name": "experts prefill", "kind": "experts", "tokens": 4510, "experts": 256, "top": 8, "n": 1024, "k": 2048},
        # routing of a decode batch, from FP32 logits: latency
        {"name": "route decode", "kind": "route", "tokens": 16, "experts": 256, "top": 8, "dtype": "f32", "padded": False, "train": False},
        # routing of a padded prompt in training, with the gradient
        {"name": "route prompt", "kind": "route", "tokens": 4510, "experts": 256, "top": 8, "dtype": "bf16", "padded": True, "train": True},
        # a large training batch
        {"name": "route batch", "kind": "route", "tokens": 65536, "experts": 256, "top": 8, "dtype": "bf16", "padded": False, "train": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(("quantise", "linear", "linear", "experts", "route"))
    if kind == "quantise":
        k = BLOCK * _spread(rng, 1, 512)
        return {"kind": kind, "rows": _spread(rng, 1, min(65536, 5120 * 11008 // k)), "k": k, "dtype": rng.choice(("bf16", "f32"))}
    if kind == "linear":
        rows, k = _spread(rng, 1, 5120), BLOCK * _spread(rng, 2, 512)
        n = _spread(rng, 64, max(64, min(12288, 4096 * 4096 * 8192 // (rows * k))))
        return {"kind": kind, "rows": rows, "n": n, "k": k, "dtype": rng.choice(("bf16", "f32"))}
    if kind == "experts":
        e = _spread(rng, 8, 256)
        return {"kind": kind, "tokens": _spread(rng, 1, 4510), "experts": e, "top": rng.randint(1, 8), "n": _spread(rng, 64, 1024), "k": BLOCK * _spread(rng, 4, 64)}
    e = _spread(rng, 4, 512)
    return {"kind": kind, "tokens": _spread(rng, 1, 65536 * 256 // max(e, 256)), "experts": e, "top": rng.randint(1, min(8, e)), "dtype": rng.choice(("bf16", "f32")),
            "padded": rng.random() < 0.5, "train": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _quantised(x):
    """(E2M1 codes [.., K], E8M0 bytes [.., K/32]) of x: the shared exponent is
    that of the block's largest magnitude less EMAX, elements to the nearest
    E2M1 value (ties to the even code), at most 6."""
    v = x.float().unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 1 - EMAX, torch.full_like(top, -127, dtype=torch.int32)).clamp(-127, 127)
    y = torch.ldexp(v, -e)
    a = y.abs()
    # between codes c and c + 1 the border itself belongs to the even one
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    return (c + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)


def _packed(codes):
    """Two codes a byte, the even element in the low nibble."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpacked(packed):
    return torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


def _values(codes, scales, dtype=torch.float32):
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=dtype, device=codes.device)
    power = torch.exp2(scales.to(dtype) - 127)
    return (table[codes.int()].unflatten(-1, (-1, BLOCK)) * power.unsqueeze(-1)).flatten(-2)


def _plain_quantise(s):
    codes, scales = _quantised(s["x"])
    return {"values": _values(codes, scales).bfloat16(), "scales": scales}


def _plain_linear(s):
    a = _values(*_quantised(s["x"]))
    b = _values(_unpacked(s["w"]), s["sw"])
    return {"y": torch.matmul(a, b.t()).bfloat16()}


def _plain_experts(s):
    e, places = s["w"].shape[0], s["rows"].numel()
    first = s["offsets"].long()
    a = _values(*_quantised(s["x"][s["rows"].long()]))
    i = torch.arange(places, device=a.device)
    of = torch.searchsorted(first[1:].contiguous(), i, right=True)      # the expert of every place
    at = of * s["most"] + i - first[of]
    groups = torch.zeros(e * s["most"], a.shape[1], device=a.device)
    groups[at] = a
    b = _values(_unpacked(s["w"]), s["sw"]).transpose(1, 2).contiguous()
    y = torch.matmul(groups.view(e, s["most"], -1), b)
    return {"y": y.view(e * s["most"], -1)[at].bfloat16()}


def _plain_route(s):
    logits, k = s["logits"].float(), s["top"]
    t, e = logits.shape
    live = s["valid"] if s["valid"] is not None else torch.ones(t, dtype=torch.bool, device=logits.device)
    n = live.sum()
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]       # ties: lowest index
    chosen = torch.gather(p, 1, order)
    w = torch.where(live[:, None], chosen / chosen.sum(1, keepdim=True), torch.zeros_like(chosen))
    ids = torch.where(live[:, None], order, torch.full_like(order, -1))
    p = torch.where(live[:, None], p, torch.zeros_like(p))

    slot = torch.where(ids < 0, torch.full_like(ids, e), ids).flatten()                  # e: not dispatched
    counts = (torch.zeros(e + 1, dtype=torch.int64, device=p.device).index_add_(0, slot, torch.ones_like(slot)))[:e]
    offsets = torch.cat((torch.zeros_like(counts[:1]), counts.cumsum(0)))
    sorted_slot, by_expert = torch.sort(slot, stable=True)
    rows = torch.where(sorted_slot < e, by_expert // k, torch.full_like(by_expert, -1))
    pos = torch.empty_like(slot)
    pos[by_expert] = torch.arange(t * k, device=p.device)
    pos = torch.where(slot < e, pos, torch.full_like(pos, -1)).view(t, k)

    mean = (p.double().sum(0) / n).float()
    loss = (e / (k * n.double()) * (counts * p.double().sum(0) / n).sum()).float()
    out = {"ids": ids.int(), "weights": w, "counts": counts.int(), "offsets": offsets.int(), "rows": rows.int(), "pos": pos.int(), "mean_probs": mean, "loss": loss}
    if s["dloss"] is not None:
        c = s["dloss"] * e * counts.float() / (k * n.float() * n.float())
        d = p * (c - (p * c).sum(1, keepdim=True))
        dw = s["dweights"]
        d = d.scatter_add(1, order, torch.where(live[:, None], w * (dw - (w * dw).sum(1, keepdim=True)), torch.zeros_like(w)))
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    import block_scaled_fp4_gemm_amd as bg

    if s["kind"] == "quantise":
        codes, scales = bg.mxfp4_quantize(s["x"])
        return {"values": bg.mxfp4_dequantize(codes, scales), "scales": scales}
    if s["kind"] == "linear":
        codes, scales = bg.mxfp4_quantize(s["x"])
        return {"y": bg.gemm_mxfp4(codes, scales, s["w"], s["sw"])}
    if s["kind"] == "experts":
        codes, scales = bg.mxfp4_quantize(s["x"], rows=s["rows"])
        return {"y": bg.gemm_mxfp4_grouped(codes, scales, s["w"], s["sw"], s["offsets"])}
    r = bg.moe_route(s["logits"], s["top"], valid=s["valid"])
    out = {"ids": r.ids, "weights": r.weights, "counts": r.counts, "offsets": r.offsets, "rows": r.rows, "pos": r.pos, "mean_probs": r.mean_probs, "loss": r.loss}
    if s["dloss"] is not None:
        out["dlogits"] = bg.moe_route_backward(s["logits"], r, dweights=s["dweights"], dloss=s["dloss"])
    return out


PLAIN = {"quantise": _plain_quantise, "linear": _plain_linear, "experts": _plain_experts, "route": _plain_route}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["kind"]](state)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _activations(g, rows, k, dtype):
    """N(0, 1) with a few channels twenty times larger, as hidden states have them."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    x *= torch.where(torch.rand(k, generator=g, device="cuda") < 0.004, 20.0, 1.0)
    return x.bfloat16() if dtype == "bf16" else x


def _weights(g, n, k):
    """N(0, 0.02) weights held in MXFP4."""
    codes, scales = _quantised(torch.randn(n, k, generator=g, device="cuda") * 0.02)
    return _packed(codes), scales


def _logits(g, tokens, experts, dtype):
    """A router's outputs: a spread of about one, and a lean towards some experts."""
    x = torch.randn(tokens, experts, generator=g, device="cuda") + 0.5 * torch.randn(experts, generator=g, device="cuda")
    return x.bfloat16() if dtype == "bf16" else x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, s = case["kind"], {"kind": case["kind"]}
    if kind == "quantise":
        s["x"] = _activations(g, case["rows"], case["k"], case["dtype"])
    elif kind == "linear":
        s["x"] = _activations(g, case["rows"], case["k"], case["dtype"])
        s["w"], s["sw"] = _weights(g, case["n"], case["k"])
    elif kind == "experts":
        t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        s["x"] = _activations(g, t, k, "bf16")
        s["w"] = torch.empty(e, n, k // 2, dtype=torch.uint8, device="cuda")
        s["sw"] = torch.empty(e, n, k // BLOCK, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (n * k))
        for i in range(0, e, step):
            w, sw = _weights(g, n * min(step, e - i), k)
            s["w"][i:i + step] = w.view(-1, n, k // 2)
            s["sw"][i:i + step] = sw.view(-1, n, k // BLOCK)
        # the plan of this batch: every token's experts, and its places sorted by them
        ids = torch.topk(_logits(g, t, e, "f32"), case["top"], dim=1).indices.flatten()
        by_expert = torch.sort(ids, stable=True).indices
        counts = torch.bincount(ids, minlength=e)
        s["rows"] = (by_expert // case["top"]).int()
        s["offsets"] = torch.cat((torch.zeros_like(counts[:1]), counts.cumsum(0))).int()
        s["most"] = int(counts.max())
    else:
        t, e = case["tokens"], case["experts"]
        s["top"] = case["top"]
        s["logits"] = _logits(g, t, e, case["dtype"])
        # a padded batch: sequences that end at different places (the first row is never padding)
        ends = torch.randint(t // 2 + 1, t + 1, (1,), generator=g, device="cuda")
        s["valid"] = ((torch.arange(t, device="cuda") < ends) | (torch.rand(t, generator=g, device="cuda") < 0.25)) if case["padded"] else None
        s["dweights"] = torch.randn(t, case["top"], generator=g, device="cuda") if case["train"] else None
        s["dloss"] = torch.rand(1, generator=g, device="cuda") + 0.5 if case["train"] else None
    return s


def work(case):
    """What no form can do without: every input read once, every output written once."""
    kind = case["kind"]
    if kind == "route":
        t, e, k = case["tokens"], case["experts"], case["top"]
        size = 2 if case["dtype"] == "bf16" else 4
        nbytes = t * e * size + t * (1 if case["padded"] else 0) + t * k * 16 + e * 16
        if case["train"]:
            nbytes += t * e * size + t * k * 4
        return {"bytes": nbytes, "flops": t * e * (10 if case["train"] else 4)}
    k = case["k"]
    if kind == "quantise":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["rows"] * (k * size + k * 2 + k // BLOCK), "flops": 3 * case["rows"] * k}
    held = k // 2 + k // BLOCK
    if kind == "linear":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["rows"] * k * size + case["n"] * held + 2 * case["rows"] * case["n"], "flops": 2 * case["rows"] * case["n"] * k}
    places = case["tokens"] * case["top"]
    # the experts that evenly drawn tokens reach
    reached = case["experts"] * (1 - (1 - case["top"] / case["experts"]) ** case["tokens"]) if case["top"] < case["experts"] else case["experts"]
    return {"bytes": int(case["tokens"] * k * 2 + reached * case["n"] * held + places * (4 + 2 * case["n"])), "flops": 2 * places * case["n"] * k}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_values(x):
    """x in MXFP4, as FP64 values, and the E8M0 bytes. Each element is rounded
    on the grid of its own binade (steps of 1/2 below 2, 1 below 4, 2 above)."""
    x = x.double()
    rows, k = x.shape
    x = x.reshape(rows * k // BLOCK, BLOCK)
    top = x.abs().max(1, keepdim=True).values
    e = torch.floor(torch.log2(top))
    e = torch.where(torch.exp2(e) > top, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)
    e = torch.where(top == 0, torch.full_like(e, -127.0), e - 2).clamp(-127, 127)
    unit = torch.exp2(e)
    m = x.abs() / unit
    step = 0.5 * (1 + (m >= 2).double() + 2 * (m >= 4).double())
    q = torch.minimum(torch.round(m / step) * step, torch.full_like(m, 6.0))        # round: half to even
    return (torch.sign(x) * q * unit).reshape(rows, k), (e.reshape(rows, k // BLOCK) + 127).to(torch.uint8)


def _exact_weights(packed, scales):
    n, half = packed.shape
    nib = torch.empty(n, half, 2, dtype=torch.uint8, device=packed.device)
    nib[..., 0], nib[..., 1] = packed % 16, packed // 16
    nib = nib.reshape(n, 2 * half).double()
    sign, c = 1 - 2 * (nib >= 8).double(), nib % 8
    exp, man = torch.floor(c / 2), c % 2
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * torch.exp2(exp - 1))
    return sign * mag * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantise":
        v, scales = _exact_values(s["x"])
        return {"values": v, "scales": scales}
    if kind == "linear":
        return {"y": _exact_values(s["x"])[0] @ _exact_weights(s["w"], s["sw"]).t()}
    if kind == "experts":
        first, rows = s["offsets"].tolist(), s["rows"].long()
        y = torch.empty(rows.numel(), case["n"], dtype=torch.float64, device="cuda")
        x = _exact_values(s["x"])[0]
        for e in range(case["experts"]):
            lo, hi = first[e], first[e + 1]
            if hi > lo:
                y[lo:hi] = x[rows[lo:hi]] @ _exact_weights(s["w"][e], s["sw"][e]).t()
        return {"y": y}
    # route: in numpy
    x = s["logits"].double().cpu().numpy()
    t, e = x.shape
    k = case["top"]
    live = s["valid"].cpu().numpy() if s["valid"] is not None else np.ones(t, bool)
    n = int(live.sum())
    z = np.exp(x - x.max(1, keepdims=True))
    p = z / z.sum(1, keepdims=True)
    best = np.argsort(-x, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, best, 1)
    w = w / w.sum(1, keepdims=True)
    best[~live], w[~live], p[~live] = -1, 0, 0
    hot = [np.nonzero((best == i).any(1))[0] for i in range(e)]        # the tokens of every expert, in order
    counts = np.array([len(h) for h in hot])
    offsets = np.concatenate(([0], np.cumsum(counts)))
    rows, pos = np.full(t * k, -1), np.full((t, k), -1)
    rows[: offsets[-1]] = np.concatenate(hot)
    for i, h in enumerate(hot):
        pos[h, (best[h] == i).argmax(1)] = offsets[i] + np.arange(len(h))
    mean = p.sum(0) / n
    out = {"ids": best.astype(np.int32), "weights": w, "counts": counts.astype(np.int32), "offsets": offsets.astype(np.int32), "rows": rows.astype(np.int32),
           "pos": pos.astype(np.int32), "mean_probs": mean, "loss": np.float64(e * (counts / (k * n) * mean).sum())}
    if s["dloss"] is not None:
        c = float(s["dloss"].double()) * e / k * counts / n / n
        dw = s["dweights"].double().cpu().numpy()
        d = p * c - p * (p @ c)[:, None]
        inner = (w * dw).sum(1)
        i = np.nonzero(live)[0]
        for j in range(k):
            d[i, best[i, j]] += w[i, j] * (dw[i, j] - inner[i])
        out["dlogits"] = d
    return out
