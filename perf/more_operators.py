"""Measured cases of the gated MLP block: its training step in BF16, and single
tokens through weights held in 4 bits.

Five kinds of case, each through the calls a user makes:
  gated       h = act(x W0^T) * (x W1^T), the block's forward pass at prefill
              (gemm_bf16_gated);
  train       the same with what the gradient needs kept, then the gradient
              (gemm_bf16_gated, gemm_bf16_gated_backward);
  gradient    a projection's gradients, dx = dy W and dW = dy^T x
              (gemm_bf16_nn, gemm_bf16_tn);
  gemv        few rows times weights in 4 bits with group scales (gemv_w4);
  gated gemv  the gated block of few rows with weights in 4 bits
              (gemv_w4_gated).

With `own` false the same results come from elementary torch operations in 32
bits. Weights in 4 bits are packed two a byte, the even element in the low
nibble:
  int4   s * (q - z), s BF16 and z a byte for every `group` elements of a row
         (z = 8 where there are no zero points);
  mxfp4  E2M1 times 2^(s - 127), s a byte for 32 elements;
  nvfp4  E2M1 times s, s E4M3 for 16 elements, times one FP32 scale.
"""
import math

import torch

own = False

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = {"mxfp4": 32, "nvfp4": 16}


def listed():
    return [
        # the gate and up projections of an MLP at prefill
        {"name": "gated prefill", "kind": "gated", "m": 5120, "n": 11008, "k": 2048, "act": "silu"},
        # a ragged prompt, a width that no tile divides, a K that ends inside a step
        {"name": "gated ragged", "kind": "gated", "m": 1015, "n": 5461, "k": 2088, "act": "gelu_tanh"},
        # a decode batch, BF16 weights: their bytes are the time
        {"name": "gated decode batch", "kind": "gated", "m": 64, "n": 11008, "k": 2048, "act": "silu"},
        # the training step of the MLP's first half
        {"name": "train step", "kind": "train", "m": 5120, "n": 11008, "k": 2048, "act": "silu"},
        # the same of a small model on a ragged batch
        {"name": "train small", "kind": "train", "m": 1015, "n": 1407, "k": 520, "act": "gelu_tanh"},
        # the down projection's gradients
        {"name": "gradient down", "kind": "gradient", "m": 5120, "n": 2048, "k": 11008},
        # the key and value projections' gradients: few output tiles, a long sum over tokens
        {"name": "gradient narrow", "kind": "gradient", "m": 5120, "n": 512, "k": 2048},
        # one token through a projection
        {"name": "gemv one token", "kind": "gemv", "rows": 1, "n": 4096, "k": 7168, "format": "int4", "group": 128, "zeros": True},
        # a decode batch through a large projection
        {"name": "gemv batch", "kind": "gemv", "rows": 16, "n": 7168, "k": 16384, "format": "nvfp4", "group": 16, "zeros": False},
        # three drafted tokens, an odd width and a K of an odd number of blocks
        {"name": "gemv ragged", "kind": "gemv", "rows": 3, "n": 12287, "k": 2080, "format": "mxfp4", "group": 32, "zeros": False},
        # one token through the gated block
        {"name": "gated gemv one token", "kind": "gated gemv", "rows": 1, "n": 11008, "k": 2048, "format": "int4", "group": 64, "zeros": False, "act": "silu"},
        # a small batch through the gated block
        {"name": "gated gemv batch", "kind": "gated gemv", "rows": 8, "n": 11008, "k": 4096, "format": "mxfp4", "group": 32, "zeros": False, "act": "gelu_tanh"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(("gated", "gated", "train", "gradient", "gemv", "gemv", "gated gemv"))
    if kind in ("gated", "train"):
        return {"kind": kind, "m": _spread(rng, 1, 5120), "n": _spread(rng, 64, 11008), "k": 8 * _spread(rng, 8, 256),
                "act": rng.choice(("silu", "gelu_tanh"))}
    if kind == "gradient":
        return {"kind": kind, "m": _spread(rng, 16, 5120), "n": 8 * _spread(rng, 8, 1376), "k": 8 * _spread(rng, 8, 256)}
    form = rng.choice(("int4", "mxfp4", "nvfp4"))
    group = GROUP.get(form) or rng.choice((32, 64, 128))
    k = _spread(rng, 256, 16384) // max(group, 32) * max(group, 32)
    case = {"kind": kind, "rows": rng.choice((1, 1, rng.randint(1, 16))), "n": _spread(rng, 64, min(12288, 7168 * 16384 // (2 * k))), "k": k,
            "format": form, "group": group, "zeros": form == "int4" and rng.random() < 0.5}
    if kind == "gated gemv":
        case["act"] = rng.choice(("silu", "gelu_tanh"))
    return case


# ---------------------------------------------------------------------------
# Plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _sigmoid_and_slope(g, act):
    """(s, z') of act(g) = g s(z(g))."""
    if act == "silu":
        return 1 / (1 + torch.exp(-g)), torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return 1 / (1 + torch.exp(-c * (g + 0.044715 * g * g * g))), c * (1 + 3 * 0.044715 * g * g)


def _plain_gated(s):
    x, w0, w1 = s["x"].float(), s["w0"].float(), s["w1"].float()
    g, u = x @ w0.t(), x @ w1.t()
    sig, slope = _sigmoid_and_slope(g, s["act"])
    out = {"h": (g * sig * u).bfloat16()}
    if s["kind"] == "train":
        dh = s["dh"].float()
        du = dh * (g * sig)
        dg = dh * u * (sig + g * slope * sig * (1 - sig))
        out["dx"] = (dg @ w0 + du @ w1).bfloat16()
        out["dw0"] = (dg.t() @ x).bfloat16()
        out["dw1"] = (du.t() @ x).bfloat16()
    return out


def _plain_gradient(s):
    dy = s["dy"].float()
    return {"dx": (dy @ s["w"].float()).bfloat16(), "dw": (dy.t() @ s["x"].float()).bfloat16()}


def _plain_weights(w):
    """The values [N, K] of weights in 4 bits."""
    q = torch.stack((w["codes"] & 15, w["codes"] >> 4), -1).flatten(-2)
    q = q.unflatten(-1, (-1, w["group"]))
    if w["format"] == "int4":
        z = w["zeros"].float().unsqueeze(-1) if w["zeros"] is not None else 8.0
        return ((q.float() - z) * w["scales"].float().unsqueeze(-1)).flatten(-2)
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=q.device)
    scale = torch.exp2(w["scales"].float() - 127) if w["format"] == "mxfp4" else w["scales"].view(torch.float8_e4m3fn).float() * w["scale_2"]
    return (table[q.int()] * scale.unsqueeze(-1)).flatten(-2)


def _plain_gemv(s):
    x = s["x"].float()
    y = [x @ _plain_weights(w).t() for w in s["weights"]]
    if s["kind"] == "gemv":
        return {"y": y[0].bfloat16()}
    return {"h": (y[0] * _sigmoid_and_slope(y[0], s["act"])[0] * y[1]).bfloat16()}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    import block_scaled_fp4_gemm_amd as bg

    kind = s["kind"]
    if kind == "gated":
        return {"h": bg.gemm_bf16_gated(s["x"], s["w0"], s["w1"], act=s["act"])}
    if kind == "train":
        h, g, u = bg.gemm_bf16_gated(s["x"], s["w0"], s["w1"], act=s["act"], save=True)
        dx, dw0, dw1 = bg.gemm_bf16_gated_backward(s["dh"], s["x"], s["w0"], s["w1"], g, u, act=s["act"])
        return {"h": h, "dx": dx, "dw0": dw0, "dw1": dw1}
    if kind == "gradient":
        return {"dx": bg.gemm_bf16_nn(s["dy"], s["w"]), "dw": bg.gemm_bf16_tn(s["dy"], s["x"])}
    held = [bg.W4Weights(w["codes"], w["scales"], w["format"], group=w["group"], zeros=w["zeros"], scale_2=w["scale_2"]) for w in s["weights"]]
    if kind == "gemv":
        return {"y": bg.gemv_w4(s["x"], held[0])}
    return {"h": bg.gemv_w4_gated(s["x"], held[0], held[1], act=s["act"])}


PLAIN = {"gated": _plain_gated, "train": _plain_gated, "gradient": _plain_gradient, "gemv": _plain_gemv, "gated gemv": _plain_gemv}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["kind"]](state)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _activations(g, rows, k):
    """N(0, 1) with a few channels ten times larger, as hidden states have them."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    x *= torch.where(torch.rand(k, generator=g, device="cuda") < 0.004, 10.0, 1.0)
    return x.bfloat16()


def _matrix(g, n, k, size):
    return (torch.randn(n, k, generator=g, device="cuda") * size).bfloat16()


def _codes(v):
    """E2M1 codes of values already divided by their scale."""
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    return c + 8 * torch.signbit(v).to(torch.uint8)


def _quantised(g, n, k, form, group, zeros):
    """A layer's weights, N(0, 0.02), in 4 bits."""
    codes, scales, points = [], [], []
    step = max(1, (1 << 25) // k)
    for i in range(0, n, step):
        v = (torch.randn(min(step, n - i), k, generator=g, device="cuda") * 0.02).unflatten(-1, (-1, group))
        if form == "int4":
            if zeros:
                lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
                s = ((hi - lo) / 15).bfloat16()
                z = torch.round(-lo / s.float()).clamp(0, 15)
                points.append(z.squeeze(-1).to(torch.uint8))
            else:
                s, z = (v.abs().amax(-1, keepdim=True) / 7).bfloat16(), 8.0
            q = torch.round(v / s.float() + z).clamp(0, 15).to(torch.uint8)
            scales.append(s.squeeze(-1))
        else:
            top = v.abs().amax(-1, keepdim=True)
            if form == "mxfp4":
                e = (torch.floor(torch.log2(top)) - 2).clamp(-127, 127)
                s = torch.exp2(e)
                scales.append((e.squeeze(-1) + 127).to(torch.uint8))
            else:
                held = (top / (6 * 2.0 ** -10)).to(torch.float8_e4m3fn)
                s = held.float() * 2.0 ** -10
                scales.append(held.squeeze(-1).view(torch.uint8))
            q = _codes(v / s)
        q = q.flatten(-2)
        codes.append(q[..., 0::2] | (q[..., 1::2] << 4))
    return {"codes": torch.cat(codes), "scales": torch.cat(scales), "format": form, "group": group,
            "zeros": torch.cat(points) if points else None, "scale_2": 2.0 ** -10 if form == "nvfp4" else 1.0}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]
    s = {"kind": kind, "act": case.get("act")}
    if kind in ("gated", "train"):
        m, n, k = case["m"], case["n"], case["k"]
        s["x"], s["w0"], s["w1"] = _activations(g, m, k), _matrix(g, n, k, 0.02), _matrix(g, n, k, 0.02)
        if kind == "train":
            s["dh"] = _matrix(g, m, n, 1e-2)
    elif kind == "gradient":
        m, n, k = case["m"], case["n"], case["k"]
        s["dy"], s["w"], s["x"] = _matrix(g, m, n, 1e-2), _matrix(g, n, k, 0.02), _activations(g, m, k)
    else:
        s["x"] = _activations(g, case["rows"], case["k"])
        s["weights"] = [_quantised(g, case["n"], case["k"], case["format"], case["group"], case["zeros"]) for _ in range(2 if kind == "gated gemv" else 1)]
    return s


def work(case):
    """What no form can do without: every input read once, every output written once."""
    kind = case["kind"]
    if kind in ("gated", "train", "gradient"):
        m, n, k = case["m"], case["n"], case["k"]
        if kind == "gradient":
            return {"bytes": 2 * (m * n + 2 * n * k + 2 * m * k), "flops": 4 * m * n * k}
        if kind == "gated":
            return {"bytes": 2 * (m * k + 2 * n * k + m * n), "flops": 4 * m * n * k}
        return {"bytes": 2 * (2 * m * k + 4 * n * k + 2 * m * n), "flops": 12 * m * n * k}
    rows, n, k, group = case["rows"], case["n"], case["k"], case["group"]
    held = n * k // 2 + n * (k // group) * ((2 if case["format"] == "int4" else 1) + (1 if case["zeros"] else 0))
    count = 2 if kind == "gated gemv" else 1
    return {"bytes": count * held + 2 * rows * (n + k), "flops": count * 2 * rows * n * k}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        z, dz = g, torch.ones_like(g)
        a = g * torch.sigmoid(z)
        return a, torch.sigmoid(z) * (1 + g * torch.sigmoid(-z))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g ** 2)


def _exact_weights(w):
    n, half = w["codes"].shape
    nib = torch.empty(n, half, 2, dtype=torch.float64, device=w["codes"].device)
    nib[..., 0], nib[..., 1] = w["codes"] % 16, w["codes"] // 16
    nib = nib.reshape(n, 2 * half)
    if w["format"] == "int4":
        s = w["scales"].double().repeat_interleave(w["group"], 1)
        z = w["zeros"].double().repeat_interleave(w["group"], 1) if w["zeros"] is not None else 8
        return s * (nib - z)
    sign, c = 1 - 2 * (nib >= 8).double(), nib % 8
    exp, man = torch.floor(c / 2), c % 2
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * torch.exp2(exp - 1))
    b = w["scales"].double()
    if w["format"] == "mxfp4":
        s = torch.exp2(b - 127)
    else:
        exp, man = torch.floor((b % 128) / 8), b % 8
        s = torch.where(exp == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(exp - 7)) * (1 - 2 * (b >= 128).double()) * w["scale_2"]
    return sign * mag * s.repeat_interleave(w["group"], 1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("gated", "train"):
        x, w0, w1 = s["x"].double(), s["w0"].double(), s["w1"].double()
        g, u = torch.mm(x, w0.t().contiguous()), torch.mm(x, w1.t().contiguous())
        a, slope = _exact_act(g, case["act"])
        out = {"h": a * u}
        if kind == "train":
            dh = s["dh"].double()
            du, dg = dh * a, dh * u * slope
            out["dx"] = torch.mm(dg, w0) + torch.mm(du, w1)
            out["dw0"], out["dw1"] = torch.mm(dg.t().contiguous(), x), torch.mm(du.t().contiguous(), x)
        return out
    if kind == "gradient":
        dy = s["dy"].double()
        return {"dx": torch.mm(dy, s["w"].double()), "dw": torch.mm(dy.t().contiguous(), s["x"].double())}
    y = [torch.mm(s["x"].double(), _exact_weights(w).t().contiguous()) for w in s["weights"]]
    if kind == "gemv":
        return {"y": y[0]}
    return {"h": _exact_act(y[0], case["act"])[0] * y[1]}
