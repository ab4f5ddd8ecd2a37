"""The gated MLP block and its gradient, written out in FP64 (test
infrastructure only). Works on numpy arrays and on torch FP64 tensors alike:
only operators, `exp` of the array's own library and transposes are used."""
from __future__ import annotations

import math

import numpy as np


def _exp(x):
    if isinstance(x, np.ndarray):
        with np.errstate(over="ignore"):
            return np.exp(x)
    return x.exp()


def gate(g, act: str):
    """(act(g), act'(g)): silu is g / (1 + e^-g), gelu_tanh 0.5 g (1 + tanh t)
    with t = sqrt(2 / pi) (g + 0.044715 g^3), and (1 + tanh t) / 2 is 1 / (1 + e^-2t)."""
    if act == "silu":
        z, dz = g, 1.0
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1.0 + 3.0 * 0.044715 * g ** 2)
    s, r = 1.0 / (1.0 + _exp(-z)), 1.0 / (1.0 + _exp(z))       # r = 1 - s
    return g * s, s + g * dz * s * r


def gated(a, b0, b1, act: str):
    """(h, g, u) of a [M, K], b0 and b1 [N, K]."""
    g, u = a @ b0.T, a @ b1.T
    return gate(g, act)[0] * u, g, u


def gate_grad(dh, g, u, act: str):
    """(dg, du) of h = act(g) u."""
    v, slope = gate(g, act)
    return dh * u * slope, dh * v


def gated_backward(dh, a, b0, b1, g, u, act: str):
    """(da, db0, db1) for given g and u."""
    dg, du = gate_grad(dh, g, u, act)
    return dg @ b0 + du @ b1, dg.T @ a, du.T @ a
