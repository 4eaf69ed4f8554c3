"""Gated feed-forward in float64 on the CPU, from the formulas."""

import math

import torch


def act(g, name):
    """act(g), act'(g)."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s + g * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    v = c * (g + 0.044715 * g ** 3)
    # (1 + tanh(v)) / 2 as a logistic function: 1 + tanh(v) itself loses its
    # digits to cancellation below v = -18, in float64 too
    s = 1 / (1 + torch.exp(-2 * v))
    return g * s, s + g * 2 * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def fwd(x, wg, wu, name):
    G, U = x @ wg.t(), x @ wu.t()
    return act(G, name)[0] * U, G, U


def bwd(dh, x, wg, wu, name):
    """dx, dwg, dwu, dG, dU."""
    _, G, U = fwd(x, wg, wu, name)
    a, da = act(G, name)
    dG, dU = dh * U * da, dh * a
    return dG @ wg + dU @ wu, dG.t() @ x, dU.t() @ x, dG, dU
