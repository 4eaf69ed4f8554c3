"""Rotary positions and query/key norms in float64 on the CPU, written from
the formulas: pairs as 2 x 2 rotations applied to each head, and the norm's
gradient from its Jacobian.  Shared by the CPU and GPU tests."""

import torch

EPS = 1e-6


def angles(pos, freqs):
    """pos [.., N, axes] int, freqs [axes, pairs] -> [.., N, pairs]."""
    return pos.double().cpu() @ torch.as_tensor(freqs, dtype=torch.float64)


def pair_index(pairs, layout):
    """The two features of every pair."""
    j = torch.arange(pairs)
    return (2 * j, 2 * j + 1) if layout == "interleaved" else (j, j + pairs)


def rotate(x, ang, layout, sign=1.0):
    """x [B, N, H, d] float64, ang [N or B,N, pairs]."""
    u, v = pair_index(ang.shape[-1], layout)
    c, s = torch.cos(ang).unsqueeze(-2), sign * torch.sin(ang).unsqueeze(-2)
    if ang.dim() == 2:
        c, s = c.unsqueeze(0), s.unsqueeze(0)
    y = x.clone()
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    return y


def qk_fwd(x, w, ang, layout, eps=EPS):
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return rotate(x * r * w, ang, layout)


def qk_bwd(dy, x, w, ang, layout, eps=EPS):
    """dx, dw, and the sum of |terms| of dw (for tolerances)."""
    t = rotate(dy, ang, layout, -1.0)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    g = t * w
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (t * xh).sum((0, 1, 2)), (t * xh).abs().sum((0, 1, 2))
