"""Reference of linear attention with a decay for each head, in 64 bits: every
pair of tokens, each sample and head by itself."""

import torch


def _pairs(N, g, reverse=False):
    t = torch.arange(N, dtype=torch.float64)
    e = t[:, None] - t
    return torch.where(e >= 0, torch.exp(g * e.clamp(min=0)), 0.0), e.clamp(min=0)


def forward(q, k, v, log_decay, scale, state=None, sums=False):
    """q, k, v [N, H, d] of one sequence; returns o [N, H, d] and the state
    behind.  sums: the sums of the terms' absolute values instead, each term
    times 1 + |log_decay| * distance, which its power's error goes with."""
    q, k, v = q.double(), k.double(), v.double()
    if sums:
        q, k, v = q.abs(), k.abs(), v.abs()
        scale = abs(scale)
    N, H, d = q.shape
    o, out = torch.zeros_like(q), torch.zeros(H, d, d, dtype=torch.float64)
    t = torch.arange(N, dtype=torch.float64)
    for h in range(H):
        g = float(max(log_decay[h].double(), torch.tensor(-1e30)))
        D, e = _pairs(N, g)
        first, last = torch.exp(g * (t + 1)), torch.exp(g * (N - 1 - t))
        over = torch.exp(torch.tensor(g * N, dtype=torch.float64))
        if sums:
            D = D * (1 + abs(g) * e)
            first = first * (1 + abs(g) * (t + 1))
            last = last * (1 + abs(g) * (N - 1 - t))
            over = over * (1 + abs(g) * N)
            D, first, last = (torch.nan_to_num(x) for x in (D, first, last))
        S0 = torch.zeros(d, d, dtype=torch.float64) if state is None else \
            state[h].double()
        if sums:
            S0 = S0.abs()
        o[:, h] = scale * (((q[:, h] @ k[:, h].T) * D) @ v[:, h]
                           + first[:, None] * (q[:, h] @ S0))
        out[h] = over * S0 + (k[:, h] * last[:, None]).T @ v[:, h]
    return o, out


def backward(do, q, k, v, log_decay, scale, state=None, dstate_out=None,
             sums=False):
    """dq, dk, dv [N, H, d] and dstate, or the sums of absolute values."""
    t = (lambda s: None if s is None else s.transpose(-1, -2))
    dq, _ = forward(do, v, k, log_decay, scale, t(state), sums)
    # backwards in time; the last token takes dstate_out as it is
    do, q, k, v = (x.double().flip(0) for x in (do, q, k, v))
    N, H, d = q.shape
    zero = torch.zeros(H, d, d, dtype=torch.float64)
    dS = zero if dstate_out is None else dstate_out.double()
    dk, _ = forward(v, do, q, log_decay, scale, None, sums)
    dv, own = forward(k, q, do, log_decay, scale, None, sums)
    g = log_decay.double().clamp(min=-1e30)
    n = torch.arange(N, dtype=torch.float64)
    pw = torch.exp(g * n[:, None])
    one, over = torch.exp(g), torch.exp(g * N)
    if sums:
        pw = torch.nan_to_num(pw * (1 + g.abs() * n[:, None]))
        one = torch.nan_to_num(one * (1 + g.abs()))
        over = torch.nan_to_num(over * (1 + g.abs() * N))
        dS, k, v, scale = dS.abs(), k.abs(), v.abs(), abs(scale)
    dk += pw[..., None] * torch.stack([v[:, h] @ dS[h].T for h in range(H)], 1)
    dv += pw[..., None] * torch.stack([k[:, h] @ dS[h] for h in range(H)], 1)
    dstate = over[:, None, None] * dS + scale * one[:, None, None] * own
    return dq, dk.flip(0), dv.flip(0), dstate
