"""Reference of the way to the experts and back, in 64 bits, choice by choice."""

import torch


def plan(expert, E):
    T, k = expert.shape
    e = expert.tolist()
    offsets, slot = [0], [[-1] * k for _ in range(T)]
    n = 0
    lists = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if 0 <= e[t][j] < E:
                lists[e[t][j]].append((t, j))
    for part in lists:
        for t, j in part:
            slot[t][j] = n
            n += 1
        offsets.append(n)
    return (torch.tensor(offsets, dtype=torch.int32),
            torch.tensor(slot, dtype=torch.int32).reshape(T, k))


def _each(slot):
    """(choice number, tokens that have it, their sorted rows)."""
    for j in range(slot.shape[1]):
        t = torch.nonzero(slot[:, j] >= 0).flatten()
        yield j, t, slot[t, j].long()


def sort_fwd(x, slot, xs):
    xs = xs.clone()
    for _, t, r in _each(slot):
        xs[r] = x[t]
    return xs


def sort_bwd(dxs, slot):
    return join_fwd(dxs, slot, torch.ones(slot.shape, dtype=torch.float64))


def join_fwd(ys, slot, w):
    y = torch.zeros(slot.shape[0], ys.shape[1], dtype=torch.float64)
    for j, t, r in _each(slot):
        y[t] += w[t, j, None].double() * ys[r].double()
    return y


def join_bwd(dy, ys, slot, w, dys):
    dys, dw = dys.double().clone(), torch.zeros(slot.shape, dtype=torch.float64)
    for j, t, r in _each(slot):
        dys[r] = w[t, j, None].double() * dy[t].double()
        dw[t, j] = (dy[t].double() * ys[r].double()).sum(-1)
    return dys, dw
