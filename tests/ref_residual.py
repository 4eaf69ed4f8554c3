"""Reference of the gated join and its dropout, in numpy and 64 bits."""

import numpy as np
import torch

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Philox 4x32-10: counter [..., 4] and key (two words) to [..., 4]."""
    x = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    lo = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = x[0] * np.uint64(M0), x[2] * np.uint64(M1)
        x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), b & lo,
             (a >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + W0) % 2 ** 32, (k[1] + W1) % 2 ** 32]
    return np.stack(x, -1).astype(np.uint32)


def keep_mask(rows, D, p, rng, row0=0):
    """bool [rows, D] and the factor of what is kept, from the documented
    numbering."""
    limit = int(np.floor((1 - p) * 65536 + 0.5))
    per = -(-D // 8)
    block = np.arange(row0 * per, (row0 + rows) * per, dtype=np.uint64)
    seed, call = (int(v) % 2 ** 64 for v in rng)
    ctr = np.stack([block & np.uint64(0xFFFFFFFF), block >> np.uint64(32),
                    np.full_like(block, call % 2 ** 32),
                    np.full_like(block, call // 2 ** 32)], -1)
    w = philox(ctr, (seed % 2 ** 32, seed // 2 ** 32))
    bits = np.stack([w & 0xFFFF, w >> 16], -1).reshape(rows, per * 8)[:, :D]
    return torch.from_numpy(bits < limit), 65536 / limit


def forward(x, h, gate, p, rng, mod=None):
    """x, h [rows, D] (x may be None), gate [nmod, D] or None, mod [rows]."""
    h = h.double()
    g = torch.ones_like(h) if gate is None else gate.double()[mod]
    y = g * h
    x = torch.zeros_like(h) if x is None else x.double()
    if p > 0:
        keep, s = keep_mask(*h.shape, p, rng)
        return torch.where(keep, x + s * y, x)
    return x + y


def backward(dy, h, gate, p, rng, mod=None, nmod=0):
    """(dh, dgate, the sum of the absolute terms of dgate)."""
    dy, h = dy.double(), h.double()
    g = torch.ones_like(h) if gate is None else gate.double()[mod]
    f = torch.ones_like(h)
    if p > 0:
        keep, s = keep_mask(*h.shape, p, rng)
        f = keep.double() * s
    dh = torch.where(f > 0, dy * g * f, 0.0)
    if gate is None:
        return dh, None, None
    terms = torch.where(f > 0, dy * h * f, 0.0)
    zero = torch.zeros(nmod, h.shape[1], dtype=torch.float64)
    return (dh, zero.index_add(0, mod, terms),
            zero.index_add(0, mod, terms.abs()))
