"""The gated feed-forward's products at sizes that reach every way they are
launched, as whole numbers, bit for bit (see tests/test_glu_gpu.py)."""

import pytest
import torch

import adaln_fwd_amd as A
from tests.glu_sizes import BF16, SIZES

pytestmark = pytest.mark.gpu


def _whole(M, D, F, seed, dt):
    """G = 64 + a few, U a few, dh in -1, 0, 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda",
                             dtype=torch.int8).to(dt)

    def sparse(r, c, p):
        keep = torch.rand(r, c, generator=g, device="cuda") < p
        return (integers(0, 2, r, c) * 2 - 1) * keep

    # about 8 terms of +-1 in each G and U
    p = min(1.0, (8 / max(D - 1, 1)) ** 0.5)
    x, wg, wu = sparse(M, D, p), sparse(F, D, p), sparse(F, D, p)
    x[:, 0], wg[:, 0], wu[:, 0] = 8, 8, 0
    return integers(-1, 2, M, F), x, wg, wu


def _once(v, dt):
    """Whole numbers below 2^24, rounded once."""
    assert v.abs().max() < 2 ** 24
    return v.float().to(dt)


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_whole_numbers_exact(size):
    code, M, D, F = size
    dt = torch.bfloat16 if code == BF16 else torch.float32
    act = "gelu" if M % 2 else "silu"
    print(f"[glu] launches {size} {act}", flush=True)
    dh, x, wg, wu = _whole(M, D, F, M + D + F, dt)
    h, saved = A.glu_fwd(x, wg, wu, act=act, save=True)
    assert torch.equal(A.glu_fwd(x, wg, wu, act=act), h)
    xd, wgd, wud, dhd = [t.double() for t in (x, wg, wu, dh)]
    G, U = xd @ wgd.t(), xd @ wud.t()
    assert G.min() >= 32 and G.max() < 256 and U.abs().max() < 256
    assert torch.equal(saved[0].double(), G)
    assert torch.equal(saved[1].double(), U)
    assert torch.equal(h, _once(G * U, dt))
    dG, dU = dhd * U, dhd * G
    # no partial sum reaches 2^24 either, in any order
    for terms in (dG.abs() @ wgd.abs() + dU.abs() @ wud.abs(),
                  dG.abs().t() @ xd.abs(), dU.abs().t() @ xd.abs()):
        assert terms.max() < 2 ** 24
    want = [_once(v, dt) for v in (dG @ wgd + dU @ wud, dG.t() @ xd,
                                   dU.t() @ xd)]
    del G, U, dG, dU, terms
    for s in (saved, None):
        got = A.glu_bwd(dh, x, wg, wu, s, act=act)
        for a, b, n in zip(got, want, ("dx", "dwg", "dwu")):
            assert torch.equal(a, b), (n, s is None, int((a != b).sum()))
